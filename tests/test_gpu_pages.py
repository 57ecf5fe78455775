"""The paged-cache operators against their formulas in 64 bits.

Bounds.  A bf16 output is off by half a step of its own (2^-8 relative) and by
that of each softmax weight, 2^-8 sum p|v|.  fp32 parts: a logit is a sum of D
products, off by at most (D + 8) 2^-24 scale sum |q||k| (the fused sum, its
scaling) plus 4 * 2^-24 |z| (reading it in base 2, the exponential), which moves
each weight and the sum of weights by that relative amount; sums of n weights or
values in any order by n 2^-24; joining parts by less than 64 * 2^-24.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from kv_cache_eviction_h2o_gb300 import binding as L   # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U24 = 2.0 ** -24


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


class Cache:
    """A pool, block tables of random pages, and requests of given lengths."""

    def __init__(self, lengths, heads, d, ps, dtype, seed=0, extra=3, width=None, kscale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.ps, self.heads, self.d, self.dtype = ps, heads, d, dtype
        self.lengths = list(lengths)
        owned = [-(-n // ps) for n in lengths]
        self.width = width or max(1, max(owned))
        pages = sum(owned) + extra
        perm = torch.randperm(pages, generator=g).numpy()
        self.table = np.full((len(lengths), self.width), -1, np.int32)
        at = 0
        for i, n in enumerate(owned):
            self.table[i, :n] = perm[at:at + n]
            at += n
        self.spare = perm[at:].astype(np.int32)
        shape = (pages, heads, ps, d)
        self.K = (kscale * (torch.randn(shape, generator=g) + torch.randn((pages, heads, 1, d), generator=g))).to(dtype)
        self.V = torch.randn(shape, generator=g).to(dtype)
        # what no request holds is never to be seen
        live = torch.zeros(pages, ps, dtype=torch.bool)
        for i, n in enumerate(self.lengths):
            for t in range(n):
                live[self.table[i, t // ps], t % ps] = True
        dead = (~live)[:, None, :, None].expand(shape)
        self.K[dead] = float("nan")
        self.V[dead] = float("inf")

    def bounds(self):
        return torch.stack([self.K.amin(2), self.K.amax(2)], 2)

    def rows(self, pages, head, n):
        """The first n keys and values of one head on these pages, fp64."""
        p = torch.as_tensor(np.asarray(pages)).long()
        return tuple(x[p, head].reshape(-1, self.d)[:n].double() for x in (self.K, self.V))


def _attention(q, k, v, scale):
    """softmax(scale q.k) v for q [G][D], and sum p|v|, max |z|, scale max sum |q||k|."""
    if k.shape[0] == 0:
        z = torch.zeros_like(q)
        return z, z, 0.0, 0.0
    z = (q @ k.T) * scale
    p = torch.softmax(z, -1)
    return p @ v, p @ v.abs(), z.abs().max().item(), scale * (q.abs() @ k.abs().T).max().item()


def _tolerance(dtype, d, n, y, av, zmax, smax):
    t = U24 * (2 * ((d + 8) * smax + 4 * zmax) + 2 * n + 64) * av
    if dtype is BF16:
        t = t * (1 + 2.0 ** -7) + 2.0 ** -8 * (y.abs() + av * (1 + 2.0 ** -7))
    return t + U24 * y.abs() + 1e-30


def _check(got, want, what):
    y, tol = want
    off = (got.double().cpu() - y).abs()
    assert torch.isfinite(got).all(), what
    worst = (off - tol).max().item()
    assert worst <= 0, "%s: %g beyond its bound (largest error %g)" % (what, worst, off.max().item())


def _picks(q, bounds, pages, head, budget, recent):
    """Indexes of the pages one row reads of one head (q [G][D])."""
    n = len(pages)
    if n <= budget:
        return np.arange(n)
    b = bounds[torch.as_tensor(pages[:n - recent]).long(), head].double()
    s = torch.maximum(q[:, None] * b[None, :, 0], q[:, None] * b[None, :, 1]).sum((0, 2))
    s = torch.where(s.isnan(), torch.full_like(s, float("inf")), s).numpy()
    best = np.lexsort((np.arange(n - recent), -s))[:budget - recent]
    return np.concatenate([np.sort(best), np.arange(n - recent, n)])


def _sparse_ref(c, q, seq, pos, budget, recent, scale):
    rows, hq, d = q.shape
    G = hq // c.heads
    b = c.bounds()
    y, tol = torch.zeros(rows, hq, d, dtype=torch.float64), torch.zeros(rows, hq, d, dtype=torch.float64)
    picked = np.full((rows, c.heads, budget), -1, np.int32)
    for r in range(rows):
        if seq[r] < 0 or pos[r] < 0:
            continue
        mine = c.table[seq[r], :pos[r] // c.ps + 1]
        for h in range(c.heads):
            qh = q[r, h * G:(h + 1) * G].double()
            at = _picks(qh, b, mine, h, budget, recent)
            picked[r, h, :len(at)] = at
            n = (len(at) - 1) * c.ps + pos[r] % c.ps + 1
            a = _attention(qh, *c.rows(mine[at], h, n), scale)
            y[r, h * G:(h + 1) * G] = a[0]
            tol[r, h * G:(h + 1) * G] = _tolerance(c.dtype, d, n, *a)
    return (y, tol), picked


def _sparse(c, q, seq, pos, budget, recent, scale, out=None, picked=None, stream=None, bounds=True):
    out = torch.full(q.shape, 7.0, dtype=c.dtype, device="cuda") if out is None else out
    picked = torch.full((q.shape[0], c.heads, budget), -7, dtype=torch.int32, device="cuda") if picked is None else picked
    L.h2o_page_attend(q, _i32(seq), _i32(pos), c.K.cuda(), c.V.cuda(), c.bounds().cuda() if bounds else None, _i32(c.table),
                      budget, recent, scale, out, picked, stream or torch.cuda.current_stream())
    return out, picked


def _queries(rows, hq, d, dtype, seed):
    return torch.randn(rows, hq, d, generator=torch.Generator().manual_seed(seed)).to(dtype)


SHAPES = [  # heads, groups, d, page size
    (4, 1, 64, 16), (2, 4, 128, 16), (1, 16, 128, 32), (3, 5, 64, 64), (2, 8, 128, 128), (1, 2, 64, 128), (2, 9, 128, 64), (5, 3, 128, 16),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,groups,d,ps", SHAPES)
def test_sparse(dtype, heads, groups, d, ps):
    # one token, a page to its end, one more, an odd long one; several rows of one request; few and many pages
    lengths = [1, ps, ps + 1, 7 * ps + 5, 40 * ps + ps // 2 + 1]
    c = Cache(lengths, heads, d, ps, dtype, seed=heads * d)
    seq = [0, 1, 2, 3, 3, 4, 4, 4, 4]
    pos = [0, ps - 1, ps, 7 * ps + 4, 3 * ps - 1, 40 * ps + ps // 2, 39 * ps - 1, 20 * ps, 11 * ps + 1]
    q = _queries(len(seq), heads * groups, d, dtype, 3)
    for budget, recent in ((2, 1), (6, 6), (11, 3), (40, 2), (64, 1)):
        want, picked = _sparse_ref(c, q, seq, pos, budget, recent, d ** -0.5)
        out, got = _sparse(c, q.cuda(), seq, pos, budget, recent, d ** -0.5)
        np.testing.assert_array_equal(got.cpu().numpy(), picked, err_msg="budget %d" % budget)
        _check(out, want, "budget %d" % budget)


def test_sparse_long_request_picks_exactly():
    # thousands of pages, most of them close to the border
    c = Cache([16 * 4093 + 3], 2, 64, 16, BF16, seed=5)
    q = _queries(3, 8, 64, BF16, 9)
    seq, pos = [0, 0, 0], [16 * 4093 + 2, 16 * 3001, 16 * 100 + 15]
    want, picked = _sparse_ref(c, q, seq, pos, 300, 10, 0.125)
    out, got = _sparse(c, q.cuda(), seq, pos, 300, 10, 0.125)
    np.testing.assert_array_equal(got.cpu().numpy(), picked)
    _check(out, want, "long")


@pytest.mark.parametrize("dtype,d,groups,pages", [(BF16, 64, 2, 16384), (F32, 128, 16, 16384), (BF16, 128, 16, 9000), (F32, 64, 1, 4097)])
def test_sparse_at_the_widest_table(dtype, d, groups, pages):
    # a table may list a page more than once: scores tie over and over, and the lowest entries win
    c = Cache([40 * 16], 1, d, 16, dtype, seed=d)
    table = np.tile(c.table, (1, -(-pages // 40)))[:, :pages]
    c.table = np.concatenate([table, np.full((1, 16384 - pages), -1, np.int32)], 1)
    q = _queries(2, groups, d, dtype, 4)
    for budget, recent in ((4096, 7), (100, 1)):
        seq, pos = [0, 0], [16 * pages - 1, 16 * (pages // 2) + 3]
        want, picked = _sparse_ref(c, q, seq, pos, budget, recent, d ** -0.5)
        out, got = _sparse(c, q.cuda(), seq, pos, budget, recent, d ** -0.5)
        np.testing.assert_array_equal(got.cpu().numpy(), picked, err_msg="budget %d" % budget)
        _check(out, want, "budget %d" % budget)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["same", "pairs", "zero", "last bit"])
def test_sparse_ties_go_to_the_lowest_page(dtype, kind):
    ps, n = 16, 70
    c = Cache([n * ps], 2, 64, ps, dtype, seed=1)
    q = _queries(1, 4, 64, dtype, 2)
    pages = torch.as_tensor(c.table[0]).long()
    if kind == "same":
        c.K[pages] = c.K[pages[:1]]
    elif kind == "pairs":
        c.K[pages[1::2]] = c.K[pages[::2]]
    elif kind == "zero":
        q.zero_()
    else:
        # scores that differ in the last bit of one key's smallest channel: fp32 sums cannot tell them apart
        c.K[pages] = c.K[pages[:1]]
        step = 2.0 ** -20 if dtype is F32 else 2.0 ** -7
        q[..., 5] = 2.0 ** -16
        c.K[pages, :, :, 5] = (1 + step * (torch.randperm(n, generator=torch.Generator().manual_seed(0)) % 16)).to(dtype)[:, None, None]
    for budget, recent in ((8, 1), (31, 5), (69, 2)):
        want, picked = _sparse_ref(c, q, [0], [n * ps - 1], budget, recent, 0.125)
        out, got = _sparse(c, q.cuda(), [0], [n * ps - 1], budget, recent, 0.125)
        np.testing.assert_array_equal(got.cpu().numpy(), picked, err_msg="%s %d" % (kind, budget))
        _check(out, want, "%s %d" % (kind, budget))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sparse_infinite_and_nan_keys(dtype):
    ps, n = 32, 20
    c = Cache([n * ps], 1, 128, ps, dtype, seed=4)
    q = _queries(1, 2, 128, dtype, 5).abs() + 0.5
    c.K[int(c.table[0, 3]), 0, 1, 7] = float("nan")         # ranks first
    c.K[int(c.table[0, 9]), 0, 0, 2] = float("-inf")        # as a minimum: q > 0 never takes it
    _, picked = _sparse_ref(c, q, [0], [n * ps - 1], 5, 2, 0.1)
    out, got = _sparse(c, q.cuda(), [0], [n * ps - 1], 5, 2, 0.1)
    np.testing.assert_array_equal(got.cpu().numpy(), picked)
    assert 3 in picked[0, 0]
    assert out.isnan().all()
    # a key of -inf logit in a page that is read takes no weight
    c = Cache([40], 1, 128, ps, dtype, seed=4)
    c.K[int(c.table[0, 0]), 0, 1] = float("-inf")
    ref = Cache([40], 1, 128, ps, dtype, seed=4)
    keep = [t for t in range(40) if t != 1]
    k, v = ref.rows(ref.table[0], 0, 40)
    a = _attention(q[0].double(), k[keep], v[keep], 0.1)
    out, _ = _sparse(c, q.cuda(), [0], [39], 5, 2, 0.1)
    _check(out[0], (a[0], _tolerance(dtype, 128, 40, *a)), "-inf key")
    # every logit -inf: nothing to attend to
    c.K[:] = float("-inf")
    out, _ = _sparse(c, q.cuda(), [0], [39], 5, 2, 0.1)
    assert (out == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kscale", [3e35, 8e35, 3e36])      # sums of |w||bound| below, about and above fp32's largest
def test_sparse_scores_near_the_end_of_fp32(dtype, kscale):
    ps, n = 16, 60
    c = Cache([n * ps], 2, 64, ps, dtype, seed=21, kscale=kscale)
    q = _queries(1, 2, 64, dtype, 22)
    want, picked = _sparse_ref(c, q, [0], [n * ps - 1], 9, 2, 1 / (8 * kscale))
    out, got = _sparse(c, q.cuda(), [0], [n * ps - 1], 9, 2, 1 / (8 * kscale))
    np.testing.assert_array_equal(got.cpu().numpy(), picked)
    _check(out, want, "large scores")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sparse_large_logits(dtype):
    # one key takes all the weight, whatever the scale of the logits
    c = Cache([500], 2, 64, 16, dtype, seed=8, kscale=40.0)
    q = (_queries(1, 4, 64, dtype, 1) * 30).to(dtype)
    want, picked = _sparse_ref(c, q, [0], [499], 12, 4, 0.5)
    out, got = _sparse(c, q.cuda(), [0], [499], 12, 4, 0.5)
    np.testing.assert_array_equal(got.cpu().numpy(), picked)
    _check(out, want, "large logits")


def test_rows_that_are_padding_empty_or_bad():
    ps = 16
    c = Cache([100, 50], 2, 64, ps, BF16, seed=2)
    seq, pos = [0, -1, 1, 0, 2, 1, -5, 0], [99, 10, -1, 5, 3, ps * c.width, 0, -(1 << 31)]
    q = _queries(len(seq), 4, 64, BF16, 1)
    want, picked = _sparse_ref(c, q[[0, 3]], [0, 0], [99, 5], 3, 1, 0.125)
    for call in ("sparse", "prefix"):
        if call == "sparse":
            out, got = _sparse(c, q.cuda(), seq, pos, 3, 1, 0.125)
            np.testing.assert_array_equal(got.cpu().numpy()[[0, 3]], picked)
            assert (got[1] == -7).all() and (got[6] == -7).all() and (got[2] == -1).all() and (got[4] == -1).all()
            _check(out[[0, 3]], want, "live rows")
        else:
            out = _prefix(c, q.cuda(), seq, pos, [], 0, 0.125)
            _check(out[[0, 3]], _prefix_ref(c, q[[0, 3]], [0, 0], [99, 5], [], 0, 0.125), "live rows")
        assert (out[1] == 7).all() and (out[6] == 7).all(), "padding rows are left as they were"
        assert (out[2] == 0).all() and (out[7] == 0).all(), "no keys: zero"
        assert out[4].isnan().all() and out[5].isnan().all(), "a row outside the tables is NaN"


def test_table_entries_outside_the_pool():
    c = Cache([200, 200], 2, 64, 16, BF16, seed=2)
    q = _queries(2, 4, 64, BF16, 1)
    good, _ = _sparse(c, q.cuda(), [0, 1], [199, 199], 4, 1, 0.125)
    for entry in (-1, c.K.shape[0], 1 << 30):
        bad = Cache([200, 200], 2, 64, 16, BF16, seed=2)
        bad.table[0, 5] = entry                              # ranked: must show
        out, _ = _sparse(bad, q.cuda(), [0, 1], [199, 199], 4, 1, 0.125)
        assert out[0].isnan().all() and torch.equal(out[1], good[1])
        out = _prefix(bad, q.cuda(), [0, 1], [199, 199], bad.table[1, :3], 40, 0.125)
        assert out[0].isnan().all() and out[1].isfinite().all()
        out = _prefix(bad, q.cuda(), [0, 1], [30, 30], bad.table[0, :6], 90, 0.125)
        assert out.isnan().all()


# ------------------------------------------------------------ shared prefix


def _prefix(c, q, seq, pos, ptable, plen, scale, out=None, stream=None):
    out = torch.full(q.shape, 7.0, dtype=c.dtype, device="cuda") if out is None else out
    rows, hq, d = q.shape
    n = L.h2o_prefix_work_bytes(rows, c.heads, hq // c.heads, d, plen, L.H2O_BF16 if c.dtype is BF16 else L.H2O_F32)
    work = torch.full((n,), 255, dtype=torch.uint8, device="cuda")       # NaN wherever it is read unwritten
    L.h2o_prefix_attend(q, _i32(seq), _i32(pos), c.K.cuda(), c.V.cuda(), _i32(ptable) if plen else None, plen, _i32(c.table), scale,
                        out, work, stream or torch.cuda.current_stream())
    return out


def _prefix_ref(c, q, seq, pos, ptable, plen, scale):
    rows, hq, d = q.shape
    G = hq // c.heads
    y, tol = torch.zeros(rows, hq, d, dtype=torch.float64), torch.zeros(rows, hq, d, dtype=torch.float64)
    for h in range(c.heads):
        pk, pv = c.rows(ptable, h, plen)
        for r in range(rows):
            k, v = c.rows(c.table[seq[r], :pos[r] // c.ps + 1] if pos[r] >= 0 else [], h, max(0, pos[r] + 1))
            a = _attention(q[r, h * G:(h + 1) * G].double(), torch.cat([pk, k]), torch.cat([pv, v]), scale)
            y[r, h * G:(h + 1) * G] = a[0]
            tol[r, h * G:(h + 1) * G] = _tolerance(c.dtype, d, plen + pos[r] + 1, *a)
    return y, tol


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,groups,d,ps", SHAPES)
def test_prefix(dtype, heads, groups, d, ps):
    lengths = [1, ps + 1, 3 * ps, 77, 1000]                  # the last request's pages are the prefix
    c = Cache(lengths, heads, d, ps, dtype, seed=heads * d + 1)
    seq, pos = [0, 1, 1, 2, 3, 3, 0], [0, ps, ps - 1, 3 * ps - 1, 76, 0, -1]
    q = _queries(len(seq), heads * groups, d, dtype, 6)
    for plen in (0, 1, 15, ps, 130, 1000):
        want = _prefix_ref(c, q, seq, pos, c.table[4], plen, d ** -0.5)
        _check(_prefix(c, q.cuda(), seq, pos, c.table[4], plen, d ** -0.5), want, "prefix %d" % plen)


@pytest.mark.parametrize("dtype,rows,heads,groups,d,plen", [
    (BF16, 1, 1, 1, 128, 4099), (BF16, 129, 1, 1, 128, 700), (BF16, 40, 2, 8, 128, 2500), (BF16, 67, 1, 8, 64, 1111),
    (BF16, 300, 3, 1, 64, 257), (BF16, 33, 1, 16, 128, 129), (BF16, 1000, 1, 16, 64, 300), (F32, 70, 2, 4, 64, 600), (F32, 65, 1, 1, 128, 333),
])
def test_prefix_many_rows(dtype, rows, heads, groups, d, plen):
    g = np.random.default_rng(rows)
    own = [int(x) for x in g.integers(1, 50, 9)] + [plen]
    c = Cache(own, heads, d, 32, dtype, seed=rows)
    seq = [int(x) for x in g.integers(0, 9, rows)]
    pos = [int(g.integers(-1, own[s])) for s in seq]
    q = _queries(rows, heads * groups, d, dtype, 6)
    want = _prefix_ref(c, q, seq, pos, c.table[9], plen, d ** -0.5)
    _check(_prefix(c, q.cuda(), seq, pos, c.table[9], plen, d ** -0.5), want, "rows %d" % rows)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [3, 130])                  # one and two tiles of 128 query rows
def test_prefix_many_tiles_a_block(rows, d):
    # as many cache heads as fill the GPU with few ranges each, so that a block sweeps many key tiles
    heads, ps, plen, scale = 40, 32, 5077, d ** -0.5
    c = Cache([1, plen], heads, d, ps, BF16, seed=d + rows)
    q = _queries(rows, heads, d, BF16, 11)
    out = _prefix(c, q.cuda(), [0] * rows, [-1] * rows, c.table[1], plen, scale)
    for h in range(heads):
        k, v = c.rows(c.table[1], h, plen)
        a = _attention(q[:, h].double().cuda(), k.cuda(), v.cuda(), scale)
        _check(out[:, h], (a[0].cpu(), _tolerance(BF16, d, plen, *a).cpu()), "head %d" % h)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefix_large_and_infinite_logits(dtype):
    c = Cache([60, 700], 1, 128, 64, dtype, seed=3, kscale=20.0)
    q = (_queries(2, 4, 128, dtype, 1) * 10).to(dtype)
    want = _prefix_ref(c, q, [0, 0], [59, 20], c.table[1], 650, 0.3)
    _check(_prefix(c, q.cuda(), [0, 0], [59, 20], c.table[1], 650, 0.3), want, "large logits")
    # keys of -inf logit take no weight; prefix rows all of -inf leave the own part, and all of them zero
    q = q.abs() + 0.5
    c.K[torch.as_tensor(c.table[1, :11]).long()] = float("-inf")
    want = _prefix_ref(c, q, [0, 0], [59, 20], [], 0, 0.3)
    _check(_prefix(c, q.cuda(), [0, 0], [59, 20], c.table[1], 650, 0.3), want, "own part alone")
    assert (_prefix(c, q.cuda(), [0, 0], [-1, -1], c.table[1], 650, 0.3) == 0).all()


# --------------------------------------------------------- tables and writes


def _tables_ref(before, new, free, ps, table, cap):
    n, width = len(before), table.shape[1]
    need = [-(-(b + t) // ps) - -(-b // ps) for b, t in zip(before, new)]
    err = 0
    if any(b < 0 or t < 0 for b, t in zip(before, new)):
        err |= 1
        need = [x if b >= 0 and t >= 0 else 0 for x, b, t in zip(need, before, new)]
        new_ok = [t if b >= 0 and t >= 0 else 0 for b, t in zip(before, new)]
    else:
        new_ok = list(new)
    if sum(new_ok) > cap:
        err |= 2
    if sum(need) > len(free):
        err |= 4
    if any(b >= 0 and t >= 0 and -(-(b + t) // ps) > width for b, t in zip(before, new)):
        err |= 8
    table, free = table.copy(), list(free)
    start, seq, pos, slot, after = [0], [], [], [], list(before)
    if err:
        start = [0] * (n + 1)
    else:
        taken = 0
        for i, (b, t) in enumerate(zip(before, new)):
            for p in range(-(-b // ps), -(-(b + t) // ps)):
                table[i, p] = free[taken]
                taken += 1
            for x in range(b, b + t):
                seq.append(i)
                pos.append(x)
                slot.append(table[i, x // ps] * ps + x % ps)
            after[i] = b + t
            start.append(start[-1] + t)
    pad = [-1] * (cap - len(seq))
    status = [0, 0, 0, err] if err else [start[-1], sum(need), max(after), 0]
    return table, after, start, seq + pad, pos + pad, slot + pad, status


def _tables(before, new, free, ps, table, cap, stream=None):
    n = len(before)
    shift = n % 3                                             # int arrays start anywhere
    out = [_i32(table)] + [torch.full((k + shift,), -9, dtype=torch.int32, device="cuda")[shift:] for k in (n, n + 1, cap, cap, cap, 4)]
    L.h2o_page_tables(_i32(before), _i32(new), _i32(free), ps, out[0], *out[1:], stream or torch.cuda.current_stream())
    return [x.cpu().numpy() for x in out]


@pytest.mark.parametrize("n,ps,most_before,most_new,cap_more", [
    (1, 16, 0, 1, 0), (1, 128, 1000, 5000, 3), (3, 16, 40, 40, 1), (64, 32, 700, 1, 0), (300, 64, 100, 90, 77), (1025, 16, 33, 7, 0),
    (16384, 16, 30, 3, 5),
])
def test_tables(n, ps, most_before, most_new, cap_more):
    g = np.random.default_rng(n)
    before, new = g.integers(0, most_before + 1, n), g.integers(0, most_new + 1, n)
    width = int(-(-(before + new).max() // ps)) + 2
    table = np.full((n, max(1, width)), -3, np.int32)
    ids = g.permutation(n * width + 5).astype(np.int32)
    at = 0
    for i, b in enumerate(before):
        k = -(-int(b) // ps)
        table[i, :k] = ids[at:at + k]
        at += k
    for got, want in zip(_tables(before, new, ids[at:], ps, table, int(new.sum()) + cap_more),
                         _tables_ref(before.tolist(), new.tolist(), ids[at:], ps, table, int(new.sum()) + cap_more)):
        np.testing.assert_array_equal(got, np.asarray(want, np.int32))


@pytest.mark.parametrize("change,bit", [("none", 0), ("count", 1), ("before", 1), ("rows", 2), ("pages", 4), ("width", 8), ("huge", 14)])
def test_tables_takes_all_or_nothing(change, bit):
    ps, before, new = 16, [20, 0, 31, 16], [5, 17, 2, 0]
    table = np.arange(100, 120, dtype=np.int32).reshape(4, 5)
    free, cap = np.arange(50, 53, dtype=np.int32), 24         # takes 3 pages, 24 rows
    if change == "count":
        new[1] = -1
    elif change == "before":
        before[2] = -31
    elif change == "rows":
        cap = 23
    elif change == "pages":
        free = free[:2]
    elif change == "width":
        new[0], free, cap = 61, np.arange(50, 70, dtype=np.int32), 100
    elif change == "huge":
        new[0], before[0], free, cap = 2 ** 31 - 1, 2 ** 31 - 1, np.arange(50, 70, dtype=np.int32), 100
    want = _tables_ref(before, new, free, ps, table, cap)
    assert want[-1][3] == bit
    for got, w in zip(_tables(before, new, free, ps, table, cap), want):
        np.testing.assert_array_equal(got, np.asarray(w, np.int32))


def test_tables_entry_that_is_no_page_gives_no_slot():
    table = np.array([[-4, -1, -1]], np.int32)
    out = _tables([3], [30], [1 << 30, 5], 16, table, 30)
    np.testing.assert_array_equal(out[5], [-1] * 29 + [5 * 16])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,d,ps,before,new", [
    (1, 64, 16, [0], [1]), (3, 128, 16, [15, 0, 16, 31, 5], [1, 16, 1, 40, 0]), (8, 128, 64, [10, 63], [500, 1]),
    (2, 64, 128, [127, 1, 100], [1, 300, 27]), (5, 64, 32, [0] * 33, [1] * 33),
])
def test_write(dtype, heads, d, ps, before, new):
    n = [b + t for b, t in zip(before, new)]
    c = Cache([max(1, x) for x in n], heads, d, ps, dtype, seed=d)
    slots = [c.table[i, x // ps] * ps + x % ps for i in range(len(n)) for x in range(before[i], n[i])]
    rows = len(slots)
    g = torch.Generator().manual_seed(1)
    fused = torch.randn(rows, 3 * heads, d, generator=g).to(dtype)    # k and v are slices of one projection
    fused[0, heads, 3] = float("nan")
    fused[-1, heads, 0] = float("inf")
    bounds = torch.full((c.K.shape[0], heads, 2, d), 5.0).to(dtype)
    K, V, B = c.K.clone(), c.V.clone(), bounds.clone()
    for r, s in enumerate(slots):
        K[s // ps, :, s % ps], V[s // ps, :, s % ps] = fused[r, heads:2 * heads], fused[r, 2 * heads:]
    for s in slots:
        if s % ps == ps - 1:
            B[s // ps] = torch.stack([K[s // ps].amin(1), K[s // ps].amax(1)], 1)
    # padding rows and slots outside the pool write nothing
    pad = torch.zeros(4, 3 * heads, d).to(dtype)
    f = torch.cat([fused, pad]).cuda()
    gk, gv, gb = c.K.cuda(), c.V.cuda(), bounds.cuda()
    L.h2o_page_write(f[:, heads:2 * heads], f[:, 2 * heads:], _i32(slots + [-1, -2 ** 31, c.K.shape[0] * ps, 2 ** 31 - 1]), gk, gv, gb,
                     torch.cuda.current_stream())
    for got, want in ((gk, K), (gv, V), (gb, B)):
        torch.testing.assert_close(got.cpu(), want, rtol=0, atol=0, equal_nan=True)


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_batch_is_served(dtype):
    """Prompts behind a common prefix, then decode steps with a request that has
    drafts taken back: tables, writes and both attentions, from nothing but the
    calls' own results, against attention over the tokens themselves."""
    heads, G, d, ps, plen, n = 2, 4, 64, 16, 75, 5
    g = torch.Generator().manual_seed(11)
    pages, width = 64, 8
    K, V = (torch.full((pages, heads, ps, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    bounds = torch.full((pages, heads, 2, d), float("nan"), dtype=dtype, device="cuda")
    free = torch.randperm(pages, generator=g).to(torch.int32).cuda()
    stream = torch.cuda.current_stream()
    scale = d ** -0.5

    def step(table, before, new, k, v, cap):
        nonlocal free
        m = before.shape[0]
        out = [torch.empty(x, dtype=torch.int32, device="cuda") for x in (m, m + 1, cap, cap, cap, 4)]
        L.h2o_page_tables(before, new, free, ps, table, *out, stream)
        after, _, seq, pos, slot, status = out
        L.h2o_page_write(k, v, slot, K, V, bounds, stream)
        rows, taken, _, err = status.tolist()
        assert err == 0 and rows == int(new.sum())
        free = free[taken:]                                   # no copy: int arrays start anywhere
        return after, seq, pos

    rand = lambda t: torch.randn(t, heads, d, generator=g).to(dtype)   # noqa: E731
    pk, pv = rand(plen), rand(plen)
    ptable = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    step(ptable, _i32([0]), _i32([plen]), pk.cuda(), pv.cuda(), plen)
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    length = _i32([0] * n)
    ref_k, ref_v = ([pk.new_zeros(0, heads, d) for _ in range(n)] for _ in range(2))   # the tokens of each request
    for t, new in enumerate([[30, 1, 16, 0, 47], [1, 4, 1, 1, 1], [1, 2, 1, 1, 1], [15, 1, 1, 20, 1]]):
        if t == 2:                                            # three of request 1's drafts are rejected
            length = length - _i32([0, 3, 0, 0, 0])
            ref_k[1], ref_v[1] = ref_k[1][:-3], ref_v[1][:-3]
        cap = sum(new) + 3                                    # padded, as a captured step would be
        k, v = rand(cap), rand(cap)
        length, seq, pos = step(table, length, _i32(new), k.cuda(), v.cuda(), cap)
        at = 0
        for i, x in enumerate(new):
            ref_k[i], ref_v[i] = torch.cat([ref_k[i], k[at:at + x]]), torch.cat([ref_v[i], v[at:at + x]])
            at += x
        assert length.tolist() == [x.shape[0] for x in ref_k]
        q = torch.randn(cap, heads * G, d, generator=g).to(dtype)
        out = torch.zeros(cap, heads * G, d, dtype=dtype, device="cuda")
        work = torch.empty(L.h2o_prefix_work_bytes(cap, heads, G, d, plen, L._CODES[str(dtype)]), dtype=torch.uint8, device="cuda")
        L.h2o_prefix_attend(q.cuda(), seq, pos, K, V, ptable[0], plen, table, scale, out, work, stream)
        sparse = torch.zeros_like(out)
        picked = torch.empty(cap, heads, 3, dtype=torch.int32, device="cuda")
        L.h2o_page_attend(q.cuda(), seq, pos, K, V, bounds, table, 3, 1, scale, sparse, picked, stream)
        for r in range(sum(new)):
            i, p = int(seq[r]), int(pos[r])
            for h in range(heads):
                qh = q[r, h * G:(h + 1) * G].double()
                mk, mv = (x[i][:p + 1, h].double() for x in (ref_k, ref_v))
                a = _attention(qh, torch.cat([pk[:, h].double(), mk]), torch.cat([pv[:, h].double(), mv]), scale)
                _check(out[r, h * G:(h + 1) * G], (a[0], _tolerance(dtype, d, plen + p + 1, *a)), "step %d row %d" % (t, r))
                npg = p // ps + 1
                full = [torch.stack([mk[x * ps:x * ps + ps].amin(0), mk[x * ps:x * ps + ps].amax(0)]) for x in range(npg)]
                b = torch.stack(full)[:, None]
                want = _picks(qh, b, np.arange(npg), 0, 3, 1)
                assert [x for x in picked[r, h].tolist() if x >= 0] == want.tolist()
                keep = torch.as_tensor([x * ps + o for x in want for o in range(ps) if x * ps + o <= p])
                a = _attention(qh, mk[keep], mv[keep], scale)
                _check(sparse[r, h * G:(h + 1) * G], (a[0], _tolerance(dtype, d, len(keep), *a)), "sparse step %d row %d" % (t, r))
        assert (out[sum(new):] == 0).all() and (sparse[sum(new):] == 0).all()


def test_strided_rows_and_another_stream():
    c = Cache([300, 200, 500], 2, 128, 32, BF16, seed=3)
    fused = _queries(4, 3 * 8, 128, BF16, 2)
    seq, pos = [0, 1, 1, 0], [299, 150, 199, 17]
    q = fused[:, 8:16]
    side = torch.cuda.Stream()
    hold = torch.full((4, 2 * 8, 128), 3.0, dtype=BF16, device="cuda")
    fq = fused.cuda()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _sparse(c, fq[:, 8:16], seq, pos, 4, 1, 0.1, out=hold[:, 8:], stream=side)
    side.synchronize()
    _check(hold[:, 8:], _sparse_ref(c, q, seq, pos, 4, 1, 0.1)[0], "sparse")
    with torch.cuda.stream(side):
        _prefix(c, fq[:, 8:16], seq, pos, c.table[2], 490, 0.1, out=hold[:, 8:], stream=side)
    side.synchronize()
    _check(hold[:, 8:], _prefix_ref(c, q, seq, pos, c.table[2], 490, 0.1), "prefix")
    assert (hold[:, :8] == 3).all()


def test_outputs_in_the_place_of_queries():
    c = Cache([300, 200, 500], 2, 128, 32, BF16, seed=3)
    seq, pos = [0, 1, 1, 0], [299, 150, 199, 17]
    q = _queries(4, 8, 128, BF16, 2)
    a, b = q.cuda(), q.cuda()
    _sparse(c, a, seq, pos, 4, 1, 0.1, out=a)
    _prefix(c, b, seq, pos, c.table[2], 490, 0.1, out=b)
    assert torch.equal(a, _sparse(c, q.cuda(), seq, pos, 4, 1, 0.1)[0])
    assert torch.equal(b, _prefix(c, q.cuda(), seq, pos, c.table[2], 490, 0.1))


def test_calls_on_two_streams_at_once():
    c = Cache([3000, 2000, 5000], 2, 128, 32, BF16, seed=6)
    K, V, B, table = c.K.cuda(), c.V.cuda(), c.bounds().cuda(), _i32(c.table)
    seq, pos = _i32([0, 1, 1, 0] * 8), _i32([2999, 1500, 1999, 170] * 8)
    q = _queries(32, 8, 128, BF16, 2).cuda()
    n = L.h2o_prefix_work_bytes(32, 2, 4, 128, 4900, L.H2O_BF16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    bufs = [(torch.empty_like(q), torch.empty_like(q), torch.empty(n, dtype=torch.uint8, device="cuda")) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, (a, b, w) in zip(streams, bufs):
            L.h2o_page_attend(q, seq, pos, K, V, B, table, 9, 2, 0.1, a, None, st)
            L.h2o_prefix_attend(q, seq, pos, K, V, table[2], 4900, table, 0.1, b, w, st)
    torch.cuda.synchronize()
    assert torch.equal(bufs[0][0], bufs[1][0]) and torch.equal(bufs[0][1], bufs[1][1])
    want = _sparse_ref(c, q[:4].cpu(), [0, 1, 1, 0], [2999, 1500, 1999, 170], 9, 2, 0.1)[0]
    _check(bufs[0][0][:4], want, "sparse")
    _check(bufs[0][1][:4], _prefix_ref(c, q[:4].cpu(), [0, 1, 1, 0], [2999, 1500, 1999, 170], c.table[2], 4900, 0.1), "prefix")


@pytest.mark.parametrize("dtype,pages", [(BF16, 40000), (F32, 36000)])
def test_offsets_beyond_32_bits(dtype, pages):
    """The pool holds more than 2^31 elements, the request its last pages: the
    bits are those of a small pool with the same pages."""
    heads, ps, d, n = 8, 64, 128, 11
    assert pages * heads * ps * d > 2 ** 31
    K, V = (torch.empty(pages, heads, ps, d, dtype=dtype, device="cuda") for _ in range(2))
    B = torch.empty(pages, heads, 2, d, dtype=dtype, device="cuda")
    k, v, q = (_queries(n * ps, h, d, dtype, i).cuda() for i, h in enumerate((heads, heads, 16)))
    stream = torch.cuda.current_stream()
    got = []
    for first, (pk, pv, pb) in ((pages - n, (K, V, B)), (0, tuple(torch.empty(n, *x.shape[1:], dtype=dtype, device="cuda") for x in (K, V, B)))):
        slot = torch.arange(first * ps, (first + n) * ps, dtype=torch.int32, device="cuda")
        L.h2o_page_write(k, v, slot, pk, pv, pb, stream)
        table = torch.arange(first, first + n, dtype=torch.int32, device="cuda")[None]
        seq, pos = _i32([0] * 5), _i32([n * ps - 1, 400, 64, 63, 0])
        a, b = torch.empty_like(q[:5]), torch.empty_like(q[:5])
        picked = torch.empty(5, heads, 3, dtype=torch.int32, device="cuda")
        L.h2o_page_attend(q[:5], seq, pos, pk, pv, pb, table, 3, 1, 0.1, a, picked, stream)
        w = torch.empty(L.h2o_prefix_work_bytes(5, heads, 2, d, 600, L._CODES[str(dtype)]), dtype=torch.uint8, device="cuda")
        L.h2o_prefix_attend(q[:5], seq, pos, pk, pv, table[0], 600, table, 0.1, b, w, stream)
        got.append((pk[first:first + n].clone(), pb[first:first + n].clone(), a, picked, b))
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_captured_steps_read_what_their_buffers_hold_then():
    """Tables, write and both attentions in one graph, replayed with other
    lengths and rows: results follow the buffers, and a second replay gives the
    same bits."""
    c = Cache([100, 40, 64], 2, 64, 16, BF16, seed=9, extra=8)
    K, V, bounds, table = c.K.cuda(), c.V.cuda(), c.bounds().cuda(), _i32(np.pad(c.table, ((0, 0), (0, 2)), constant_values=-1))
    before, new, free = _i32([99, 39, 63]), _i32([1, 1, 1]), _i32(c.spare)
    cap, plen = 8, 50
    after, start, seq, pos, slot, status = (torch.zeros(x, dtype=torch.int32, device="cuda") for x in (3, 4, cap, cap, cap, 4))
    k, v, q = (torch.randn(cap, h, 64, device="cuda").to(BF16) for h in (2, 2, 8))
    sparse, full = (torch.zeros(cap, 8, 64, dtype=BF16, device="cuda") for _ in range(2))
    work = torch.empty(L.h2o_prefix_work_bytes(cap, 2, 4, 64, plen, L.H2O_BF16), dtype=torch.uint8, device="cuda")
    ptable = table[0].clone()

    def step():
        s = torch.cuda.current_stream()
        L.h2o_page_tables(before, new, free, 16, table, after, start, seq, pos, slot, status, s)
        L.h2o_page_write(k, v, slot, K, V, bounds, s)
        L.h2o_page_attend(q, seq, pos, K, V, bounds, table, 4, 2, 0.125, sparse, None, s)
        L.h2o_prefix_attend(q, seq, pos, K, V, ptable, plen, table, 0.125, full, work, s)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for b, t in (([99, 39, 63], [1, 1, 1]), ([100, 40, 64], [1, 3, 2]), ([101, 43, 66], [0, 5, 3])):
        before.copy_(_i32(b))
        new.copy_(_i32(t))
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        got = sparse.clone(), full.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], sparse) and torch.equal(got[1], full)
        now = Cache([1], 2, 64, 16, BF16)
        now.K, now.V, now.table = K.cpu(), V.cpu(), table.cpu().numpy()
        n = sum(t)
        sq, ps = seq[:n].tolist(), pos[:n].tolist()
        _check(sparse[:n], _sparse_ref(now, q[:n].cpu(), sq, ps, 4, 2, 0.125)[0], "sparse")
        _check(full[:n], _prefix_ref(now, q[:n].cpu(), sq, ps, ptable.cpu().numpy(), plen, 0.125), "prefix")


def test_injected_launch_failure(monkeypatch):
    c = Cache([20], 1, 64, 16, F32)
    q = _queries(1, 1, 64, F32, 0).cuda()
    monkeypatch.setenv("H2O_FAULT", "launch")
    with pytest.raises(L.H2OError) as e:
        _sparse(c, q, [0], [19], 2, 1, 0.1)
    assert e.value.code == L.H2O_ERR_CUDA
    with pytest.raises(L.H2OError):
        _prefix(c, q, [0], [19], [], 0, 0.1)
    monkeypatch.delenv("H2O_FAULT")
    assert _sparse(c, q, [0], [19], 2, 1, 0.1)[0].isfinite().all()


@pytest.mark.parametrize("d", [64, 128])
def test_prefix_tiles_that_arrive_out_of_order(d):
    # one tile of query rows over key tiles by turns on the same few pages, which the L2 cache holds, and on pages far
    # apart, which it does not: a tile may be there before the one that was asked for earlier
    heads, ps, pages, tiles, rows, scale = 40, 32, 6000, 40, 3, d ** -0.5
    plen = tiles * 128 - 43
    g = torch.Generator(device="cuda").manual_seed(d)
    K, V = (torch.randn(pages, heads, ps, d, dtype=BF16, device="cuda", generator=g) for _ in range(2))
    far = torch.randperm(pages - 4, device="cuda", generator=g)[:tiles // 2 * 4].view(-1, 4) + 4
    ptable = torch.stack([torch.arange(4, device="cuda").expand_as(far), far], 1).reshape(-1).to(torch.int32)
    q = torch.randn(rows, heads, d, dtype=BF16, device="cuda", generator=g)
    seq, pos, table = _i32([0] * rows), _i32([-1] * rows), _i32([[0]])
    work = torch.empty(L.h2o_prefix_work_bytes(rows, heads, 1, d, plen, L.H2O_BF16), dtype=torch.uint8, device="cuda")
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(20):
        out = torch.zeros_like(q)
        flush.zero_()
        L.h2o_prefix_attend(q, seq, pos, K, V, ptable, plen, table, scale, out, work, torch.cuda.current_stream())
        first = out if first is None else first
        assert torch.equal(out, first)
    at = ptable.long()
    for h in range(heads):
        k, v = (x[at, h].reshape(-1, d)[:plen].double() for x in (K, V))
        a = _attention(q[:, h].double(), k, v, scale)
        _check(out[:, h], (a[0].cpu(), _tolerance(BF16, d, plen, *a).cpu()), "head %d" % h)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [3, 130])                  # one and two tiles of 128 query rows
def test_prefix_maximum_raised_by_every_part_of_a_tile(rows, d):
    # logits grow by 2^9 every 64 keys, and values shrink by as much, so that each of the last 13 parts has an equal share
    heads, ps, parts, scale = 40, 32, 79, 0.125
    plen = parts * 64 - 21
    g = torch.Generator().manual_seed(d + rows)
    c = Cache([1, plen], heads, d, ps, BF16, seed=d)
    part = torch.arange(plen) // 64
    k, v = (0.3 * torch.randn(plen, heads, d, generator=g) for _ in range(2))
    k[..., 0] = 8.0 * part[:, None]
    v = v * torch.exp2(9.0 * (parts - 1 - part).clamp(max=12))[:, None, None]
    q = 0.3 * torch.randn(rows, heads, d, generator=g)
    q[..., 0] = 6.25                                         # 6.25 * 8 * scale * log2(e) = 9.02
    slot = _i32([int(c.table[1, t // ps]) * ps + t % ps for t in range(plen)])
    K, V = c.K.cuda(), c.V.cuda()
    L.h2o_page_write(k.to(BF16).cuda(), v.to(BF16).cuda(), slot, K, V, torch.empty(K.shape[0], heads, 2, d, dtype=BF16, device="cuda"),
                     torch.cuda.current_stream())
    c.K, c.V = K.cpu(), V.cpu()
    q = q.to(BF16)
    out = _prefix(c, q.cuda(), [0] * rows, [-1] * rows, c.table[1], plen, scale)
    for h in range(heads):
        kk, vv = c.rows(c.table[1], h, plen)
        a = _attention(q[:, h].double().cuda(), kk.cuda(), vv.cuda(), scale)
        _check(out[:, h], (a[0].cpu(), _tolerance(BF16, d, plen, *a).cpu()), "head %d" % h)


def test_tables_of_any_size_in_a_fresh_process():
    # what a kernel may use of shared memory is set once a process: sizes about 48 KB, none larger before them
    import os
    import subprocess
    import sys
    code = """
import torch
from kv_cache_eviction_h2o_gb300 import binding as L
for n in (4035, 4039, 4040, 4092, 4095):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    seq, pos, slot, status = i32(n), i32(n), i32(n), i32(4)
    L.h2o_page_tables(i32(n) + 7, i32(n) + 1, i32(0), 16, torch.arange(n, dtype=torch.int32, device="cuda")[:, None], i32(n),
                      i32(n + 1), seq, pos, slot, status, torch.cuda.current_stream())
    assert status.tolist() == [n, 0, 8, 0]
    assert (slot == 16 * torch.arange(n, device="cuda") + 7).all() and (pos == 7).all()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,d,ps,pages", [(1, 64, 16, 1), (3, 128, 16, 40), (8, 128, 64, 60), (2, 64, 128, 30), (5, 128, 32, 9)])
def test_write_leaves_slots_out(dtype, heads, d, ps, pages):
    # rows of a page in the order of their slots, some of which keep what they held
    g = np.random.default_rng(ps + pages)
    c = Cache([ps * pages], heads, d, ps, dtype, seed=d)
    bounds = torch.full((pages + 3, heads, 2, d), 5.0).to(dtype)
    K, V, B = c.K.clone(), c.V.clone(), bounds.clone()
    slots = []
    for i, p in enumerate(c.table[0]):
        n = int(g.integers(1, ps + 1))
        at = [12, 14, 15] if i == 0 and ps == 16 else sorted(g.choice(ps, n, replace=False))
        if i % 4 != 3 and at[-1] != ps - 1:
            at[-1] = ps - 1
        slots += [int(p) * ps + int(x) for x in at]
    k, v = (torch.randn(len(slots), heads, d, generator=torch.Generator().manual_seed(i)).to(dtype) * 3 for i in (1, 2))
    for r, s in enumerate(slots):
        K[s // ps, :, s % ps], V[s // ps, :, s % ps] = k[r], v[r]
    for s in slots:
        if s % ps == ps - 1:
            B[s // ps] = torch.stack([K[s // ps].amin(1), K[s // ps].amax(1)], 1)
    gk, gv, gb = c.K.cuda(), c.V.cuda(), bounds.cuda()
    L.h2o_page_write(k.cuda(), v.cuda(), _i32(slots), gk, gv, gb, torch.cuda.current_stream())
    for got, want in ((gk, K), (gv, V), (gb, B)):
        torch.testing.assert_close(got.cpu(), want, rtol=0, atol=0, equal_nan=True)


def test_calls_without_a_stream_are_captured():
    # on the current stream, which a capture wants them on
    c = Cache([100, 60], 2, 64, 16, BF16, seed=4, extra=4)
    K, V, B, table = c.K.cuda(), c.V.cuda(), c.bounds().cuda(), _i32(np.pad(c.table, ((0, 0), (0, 1)), constant_values=-1))
    before, new, free = _i32([99, 59]), _i32([1, 1]), _i32(c.spare)
    after, start, seq, pos, slot, status = (torch.zeros(x, dtype=torch.int32, device="cuda") for x in (2, 3, 2, 2, 2, 4))
    k, v, q = (_queries(2, h, 64, BF16, i).cuda() for i, h in enumerate((2, 2, 8)))
    sparse, full = torch.zeros_like(q), torch.zeros_like(q)
    work = torch.empty(L.h2o_prefix_work_bytes(2, 2, 4, 64, 40, L.H2O_BF16), dtype=torch.uint8, device="cuda")
    ptable = table[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.h2o_page_tables(before, new, free, 16, table, after, start, seq, pos, slot, status)
        L.h2o_page_write(k, v, slot, K, V, B)
        L.h2o_page_attend(q, seq, pos, K, V, B, table, 4, 2, 0.125, sparse)
        L.h2o_prefix_attend(q, seq, pos, K, V, ptable, 40, table, 0.125, full, work)
    graph.replay()
    torch.cuda.synchronize()
    c.K, c.V, c.table = K.cpu(), V.cpu(), table.cpu().numpy()
    assert status.tolist() == [2, 0, 100, 0]
    _check(sparse, _sparse_ref(c, q.cpu(), [0, 1], [99, 59], 4, 2, 0.125)[0], "sparse")
    _check(full, _prefix_ref(c, q.cpu(), [0, 1], [99, 59], c.table[0], 40, 0.125), "prefix")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,ps,low", [(64, 16, 2.0 ** -50), (128, 32, 2.0 ** -52), (128, 16, 2.0 ** -50)])
def test_sparse_ranks_by_all_bits_of_fp64(dtype, d, ps, low):
    # two pages whose scores are sums of four queries each and differ in one of fp64's last bits; the better one comes second
    c = Cache([4 * ps], 1, d, ps, dtype, seed=2)
    pages = torch.as_tensor(c.table[0]).long()
    c.K[pages] = 0.0
    c.K[pages[0], :, :, 7] = 1.0
    c.K[pages[1], :, :, 9] = 1.0
    q = torch.zeros(1, 4, d, dtype=dtype)
    q[0, :, 7] = torch.tensor([1.0, 2.0 ** -25, 2.0 ** -48, 0.0])
    q[0, :, 9] = torch.tensor([1.0, 2.0 ** -25, 2.0 ** -48, low])
    want, picked = _sparse_ref(c, q, [0], [4 * ps - 1], 2, 1, 0.125)
    assert picked[0, 0].tolist() == [1, 3]
    out, got = _sparse(c, q.cuda(), [0], [4 * ps - 1], 2, 1, 0.125)
    np.testing.assert_array_equal(got.cpu().numpy(), picked)
    _check(out, want, "picked")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_rows_without_weight_are_zero_whatever_the_values(dtype, value):
    c = Cache([60, 300], 2, 64, 16, dtype, seed=3)
    c.K[:], c.V[:] = float("-inf"), value
    q = _queries(3, 8, 64, dtype, 1).abs() + 0.5
    out, _ = _sparse(c, q.cuda(), [0, 1, 1], [59, 299, 17], 3, 1, 0.125)
    assert (out == 0).all()
    assert (_prefix(c, q.cuda(), [0, 0, 0], [59, -1, 5], c.table[1], 290, 0.125) == 0).all()
    assert (_prefix(c, q.cuda(), [0, 1, 1], [59, 299, 17], [], 0, 0.125) == 0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("groups", [3, 16])
def test_weights_of_own_pages_keep_two_parts(d, groups):
    # Attention to own pages multiplies each softmax weight in two bf16 parts, off by 2^-16 of it, so that an output is off by
    # its own rounding, and by those 2^-16 and the fp32 terms above (twice the products: 4 n) of sum p|v|.  With small keys and
    # some hundred tokens these are far below what weights of one part leave.
    c = Cache([150, 90, 33], 2, d, 32, BF16, seed=7, kscale=0.1)
    seq, pos = [0, 1, 2, 0], [149, 89, 32, 101]
    q = _queries(4, 2 * groups, d, BF16, 5)
    b, scale, one_part_fails = c.bounds(), d ** -0.5, False
    for budget in (c.width, 3, 0):
        if budget:
            out, _ = _sparse(c, q.cuda(), seq, pos, budget, 1, scale)
        else:
            out = _prefix(c, q.cuda(), seq, pos, [], 0, scale)
        for r in range(4):
            mine = c.table[seq[r], :pos[r] // 32 + 1]
            for h in range(2):
                qh = q[r, h * groups:(h + 1) * groups].double()
                at = _picks(qh, b, mine, h, budget or c.width, 1)
                n = (len(at) - 1) * 32 + pos[r] % 32 + 1
                k, v = c.rows(mine[at], h, n)
                y, av, zmax, smax = _attention(qh, k, v, scale)
                tol = (U24 * (2 * ((d + 8) * smax + 4 * zmax) + 4 * n + 64) + 2.0 ** -16) * av * (1 + 2.0 ** -7) + (2.0 ** -8 + U24) * y.abs()
                _check(out[r, h * groups:(h + 1) * groups], (y, tol), "budget %d row %d" % (budget, r))
                z = (qh @ k.T) * scale
                e = torch.exp(z - z.amax(1, keepdim=True))
                rough = ((e.to(BF16).double() @ v) / e.sum(1, keepdim=True)).to(BF16).double()
                one_part_fails |= bool(((rough - y).abs() > tol).any())
    assert one_part_fails, "the bound tells one part from two"


@pytest.mark.parametrize("d,groups", [(64, 1), (128, 4), (128, 16)])
def test_sparse_with_many_units_of_few_tiles(d, groups):
    # a decode batch: more units than two-warp CTAs fit, each of which picks
    g = np.random.default_rng(d)
    lengths = [int(x) for x in g.integers(1, 700, 90)]
    c = Cache(lengths, 8, d, 16, BF16, seed=d + groups)
    seq, pos = list(range(90)), [n - 1 for n in lengths]
    q = _queries(90, 8 * groups, d, BF16, 3)
    for budget, recent in ((7, 2), (20, 20)):
        want, picked = _sparse_ref(c, q, seq, pos, budget, recent, d ** -0.5)
        out, got = _sparse(c, q.cuda(), seq, pos, budget, recent, d ** -0.5)
        np.testing.assert_array_equal(got.cpu().numpy(), picked)
        _check(out, want, "budget %d" % budget)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", [300, 4096, 16384])
def test_tables_much_wider_than_the_requests(dtype, width):
    lengths = [1, 40, 16 * 9, 16 * 21 + 5]
    c = Cache(lengths, 2, 128, 16, dtype, seed=1, width=width)
    seq, pos = [0, 1, 2, 3, 3], [0, 39, 16 * 9 - 1, 16 * 21 + 4, 100]
    q = _queries(5, 6, 128, dtype, 2)
    for budget, recent in ((4, 1), (19, 3)):
        want, picked = _sparse_ref(c, q, seq, pos, budget, recent, 0.09)
        out, got = _sparse(c, q.cuda(), seq, pos, budget, recent, 0.09)
        np.testing.assert_array_equal(got.cpu().numpy(), picked)
        _check(out, want, "budget %d" % budget)
    for plen in (0, 140):
        _check(_prefix(c, q.cuda(), seq, pos, c.table[2], plen, 0.09), _prefix_ref(c, q, seq, pos, c.table[2], plen, 0.09), "prefix %d" % plen)


@pytest.mark.parametrize("dtype,d,groups", [(BF16, 128, 4), (BF16, 64, 1), (F32, 64, 2)])
def test_one_long_request_among_short_ones(dtype, d, groups):
    g = np.random.default_rng(d)
    lengths = [int(x) for x in g.integers(1, 90, 40)]
    lengths[17] = 20011
    c = Cache(lengths, 4, d, 32, dtype, seed=d)
    seq, pos = list(range(40)), [n - 1 for n in lengths]
    q = _queries(40, 4 * groups, d, dtype, 2)
    for budget, recent in ((30, 4), (500, 1)):
        want, picked = _sparse_ref(c, q, seq, pos, budget, recent, d ** -0.5)
        out, got = _sparse(c, q.cuda(), seq, pos, budget, recent, d ** -0.5)
        np.testing.assert_array_equal(got.cpu().numpy(), picked)
        _check(out, want, "budget %d" % budget)
    for plen in (0, 70):
        _check(_prefix(c, q.cuda(), seq, pos, c.table[17], plen, d ** -0.5), _prefix_ref(c, q, seq, pos, c.table[17], plen, d ** -0.5),
               "prefix %d" % plen)
