"""Rotary positions, prompt attention and quantised paged caches against their
formulas in 64 bits.

Bounds (U = 2^-24, an fp32 half step).
Rotary: the angle is off by 3 U times at most pi / 4 (its conversion, 2 pi 2^-32
in fp32, their product), sine and cosine by 3 U more (the last two steps of their
sums, what lies before them and the next term), by 2 U for the amplitude and its
product; with the two roundings of x cos - y sin: 10 U A (|a| + |b|).  bf16 then
by 2^-8 of the value.
Attention: a logit is a sum of D products, off by (D + 8) U scale sum |q||k| (the
sum, its scaling; twice that where a tensor core's sums drop what lies below
2^-23 of their largest term) and 4 U |z| (reading it in base 2, the
exponential), which moves each weight and the weights' sum by that relative
amount; sums of n weights or values in any order by n U, twice on a tensor core; joining parts by 64 U.
A weight rounded to bf16 is off by 2^-8, to fp16 by 2^-12 where it is not
among the smallest (the row's largest is 2^6 or more, fp16's steps 2^-24 at
least: 2^-31 of the largest weight times its value).  bf16 outputs by 2^-8 of themselves.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from kv_cache_eviction_h2o_gb300 import binding as L   # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def _inside(got, y, tol, what=""):
    got = got.double().cpu()
    assert torch.equal(got.isnan(), y.isnan()), what
    assert torch.equal(got.isinf(), y.isinf()), what
    fine = y.isfinite()
    off = ((got - y).abs() - tol)[fine]
    assert off.numel() == 0 or off.max() <= 0, "%s: %g beyond its bound" % (what, off.max())


# -------------------------------------------------------------- rotary positions

def _rope_ref(x, pos, table, form, amp):
    """y and its bound for x [rows][heads][d]."""
    n = len(table)
    turn = np.array([[((p * int(t)) % 2 ** 64) / 2.0 ** 64 for t in table] for p in pos])
    ang = torch.as_tensor(2 * math.pi * turn)[:, None]
    c, s = amp * torch.cos(ang), amp * torch.sin(ang)
    a, b = (slice(0, n), slice(n, 2 * n)) if form == L.H2O_ROPE_HALF else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    y, tol = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    xa, xb = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    size = 10 * U * abs(amp) * (xa.abs() + xb.abs())
    tol[..., a], tol[..., b] = size, size
    if x.dtype is BF16:
        tol[..., : 2 * n] += 2.0 ** -8 * (y[..., : 2 * n].abs() + tol[..., : 2 * n])
    return y, tol + 1e-37


ROPES = [(128, 128, 1), (64, 64, 1), (128, 64, 1), (128, 24, 1), (64, 12, 1), (64, 6, 1), (128, 2, 1), (128, 32, 4), (64, 16, 7)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("form", [L.H2O_ROPE_HALF, L.H2O_ROPE_PAIRS])
@pytest.mark.parametrize("d,rot,step", ROPES)
def test_rope(dtype, form, d, rot, step):
    rows, heads, kv = 37, 6, 3 * step
    g = _gen(rot)
    table = L.h2o_rope_table(rot)
    pos = torch.randint(0, 1 << 20, (rows,), generator=g).tolist()
    pos[:6] = [0, 1, -1, 2 ** 31 - 1, 7, -5]
    q, k = torch.randn(rows, heads, d, generator=g).to(dtype), torch.randn(rows, kv, d, generator=g).to(dtype)
    qo, ko = torch.full((rows, heads, d), 7.0, dtype=dtype, device="cuda"), torch.full((rows, kv, d), 7.0, dtype=dtype, device="cuda")
    L.h2o_rope(q.cuda(), k.cuda(), _i32(pos), torch.as_tensor(table).cuda(), form, 1.25, qo, ko)
    live = [i for i in range(rows) if pos[i] >= 0]
    for x, got in ((q, qo), (k, ko)):
        y, tol = _rope_ref(x[live], [pos[i] for i in live], table, form, 1.25)
        _inside(got[live], y, tol)
        assert torch.equal(got[live][..., rot:].cpu(), x[live][..., rot:])
        assert (got[[2, 5]] == 7).all()                    # padding rows
    # turning back gives what there was; in place, in rows of a wider buffer
    wide = torch.zeros(rows, heads + kv + 1, d, dtype=dtype, device="cuda")
    wide[:, :heads], wide[:, heads:heads + kv], wide[:, -1] = q.cuda(), k.cuda(), 3.0
    qs, ks = wide[:, :heads], wide[:, heads:heads + kv]
    L.h2o_rope(qs, ks, _i32(pos), torch.as_tensor(table).cuda(), form, 1.25, qs, ks)
    assert torch.equal(qs[live], qo[live]) and torch.equal(ks[live], ko[live])
    assert torch.equal(qs[[2, 5]].cpu(), q[[2, 5]]) and (wide[:, -1] == 3).all()
    L.h2o_rope(qs, ks, _i32(pos), torch.as_tensor(-table).cuda(), form, 0.8, qs, ks)
    for x, got in ((q, qs), (k, ks)):
        z = x.double()
        # both turns' own errors, and what the first's rounding is after the second
        most = z.abs().amax(-1, keepdim=True)
        _inside(got, z, 60 * U * most + (2.0 ** -8 * 4.1 * most if dtype is BF16 else 0))


def test_rope_queries_alone_and_special_values():
    q = torch.randn(5, 2, 64, generator=_gen(1)).cuda()
    q[0, 0, 40], q[1, 1, 3], q[2, 0, 17] = float("nan"), float("inf"), float("-inf")
    table = torch.as_tensor(L.h2o_rope_table(32)).cuda()
    for form in (L.H2O_ROPE_HALF, L.H2O_ROPE_PAIRS):
        out = torch.empty_like(q)
        L.h2o_rope(q, None, _i32([3, 4, 5, 6, 7]), table, form, 1.0, out, None)
        # a NaN among the channels that stay touches no other
        assert out[0, 0, 40].isnan() and out[0].isnan().sum() == 1
        assert out[1].isfinite().logical_not().sum() == 2 and out[2].isfinite().logical_not().sum() == 2
        assert torch.equal(out[..., 32:].nan_to_num(), q[..., 32:].nan_to_num())


def test_rope_gradient_is_the_turn_back():
    # d loss / d x for loss = sum(w rope(x)) is rope of w with the negated table; against differences of the operator itself
    g = _gen(4)
    rows, heads, d, rot, amp = 4, 2, 64, 32, 1.5
    x, w = torch.randn(rows, heads, d, generator=g).cuda(), torch.randn(rows, heads, d, generator=g).cuda()
    pos, table = _i32([0, 5, 1000, 123456]), torch.as_tensor(L.h2o_rope_table(rot)).cuda()
    for form in (L.H2O_ROPE_HALF, L.H2O_ROPE_PAIRS):
        def f(z):
            out = torch.empty_like(z)
            L.h2o_rope(z, None, pos, table, form, amp, out, None)
            return out
        grad = torch.empty_like(w)
        L.h2o_rope(w, None, pos, -table, form, amp, grad, None)
        y, tol = _rope_ref(w.cpu(), [-p for p in pos.tolist()], table.tolist(), form, amp)
        _inside(grad, y, tol)
        for i in range(0, d, 7):
            step = torch.zeros_like(x)
            step[..., i] = 1.0                             # the operator is linear: a whole step is exact but for roundings
            diff = ((f(x + step) - f(x)).double() * w.double()).sum(-1)
            assert ((diff - grad[..., i].double()).abs() <= 400 * U * (w.abs().sum(-1) * (x.abs().amax() + 1)).double()).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rope_many_rows(dtype):
    rows, heads, kv, d = 5001, 32, 8, 128
    g = _gen(9)
    q, k = torch.randn(rows, heads, d, generator=g).to(dtype), torch.randn(rows, kv, d, generator=g).to(dtype)
    pos = torch.randint(0, 1 << 17, (rows,), generator=g)
    table = L.h2o_rope_table(128, kind=L.H2O_ROPE_PARTS, factor=8.0, original_len=4096.0, low=1.0, high=32.0)
    qo, ko = q.cuda(), k.cuda()
    L.h2o_rope(qo, ko, _i32(pos), torch.as_tensor(table).cuda(), L.H2O_ROPE_HALF, 1.0, qo, ko)
    at = torch.cat([torch.arange(0, rows, 97), torch.tensor([rows - 1])])
    for x, got in ((q, qo), (k, ko)):
        y, tol = _rope_ref(x[at], pos[at].tolist(), table, L.H2O_ROPE_HALF, 1.0)
        _inside(got[at.cuda()], y, tol)


# ------------------------------------------------------------- prompt attention

def _softmax_rows(q, k, v, scale, seen):
    """softmax(scale q.k) v over the first seen[x] keys of each row x of q, with sum p|v|, max |z| and scale max |q||k| of each, fp64."""
    n, d = q.shape
    y, av = torch.zeros(n, d, dtype=torch.float64, device=q.device), torch.zeros(n, d, dtype=torch.float64, device=q.device)
    seen = torch.as_tensor(seen, device=q.device)
    hide = torch.arange(k.shape[0], device=q.device) >= seen[:, None]
    if k.shape[0] == 0:
        return y, av, y[:, :1], y[:, :1]
    k0 = torch.where(hide.all(0)[:, None], 0.0, k)         # keys that nobody sees may hold anything
    v0 = torch.where(hide.all(0)[:, None], 0.0, v)
    z = ((q @ k0.T) * scale).masked_fill(hide, -math.inf)
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
    p = e / e.sum(1, keepdim=True)
    p = torch.where(e.sum(1, keepdim=True) == 0, 0.0, p)
    if v0.isfinite().all():
        y, av = p @ v0, p @ v0.abs()
    else:
        for x in range(n):
            m = int(seen[x])
            y[x], av[x] = p[x, :m] @ v0[:m], p[x, :m] @ v0[:m].abs()
    s = scale * (q.abs() @ k0.abs().T).masked_fill(hide, 0.0).amax(1, keepdim=True)
    return y, av, z.masked_fill(hide, 0.0).abs().amax(1, keepdim=True), s


def _bound(dtype, d, n, y, av, zmax, smax, half=2.0 ** -8):
    t = U * (2 * (2 * (d + 8) * smax + 4 * zmax) + 4 * n + 64) * av
    if dtype is BF16:
        t = t * (1 + 2.0 ** -7) + half * av + 2.0 ** -8 * (y.abs() + t + half * av)
    return t + U * y.abs() + 1e-30


def _prompt_ref(q, k, v, qs, ks, scale, half=2.0 ** -8):
    dtype, (rows, hq, d), heads = q.dtype, q.shape, k.shape[1]
    G = hq // heads
    y, tol = (torch.full(q.shape, 7.0, dtype=torch.float64) for _ in range(2))
    q, k, v = (x.cuda().double() for x in (q, k, v))
    for i in range(len(qs) - 1):
        nq, nk = qs[i + 1] - qs[i], ks[i + 1] - ks[i]
        if nq <= 0:
            continue
        seen = np.clip(nk - nq + np.arange(nq) + 1, 0, nk)
        for j in range(hq):
            a = _softmax_rows(q[qs[i]:qs[i + 1], j], k[ks[i]:ks[i + 1], j // G], v[ks[i]:ks[i + 1], j // G], scale, seen)
            y[qs[i]:qs[i + 1], j] = a[0].cpu()
            tol[qs[i]:qs[i + 1], j] = _bound(dtype, d, nk, *a, half).cpu()
    return y, tol


def _starts(lengths, first=0):
    return np.concatenate([[first], first + np.cumsum(lengths)]).astype(np.int32)


def _prompt(q, k, v, qs, ks, scale, out=None, stream=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
    L.h2o_prompt_attend(q.cuda(), k.cuda(), v.cuda(), _i32(qs), None if ks is None else _i32(ks), scale, out, stream)
    return out


def _packed(rows, keys, heads, G, d, dtype, seed, spread=1.0):
    g = _gen(seed)
    return (spread * torch.randn(rows, heads * G, d, generator=g)).to(dtype), torch.randn(keys, heads, d, generator=g).to(dtype), \
        torch.randn(keys, heads, d, generator=g).to(dtype)


HEADS = [(4, 1, 64), (2, 4, 128), (1, 16, 128), (2, 3, 64), (1, 5, 128), (2, 7, 64), (1, 8, 128), (1, 9, 64), (3, 1, 128), (1, 11, 128), (1, 13, 64),
         (1, 15, 64), (1, 2, 128), (1, 6, 64), (1, 10, 64), (1, 12, 128), (1, 14, 128)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,G,d", HEADS)
def test_prompt(dtype, heads, G, d):
    lengths = [1, 5, 130, 0, 64, 257, 2]
    rows = sum(lengths)
    q, k, v = _packed(rows, rows, heads, G, d, dtype, heads * G)
    qs = _starts(lengths)
    _inside(_prompt(q, k, v, qs, None, d ** -0.5), *_prompt_ref(q, k, v, qs, qs, d ** -0.5))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [127, 128, 129, 255, 256, 257, 383, 385, 511, 513, 640, 1025])
def test_prompt_lengths_about_a_tile(dtype, n):
    for heads, G, d in ((2, 1, 64), (1, 4, 128)):
        q, k, v = _packed(n, n, heads, G, d, dtype, n)
        _inside(_prompt(q, k, v, [0, n], [0, n], d ** -0.5), *_prompt_ref(q, k, v, [0, n], [0, n], d ** -0.5))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 7])
def test_prompt_behind_earlier_tokens(dtype, d, G):
    new = [1, 33, 7, 200, 1, 300, 128, 3]
    before = [0, 1000, 129, 57, 2000, 1, 128, 0]
    keys = [a + b for a, b in zip(new, before)]
    keys[-1] = 1                                           # 3 queries, 1 key: two rows see none
    q, k, v = _packed(sum(new) + 9, sum(keys) + 20, 2, G, d, dtype, G)
    qs, ks = _starts(new, 4), _starts(keys, 11)
    out = _prompt(q, k, v, qs, ks, d ** -0.5)
    y, tol = _prompt_ref(q, k, v, qs, ks, d ** -0.5)
    _inside(out, y, tol)
    assert (out[:4] == 7).all() and (out[qs[-1]:] == 7).all() and (out[qs[-1] - 3:qs[-1] - 1] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_does_not_see_what_is_masked(dtype):
    # NaN and infinities behind the last request, before the first, and in tokens that come after
    new, d = [70, 300, 150], 128
    for value in (float("nan"), float("inf"), -float("inf")):
        q, k, v = _packed(540, 560, 2, 2, d, dtype, 5)
        qs, ks = _starts(new, 2), _starts(new, 3)
        k[:3], v[:3], k[523:], v[523:], q[522:], q[:2] = (value,) * 6
        clean = _prompt_ref(q[2:522], k[3:523], v[3:523], _starts(new), _starts(new), d ** -0.5)
        out = _prompt(q, k, v, qs, ks, d ** -0.5)
        _inside(out[2:522], *clean)
        # from token 200 of the second request on
        v[3 + 70 + 200] = value
        out = _prompt(q, k, v, qs, ks, d ** -0.5)
        late = torch.zeros(520, dtype=torch.bool)
        late[70 + 200:70 + 300] = True
        _inside(out[2:522][~late], clean[0][~late], clean[1][~late])
        got = out[2:522][late]
        assert got.isnan().all() if value != value else (got == value).all()
        v[3 + 70 + 200] = 1.0
        k[3 + 70 + 200, :, 5] = value
        out = _prompt(q, k, v, qs, ks, d ** -0.5)
        _inside(out[2:522][~late], clean[0][~late], clean[1][~late])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("spread", [0.0, 30.0, 3000.0])
def test_prompt_flat_and_large_logits(dtype, spread):
    n, d = 600, 64
    q, k, v = _packed(n, n, 2, 2, d, dtype, 8, spread)
    k[::50] *= 4                                           # maxima that rise along the row
    _inside(_prompt(q, k, v, [0, n], None, 0.5), *_prompt_ref(q, k, v, [0, n], [0, n], 0.5))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_numbers_that_are_none_stay_in_their_channel(dtype):
    # NaN among a row's own values, and among those of its tile that it does not see
    n, d, heads, G = 700, 64, 2, 4
    q, k, v = _packed(n, n, heads, G, d, dtype, 12)
    y, tol = _prompt_ref(q, k, v, [0, n], [0, n], d ** -0.5)
    none = torch.zeros(n, heads, d, dtype=torch.bool)
    for token, h, c in ((3, 0, 5), (130, 0, 6), (131, 1, 0), (132, 1, 63), (500, 0, 5), (n - 1, 1, 30)):
        v[token, h, c] = float("nan")
        none[token:, h, c] = True
    none = none.repeat_interleave(G, 1)
    out = _prompt(q, k, v, [0, n], None, d ** -0.5)
    assert torch.equal(out.isnan().cpu(), none)
    _inside(out.cpu()[~none], y[~none], tol[~none])


def test_prompt_values_near_the_end_of_the_range():
    # weights are up to 2^8 before they are divided: 64 of 2^7.5 times 1e36 are no number, their mean is
    n, d = 128, 64
    q, k, v = _packed(n, n, 1, 1, d, BF16, 13)
    q[:], k[:], v = 0.0, 0.0, v * 1e36
    q[:, :, 0], k[64:, :, 0] = 1.0, 41.5
    _inside(_prompt(q, k, v, [0, n], None, 0.125), *_prompt_ref(q, k, v, [0, n], [0, n], 0.125))


def test_prompt_rows_made_again_for_longer_than_a_wait():
    # 256 queries behind 400000 keys without a number: two seconds of one CTA, whose next requests are as they should be
    n, few, d = 400_000, 400, 64
    g = _gen(14)
    q = torch.randn(256 + few, 1, d, generator=g).to(BF16)
    kv = torch.zeros(2, n + few, 1, d, dtype=BF16, device="cuda")
    kv[1, :n] = float("nan")
    v = torch.randn(few, 1, d, generator=g).to(BF16)
    kv[1, n:] = v.cuda()
    for first in (True, False):                            # (the long request before the others, or behind them)
        if not first:
            kv = torch.cat([kv[:, n:], kv[:, :n]], 1)
        out = _prompt(q, kv[0], kv[1], _starts([256] + [1] * few if first else [1] * few + [256]),
                      _starts([n] + [1] * few if first else [1] * few + [n]), 0.125).cpu()
        long, short = (out[:256], out[256:]) if first else (out[few:], out[:few])
        assert long.isnan().all() and torch.equal(short, v)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_rows_without_weight_are_zero(dtype):
    n, d = 140, 64
    q, k, v = _packed(n, n, 1, 1, d, dtype, 3)
    q[:, :, 0], k[:, :, 0] = 1.0, 0.0
    k[:9, :, 0] = -float("inf")                            # the first nine rows see nothing else
    v[4] = float("inf")
    out = _prompt(q, k, v, [0, n], None, 0.5)
    assert (out[:9] == 0).all()
    y, tol = _prompt_ref(q[9:], k[9:], v[9:], [0, n - 9], [0, n - 9], 0.5)
    assert out[9:].isnan().all()                           # 0 times the infinite value, as in the formula
    v[4] = 1.0
    _inside(_prompt(q, k, v, [0, n], None, 0.5)[9:], y, tol)


def test_prompt_starts_that_are_none_leave_their_rows():
    q, k, v = _packed(300, 300, 2, 2, 64, BF16, 6)
    for qs, ks, live in (([0, 100, 400], None, slice(0, 100)), ([0, 100, 300], [0, 100, 301], slice(0, 100)),
                         ([0, 100, 300], [0, 100, 20], slice(0, 100)), ([0, 100, 300], [-5, 100, 20], slice(0, 0)), ([-3, 100, 100], None, slice(0, 0))):
        out = _prompt(q, k, v, qs, ks, 0.125)
        y, tol = _prompt_ref(q[live], k[live], v[live], [0, live.stop], [0, live.stop], 0.125)
        _inside(out[live], y, tol)
        assert (out[live.stop:] == 7).all()
    # starts that descend: whatever rows are written, nothing behind them is
    whole = torch.full((400, 4, 64), 7.0, dtype=BF16, device="cuda")
    for qs in ([0, 100, 50], [300, 0, 200], [50, -100, 3000], [2 ** 31 - 1, 5, -2 ** 31]):
        L.h2o_prompt_attend(q.cuda(), k.cuda(), v.cuda(), _i32(qs), None, 0.125, whole[50:350])
        assert (whole[:50] == 7).all() and (whole[350:] == 7).all()


def test_prompt_no_tokens_at_all():
    q, k, v = _packed(5, 5, 2, 2, 64, BF16, 6)
    assert (_prompt(q, k, v, [0, 0, 0], None, 0.125) == 7).all()
    assert (_prompt(q, k[:0], v[:0], [0, 5], [0, 0], 0.125) == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_many_requests(dtype):
    lengths = [(i * 7) % 5 for i in range(3000)]
    rows = sum(lengths)
    q, k, v = _packed(rows, rows, 1, 2, 64, dtype, 2)
    qs = _starts(lengths)
    out = _prompt(q, k, v, qs, None, 0.125)
    at = [i for i in range(0, 3000, 101)] + [2999]
    for i in at:
        a, b = qs[i], qs[i + 1]
        _inside(out[a:b], *_prompt_ref(q[a:b], k[a:b], v[a:b], [0, b - a], [0, b - a], 0.125))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_strided_rows_and_another_stream(dtype):
    n, heads, G, d = 333, 2, 4, 128
    wide = torch.randn(n, heads * (G + 2) + 1, d, generator=_gen(12)).to(dtype).cuda()
    q, k, v = wide[:, :heads * G], wide[:, heads * G:heads * (G + 1)], wide[:, heads * (G + 1):heads * (G + 2)]
    other = torch.full((n, heads * G + 2, d), 7.0, dtype=dtype, device="cuda")
    out = other[:, 1:-1]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    L.h2o_prompt_attend(q, k, v, _i32([0, 100, n]), None, d ** -0.5, out, s)
    s.synchronize()
    _inside(out, *_prompt_ref(q.cpu(), k.cpu(), v.cpu(), [0, 100, n], [0, 100, n], d ** -0.5))
    assert (other[:, 0] == 7).all() and (other[:, -1] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_same_bits_every_time(dtype):
    q, k, v = (x.cuda() for x in _packed(700, 1500, 2, 4, 128, dtype, 1))
    runs = [_prompt(q, k, v, [0, 300, 700], [0, 900, 1500], 0.1) for _ in range(3)]
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


@pytest.mark.parametrize("dtype,before", [(BF16, 30000), (F32, 3000)])
@pytest.mark.parametrize("new", [1, 5, 40, 300])
def test_prompt_few_queries_behind_many_keys(dtype, before, new):
    for heads, G, d in ((1, 1, 128), (2, 8, 128), (1, 3, 64)):
        q, k, v = _packed(new, before + new, heads, G, d, dtype, new)
        _inside(_prompt(q, k, v, [0, new], [0, before + new], d ** -0.5), *_prompt_ref(q, k, v, [0, new], [0, before + new], d ** -0.5))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("G,d", [(1, 128), (4, 64), (7, 128)])
def test_prompt_few_unequal_requests_with_many_keys(dtype, G, d):
    # long and short key ranges shared by several CTAs, requests without queries, keys or either, rows that see none
    new, keys = [5, 10, 0, 3, 1, 40], [6000, 4, 100, 0, 3001, 777]
    q, k, v = _packed(sum(new), sum(keys) + 30, 1, G, d, dtype, G)
    k[-30:], v[-30:] = float("nan"), float("inf")
    qs, ks = _starts(new), _starts(keys)
    out = _prompt(q, k, v, qs, ks, d ** -0.5)
    _inside(out, *_prompt_ref(q, k, v, qs, ks, d ** -0.5))
    assert (out[5:11] == 0).all() and (out[15:18] == 0).all()
    # values that are no numbers, before and after what a row sees
    v[5998], v[9105 + 770] = float("inf"), float("nan")
    y, tol = _prompt_ref(q, k, v, qs, ks, d ** -0.5)
    out = _prompt(q, k, v, qs, ks, d ** -0.5)
    clean = torch.ones(sum(new), dtype=torch.bool)
    clean[3:5] = False                                     # the rows from those keys on
    clean[19 + 33:] = False
    _inside(out[clean], y[clean], tol[clean])
    assert not out[3:5].isfinite().any()


def test_prompt_offsets_beyond_32_bits():
    # 2^31 elements lie before the request's keys
    keys, heads, d, n = (1 << 19) + 300, 32, 128, 200
    k = torch.zeros(keys, heads, d, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    q, kk, vv = _packed(n, 300, heads, 1, d, BF16, 15)
    k[-300:], v[-300:] = kk.cuda(), vv.cuda()
    out = _prompt(q, k, v, [0, n], [keys - 300, keys], 0.1)
    y, tol = _prompt_ref(q[:, ::8], kk[:, ::8], vv[:, ::8], [0, n], [0, 300], 0.1)
    _inside(out[:, ::8], y, tol)


def test_prompt_captured_and_replayed_with_other_lengths():
    n, d = 500, 64
    q, k, v = (x.cuda() for x in _packed(n, n, 2, 4, d, BF16, 21))
    qs, out = _i32([0, 10, 500]), torch.full((n, 8, d), 7.0, dtype=BF16, device="cuda")
    L.h2o_prompt_attend(q, k, v, qs, None, 0.125, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.h2o_prompt_attend(q, k, v, qs, None, 0.125, out)
    for cut in (10, 256, 499):
        qs.copy_(_i32([0, cut, 500]))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        _inside(out, *_prompt_ref(q.cpu(), k.cpu(), v.cpu(), [0, cut, 500], [0, cut, 500], 0.125))


# ------------------------------------------------------------ quantised pools

def _quantise(x, bits):
    """Codes and scales of rows by the rule, in numpy's fp32."""
    x = x.float().numpy()
    top = np.float32(2 ** (bits - 1) - 1)
    amax = np.abs(x).max(-1, keepdims=True)
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(amax)
        inv = np.where(amax > 0, top / amax, np.float32(0)).astype(np.float32)
        code = np.clip(np.nan_to_num(np.rint(x * inv)), -top, top)
        scale = (amax / top).astype(np.float32)
    code = np.where(bad, 0, code).astype(np.int8)
    return code, np.where(bad, np.float32("nan"), scale)[..., 0].astype(np.float32)


def _pack(code, bits):
    if bits == 8:
        return torch.as_tensor(code)
    u = (code.astype(np.int16) + 8).astype(np.uint8)
    return torch.as_tensor(u[..., 0::2] | u[..., 1::2] << 4)


class Pool:
    def __init__(self, pages, heads, ps, d, bits, fill=None):
        self.pages, self.heads, self.ps, self.d, self.bits = pages, heads, ps, d, bits
        shape = (pages, heads, ps, d * bits // 8)
        dt = torch.int8 if bits == 8 else torch.uint8
        self.K, self.V = (torch.full(shape, 0x55, dtype=dt, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.full((pages, heads, ps), 9.0, device="cuda") for _ in range(2))

    def args(self):
        return self.K, self.V, self.ks, self.vs


SIZES = [(1, 64, 16, 1), (3, 128, 16, 40), (8, 128, 64, 100), (2, 64, 128, 300), (5, 128, 32, 77), (32, 64, 32, 65)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("heads,d,ps,rows", SIZES)
def test_quantised_write_and_read(dtype, bits, heads, d, ps, rows):
    g = _gen(rows)
    pages = -(-rows // ps) + 2
    slot = torch.randperm(pages * ps, generator=g)[:rows].to(torch.int32)
    k, v = (torch.randn(rows, heads, d, generator=g) * torch.exp(2 * torch.randn(rows, heads, 1, generator=g)) for _ in range(2))
    k, v = k.to(dtype), v.to(dtype)
    special = min(rows - 1, 8)
    for i, x in enumerate([0.0, float("nan"), float("inf"), -float("inf"), 1e-39, 3e38, 1e-30, 2.0][:special]):
        k[i, 0] = 0.0 if x == x and abs(x) < 1 else k[i, 0]
        k[i, 0, i] = x
    if rows > 10:
        slot[9], slot[10] = -1, pages * ps                 # padding rows
    p = Pool(pages, heads, ps, d, bits)
    want = Pool(pages, heads, ps, d, bits)
    L.h2o_page_quant_write(k.cuda(), v.cuda(), slot.cuda(), *p.args())
    live = [i for i in range(rows) if 0 <= slot[i] < pages * ps]
    at = slot[live].long()
    for x, pool, scales in ((k, want.K, want.ks), (v, want.V, want.vs)):
        code, scale = _quantise(x, bits)
        pool[at.cuda() // ps, :, at.cuda() % ps] = _pack(code, bits)[live].cuda()
        scales[at.cuda() // ps, :, at.cuda() % ps] = torch.as_tensor(scale)[live].cuda()
    for a, b in zip(p.args(), want.args()):
        assert torch.equal(a.nan_to_num(-1.0) if a.is_floating_point() else a, b.nan_to_num(-1.0) if b.is_floating_point() else b)
    # and back, one slot twice, into slices of a wider buffer
    again = torch.cat([slot, slot[-1:]])
    wide = torch.full((rows + 1, 2 * heads + 1, d), 7.0, dtype=dtype, device="cuda")
    ko, vo = wide[:, :heads], wide[:, heads + 1:]
    L.h2o_page_quant_read(*p.args(), again.cuda(), ko, vo)
    for x, got in ((k, ko), (v, vo)):
        code, scale = _quantise(x, bits)
        y = (torch.as_tensor(code).float() * torch.as_tensor(scale)[..., None]).to(dtype)
        dead = [i for i in range(rows) if i not in live]
        assert torch.equal(got[:rows][live].cpu().nan_to_num(-1.0), y[live].nan_to_num(-1.0))
        assert torch.equal(got[rows], got[rows - 1]) and (got[dead] == 7).all()
    assert (wide[:, heads] == 7).all()
    # a row is off by half a code's step at most (a product and a quotient of its own in fp32)
    off = (ko[:rows][live].double().cpu() - k[live].double()).abs()
    amax = k[live].double().abs().amax(-1, keepdim=True)
    step = amax / (2 ** (bits - 1) - 1)
    fine = amax.isfinite() & (amax > 1e-36)
    near = step * (0.5 + 2.0 ** -14) + (2.0 ** -8 * (k[live].double().abs() + step) if dtype is BF16 else 0)
    assert (torch.where(fine, off - near, torch.full_like(off, -1.0)) <= 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("heads,d,ps,rows", [(7, 128, 64, 24000), (100, 64, 16, 3100), (1, 64, 32, 200001), (8, 128, 128, 20003)])
def test_quantised_many_rows(dtype, bits, heads, d, ps, rows):
    # several rows a thread; the rule's steps as torch's (a tensor over a tensor is one rounding)
    g = torch.Generator(device="cuda").manual_seed(rows)
    pages = -(-rows // ps) + 1
    slot = torch.randperm(pages * ps, generator=g, device="cuda")[:rows].to(torch.int32)
    slot[::97] = -1
    k, v = (torch.randn(rows, heads, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    k[5], v[7, 0, 3], k[11, 0, 0], v[13] = 0.0, float("nan"), float("inf"), 1e-38
    p = Pool(pages, heads, ps, d, bits)
    L.h2o_page_quant_write(k, v, slot, *p.args())
    live = slot >= 0
    at = slot[live].long()
    back = [torch.full_like(k, 7.0) for _ in range(2)]
    L.h2o_page_quant_read(*p.args(), slot, *back)
    for x, pool, scales, got in ((k, p.K, p.ks, back[0]), (v, p.V, p.vs, back[1])):
        x = x[live].float()
        amax = x.abs().amax(-1, keepdim=True)
        odd = ~amax.isfinite()
        top = torch.full_like(amax, 2 ** (bits - 1) - 1)
        inv = torch.where(amax > 0, top / amax, 0.0)
        code = torch.where(odd, 0.0, torch.round(x * inv).nan_to_num().clamp(-top, top))
        scale = torch.where(odd, torch.nan, amax / top)[..., 0]
        stored = pool[at // ps, :, at % ps]
        if bits == 4:
            stored = torch.stack([stored & 15, stored >> 4], -1).flatten(-2).float() - 8
        assert torch.equal(stored.float(), code)
        assert torch.equal(scales[at // ps, :, at % ps].nan_to_num(-1.0), scale.nan_to_num(-1.0))
        assert torch.equal(got[live].nan_to_num(-1.0), (code * scale[..., None]).to(dtype).nan_to_num(-1.0))
        assert (got[~live] == 7).all()
    rest = torch.ones(pages * ps, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (p.ks.transpose(1, 2).reshape(-1, heads)[rest] == 9.0).all() and (p.K.transpose(1, 2).reshape(pages * ps, -1)[rest] == 0x55).all()


def test_quantised_rows_strided_on_another_stream():
    rows, heads, d = 50, 4, 128
    wide = torch.randn(rows, 3 * heads, d, generator=_gen(3)).to(BF16).cuda()
    p = Pool(8, heads, 16, d, 8)
    slot = torch.randperm(128, generator=_gen(2))[:rows].to(torch.int32).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    L.h2o_page_quant_write(wide[:, heads:2 * heads], wide[:, 2 * heads:], slot, *p.args(), s)
    out = torch.zeros_like(wide)
    s.wait_stream(torch.cuda.current_stream())
    L.h2o_page_quant_read(*p.args(), slot, out[:, heads:2 * heads], out[:, 2 * heads:], s)
    s.synchronize()
    code, scale = _quantise(wide.cpu(), 8)
    y = (torch.as_tensor(code).float() * torch.as_tensor(scale)[..., None]).to(BF16)
    assert torch.equal(out[:, heads:].cpu(), y[:, heads:]) and (out[:, :heads] == 0).all()


# ------------------------------------------------- attention over quantised pools

class Cache:
    """A quantised pool, block tables of random pages, and requests of given lengths."""

    def __init__(self, lengths, heads, d, ps, bits, seed=0, extra=3, width=None):
        g = _gen(seed)
        self.ps, self.heads, self.d, self.bits, self.lengths = ps, heads, d, bits, list(lengths)
        owned = [-(-n // ps) for n in lengths]
        self.width = width or max(1, max(owned))
        pages = sum(owned) + extra
        perm = torch.randperm(pages, generator=g).numpy()
        self.table = np.full((len(lengths), self.width), -1, np.int32)
        at = 0
        for i, n in enumerate(owned):
            self.table[i, :n] = perm[at:at + n]
            at += n
        top = 2 ** (bits - 1) - 1
        self.kc, self.vc = (torch.randint(-top, top + 1, (pages, heads, ps, d), generator=g, dtype=torch.int8) for _ in range(2))
        self.ks, self.vs = (torch.exp(0.7 * torch.randn(pages, heads, ps, generator=g)) * 2 / top for _ in range(2))
        live = torch.zeros(pages, ps, dtype=torch.bool)
        for i, n in enumerate(self.lengths):
            for t in range(n):
                live[self.table[i, t // ps], t % ps] = True
        dead = (~live)[:, None].expand(pages, heads, ps)   # what no request holds is never to be seen
        self.ks[dead], self.vs[dead] = float("nan"), float("inf")

    def pool(self):
        return _pack(self.kc.numpy(), self.bits).cuda(), _pack(self.vc.numpy(), self.bits).cuda(), self.ks.cuda(), self.vs.cuda()

    def rows(self, i, head, n):
        p = torch.as_tensor(self.table[i, :-(-n // self.ps)]).long()
        return tuple((c[p, head].double() * s[p, head].double()[..., None]).reshape(-1, self.d)[:n] for c, s in ((self.kc, self.ks), (self.vc, self.vs)))


def _attend(c, q, seq, pos, scale, out=None, stream=None, table=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
    L.h2o_page_quant_attend(q.cuda(), _i32(seq), _i32(pos), *c.pool(), _i32(c.table if table is None else table), scale, out, stream)
    return out


def _attend_ref(c, q, seq, pos, scale):
    rows, hq, d = q.shape
    G = hq // c.heads
    y, tol = torch.zeros(rows, hq, d, dtype=torch.float64), torch.zeros(rows, hq, d, dtype=torch.float64)
    for r in range(rows):
        if seq[r] < 0 or pos[r] < 0:
            continue
        for h in range(c.heads):
            k, v = c.rows(seq[r], h, pos[r] + 1)
            qq = q[r, h * G:(h + 1) * G].double()
            # queries are fp16 numbers apart from the row's largest: as if all their channels were off by 2^-23 of it
            most = qq.abs().amax(1, keepdim=True)
            a = _softmax_rows(qq, k, v, scale, [pos[r] + 1] * G)
            smax = scale * (most * k.abs().sum(1).amax())
            w = torch.softmax((qq @ k.T) * scale, 1) * (v.abs().amax(1))
            small = 2.0 ** -31 * (pos[r] + 1) * w.amax(1, keepdim=True)
            t = _bound(q.dtype, d, pos[r] + 1, a[0], a[1], a[2], smax, 2.0 ** -12)
            y[r, h * G:(h + 1) * G] = a[0]
            tol[r, h * G:(h + 1) * G] = t + small
    return y, tol


def _queries(rows, hq, d, dtype, seed):
    return torch.randn(rows, hq, d, generator=_gen(seed)).to(dtype)


SHAPES = [  # heads, groups, d, page size
    (4, 1, 64, 16), (2, 4, 128, 16), (1, 16, 128, 32), (3, 5, 64, 64), (2, 8, 128, 128), (1, 2, 64, 128), (2, 9, 128, 64), (5, 3, 128, 16), (1, 13, 64, 32),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("heads,G,d,ps", SHAPES)
def test_attend(dtype, bits, heads, G, d, ps):
    lengths = [1, 15, 16, 17, 300, 2 * ps, 2 * ps + 1, 130]
    c = Cache(lengths, heads, d, ps, bits, seed=G)
    seq, pos = [], []
    for i, n in enumerate(lengths):
        for t in {n - 1, n // 2, 0}:
            seq.append(i)
            pos.append(t)
    q = _queries(len(seq), heads * G, d, dtype, 1)
    _inside(_attend(c, q, seq, pos, d ** -0.5), *_attend_ref(c, q, seq, pos, d ** -0.5))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("heads,G,d,n", [(1, 1, 128, 20000), (2, 8, 128, 9001), (8, 2, 64, 5000), (1, 16, 64, 33333)])
def test_attend_long_requests(dtype, bits, heads, G, d, n):
    c = Cache([n, 3], heads, d, 32, bits, seed=n)
    q = _queries(3, heads * G, d, dtype, 2)
    _inside(_attend(c, q, [0, 1, 0], [n - 1, 2, n - 2], d ** -0.5), *_attend_ref(c, q, [0, 1, 0], [n - 1, 2, n - 2], d ** -0.5))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
def test_attend_many_units(dtype, bits):
    lengths = [(i * 37) % 500 + 1 for i in range(200)]
    c = Cache(lengths, 8, 128, 16, bits, seed=4, width=60)
    q = _queries(200, 16, 128, dtype, 3)
    pos = [n - 1 for n in lengths]
    out = _attend(c, q, list(range(200)), pos, 0.1)
    at = list(range(0, 200, 9))
    y, tol = _attend_ref(c, q[at], at, [pos[i] for i in at], 0.1)
    _inside(out[at], y, tol)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
def test_attend_rows_that_are_padding_empty_or_bad(dtype, bits):
    c = Cache([100, 60], 2, 128, 16, bits, seed=9)
    q = _queries(9, 8, 128, dtype, 5)
    seq, pos = [0, -1, 1, 0, 2, 0, 1, 1, -7], [99, 5, -1, 7 * 16, 3, 50, 59, -9, -7]
    out = _attend(c, q, seq, pos, 0.1)
    assert (out[[1, 8]] == 7).all() and (out[[2, 7]] == 0).all() and out[[3, 4]].isnan().all()
    at = [0, 5, 6]
    y, tol = _attend_ref(c, q[at], [seq[i] for i in at], [pos[i] for i in at], 0.1)
    _inside(out[at], y, tol)
    # entries that are no page: NaN in the rows that read them, and in no other
    table = c.table.copy()
    table[0, 4], table[1, 3] = c.kc.shape[0], -1
    out = _attend(c, q[:4], [0, 0, 1, 1], [99, 63, 59, 47], 0.1, table=table)
    assert out[[0, 2]].isnan().all()
    _inside(out[[1, 3]], *_attend_ref(c, q[[1, 3]], [0, 1], [63, 47], 0.1))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
def test_attend_sizes_far_apart(dtype, bits):
    # queries and scales over many powers of two, and rows of zeros
    n, d = 400, 64
    c = Cache([n], 2, d, 16, bits, seed=6)
    q = _queries(6, 4, d, dtype, 6)
    for i, s in enumerate([1e-30, 1e30, 1e-4, 3e4, 1.0, 1.0]):
        q[i] *= s
    q[5] = 0.0
    pages = torch.as_tensor(c.table[0]).long()
    for i, (ks, vs) in enumerate([(1e30, 1.0), (1e-30, 1e-20), (1e3, 1e20), (1e-5, 1.0), (1.0, 1.0), (1.0, 1e-3)]):
        e = Cache([n], 2, d, 16, bits, seed=6)
        e.ks *= ks
        e.vs *= vs
        e.vs[pages[:3], 0] = 0.0
        e.vs[pages[5]] *= 1e5                              # a page whose values are far larger
        e.ks[pages[4], 1] = 0.0
        _inside(_attend(e, q[i:i + 1], [0], [n - 1], 0.125), *_attend_ref(e, q[i:i + 1], [0], [n - 1], 0.125))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
def test_attend_large_logits_and_special_values(dtype, bits):
    n, d = 777, 128
    c = Cache([n], 2, d, 32, bits, seed=2)
    q = 40 * _queries(4, 4, d, dtype, 8)
    _inside(_attend(c, q, [0] * 4, [n - 1] * 4, 0.5), *_attend_ref(c, q, [0] * 4, [n - 1] * 4, 0.5))
    # a row stored as NaN: seen by the rows behind it, in its head
    pages = torch.as_tensor(c.table[0]).long()
    c.ks[pages[3], 0, 7] = float("nan")
    out = _attend(c, q[:2], [0, 0], [n - 1, 3 * 32 + 6], 0.5)
    assert out[0, :2].isnan().all() and out[0, 2:].isfinite().all() and out[1].isfinite().all()
    c.ks[pages[3], 0, 7], c.vs[pages[3], 1, 7] = 1.0, float("nan")
    out = _attend(c, q[:2], [0, 0], [n - 1, 3 * 32 + 6], 0.5)
    assert out[0, 2:].isnan().all() and out[0, :2].isfinite().all() and out[1].isfinite().all()
    # queries that are no numbers
    q[0, 1, 3], q[1, 0, 0] = float("nan"), float("inf")
    out = _attend(c, q[:2], [0, 0], [90, 90], 0.5)
    assert out[0, 1].isnan().all() and out[1, 0].isnan().all() and out[0, [0, 2, 3]].isfinite().all() and out[1, 1:].isfinite().all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", [300, 4096, 16384])
@pytest.mark.parametrize("requests,heads", [(2, 3), (40, 4), (150, 8)])
def test_attend_tables_much_wider_than_the_requests(dtype, width, requests, heads):
    lengths = [(i * 53) % 700 + 1 for i in range(requests)]
    c = Cache(lengths, heads, 64, 16, 4, seed=width, width=width)
    q = _queries(requests, 2 * heads, 64, dtype, 3)
    pos = [n - 1 for n in lengths]
    out = _attend(c, q, list(range(requests)), pos, 0.1)
    at = list(range(0, requests, 17))
    y, tol = _attend_ref(c, q[at], at, [pos[i] for i in at], 0.1)
    _inside(out[at], y, tol)


def test_attend_captured_and_replayed():
    c = Cache([400, 90], 2, 128, 32, 8, seed=3, width=40)
    pool, table = c.pool(), _i32(c.table)
    q, seq, pos = _queries(2, 8, 128, BF16, 1).cuda(), _i32([0, 1]), _i32([10, 20])
    out = torch.empty_like(q)
    L.h2o_page_quant_attend(q, seq, pos, *pool, table, 0.1, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.h2o_page_quant_attend(q, seq, pos, *pool, table, 0.1, out)
    for a, b in ((399, 89), (0, -1), (200, 33)):
        pos.copy_(_i32([a, b]))
        graph.replay()
        torch.cuda.synchronize()
        _inside(out, *_attend_ref(c, q.cpu(), [0, 1], [a, b], 0.1))


@pytest.mark.parametrize("bits,pages", [(8, 70000), (4, 140000)])
def test_attend_offsets_beyond_32_bits(bits, pages):
    # pages of 4 x 128 x 128 codes: beyond 4 GB of each
    heads, ps, d, n = 4, 128, 128, 300
    c = Cache([n], heads, d, ps, bits, seed=3, extra=0)
    K, V, ks, vs = c.pool()
    bigK, bigV = (torch.empty(pages, *K.shape[1:], dtype=K.dtype, device="cuda") for _ in range(2))
    bks, bvs = (torch.empty(pages, heads, ps, device="cuda") for _ in range(2))
    at = [pages - 1, pages - 3, 5]
    for i, p in enumerate(c.table[0]):
        bigK[at[i]], bigV[at[i]], bks[at[i]], bvs[at[i]] = K[p], V[p], ks[p], vs[p]
    q = _queries(1, 8, d, BF16, 4)
    out = torch.empty_like(q).cuda()
    L.h2o_page_quant_attend(q.cuda(), _i32([0]), _i32([n - 1]), bigK, bigV, bks, bvs, _i32([at]), 0.1, out)
    _inside(out, *_attend_ref(c, q, [0], [n - 1], 0.1))
    # writes and reads there
    k = torch.randn(3, heads, d, generator=_gen(7)).to(BF16)
    slot = _i32([(pages - 1) * ps + 127, 4, (pages - 2) * ps])
    L.h2o_page_quant_write(k.cuda(), k.cuda(), slot, bigK, bigV, bks, bvs)
    ko, vo = torch.empty_like(k).cuda(), torch.empty_like(k).cuda()
    L.h2o_page_quant_read(bigK, bigV, bks, bvs, slot, ko, vo)
    code, scale = _quantise(k, bits)
    y = (torch.as_tensor(code).float() * torch.as_tensor(scale)[..., None]).to(BF16)
    assert torch.equal(ko.cpu(), y) and torch.equal(vo.cpu(), y)


def test_attend_strided_in_place_and_on_two_streams():
    c = Cache([500, 20, 333], 2, 128, 16, 4, seed=1)
    pool, table = c.pool(), _i32(c.table)
    wide = torch.randn(3, 8 + 4, 128, generator=_gen(5)).to(BF16).cuda()
    q = wide[:, :8]
    y, tol = _attend_ref(c, q.cpu(), [0, 1, 2], [499, 19, 332], 0.1)
    outs, streams = [torch.empty(3, 8, 128, dtype=BF16, device="cuda") for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    seq, pos = _i32([0, 1, 2]), _i32([499, 19, 332])
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip(streams, outs):
            L.h2o_page_quant_attend(q, seq, pos, *pool, table, 0.1, o, s)
    torch.cuda.synchronize()
    for o in outs:
        _inside(o, y, tol)
    assert torch.equal(outs[0], outs[1])
    L.h2o_page_quant_attend(q, seq, pos, *pool, table, 0.1, q)      # in the place of the queries
    assert torch.equal(q, outs[0])


# ------------------------------------------------------------------- together

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
def test_a_batch_is_served(dtype, bits):
    """Prompts, single tokens, and a prompt that goes on behind its cached context: positions, codes, attention."""
    heads, G, d, ps, P, rot = 2, 4, 128, 16, 80, 64
    g = _gen(31)
    table = torch.as_tensor(L.h2o_rope_table(rot)).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    n, width = 3, 16
    blocks, length = torch.full((n, width), -1, **i32), torch.zeros(n, **i32)
    free = torch.randperm(P, generator=g).to(**i32)
    p = Pool(P, heads, ps, d, bits)
    ref = [[torch.zeros(0, heads, d, dtype=torch.float64) for _ in range(2)] for _ in range(n)]    # what each cache stands for
    scale = d ** -0.5
    for step, new in enumerate(([70, 5, 130], [1, 1, 1], [1, 0, 1], [3, 90, 2])):
        rows = sum(new)
        after, start, seq, pos, slot, status = (torch.empty(m, **i32) for m in (n, n + 1, rows, rows, rows, 4))
        L.h2o_page_tables(length, torch.tensor(new, **i32), free, ps, blocks, after, start, seq, pos, slot, status)
        assert status.tolist()[3] == 0
        qkv = torch.randn(rows, heads * (G + 2), d, generator=g).to(dtype).cuda()
        q, k, v = qkv[:, :heads * G], qkv[:, heads * G:heads * (G + 1)], qkv[:, heads * (G + 1):]
        L.h2o_rope(q, k, pos, table, L.H2O_ROPE_HALF, 1.0, q, k)
        L.h2o_page_quant_write(k, v, slot, *p.args())
        out = torch.full((rows, heads * G, d), 7.0, dtype=dtype, device="cuda")
        old = [x[0].shape[0] for x in ref]
        for i in range(n):
            a, b = int(start[i]), int(start[i + 1])
            for j, x in enumerate((k, v)):
                code, s = _quantise(x[a:b].cpu(), bits)
                ref[i][j] = torch.cat([ref[i][j], torch.as_tensor(code).double() * torch.as_tensor(s).double()[..., None]])
        if step == 0:
            # a first prompt attends to its rows as they are
            L.h2o_prompt_attend(q, k, v, start, None, scale, out)
            y, tol = _prompt_ref(q.cpu(), k.cpu(), v.cpu(), start.tolist(), start.tolist(), scale)
        elif step < 3:
            L.h2o_page_quant_attend(q, seq, pos, *p.args(), blocks, scale, out)
        else:
            # rows behind a cached context: the whole context read back
            total = after.tolist()
            t = torch.cat([torch.arange(m) for m in total]).cuda()
            i = torch.repeat_interleave(torch.arange(n), torch.tensor(total)).cuda()
            at = (blocks[i, t // ps].long() * ps + t % ps).to(torch.int32)
            kk, vv = (torch.empty(sum(total), heads, d, dtype=dtype, device="cuda") for _ in range(2))
            L.h2o_page_quant_read(*p.args(), at, kk, vv)
            ks = _starts(total)
            L.h2o_prompt_attend(q, kk, vv, start, _i32(ks), scale, out)
            y, tol = _prompt_ref(q.cpu(), kk.cpu(), vv.cpu(), start.tolist(), ks, scale)
            whole = torch.cat([r[0] for r in ref])
            assert ((kk.double().cpu() - whole).abs() <= (2.0 ** -8 if dtype is BF16 else 0) * whole.abs() + 2 * U * whole.abs()).all()
        if 0 < step < 3:
            y, tol = torch.zeros(rows, heads * G, d, dtype=torch.float64), torch.zeros(rows, heads * G, d, dtype=torch.float64)
            for r, i in enumerate(seq.tolist()):
                for j in range(heads * G):
                    qq = q[r:r + 1, j].cpu().double()
                    kk, vv = ref[i][0][:, j // G], ref[i][1][:, j // G]
                    a = _softmax_rows(qq, kk, vv, scale, [kk.shape[0]])
                    smax = scale * qq.abs().max() * kk.abs().sum(1).max()
                    y[r, j] = a[0][0]
                    tol[r, j] = (_bound(dtype, d, kk.shape[0], a[0], a[1], a[2], smax, 2.0 ** -12) + 2.0 ** -31 * kk.shape[0] * vv.abs().max())[0]
        _inside(out, y, tol, "step %d" % step)
        assert [x[0].shape[0] for x in ref] == after.tolist() and old == length.tolist()
        length, free = after, free[int(status[1]):]


def test_injected_launch_failure(monkeypatch):
    c = Cache([40], 2, 64, 16, 8)
    q = _queries(1, 4, 64, BF16, 0).cuda()
    k = torch.zeros(1, 2, 64, dtype=BF16, device="cuda")
    pool = c.pool()
    monkeypatch.setenv("H2O_FAULT", "launch")
    for call in (lambda: L.h2o_page_quant_attend(q, _i32([0]), _i32([3]), *pool, _i32(c.table), 0.1, q.clone()),
                 lambda: L.h2o_page_quant_write(k, k, _i32([3]), *pool), lambda: L.h2o_page_quant_read(*pool, _i32([3]), k, k.clone()),
                 lambda: L.h2o_prompt_attend(q, k, k, _i32([0, 1]), None, 0.1, q.clone()),
                 lambda: L.h2o_rope(q, k, _i32([0]), torch.zeros(16, dtype=torch.int64, device="cuda"), 0, 1.0, q, k)):
        with pytest.raises(L.H2OError) as e:
            call()
        assert e.value.code == L.H2O_ERR_CUDA
    monkeypatch.delenv("H2O_FAULT")
    L.h2o_page_quant_write(k, k, _i32([3]), *pool)
    torch.cuda.synchronize()
