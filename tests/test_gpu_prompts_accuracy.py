"""Prompt attention and attention over quantised pages where a wrong weight, sum
or tile shows: bounds far below the results.

Large logits are exact: queries and codes are small whole numbers and scales
powers of two, so that no path's products round (a tensor core's sums neither,
below 2^24 of their smallest unit), and what is left of the bounds in
test_gpu_prompts.py is the exponential's 4 U |z|, the sums' and the weights'
and outputs' rounding.  Values have a mean far from zero.

fp32 over long contexts with logits of size 3: a sum of N roundings of either sign, each at most half
a step, is off by sqrt(N / 3) U of itself in standard deviation.  Keys are added up in
chains of at most 2048 sums (16 products each, by one warp), weights in chains
of at most 8192, and logits of size 3 are off by 4 such deviations of their 136
roundings: sqrt(2048 / 3) U + sqrt(8192 / 3) U + 4 sqrt(136 / 3) U = 6.3e-6 at the very most; over the
independent errors of the weights only the first two stay, and those chains are
shared by at least four warps whose errors are independent: half of 78 U,
2.3e-6.  2e-6 is asked for, since what it has to tell apart (sums inside the tensor cores) was 3.2e-6
to 8.1e-6 off, and everything else larger.
"""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import test_gpu_prompts as P   # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = P.U


def _telling(got, y, tol, share, what=""):
    """Inside the bounds, which are below `share` of the results (the middle ones)."""
    assert tol.median() <= share * y.abs().median(), "%g of %g" % (tol.median(), y.abs().median())
    P._inside(got, y, tol, what)


def _whole(shape, most, seed):
    return torch.randint(-most, most + 1, shape, generator=P._gen(seed)).float()


def _values(shape, seed):
    return 1.0 + 0.4 * torch.randn(*shape, generator=P._gen(seed)) + 2.0 * (torch.arange(shape[0]) % 3 == 0).float()[:, None, None]


def _exact(dtype, n, a, half):
    """The bound without the products' rounding: `a` as _softmax_rows gives it, half: a weight's rounding."""
    y, av, zmax, _ = a
    return P._bound(dtype, 0, n, y, av, zmax, torch.zeros_like(zmax), half)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("nq,nk,G,d", [(600, 600, 2, 64), (300, 900, 4, 128), (5, 4000, 1, 128), (40, 3000, 8, 64)])
@pytest.mark.parametrize("rise", [0, 1, 40])
def test_prompt_large_exact_logits(dtype, nq, nk, G, d, rise):
    # logits up to 3000, whose maxima rise along the keys; every key has a twin, so that several count
    q, k, v = _whole((nq, G, d), 3, 1), _whole((nk, 1, d), 2, 2), _values((nk, 1, d), 3)
    q[:, :, 0] = 3.0
    k[:, 0, 0] = (rise * torch.arange(nk) // 60 % 120).float()
    k[1::2] = k[::2]
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    scale = 0.125 if rise < 40 else 4.0
    out = P._prompt(q, k, v, [0, nq], [0, nk], scale)
    seen = torch.clamp(nk - nq + torch.arange(nq) + 1, 0, nk)
    for j in range(G):
        a = P._softmax_rows(q[:, j].cuda().double(), k[:, 0].cuda().double(), v[:, 0].cuda().double(), scale, seen.cuda())
        _telling(out[:, j], a[0].cpu(), _exact(dtype, nk, a, 2.0 ** -8).cpu(), 0.02)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("heads,G,d,n", [(2, 4, 128, 777), (1, 16, 64, 3000), (1, 1, 128, 9000)])
@pytest.mark.parametrize("rise", [0, 1, 4])
def test_attend_large_exact_logits(dtype, bits, heads, G, d, n, rise):
    # codes are whole numbers, scales of keys rise by powers of two along them
    c = P.Cache([n], heads, d, 16, bits, seed=2)
    c.kc.clamp_(-7, 7)
    pages = torch.as_tensor(c.table[0]).long()
    c.ks[:] = 0.125
    for i, p in enumerate(pages.tolist()):
        c.ks[p] *= 2.0 ** (rise * (i % 64) // 32)
    c.vc.abs_()
    q = _whole((3, heads * G, d), 3, 4).to(dtype)
    pos, scale = [n - 1, n // 2, 17], 4.0 if rise == 4 else 0.25
    out = P._attend(c, q, [0] * 3, pos, scale)
    for r in range(3):
        for h in range(heads):
            k, v = c.rows(0, h, pos[r] + 1)
            a = P._softmax_rows(q[r, h * G:(h + 1) * G].double(), k, v, scale, [pos[r] + 1] * G)
            half = 2.0 ** -11 if dtype is BF16 else 2.0 ** -22
            tol = _exact(dtype, pos[r] + 1, a, half)
            if dtype is F32:
                tol = tol + half * a[1]
            w = torch.softmax((q[r, h * G:(h + 1) * G].double() @ k.T) * scale, 1) * v.abs().amax(1)
            tol = tol + 2.0 ** -30 * (pos[r] + 1) * w.amax(1, keepdim=True)
            _telling(out[r, h * G:(h + 1) * G], a[0], tol, 0.03)


@pytest.mark.parametrize("G,d,nq,n", [(1, 128, 3, 20000), (4, 64, 2, 20000), (1, 128, 200, 20000), (2, 128, 900, 4000)])
def test_prompt_fp32_error_over_many_keys(G, d, nq, n):
    q, k, v = P._packed(nq, n, 1, G, d, F32, n + G)
    v = v.abs() + 0.5
    y, _ = P._prompt_ref(q, k, v, [0, nq], [0, n], d ** -0.5)
    off = (P._prompt(q, k, v, [0, nq], [0, n], d ** -0.5).double().cpu() - y).abs().max()
    assert off <= 2e-6 * v.mean()


def _attend_error(bits, heads, G, d, flat):
    n = 32000
    c = P.Cache([n], heads, d, 32, bits, seed=n)
    c.vc.abs_()
    if flat:
        c.ks[:], c.vs[:] = (2.0 / (2 ** (bits - 1) - 1) for _ in range(2))
    q = 0.5 * P._queries(1, heads * G, d, F32, 2)
    out = P._attend(c, q, [0], [n - 1], d ** -0.5).double().cpu()
    for h in range(heads):
        k, v = c.rows(0, h, n)
        qq = q[0, h * G:(h + 1) * G].double()
        y, _, zmax, _ = P._softmax_rows(qq, k, v, d ** -0.5, [n] * G)
        yield (out[0, h * G:(h + 1) * G] - y).abs(), y, v.mean(), zmax, d ** -0.5 * qq.abs().amax(1, keepdim=True) * k.norm(dim=1).max()


ATTEND = [(1, 1, 128), (2, 4, 128), (1, 16, 64)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("heads,G,d", ATTEND)
def test_attend_fp32_error_over_many_keys(bits, heads, G, d):
    # scales far apart: logits up to 32 and single keys with most of the weight, so that two errors of one weight come on
    # top: 4 U |z|, and four deviations of what the queries' rounding, half a step of 2^-22 of the row's largest a channel, makes of a logit
    for off, y, mean, zmax, size in _attend_error(bits, heads, G, d, False):
        assert (off <= (2e-6 + 4 * U * zmax + 4 * 2.0 ** -23 * size) * torch.maximum(y, mean)).all()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("heads,G,d", ATTEND)
def test_attend_fp32_error_over_many_keys_alike(bits, heads, G, d):
    for off, y, mean, zmax, _ in _attend_error(bits, heads, G, d, True):
        assert zmax.max() <= 4 and (off <= 2e-6 * mean).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("nq,nk,heads,G,d", [(1, 20001, 2, 1, 128), (5, 20010, 1, 1, 64), (5, 3001, 1, 16, 128), (200, 2500, 2, 4, 128), (900, 900, 1, 1, 64)])
@pytest.mark.parametrize("where", [0.0, 0.37, 1.0])
def test_prompt_most_weight_in_few_keys(dtype, nq, nk, heads, G, d, where):
    # two keys at the end (of the first row's), at the start or between have half of the weight, and values of their own
    q, k, v = P._packed(nq, nk, heads, G, d, dtype, nk, 0.2)
    v = v.abs() + 0.5
    at = int(where * (nk - nq - 1)) if nk > nq else int(where * (nk - 2))
    q[:, :, 0] = 1.0
    k[:, :, 0] = 0.0
    k[at:at + 2, :, 0] = float(torch.tensor(nk / 2.0).log() * d ** 0.5)
    v[at:at + 2] += 3.0
    _telling(P._prompt(q, k, v, [0, nq], [0, nk], d ** -0.5), *P._prompt_ref(q, k, v, [0, nq], [0, nk], d ** -0.5), 0.04)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("n,heads,G,d", [(9001, 1, 1, 128), (20033, 2, 4, 128), (5000, 1, 16, 64)])
@pytest.mark.parametrize("where", [0.0, 0.61, 1.0])
def test_attend_most_weight_in_few_keys(dtype, bits, n, heads, G, d, where):
    c = P.Cache([n], heads, d, 16, bits, seed=n)
    c.vc.abs_()
    q = 0.1 * P._queries(1, heads * G, d, dtype, 7).float()
    q[:, :, 0] = 1.0
    q = q.to(dtype)
    top = 2 ** (bits - 1) - 1
    c.kc[..., 0] = 0
    for t in (int(where * (n - 2)), int(where * (n - 2)) + 1):
        p = int(c.table[0, t // 16])
        c.kc[p, :, t % 16] = 0
        c.kc[p, :, t % 16, 0], c.ks[p, :, t % 16] = top, float(torch.tensor(n / 2.0).log() * d ** 0.5) / top
        c.vs[p, :, t % 16] *= 3.0
    _telling(P._attend(c, q, [0], [n - 1], d ** -0.5), *P._attend_ref(c, q, [0], [n - 1], d ** -0.5), 0.04)


@pytest.mark.parametrize("nq,nk,G,d", [(130, 130, 2, 64), (5, 3000, 1, 128), (300, 300, 4, 128)])
def test_prompt_fp32_small_numbers(nq, nk, G, d):
    # values of 1e-36, and queries of 1e-36 with keys of 1e36: read to 2^-134, half of bf16's last step, which is 2^-14 of them.  A weight
    # moves by what its logit and the largest one do, the sums by n U (both as in test_gpu_prompts.py)
    q, k, v = P._packed(nq, nk, 1, G, d, F32, nk)
    v = (v.abs() + 0.5) * 1e-36
    seen = torch.clamp(nk - nq + torch.arange(nq) + 1, 0, nk)
    for qq, kk in ((q, k), (q * 1e-36, k * 1e36)):
        out = P._prompt(qq, kk, v, [0, nq], [0, nk], d ** -0.5).double().cpu()
        for j in range(G):
            y, av, zmax, smax = (x.cpu() for x in P._softmax_rows(qq[:, j].cuda().double(), kk[:, 0].cuda().double(), v[:, 0].cuda().double(), d ** -0.5, seen.cuda()))
            moved = d ** -0.5 * 2.0 ** -134 * (kk.double().abs().sum(2).amax() + qq[:, j].double().abs().sum(1, keepdim=True))
            tol = (U * (2 * (2 * (d + 8) * smax + 4 * zmax) + 4 * nk + 64) + 2 * moved) * av + 2.0 ** -134 + U * y
            assert ((out[:, j] - y).abs() <= tol).all() and tol.median() <= 0.005 * y.median()
