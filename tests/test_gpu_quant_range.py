"""Attention over quantised pages at the ends of fp32's range: queries beyond
what the call takes, scales near the largest there are, weights and values whose
products are near it.  Bounds as in test_gpu_prompts.py."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import test_gpu_prompts as P   # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("sign", [1, -1])
def test_queries_beyond_the_range_are_nan(dtype, bits, sign):
    # one key, whose product with the queries has either sign
    c = P.Cache([1], 1, 64, 16, bits)
    c.kc[:], c.ks[:] = sign * 5, 1.0
    q = torch.ones(5, 1, 64)
    for i, x in enumerate((2.0 ** 113, 1.5 * 2.0 ** 114, 1e36, 3e38, float("inf"))):
        q[i] *= x
    out = P._attend(c, q.to(dtype), [0] * 5, [0] * 5, 1.0).cpu()
    assert out[1:].isnan().all()
    # within the range: the only key's value
    v = c.rows(0, 0, 1)[1][0]
    assert ((out[0, 0].double() - v).abs() <= 2.0 ** -8 * v.abs()).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
def test_queries_of_zeros_whatever_the_scale(dtype, bits):
    n, d = 40, 64
    c = P.Cache([n], 1, d, 16, bits)
    q = torch.zeros(1, 2, d, dtype=dtype)
    for scale in (1e-30, 1.0, 1e36):
        P._inside(P._attend(c, q, [0], [n - 1], scale), *P._attend_ref(c, q, [0], [n - 1], scale))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("heads,G,d,n", [(2, 2, 64, 300), (1, 16, 128, 2000)])
def test_keys_near_the_largest_there_are(dtype, bits, heads, G, d, n):
    # keys up to 1.3e38 and queries of 1e-38: their products are of any size
    c = P.Cache([n], heads, d, 16, bits, seed=3)
    c.ks[:] = 1.3e38 / (2 ** (bits - 1) - 1)
    for size in (1e-38, 3e-38, 1e-30):
        q = size * P._queries(2, heads * G, d, F32, 4)
        q = q.to(dtype)
        P._inside(P._attend(c, q, [0, 0], [n - 1, n // 2], 0.5), *P._attend_ref(c, q, [0, 0], [n - 1, n // 2], 0.5))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("logit", [1.0, 5.0, 5.5, 40.0])
def test_values_near_the_largest_there_are(dtype, bits, logit):
    # one key of larger weight than the many before it, and its value times that weight beyond the range
    n, d, top = 4000, 128, 2 ** (bits - 1) - 1
    c = P.Cache([n], 1, d, 16, bits, seed=5)
    c.kc[:], c.ks[:], c.vs[:] = 0, 1.0, 1e-3
    q = torch.zeros(1, 3, d)
    q[:, :, 7] = 1.0
    at = 3203
    page = int(c.table[0, at // 16])
    c.kc[page, 0, at % 16, 7], c.ks[page, 0, at % 16], c.vs[page, 0, at % 16] = top, logit / top, 2.5e38 / top
    q = q.to(dtype)
    y, tol = P._attend_ref(c, q, [0], [n - 1], 1.0)
    assert y.isfinite().all()
    P._inside(P._attend(c, q, [0], [n - 1], 1.0), y, tol)
