"""Prompt attention with infinities and NaN among queries, keys and values: each
output is what the formula says of what its row sees, and a call with such rows
takes about the time of one without.  Bounds as in test_gpu_prompts.py."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import test_gpu_prompts as P   # noqa: E402
from kv_cache_eviction_h2o_gb300 import binding as L   # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")

# requests' queries and keys, heads, groups, d: whole prompts (two tiles of queries an item, and one), many requests, few
# queries behind many keys (clusters share them), queries that see no key
SHAPES = [([700], [700], 2, 4, 128), ([300, 90, 5], [300, 200, 5], 2, 1, 64), ([3] * 200, [40] * 200, 1, 3, 128), ([5], [5000], 1, 1, 128),
          ([40, 3], [3000, 1500], 1, 8, 64), ([9], [4], 1, 2, 64), ([260], [2600], 1, 1, 128)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("what", ["first key", "first value", "first values infinite", "a query", "all values", "all values infinite", "late value",
                                  "late infinity", "infinity then a later one", "NaN then another channel", "late key", "either sign"])
def test_rows_are_what_the_formula_says(dtype, shape, what):
    new, keys, heads, G, d = SHAPES[shape]
    q, k, v = P._packed(sum(new), sum(keys), heads, G, d, dtype, 30 + shape)
    qs, ks = P._starts(new), P._starts(keys)
    first = torch.as_tensor(ks[:-1]).long()
    # a key that some of its tile's rows see and others do not; and one after it
    late = torch.as_tensor(ks[1:]).long() - torch.as_tensor([1 + min(a // 2, b - 1) for a, b in zip(new, keys)])
    later = torch.minimum(late + 1, torch.as_tensor(ks[1:]).long() - 1)
    if what == "first key":
        k[first, 0, 3] = NAN
    elif what == "first value":
        v[first, :, 5] = NAN
    elif what == "first values infinite":
        v[first] = INF
    elif what == "a query":
        q[:: 7, 0, 1] = NAN
    elif what == "all values":
        v[:] = NAN
    elif what == "all values infinite":
        v[:] = -INF
    elif what == "late value":
        v[late, :, 9] = NAN
    elif what == "late infinity":
        v[late, :, 9:12] = -INF
    elif what == "infinity then a later one":
        v[first, :, 2], v[late, :, 2], v[late, :, 3] = INF, INF, INF
    elif what == "NaN then another channel":
        v[first, :, 2], v[late, :, 3], v[late, :, 2] = NAN, NAN, INF
    elif what == "late key":
        k[late, 0, 3] = NAN
    else:
        v[first, :, 4], v[late, :, 4], v[later, :, 6] = INF, -INF, NAN
    P._inside(P._prompt(q, k, v, qs, ks, d ** -0.5), *P._prompt_ref(q, k, v, qs, ks, d ** -0.5))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,nk,G,d", [(600, 600, 4, 128), (5, 4000, 1, 64), (70, 2000, 2, 128)])
def test_keys_of_infinities(dtype, n, nk, G, d):
    # queries whose product with the first key is -inf: that key has no weight, and they are as if it were not there
    q, k, v = P._packed(n, nk, 1, G, d, dtype, n)
    q[:, :, 3] = -q[:, :, 3].abs() - 0.1
    k[0, :, 3] = INF
    y, tol = P._prompt_ref(q, k[1:], v[1:], [0, n], [0, nk - 1], d ** -0.5)
    P._inside(P._prompt(q, k, v, [0, n], [0, nk], d ** -0.5), y, tol)
    q[n // 2] *= -1                                        # and one whose product is +inf
    out = P._prompt(q, k, v, [0, n], [0, nk], d ** -0.5)
    assert out[n // 2].isnan().all()
    rest = torch.arange(n) != n // 2
    P._inside(out[rest], y[rest], tol[rest])


def _time(f):
    f()
    torch.cuda.synchronize()
    best = 1e9
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


# (rows were made again key by key before: hundreds of times the call)
TIMED = [(BF16, 8, 2048, 2048, 8, 4, 128), (BF16, 1, 5, 20005, 8, 1, 128), (F32, 2, 1024, 1024, 8, 4, 128), (F32, 1, 5, 20005, 8, 1, 128)]


@pytest.mark.parametrize("case", range(len(TIMED)))
@pytest.mark.parametrize("what", ["key", "value", "query", "values", "channel"])
def test_rows_without_a_number_take_no_longer(case, what):
    dtype, requests, nq, nk, heads, G, d = TIMED[case]
    g = torch.Generator(device="cuda").manual_seed(case)
    q = torch.randn(requests * nq, heads * G, d, generator=g, device="cuda").to(dtype)
    k, v = (torch.randn(requests * nk, heads, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    qs, ks = (torch.arange(requests + 1, device="cuda", dtype=torch.int32) * n for n in (nq, nk))
    out = torch.empty_like(q)

    def call():
        L.h2o_prompt_attend(q, k, v, qs, ks, d ** -0.5, out)
    clean = _time(call)
    if what == "key":
        k[::nk, :, 3] = NAN
    elif what == "value":
        v[::nk] = NAN
    elif what == "query":
        q[:, :, 1] = NAN
    elif what == "values":
        v[:] = NAN
    else:
        v[::nk, :, 5] = NAN
    # (twice the time is what the second looks may take; three times leaves room for the clocks)
    assert _time(call) <= 3 * clean + 0.02
    odd = out.isnan()
    assert odd.all() if what != "channel" else odd[..., 5].all() and odd.sum() * d == odd.numel()


def test_rows_made_again_for_longer_than_a_second():
    # 128 queries behind 800000 keys, whose last value is no number and seen by the last query alone: the others are made again,
    # which takes longer than any wait of the kernel may, and the other requests are as they should be
    n, new, few, d = 800_000, 128, 400, 64
    g = P._gen(14)
    q = torch.randn(new + few, 1, d, generator=g).to(BF16)
    q[:new] = 0.0
    kv = torch.zeros(2, n + few, 1, d, dtype=BF16, device="cuda")
    v = torch.randn(few, 1, d, generator=g).to(BF16)
    kv[1, :n], kv[1, n:] = 1.5, v.cuda()
    kv[1, n - 1] = NAN
    out = P._prompt(q, kv[0], kv[1], P._starts([new] + [1] * few), P._starts([n] + [1] * few), 0.125).cpu()
    assert out[new - 1].isnan().all() and torch.equal(out[new:], v)
    # 800000 equal weights: sums off by n U at most, 0.05 of them
    assert ((out[:new - 1].float() - 1.5).abs() <= 1.5 * (n * 2.0 ** -24 + 2.0 ** -8)).all()
