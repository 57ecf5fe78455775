// prompt_rows.cuh -- what the tiled kernels of prompt attention share: one query
// row by one warp on the CUDA cores, which they leave some rows to, and the
// request of a tile.
#pragma once

#include "common.cuh"
#include "prompts.h"

namespace h2o {

// out = softmax(scale q.k) v over the n keys from k and v on (rows of one
// head, kstride and vstride elements apart): a running maximum m (base 2) and sum l,
// keys one after another, and no key beyond them is looked at.
template <typename T, int D>
__device__ __noinline__ void prompt_row(const T* q, const T* k, long long kstride, const T* v, long long vstride, int n, float qscale, T* out)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    float x[E], o[E] = {}, m = -INFINITY, l = 0.f;
    load_vec<T, E>(q + lane * E, x);
    for (int j = 0; j < n; ++j) {
        float y[E], w[E], z = 0.f;
        load_vec<T, E>(k + j * kstride + lane * E, y);
        load_vec<T, E>(v + j * vstride + lane * E, w);
#pragma unroll
        for (int e = 0; e < E; ++e) z = fmaf(x[e], y[e], z);
        z = warp_sum(z) * qscale;
        const float mn = z > m || z != z ? z : m, base = mn == -INFINITY ? 0.f : mn;
        const float a = ex2_approx(m - base), p = ex2_approx(z - base);
        m = mn;
        l = fmaf(l, a, p);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(p, w[e], o[e] * a);
    }
    const float f = 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float r = l == 0.f ? 0.f : o[e] * f;
        if constexpr (sizeof(T) == 2) out[lane * E + e] = __float2bfloat16_rn(r);
        else out[lane * E + e] = r;
    }
}

// The request of work index x, by the whole warp: the last i with f(i) = q_start[i] / per + i <= x, or -1.  f's values
// leave room for every tile of `per` positions of a request before the next one's, f(i + 1) - f(i) >= ceil(length / per),
// so x - f(i) is the tile of request i if it has as many, and all requests' tiles are within rows / per + requests.
__device__ __forceinline__ int request_at(const PackedArgs& A, int x, int per)
{
    const int lane = threadIdx.x & 31;
    auto f = [&](int i) { return min(max(A.q_start[i], 0), A.rows) / per + i; };
    int lo = 0, hi = A.requests;
    if (f(0) > x) return -1;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, i = lo + lane * step;
        const unsigned in = __ballot_sync(0xffffffffu, i < hi && f(i) <= x);
        const int k = in == 0xffffffffu ? 32 : max(1, __ffs(~in) - 1);
        lo += (k - 1) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

}  // namespace h2o
