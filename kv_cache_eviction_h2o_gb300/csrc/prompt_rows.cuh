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

// The last of the rows 0 .. n - 1 from v on that holds an infinity or a NaN, or -1: by one warp.
template <typename T, int D>
__device__ __noinline__ int last_odd(const T* v, long long stride, int n)
{
    constexpr int E = D / 32, U = 8;
    const int lane = threadIdx.x & 31;
    for (int j = n - 1; j >= 0; j -= U) {
        unsigned odd = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[E];
            load_vec<T, E>(v + (long long)max(j - u, 0) * stride + lane * E, x);
#pragma unroll
            for (int e = 0; e < E; ++e) odd |= fabsf(x[e]) < INFINITY ? 0u : 1u << u;
        }
        odd = __reduce_or_sync(0xffffffffu, odd);
        if (odd) return max(j - (__ffs(odd) - 1), 0);
    }
    return -1;
}

// The request of work index x, by the whole warp: the last i with f(i) = q_start[i] / per + i <= x, or -1.  f's values
// leave room for every tile of `per` positions of a request before the next one's, f(i + 1) - f(i) >= ceil(length / per),
// so x - f(i) is the tile of request i if it has as many, and all requests' tiles are within rows / per + requests.
__device__ __forceinline__ int request_at(const PackedArgs& A, int x, int per)
{
    const int lane = threadIdx.x & 31;
    auto f = [&](int i) { return min(max(A.q_start[i], 0), A.rows) / per + i; };
    int lo = 0, hi = A.requests;
    if (hi > 1 && f(0) > x) return -1;                     // (one request: its caller sees to it)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, i = lo + lane * step;
        const unsigned in = __ballot_sync(0xffffffffu, i < hi && f(i) <= x);
        const int k = in == 0xffffffffu ? 32 : max(1, __ffs(~in) - 1);
        lo += (k - 1) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// CTAs of a cluster that shares a tile's keys: as many as leave all `items` clusters at once on the GPU, per_sm CTAs an
// SM, and each CTA `least` keys.  (A cluster's CTAs are on one group of SMs, of which there are eight: 16 of 7 or more CTAs, or
// 32 of 5, take turns.  5 queries behind 20000 tokens of 8 heads: 138 us with one CTA, 26 with eight, 24 with twelve, 45 with
// sixteen.)
inline int key_cluster(long long items, long long keys, int per_sm, int least)
{
    constexpr int size[] = {16, 12, 8, 6, 4, 3, 2}, fit[] = {7, 8, 15, 22, 36, 48, 76};
    for (int i = 0; i < 7; ++i)
        if (items <= (long long)fit[i] * per_sm && keys >= (long long)least * size[i]) return size[i];
    return 1;
}

}  // namespace h2o
