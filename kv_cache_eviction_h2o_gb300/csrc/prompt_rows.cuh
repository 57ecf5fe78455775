// prompt_rows.cuh -- what the tiled kernels of prompt attention share: one query
// row by one warp on the CUDA cores, which they leave some rows to, and the
// request of a tile.
#pragma once

#include <climits>

#include "common.cuh"
#include "prompts.h"

namespace h2o {

// N channels from p on, 16 bytes or more, as they lie and as fp32
template <typename T, int N> struct Raw {
    static constexpr int W = N * sizeof(T) / 16;
    uint4 w[W];
    __device__ __forceinline__ void load(const T* p)
    {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ float operator[](int e) const
    {
        const uint4 x = w[e * sizeof(T) / 16];
        const int i = e % (16 / (int)sizeof(T)), j = sizeof(T) == 2 ? i / 2 : i;
        const uint32_t y = j == 0 ? x.x : j == 1 ? x.y : j == 2 ? x.z : x.w;
        return __uint_as_float(sizeof(T) == 4 ? y : i & 1 ? y & 0xffff0000u : y << 16);
    }
};

// out = softmax(scale q.k) v over the n keys from k and v on (rows of one
// head, kstride and vstride elements apart), by one warp, and no key beyond them is
// looked at.  Eight lanes take a key, U keys at a time, with a running maximum m
// (base 2) and sums l and o of their own, which are joined at the end.  A row
// all of whose channels are NaN stays so, and is left at that.
template <typename T, int D>
__device__ __noinline__ void prompt_row(const T* q, const T* k, long long kstride, const T* v, long long vstride, int n, float qscale, T* out)
{
    constexpr int E = D / 8, U = 32 / (E * (int)sizeof(T) / 4);        // (32 registers of keys, and as many of values)
    const int lane = threadIdx.x & 31, group = lane >> 3, c = (lane & 7) * E;
    float o[E] = {}, m = -INFINITY, l = 0.f;
    Raw<T, E> x;
    x.load(q + c);
#pragma unroll 1
    for (int j = group; j - group < n; j += 4 * U) {
        Raw<T, E> y[U], w[U];
        float z[U], top = m;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = min(j + 4 * u, n - 1);
            y[u].load(k + at * kstride + c);
            w[u].load(v + at * vstride + c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            z[u] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) z[u] = fmaf(x[e], y[u][e], z[u]);
        }
#pragma unroll
        for (int d = 4; d > 0; d >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u) z[u] += __shfl_xor_sync(0xffffffffu, z[u], d);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            z[u] = j + 4 * u < n ? z[u] * qscale : -INFINITY;
            top = fmaxf(top, z[u]);                        // (a NaN is in l all the same)
        }
        const float base = top == -INFINITY ? 0.f : top, a = ex2_approx(m - base);
        m = top;
        l *= a;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= a;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float p = ex2_approx(z[u] - base);
            const bool in = j + 4 * u < n;
            l += p;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(p, in ? w[u][e] : 0.f, o[e]);
        }
        bool lost = true;                                  // (of this group's keys alone)
#pragma unroll
        for (int e = 0; e < E; ++e) lost = lost && o[e] != o[e];
        const unsigned all = __ballot_sync(0xffffffffu, lost && l > 0.f);
        if (__any_sync(0xffffffffu, l != l) || ((all | all >> 8 | all >> 16 | all >> 24) & 0xffu) == 0xffu) break;
    }
    // the groups' sums: lanes 8 and 16 apart have the same channels
    float top = m;
#pragma unroll
    for (int d = 8; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float a = ex2_approx(m - (top == -INFINITY ? 0.f : top));
    l *= a;
#pragma unroll
    for (int d = 8; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    const float f = 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        float r = o[e] * a;
#pragma unroll
        for (int d = 8; d < 32; d <<= 1) r += __shfl_xor_sync(0xffffffffu, r, d);
        r = l == 0.f ? 0.f : r * f;
        if (e % 4 == group) {
            if constexpr (sizeof(T) == 2) out[c + e] = __float2bfloat16_rn(r);
            else out[c + e] = r;
        }
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

// What a warp has found out about a request's values, a row of results that is no number after the other, so that each
// value is looked at once.  Rows are asked for in ascending order of what they see.
template <int D> struct OddRows {
    static constexpr int E = D / 32;
    int last = -2;                                         // the last value row behind what the first row sees that holds an infinity or a NaN, or -1; -2: not looked for
    int to[2] = {0, 0}, first[2][E];                       // rows looked at, and the first that holds a NaN [0], either [1], in this lane's channels
    int keys = 0, key = INT_MAX;                           // key rows looked at, and the first that holds a NaN
    __device__ __forceinline__ OddRows()
    {
#pragma unroll
        for (int e = 0; e < E; ++e) first[0][e] = first[1][e] = INT_MAX;
    }
};

// Which of this lane's D / 32 channels of a row of results are no number.  (Past the L1, which does not see rows that left as boxes.)
template <typename T, int D>
__device__ __forceinline__ unsigned odd_channels(const T* out)
{
    constexpr int E = D / 32;
    const int at = (threadIdx.x & 31) * E;
    unsigned odd = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if constexpr (sizeof(T) == 2) odd |= (__ldcg(reinterpret_cast<const unsigned short*>(out) + at + e) & 0x7f80u) == 0x7f80u ? 1u << e : 0u;
        else odd |= fabsf(__ldcg(out + at + e)) < INFINITY ? 0u : 1u << e;
    }
    return odd;
}

// Whether a row of results whose weights are numbers is what its own `sees` values make it, where each lane's channels
// `odd` are no number: it stands if each of these has a NaN among them, or (bf16) an infinity or a NaN where none of the
// other values that the products took, up to row `end`, holds either.  (fp32: an infinity's bf16 parts are NaN, so
// its row is to be made again.)
template <typename T, int D>
__device__ __noinline__ bool row_stands(OddRows<D>& R, unsigned odd, const T* v, long long stride, int sees, int end)
{
    constexpr int E = D / 32, U = 16;
    const int lane = threadIdx.x & 31;
    int either = 0;
    if constexpr (sizeof(T) == 2) {
        if (R.last == -2) {
            const int i = last_odd<T, D>(v + sees * stride, stride, end - sees);
            R.last = i < 0 ? -1 : sees + i;
        }
        either = R.last < sees;
    }
    int first[E], to = R.to[either];
    bool stands;
#pragma unroll
    for (int e = 0; e < E; ++e) first[e] = R.first[either][e];
#pragma unroll 1
    for (;; to = min(to + U, sees)) {
        bool left = false;
#pragma unroll
        for (int e = 0; e < E; ++e) left |= (odd >> e & 1u) && first[e] >= sees;
        stands = !__any_sync(0xffffffffu, left);
        if (stands || to >= sees) break;
        float x[U][E];
#pragma unroll
        for (int u = 0; u < U; ++u) load_vec<T, E>(v + min(to + u, sees - 1) * stride + lane * E, x[u]);
        bool any = false;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) any |= !(fabsf(x[u][e]) < INFINITY);
        if (!any) continue;
#pragma unroll
        for (int u = U - 1; u >= 0; --u)
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (either ? !(fabsf(x[u][e]) < INFINITY) : x[u][e] != x[u][e]) first[e] = min(first[e], min(to + u, sees - 1));
    }
#pragma unroll
    for (int e = 0; e < E; ++e) R.first[either][e] = first[e];
    R.to[either] = to;
    return stands;
}

// Whether the query or one of the first `sees` keys holds a NaN, which makes a row NaN as a whole.
template <typename T, int D>
__device__ __noinline__ bool nan_logit(OddRows<D>& R, const T* q, const T* k, long long stride, int sees)
{
    constexpr int E = D / 32, U = 16;
    const int lane = threadIdx.x & 31;
    float x[U][E];
    load_vec<T, E>(q + lane * E, x[0]);
    bool none = false;
#pragma unroll
    for (int e = 0; e < E; ++e) none |= x[0][e] != x[0][e];
    if (__any_sync(0xffffffffu, none)) return true;
    for (; R.key >= sees && R.keys < sees; R.keys = min(R.keys + U, sees)) {
#pragma unroll
        for (int u = 0; u < U; ++u) load_vec<T, E>(k + min(R.keys + u, sees - 1) * stride + lane * E, x[u]);
        int at = INT_MAX;
#pragma unroll
        for (int u = U - 1; u >= 0; --u)
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (x[u][e] != x[u][e]) at = min(R.keys + u, sees - 1);
        R.key = __reduce_min_sync(0xffffffffu, at);
    }
    return R.key < sees;
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
