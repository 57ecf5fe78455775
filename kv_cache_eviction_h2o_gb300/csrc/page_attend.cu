// page_attend.cu -- attention of query rows over the pages of their requests:
// over the pages a cheap score picks (h2o_page_attend), or over all of a
// request's own pages, joined with what a shared prefix gave
// (h2o_prefix_attend).
//
// Work unit: one query row of one cache head, its G query heads together, so
// a page is read once for all of them.  Picking, per unit:
//   s_b = sum_e w+_e max_be + w-_e min_be,  w+ = sum_g max(q_g, 0),
//                                           w- = sum_g min(q_g, 0)
// is the sum over the heads of the largest q_g . k that a key within page b's
// bounds can have; summing the queries first makes it one product of length
// 2 D a page whatever G is.  The page ranks are those of the exact s: scores
// are made in fp32, whose error is at most eps = 2^-18 max_b sum |w||bound|
// (at most 32 fused multiply-adds a lane, 3 adds, 15 adds in w: 50 roundings
// of 2^-24), a page more than 2 eps from the k-th largest is decided by that,
// and the few nearer ones are scored again in fp64 and ranked by that, ties
// to the lowest page.
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "paged.h"

namespace h2o {

namespace {

constexpr int kWarps = 4;              // warps of a CTA
constexpr int kNT = kWarps * 32;
constexpr int kKeys = 16;              // keys of a tile (page sizes are its multiples)
constexpr float kEps = 3.814697e-6f;   // 2^-18
// tiles in flight per warp
template <typename T> constexpr int kStages = sizeof(T) == 2 ? 3 : 2;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool fill)
{
    // bytes not read are written as zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(fill ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void cluster_max_u32(uint32_t addr, uint32_t v)
{
    asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// A tile holds 16 rows of D elements; 16-byte chunk c of row r lies at chunk
// c ^ (r & 7), so 8 rows of one column, as well as one row, are free of bank
// conflicts.
template <typename T, int D>
__device__ __forceinline__ uint32_t tile_at(int row, int byte)
{
    return (uint32_t)(row * D * (int)sizeof(T) + (byte ^ ((row & 7) << 4)));
}

// -------------------------------------------------------------- picking

struct PickSmem {
    int warp_i[2][kWarps];
    unsigned warp_u[2][kWarps];
    unsigned amax;                     // bits of the largest sum |w||bound| (of the whole cluster)
};

// sum over the CTA, in every thread
__device__ __forceinline__ int cta_sum(PickSmem& P, int v, int& phase)
{
    v = __reduce_add_sync(0xffffffffu, v);
    phase ^= 1;
    if ((threadIdx.x & 31) == 0) P.warp_i[phase][threadIdx.x >> 5] = v;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += P.warp_i[phase][w];
    return s;
}
__device__ __forceinline__ unsigned cta_min(PickSmem& P, unsigned v, int& phase)
{
    v = __reduce_min_sync(0xffffffffu, v);
    phase ^= 1;
    if ((threadIdx.x & 31) == 0) P.warp_u[phase][threadIdx.x >> 5] = v;
    __syncthreads();
    unsigned s = ~0u;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s = min(s, P.warp_u[phase][w]);
    return s;
}

// order-preserving map of an fp64 value to an unsigned key; NaN above all
__device__ __forceinline__ unsigned long long ord_key64(double x)
{
    if (x != x) return ~0ull;
    if (x == 0.0) x = 0.0;                                 // -0 and 0 are one score
    const unsigned long long b = (unsigned long long)__double_as_longlong(x);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
__device__ __forceinline__ float ord_value(unsigned k)
{
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// Leaves s[j] >= the returned bound exactly for the `take` best of the n
// pages' scores s (0 < take < n).  `again(j)` is page j's score in fp64, made
// by a whole warp.  big: room for n keys of 64 bits; s may be overwritten.
template <class Again>
__device__ float pick_bound(PickSmem& P, float* s, int n, int take, unsigned long long* big, Again again)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int ph = 0;
    const float amax = __uint_as_float(P.amax);
    float above = INFINITY, below = -INFINITY;             // decided: s > above is in, s < below is out
    int in = 0;                                            // pages decided to be in
    if (amax < FLT_MAX) {                                  // (an infinity or NaN among the factors decides nothing)
        unsigned lo = ~0u, hi = 0u;
        for (int j = tid; j < n; j += kNT) {
            const unsigned k = ord_key(s[j]);
            lo = min(lo, k);
            hi = max(hi, k);
        }
        lo = cta_min(P, lo, ph);
        hi = ~cta_min(P, ~hi, ph);
        // the largest key that `take` keys reach
        while (lo < hi) {
            const unsigned mid = lo + (hi - lo) / 2 + 1;
            int c = 0;
            for (int j = tid; j < n; j += kNT) c += ord_key(s[j]) >= mid;
            c = cta_sum(P, c, ph);
            if (c >= take) lo = mid; else hi = mid - 1;
            if (c == take) break;
        }
        unsigned kth = ~0u;
        for (int j = tid; j < n; j += kNT) {
            const unsigned k = ord_key(s[j]);
            if (k >= lo) kth = min(kth, k);
        }
        const float t = ord_value(cta_min(P, kth, ph)), e2 = __fmaf_ru(2.f * kEps, amax, 1e-37f);
        above = __fadd_ru(t, e2);
        below = __fadd_rd(t, -e2);
        int c = 0;                                         // (in, in or open)
        for (int j = tid; j < n; j += kNT) c += (s[j] > above ? 1 : 0) + (s[j] >= below ? 1 << 16 : 0);
        c = cta_sum(P, c, ph);
        in = c & 0xffff;
        if ((c >> 16) == take) return below;
    }
    // the open pages by their fp64 scores
    for (int j = warp; j < n; j += kWarps) {
        const float x = s[j];
        const bool open = !(x > above) && !(x < below);
        unsigned long long key = 0;
        if (open) key = ord_key64(again(j));
        if (lane == 0) big[j] = open ? key : 0ull;         // no score has key 0
    }
    __syncthreads();
    const int want = take - in;
    unsigned long long lo = 0, hi = ~0ull;                 // the largest key that `want` open pages reach
    while (lo < hi) {
        const unsigned long long mid = lo + (hi - lo) / 2 + 1;
        int c = 0;
        for (int j = tid; j < n; j += kNT) c += big[j] >= mid;
        if (cta_sum(P, c, ph) >= want) lo = mid; else hi = mid - 1;
    }
    int c = 0;
    for (int j = tid; j < n; j += kNT) c += big[j] > lo;
    const int ties = want - cta_sum(P, c, ph);             // of the pages with just that key, the first ones
    int jl = 0, jh = n - 1;                                // the smallest j up to which there are `ties` of them
    while (jl < jh) {
        const int mid = (jl + jh) / 2;
        c = 0;
        for (int j = tid; j <= mid; j += kNT) c += big[j] == lo;
        if (cta_sum(P, c, ph) >= ties) jh = mid; else jl = mid + 1;
    }
    for (int j = tid; j < n; j += kNT) {
        const unsigned long long k = big[j];
        const bool is_in = k == 0 ? s[j] > above : k > lo || (k == lo && j <= jl);
        s[j] = is_in ? 1.f : -1.f;
    }
    __syncthreads();
    return 0.f;
}

// ------------------------------------------------------------ attention core

// One warp's running softmax over its tiles on the CUDA cores: lane = key
// (lane & 15) and half of D for the logits, D / 32 channels for the values.
template <typename T, int D, int GP>
struct CoreSimt {
    static constexpr int E = D / 32;
    float o[GP][E], m[GP], l[GP];

    __device__ __forceinline__ void init()
    {
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            m[g] = -INFINITY;
            l[g] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[g][e] = 0.f;
        }
    }

    __device__ __forceinline__ void tile(const unsigned char* kt, const unsigned char* vt, int valid, const float* q,
                                         float* pb, float qscale, int lane)
    {
        constexpr int N = 16 / sizeof(T);
        const int key = lane & 15, half = lane >> 4;
        float z[GP];
#pragma unroll
        for (int g = 0; g < GP; ++g) z[g] = 0.f;
#pragma unroll 4
        for (int c = 0; c < D / 2 / N; ++c) {
            const int d0 = half * (D / 2) + c * N;
            float kf[N];
            load_vec<T, N>(reinterpret_cast<const T*>(kt + tile_at<T, D>(key, d0 * (int)sizeof(T))), kf);
#pragma unroll
            for (int g = 0; g < GP; ++g)
#pragma unroll
                for (int i = 0; i < N; i += 4) {
                    const float4 w = *reinterpret_cast<const float4*>(q + g * D + d0 + i);
                    z[g] = fmaf(w.x, kf[i], z[g]);
                    z[g] = fmaf(w.y, kf[i + 1], z[g]);
                    z[g] = fmaf(w.z, kf[i + 2], z[g]);
                    z[g] = fmaf(w.w, kf[i + 3], z[g]);
                }
        }
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            z[g] = (z[g] + __shfl_xor_sync(0xffffffffu, z[g], 16)) * qscale;
            if (key >= valid) z[g] = -INFINITY;
            float t = z[g];
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
            const float mn = fmaxf(m[g], t), base = mn == -INFINITY ? 0.f : mn;
            const float a = ex2_approx(m[g] - base), p = ex2_approx(z[g] - base);
            m[g] = mn;
            l[g] = l[g] * a + (half ? 0.f : p);
#pragma unroll
            for (int e = 0; e < E; ++e) o[g][e] *= a;
            if (!half) pb[g * kKeys + key] = p;
        }
        __syncwarp();
#pragma unroll
        for (int k0 = 0; k0 < kKeys; k0 += 4) {
            float v[4][E];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const unsigned char* a = vt + tile_at<T, D>(k0 + i, lane * E * (int)sizeof(T));
                if constexpr (sizeof(T) == 2 || E == 4) load_vec<T, E>(reinterpret_cast<const T*>(a), v[i]);
                else {
                    const float2 w = *reinterpret_cast<const float2*>(a);
                    v[i][0] = w.x;
                    v[i][1] = w.y;
                }
            }
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                const float4 p = *reinterpret_cast<const float4*>(pb + g * kKeys + k0);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    o[g][e] = fmaf(p.x, v[0][e], o[g][e]);
                    o[g][e] = fmaf(p.y, v[1][e], o[g][e]);
                    o[g][e] = fmaf(p.z, v[2][e], o[g][e]);
                    o[g][e] = fmaf(p.w, v[3][e], o[g][e]);
                }
            }
        }
        __syncwarp();
    }

    // o to out [GP][D], (m, l) to ml [GP]
    __device__ __forceinline__ void finish(float* out, float2* ml, int lane, bool bad)
    {
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            const float s = warp_sum(l[g]);
#pragma unroll
            for (int e = 0; e < E; ++e) out[g * D + lane * E + e] = o[g][e];
            if (lane == 0) ml[g] = make_float2(m[g], bad ? NAN : s);
        }
    }
};

template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename T, int D, int GP>
struct alignas(16) AttendSmem {
    double w64[2 * D];                 // the page weights, minima's then maxima's
    float w[2 * D];
    float q[GP * D];                   // the queries; later this CTA's sum of values
    float p[kWarps][GP * kKeys];
    float2 wml[kWarps][GP];
    float2 ml[GP];
    PickSmem pick;
};

// Shared memory: the warps' rings (fp64 keys while picking), AttendSmem, and
// when picking the scores and the picked pages.
template <typename T, int D> constexpr int kTileBytes = kKeys * D * (int)sizeof(T);
template <typename T, int D> constexpr int kRingBytes = kStages<T> * 2 * kTileBytes<T, D>;   // a warp's

template <typename T, int D, int GP>
__global__ void __launch_bounds__(kNT) page_attend_kernel(const PagePool pool, const PageRows R, const int budget,
                                                          const int recent, int* __restrict__ picked,
                                                          const PrefixPart part, const int front, const int wpad)
{
    extern __shared__ __align__(128) unsigned char raw[];
    using S_t = AttendSmem<T, D, GP>;
    constexpr int NS = kStages<T>, TB = kTileBytes<T, D>;
    S_t& S = *reinterpret_cast<S_t*>(raw + front);
    float* scores = reinterpret_cast<float*>(raw + front + sizeof(S_t));
    int* list = reinterpret_cast<int*>(scores + wpad);
    unsigned long long* big = reinterpret_cast<unsigned long long*>(raw);
    unsigned char* ring = raw + (threadIdx.x >> 5) * kRingBytes<T, D>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
    const int u = blockIdx.x / C, row = u / pool.heads, h = u - row * pool.heads;
    const int seq = R.seq[row];
    if (seq < 0) return;                                   // a row that is not there, for the whole cluster
    const int pos = R.pos[row];
    const int sh = __ffs(pool.ps) - 1;
    const int G = R.G;
    int npages = pos < 0 ? 0 : (pos >> sh) + 1;
    bool bad = seq >= R.requests || npages > R.width;
    if (bad) npages = 0;
    const int* table = R.table + (size_t)(bad ? 0 : seq) * R.width;
    const T* qrow = static_cast<const T*>(R.q) + (size_t)row * R.q_stride + (size_t)h * G * D;
    for (int i = tid; i < GP * D; i += kNT) S.q[i] = i < G * D ? Elem<T>::to_f(qrow[i]) : 0.f;
    if (tid == 0) S.pick.amax = 0u;
    __syncthreads();

    int nlist = npages;
    const int* src = table;                                // physical page of each entry
    const int ncand = npages - recent, take = budget - recent;
    if (budget > 0 && npages > budget) {
        for (int i = tid; i < 2 * D; i += kNT) {
            double s = 0.0;
            float f = 0.f;
            const bool lo = i < D;
            for (int g = 0; g < G; ++g) {
                const float x = S.q[g * D + (lo ? i : i - D)];
                const float y = lo ? (x < 0.f || x != x ? x : 0.f) : (x > 0.f || x != x ? x : 0.f);
                s += (double)y;
                f += y;
            }
            S.w64[i] = s;
            S.w[i] = f;
        }
        __syncthreads();
        cluster_arrive();
        cluster_wait();                                    // every CTA has set its maximum
        constexpr int N = 16 / sizeof(T), NV = 2 * D / 8 / N;
        const T* bounds = static_cast<const T*>(pool.bounds);
        // eight lanes a page, four pages a warp
        float w[NV][N];
        const int sub = lane & 7;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) w[i][e] = S.w[(i * 8 + sub) * N + e];
        unsigned amax = 0u;
        for (int j0 = (rank * kWarps + warp) * 4; j0 < ncand; j0 += C * kWarps * 4) {
            const int j = j0 + (lane >> 3);
            const int pg = j < ncand ? table[j] : 0;
            const bool ok = (unsigned)pg < (unsigned)pool.pages;
            const T* b = bounds + ((size_t)(ok ? pg : 0) * pool.heads + h) * 2 * D;
            float s = 0.f, a = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float x[N];
                load_vec<T, N>(b + (i * 8 + sub) * N, x);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    s = fmaf(w[i][e], x[e], s);
                    a = fmaf(fabsf(w[i][e]), fabsf(x[e]), a);
                }
            }
#pragma unroll
            for (int d = 4; d > 0; d >>= 1) {
                s += __shfl_xor_sync(0xffffffffu, s, d);
                a += __shfl_xor_sync(0xffffffffu, a, d);
            }
            if (!ok) { s = NAN; a = NAN; }                 // no such page: picked, and its row is NaN
            if (j < ncand) {
                amax = max(amax, __float_as_uint(fabsf(a)));
                for (int c = sub; c < C; c += 8) st_cluster_f32(map_to_rank(scores + j, c), s);
            }
        }
        amax = __reduce_max_sync(0xffffffffu, amax);
        if (lane < C) cluster_max_u32(map_to_rank(&S.pick.amax, lane), amax);
        cluster_arrive();
        cluster_wait();
        const float bound = pick_bound(S.pick, scores, ncand, take, big, [&](int j) {
            const int pg = table[j];
            if ((unsigned)pg >= (unsigned)pool.pages) return (double)NAN;
            const T* b = bounds + ((size_t)pg * pool.heads + h) * 2 * D;
            double s = 0.0;
            if (__uint_as_float(S.pick.amax) < FLT_MAX) {
                for (int e = lane; e < 2 * D; e += 32) s += S.w64[e] * (double)Elem<T>::to_f(b[e]);
            } else {
                // an infinite bound on the side that no query takes counts for nothing: the maxima themselves
                for (int e = lane; e < D; e += 32)
                    for (int g = 0; g < G; ++g) {
                        const double x = S.q[g * D + e], y0 = x * (double)Elem<T>::to_f(b[e]), y1 = x * (double)Elem<T>::to_f(b[D + e]);
                        s += y0 != y0 || y1 != y1 ? (double)NAN : fmax(y0, y1);
                    }
            }
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            return s;
        });
        // the picked pages in order: each thread takes a run of pages
        const int per = (ncand + kNT - 1) / kNT, j0 = min(ncand, tid * per), j1 = min(ncand, j0 + per);
        int c = 0;
        for (int j = j0; j < j1; ++j) c += scores[j] >= bound;
        int before = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= d) before += x;
        }
        __syncthreads();
        if (lane == 31) S.pick.warp_i[0][warp] = before;
        __syncthreads();
        before -= c;
        for (int k = 0; k < warp; ++k) before += S.pick.warp_i[0][k];
        int* pick_out = picked && rank == 0 ? picked + (size_t)u * budget : nullptr;
        for (int j = j0; j < j1; ++j)
            if (scores[j] >= bound) {
                list[before] = table[j];
                if (pick_out) pick_out[before] = j;
                ++before;
            }
        for (int j = tid; j < recent; j += kNT) {
            list[take + j] = table[ncand + j];
            if (pick_out) pick_out[take + j] = ncand + j;
        }
        __syncthreads();
        nlist = budget;
        src = list;
    } else if (picked && rank == 0) {
        for (int j = tid; j < budget; j += kNT) picked[(size_t)u * budget + j] = j < npages ? j : -1;
    }

    // tiles of 16 keys, dealt to the warps of the cluster in turn
    const int tsh = sh - 4;                                // log2 of the tiles of a page
    const int ntiles = nlist ? ((nlist - 1) << tsh) + ((pos & (pool.ps - 1)) >> 4) + 1 : 0;
    const int stride = C * kWarps;
    const int t0 = rank * kWarps + warp;
    CoreSimt<T, D, GP> core;
    core.init();
    const T* K = static_cast<const T*>(pool.K);
    const T* V = static_cast<const T*>(pool.V);
    auto valid_of = [&](int t) {                           // keys of tile t up to pos
        return t == ntiles - 1 ? (pos & 15) + 1 : kKeys;
    };
    int pg_next = t0 < ntiles ? src[t0 >> tsh] : 0;        // the page of the next tile to be asked for
    auto ask = [&](int t, int stage) {
        if (t < ntiles) {
            const int pg = pg_next;
            const bool ok = (unsigned)pg < (unsigned)pool.pages;
            if (!ok) bad = true;
            const int valid = ok ? valid_of(t) : 0;
            const size_t off = (((size_t)(ok ? pg : 0) * pool.heads + h) * pool.ps + ((size_t)(t & ((1 << tsh) - 1)) << 4)) * D;
            constexpr int CH = D * (int)sizeof(T) / 16;
            const uint32_t kd = smem_u32(ring + 2 * stage * TB), vd = kd + TB;
#pragma unroll
            for (int i = lane; i < kKeys * CH; i += 32) {
                const int r = i / CH, c = i % CH;
                const bool fill = r < valid;               // keys past the newest are not read: zeros
                const size_t o = off + (fill ? (size_t)r * D + c * (16 / sizeof(T)) : 0);
                cp_async16(kd + tile_at<T, D>(r, c * 16), K + o, fill);
                cp_async16(vd + tile_at<T, D>(r, c * 16), V + o, fill);
            }
            if (t + stride < ntiles) pg_next = src[(t + stride) >> tsh];
        }
        cp_commit();
    };
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) ask(t0 + s * stride, s);
    int stage = 0;
    for (int t = t0; t < ntiles; t += stride) {
        ask(t + (NS - 1) * stride, stage == 0 ? NS - 1 : stage - 1);
        cp_wait<NS - 1>();
        __syncwarp();
        core.tile(ring + 2 * stage * TB, ring + 2 * stage * TB + TB, valid_of(t), S.q, S.p[warp], R.qscale, lane);
        stage = stage + 1 == NS ? 0 : stage + 1;
    }
    cp_wait<0>();
    __syncwarp();

    // the warps' sums, then the CTAs', then the prefix's
    float* wo = reinterpret_cast<float*>(ring);
    static_assert(kRingBytes<T, D> >= (int)sizeof(float) * GP * D, "a warp's sums lie in its ring");
    core.finish(wo, S.wml[warp], lane, bad);
    __syncthreads();
    for (int i = tid; i < GP * D; i += kNT) {
        const int g = i / D;
        float m = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, S.wml[w][g].x);
        const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float a = ex2_approx(S.wml[w][g].x - base);
            l += a * S.wml[w][g].y;
            o = fmaf(a, reinterpret_cast<const float*>(raw + w * kRingBytes<T, D>)[i], o);
        }
        S.q[i] = o;
        if (i % D == 0) S.ml[g] = make_float2(m, l);
    }
    cluster_arrive();
    cluster_wait();
    T* orow = static_cast<T*>(R.out) + (size_t)row * R.out_stride + (size_t)h * G * D;
    const size_t qrows = (size_t)R.rows * pool.heads * G, qr = (size_t)u * G;
    for (int i = rank * kNT + tid; i < G * D; i += C * kNT) {
        const int g = i / D;
        float m = -INFINITY, l = 0.f, o = 0.f;
        for (int c = 0; c < C; ++c) m = fmaxf(m, ld_cluster_f32(map_to_rank(&S.ml[g].x, c)));
        for (int s = 0; s < part.splits; ++s) m = fmaxf(m, part.ml[s * qrows + qr + g].x);
        const float base = m == -INFINITY ? 0.f : m;
        for (int c = 0; c < C; ++c) {
            const float a = ex2_approx(ld_cluster_f32(map_to_rank(&S.ml[g].x, c)) - base);
            l += a * ld_cluster_f32(map_to_rank(&S.ml[g].y, c));
            o = fmaf(a, ld_cluster_f32(map_to_rank(&S.q[i], c)), o);
        }
        for (int s = 0; s < part.splits; ++s) {
            const float2 x = part.ml[s * qrows + qr + g];
            const float a = ex2_approx(x.x - base);
            l += a * x.y;
            o = fmaf(a, part.o[(s * qrows + qr) * D + i], o);
        }
        // no key at all: zero; a bad table entry has made l NaN
        orow[i] = from_f<T>(l == 0.f ? 0.f : o / l);
    }
    cluster_arrive();
    cluster_wait();                                        // no CTA leaves while another reads its sums
}

template <typename T, int D, int GP>
cudaError_t go(const PagePool& p, const PageRows& r, int budget, int recent, int* picked, const PrefixPart& part, cudaStream_t st)
{
    const bool picks = budget > 0 && budget < r.width;
    const int wpad = picks ? (r.width + 3) & ~3 : 0;
    const int front = std::max(kWarps * kRingBytes<T, D>, 8 * wpad);
    const size_t smem = front + sizeof(AttendSmem<T, D, GP>) + 4 * ((size_t)wpad + (picks ? budget : 0));
    const auto kernel = page_attend_kernel<T, D, GP>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int C = 1;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)r.rows * p.heads * C));
    cfg.blockDim = dim3(kNT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, r, budget, recent, picked, part, front, wpad);
}

template <typename T, int D>
cudaError_t by_groups(const PagePool& p, const PageRows& r, int budget, int recent, int* picked, const PrefixPart& part, cudaStream_t st)
{
    if (r.G == 1) return go<T, D, 1>(p, r, budget, recent, picked, part, st);
    if (r.G <= 4) return go<T, D, 4>(p, r, budget, recent, picked, part, st);
    if (r.G <= 8) return go<T, D, 8>(p, r, budget, recent, picked, part, st);
    return go<T, D, 16>(p, r, budget, recent, picked, part, st);
}

}  // namespace

cudaError_t launch_page_attend(const PagePool& p, const PageRows& r, int budget, int recent, int* picked,
                               const PrefixPart& part, cudaStream_t st)
{
    if (p.dtype)
        return p.D == 64 ? by_groups<__nv_bfloat16, 64>(p, r, budget, recent, picked, part, st)
                         : by_groups<__nv_bfloat16, 128>(p, r, budget, recent, picked, part, st);
    return p.D == 64 ? by_groups<float, 64>(p, r, budget, recent, picked, part, st)
                     : by_groups<float, 128>(p, r, budget, recent, picked, part, st);
}

}  // namespace h2o
