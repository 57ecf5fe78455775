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
// are made in fp32, whose error is at most eps = 24 * 2^-24 sum |w| max |bound|
// (two chains of 16 fused multiply-adds a lane, 4 adds, one rounding of w: 21
// roundings; the bound's own are far below the rest), a page more than 2 eps from the k-th largest is decided by that,
// and the few nearer ones are scored again in fp64 and ranked by that, ties
// to the lowest page.
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "paged.h"

namespace h2o {

namespace {

constexpr int kKeys = 16;              // keys of a tile (page sizes are its multiples)
constexpr float kEps = 1.4305115e-6f;  // 24 * 2^-24
// tiles in flight per warp
template <typename T> constexpr int kStages = sizeof(T) == 2 ? 3 : 2;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool fill)
{
    // bytes not read are written as zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(fill ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

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

// A sum of fp32 values of one sign as three fp32 parts: each addition's rounding
// error goes to the next part, exactly (TwoSum), and the third's is below 2^-70
// of the sum for 16 values, of which fp64 keeps 2^-53.
struct Sum3 {
    float hi = 0.f, mid = 0.f, lo = 0.f;
    __device__ __forceinline__ static float2 two_sum(float a, float b)
    {
        const float s = a + b, bp = s - a;
        return make_float2(s, (a - (s - bp)) + (b - bp));
    }
    __device__ __forceinline__ void add(float x)
    {
        const float2 h = two_sum(hi, x), m = two_sum(mid, h.y);
        hi = h.x;
        mid = m.x;
        lo += m.y;
    }
    // the sum rounded to fp32, and what that leaves
    __device__ __forceinline__ float2 rounded() const { return two_sum(hi, mid); }
};

// the largest |x| of 16-byte vectors, NaN where one is
template <typename T> struct AbsMax;
template <> struct AbsMax<__nv_bfloat16> {
    uint32_t m = 0u;
    __device__ __forceinline__ void take(uint4 v, bool on)
    {
        const uint32_t mask = on ? 0x7fff7fffu : 0u;
        const uint32_t x[4] = {v.x & mask, v.y & mask, v.z & mask, v.w & mask};
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x[i]));
    }
    __device__ __forceinline__ float value() const
    {
        float a = __uint_as_float(m << 16), b = __uint_as_float(m & 0xffff0000u);
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
        return a;
    }
};
template <> struct AbsMax<float> {
    float m = 0.f;
    __device__ __forceinline__ void take(uint4 v, bool on)
    {
        const uint32_t mask = on ? 0x7fffffffu : 0u;
        const uint32_t x[4] = {v.x & mask, v.y & mask, v.z & mask, v.w & mask};
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(__uint_as_float(x[i])));
    }
    __device__ __forceinline__ float value() const { return m; }
};

constexpr int kHold = 16;              // scores a thread keeps in registers
constexpr int kFew = 32;               // open pages that are ranked one against another

template <int NW>
struct PickSmem {
    unsigned long long warp[2][NW];
    unsigned long long key[kFew];      // the open pages' fp64 scores, and which they are
    int at[kFew];
    int n_open;
    unsigned amax;                     // bits of sum |w| times the largest |bound| (of the whole cluster)
    int taken[NW];                     // picked pages of each warp's range
    unsigned mark[kMaxTableWidth / 32];   // which pages are picked
};

// sum over the CTA, in every thread; halves of 32 bits do not carry
template <int NW>
__device__ __forceinline__ unsigned long long cta_sum(PickSmem<NW>& P, unsigned lo, unsigned hi, int& phase)
{
    lo = __reduce_add_sync(0xffffffffu, lo);
    hi = __reduce_add_sync(0xffffffffu, hi);
    phase ^= 1;
    if ((threadIdx.x & 31) == 0) P.warp[phase][threadIdx.x >> 5] = (unsigned long long)hi << 32 | lo;
    __syncthreads();
    unsigned long long s = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) s += P.warp[phase][w];
    return s;
}
// (smallest a, largest b) over the CTA
template <int NW>
__device__ __forceinline__ uint2 cta_range(PickSmem<NW>& P, unsigned a, unsigned b, int& phase)
{
    a = __reduce_min_sync(0xffffffffu, a);
    b = __reduce_max_sync(0xffffffffu, b);
    phase ^= 1;
    if ((threadIdx.x & 31) == 0) P.warp[phase][threadIdx.x >> 5] = (unsigned long long)b << 32 | a;
    __syncthreads();
    a = ~0u;
    b = 0u;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        a = min(a, (unsigned)P.warp[phase][w]);
        b = max(b, (unsigned)(P.warp[phase][w] >> 32));
    }
    return make_uint2(a, b);
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

// f(key) for this thread's pages: from registers while all scores fit them (1900 pages: 2.1 us of search, 3.2 from
// shared memory)
template <int NT>
struct Held {
    unsigned k[kHold];
    const float* s;
    int n;
    __device__ __forceinline__ Held(const float* s_, int n_) : s(s_), n(n_)
    {
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int j = (int)threadIdx.x + i * NT;
            k[i] = j < n ? ord_key(s[j]) : 0u;             // (0: below every score)
        }
    }
    template <class F> __device__ __forceinline__ void each(F f) const
    {
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            if (i * NT >= n) break;
            f(k[i]);
        }
        for (int j = threadIdx.x + kHold * NT; j < n; j += NT) f(ord_key(s[j]));
    }
};

// Leaves s[j] >= the returned bound exactly for the `take` best of the n
// pages' scores s (0 < take < n).  `again(j)` is page j's score in fp64, made
// by a whole warp, after `wide` and a barrier.  big: room for n keys of 64 bits; s may be overwritten,
// after `settle`, which is called once.
template <int NW, class Settle, class Wide, class Again>
__device__ float pick_bound(PickSmem<NW>& P, float* s, int n, int take, unsigned long long* big, Settle settle, Wide wide, Again again)
{
    constexpr int NT = NW * 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int ph = 0;
    const float amax = __uint_as_float(P.amax);
    float above = INFINITY, below = -INFINITY;             // decided: s > above is in, s < below is out
    int in = 0;                                            // pages decided to be in
    if (amax < FLT_MAX / 2) {                              // (an infinity or NaN among the factors, or a sum, decides nothing)
        const Held<NT> held(s, n);
        unsigned a = ~0u, b = 0u;
        held.each([&](unsigned k) { a = min(a, k ? k : ~0u); b = max(b, k); });
        const uint2 r = cta_range(P, a, b, ph);
        // count(key >= lo) >= take > count(key >= hi): three keys between them a step
        unsigned long long lo = r.x, hi = (unsigned long long)r.y + 1;
        while (hi - lo > 1) {
            const unsigned long long gap = hi - lo;
            const unsigned k1 = (unsigned)(lo + max(1ull, gap / 4)), k2 = (unsigned)(lo + max(1ull, gap / 2)),
                           k3 = (unsigned)(lo + max(1ull, gap - gap / 4 - (gap < 4 ? 1 : 0)));
            unsigned c1 = 0, c2 = 0, c3 = 0;
            held.each([&](unsigned k) { c1 += k >= k1; c2 += k >= k2; c3 += k >= k3; });
            const unsigned long long c = cta_sum(P, c1 | c2 << 16, c3, ph);
            const int n1 = (int)(c & 0xffff), n2 = (int)(c >> 16 & 0xffff), n3 = (int)(c >> 32);
            if (n3 >= take) lo = k3;
            else if (n2 >= take) { lo = k2; hi = k3; }
            else if (n1 >= take) { lo = k1; hi = k2; }
            else hi = k1;
            if (n1 == take || n2 == take || n3 == take) {
                lo = n1 == take ? k1 : n2 == take ? k2 : k3;   // just the best: the border lies below the smallest of them
                break;
            }
        }
        settle();
        a = ~0u;                                           // the take-th score
        held.each([&](unsigned k) { if (k >= lo) a = min(a, k); });
        const float t = ord_value(cta_range(P, a, 0u, ph).x), e2 = __fmaf_ru(2.f * kEps, amax, 1e-37f);
        above = __fadd_ru(t, e2);
        below = __fadd_rd(t, -e2);
        unsigned ci = 0, co = 0;                           // in; in or open
        const unsigned ka = ord_key(above), kb = ord_key(below);
        held.each([&](unsigned k) { ci += k > ka; co += k >= kb; });
        const unsigned long long c = cta_sum(P, ci, co, ph);
        in = (int)(c & 0xffffffffu);
        if ((int)(c >> 32) == take) return below;
        const int open = (int)(c >> 32) - in;
        if (open <= kFew) {
            // a few: their fp64 scores, each compared with every other
            if (tid == 0) P.n_open = 0;
            wide();
            __syncthreads();
            for (int j = tid; j < n; j += NT)
                if (s[j] <= above && s[j] >= below) P.at[atomicAdd(&P.n_open, 1)] = j;
            __syncthreads();
            for (int i = warp; i < open; i += NW) {
                const unsigned long long k = ord_key64(again(P.at[i]));
                if (lane == 0) P.key[i] = k;
            }
            __syncthreads();
            if (tid < open) {
                int better = 0;
                for (int i = 0; i < open; ++i)
                    better += P.key[i] > P.key[tid] || (P.key[i] == P.key[tid] && P.at[i] < P.at[tid]);
                if (better >= take - in) s[P.at[tid]] = -INFINITY;
            }
            __syncthreads();
            return below;
        }
    } else {
        settle();
    }
    // the open pages by their fp64 scores
    wide();
    __syncthreads();
    for (int j = warp; j < n; j += NW) {
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
        for (int j = tid; j < n; j += NT) c += big[j] >= mid;
        c = (int)cta_sum(P, (unsigned)c, 0u, ph);
        if (c >= want) lo = mid; else hi = mid - 1;
        if (c == want) break;
    }
    int c = 0;
    for (int j = tid; j < n; j += NT) c += big[j] >= lo;
    int jl = n;                                            // pages of just the key lo are in up to jl
    if ((int)cta_sum(P, (unsigned)c, 0u, ph) != want) {
        c = 0;
        for (int j = tid; j < n; j += NT) c += big[j] > lo;
        const int ties = want - (int)cta_sum(P, (unsigned)c, 0u, ph);
        jl = 0;
        int jh = n - 1;                                    // the smallest j up to which there are `ties` of them
        while (jl < jh) {
            const int mid = (jl + jh) / 2;
            c = 0;
            for (int j = tid; j <= mid; j += NT) c += big[j] == lo;
            if ((int)cta_sum(P, (unsigned)c, 0u, ph) >= ties) jh = mid; else jl = mid + 1;
        }
    }
    for (int j = tid; j < n; j += NT) {
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
template <typename T, int D, int GP, int NW>
struct CoreSimt {
    static constexpr int kWarps = NW, kNT = NW * 32;
    static constexpr int E = D / 32;
    struct Shared {
        float q[GP * D];
        float p[kWarps][GP * kKeys];
    };
    float o[GP][E], m[GP], l[GP];

    // qrow: the G queries; the whole CTA calls it
    __device__ __forceinline__ void init(Shared& S, const T* qrow, int G)
    {
        for (int i = threadIdx.x; i < GP * D; i += kNT) S.q[i] = i < G * D ? Elem<T>::to_f(qrow[i]) : 0.f;
        __syncthreads();
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            m[g] = -INFINITY;
            l[g] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[g][e] = 0.f;
        }
    }

    __device__ __forceinline__ void tile(const unsigned char* kt, const unsigned char* vt, int valid, Shared& S, float qscale,
                                         int lane, int G)
    {
        const float* q = S.q;
        float* pb = S.p[threadIdx.x >> 5];
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
                load_vec<T, E>(reinterpret_cast<const T*>(a), v[i]);
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

    // o to out [G][D], (m, l) to ml [G]
    __device__ __forceinline__ void finish(float* out, float2* ml, int lane, int G, bool bad)
    {
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            const float s = warp_sum(l[g]);
            if (g >= G) continue;
#pragma unroll
            for (int e = 0; e < E; ++e) out[g * D + lane * E + e] = o[g][e];
            if (lane == 0) ml[g] = make_float2(m[g], bad ? NAN : s);
        }
    }
};

// The same on the tensor cores (bf16): the G queries are the rows of 16-row
// products, S = Q K^T with 16 keys and O += P V with P from S's registers.
// 48 products of 16 x 8 x 16 a tile, a small part of the time its 4 KB of
// keys and 4 KB of values (head_dim 128) take to arrive; tcgen05's 128 rows
// would be seven eighths padding here.  There is time for P in two bf16 parts
// (2^-16 relative a weight, far below the output's own rounding).  The maximum
// is raised only when a logit passes it by 2^8.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int NW>
struct CoreMma {
    static constexpr int kWarps = NW;
    using T = __nv_bfloat16;
    struct Shared {};
    static constexpr float kRaise = 8.f;
    uint32_t q[D / 16][4];
    float o[D / 8][4], m[2], l[2];     // rows lane / 4 and lane / 4 + 8

    __device__ __forceinline__ void init(Shared&, const T* qrow, int G)
    {
        const int lane = threadIdx.x & 31, r = lane >> 2, c = (lane & 3) * 2;
        const uint32_t* p0 = reinterpret_cast<const uint32_t*>(qrow + (size_t)r * D + c);
        const uint32_t* p1 = p0 + 4 * D;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            q[k][0] = r < G ? p0[k * 8] : 0u;
            q[k][1] = r + 8 < G ? p1[k * 8] : 0u;
            q[k][2] = r < G ? p0[k * 8 + 4] : 0u;
            q[k][3] = r + 8 < G ? p1[k * 8 + 4] : 0u;
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }

    __device__ __forceinline__ void tile(const unsigned char* kt, const unsigned char* vt, int valid, Shared&, float qscale, int lane, int G)
    {
        const int mat = lane >> 3, r8 = lane & 7;
        float z[2][4] = {};
        const uint32_t ka = smem_u32(kt) + (uint32_t)((mat >> 1) * 8 + r8) * (D * 2);
        const uint32_t va = smem_u32(vt) + (uint32_t)((mat & 1) * 8 + r8) * (D * 2);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t b[4];
            ldsm4(b, ka + (uint32_t)(((k * 2 + (mat & 1)) ^ r8) << 4));
            mma16816(z[0], q[k], b[0], b[1]);
            mma16816(z[1], q[k], b[2], b[3]);
        }
        if (valid < kKeys) {
            const int c = (lane & 3) * 2;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (i * 8 + c + (e & 1) >= valid) z[i][e] = -INFINITY;
        }
        uint32_t p[4], r[4];                               // the weights in bf16, and what that leaves of them
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            p[x] = p[x + 2] = r[x] = r[x + 2] = 0u;
            if (x == 1 && G <= 8) break;                   // rows of padding
            float t = fmaxf(fmaxf(z[0][2 * x], z[0][2 * x + 1]), fmaxf(z[1][2 * x], z[1][2 * x + 1]));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2)) * qscale;
            const bool raise = t > m[x] + kRaise;
            if (__any_sync(0xffffffffu, raise)) {
                const float a = raise ? ex2_approx(m[x] - t) : 1.f;
                if (raise) m[x] = t;
                l[x] *= a;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[i][2 * x] *= a;
                    o[i][2 * x + 1] *= a;
                }
            }
            const float base = m[x] == -INFINITY ? 0.f : m[x];
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = ex2_approx(fmaf(z[i >> 1][2 * x + (i & 1)], qscale, -base));
            l[x] += (e[0] + e[1]) + (e[2] + e[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t& hi = p[x + 2 * i];
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(e[2 * i + 1]), "f"(e[2 * i]));
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                    : "=r"(r[x + 2 * i])
                    : "f"(e[2 * i + 1] - __uint_as_float(hi & 0xffff0000u)), "f"(e[2 * i] - __uint_as_float(hi << 16)));
            }
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t b[4];
            ldsm4_t(b, va + (uint32_t)(((k * 2 + (mat >> 1)) ^ r8) << 4));
            mma16816(o[2 * k], p, b[0], b[1]);
            mma16816(o[2 * k + 1], p, b[2], b[3]);
            mma16816(o[2 * k], r, b[0], b[1]);
            mma16816(o[2 * k + 1], r, b[2], b[3]);
        }
        __syncwarp();
    }

    __device__ __forceinline__ void finish(float* out, float2* ml, int lane, int G, bool bad)
    {
        const int r = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float s = l[x];
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            const int g = r + 8 * x;
            if (g >= G) continue;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) *reinterpret_cast<float2*>(out + g * D + i * 8 + c) = make_float2(o[i][2 * x], o[i][2 * x + 1]);
            if ((lane & 3) == 0) ml[g] = make_float2(m[x], bad ? NAN : s);
        }
    }
};

// two or four floats
template <int N> __device__ __forceinline__ void load_f(const float* p, float* x)
{
    if constexpr (N == 4) {
        const float4 w = *reinterpret_cast<const float4*>(p);
        x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
    } else {
        const float2 w = *reinterpret_cast<const float2*>(p);
        x[0] = w.x; x[1] = w.y;
    }
}
template <int N> __device__ __forceinline__ void store_f(float* p, const float* x)
{
    if constexpr (N == 4) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
}
template <int N> __device__ __forceinline__ void store_out(float* p, const float* x) { store_f<N>(p, x); }
template <int N> __device__ __forceinline__ void store_out(__nv_bfloat16* p, const float* x)
{
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    if constexpr (N == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
template <int N> __device__ __forceinline__ void ld_cluster_f(uint32_t addr, float* x)
{
    if constexpr (N == 4) {
        const float4 w = ld_cluster_f4(addr);
        x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
    } else {
        const float2 w = ld_cluster_f2(addr);
        x[0] = w.x; x[1] = w.y;
    }
}

template <int D, class Core>
struct alignas(16) AttendSmem {
    float2 w[2 * D];                   // the page weights, minima's then maxima's, as w.x + w.y + w_lo; later in fp64
    typename Core::Shared core;
    float2 wml[Core::kWarps][kMaxPageGroups];
    float2 ml[kMaxPageGroups];
    PickSmem<Core::kWarps> pick;
    // (the marks are made when pages are ranked)
    __device__ __forceinline__ float* w_lo() { return reinterpret_cast<float*>(pick.mark); }
    static_assert(sizeof(pick.mark) >= 2 * D * sizeof(float), "w_lo fits");
};

// Shared memory: the warps' rings (fp64 keys while picking), AttendSmem, and
// when picking the scores and the picked pages.
template <typename T, int D> constexpr int kTileBytes = kKeys * D * (int)sizeof(T);
template <typename T, int D> constexpr int kRingBytes = kStages<T> * 2 * kTileBytes<T, D>;   // a warp's

constexpr int kMaxCluster = 16;
constexpr int kMaxSources = kMaxCluster + kMaxPrefixSplits;   // CTAs of a cluster and ranges of a prefix

// Several CTAs an SM (bf16): while one ranks its pages, or waits for its
// first keys, the others read.
template <typename T, int D, class Core>
__global__ void __launch_bounds__(Core::kWarps * 32, sizeof(T) == 2 ? 8 / Core::kWarps : 1)
    page_attend_kernel(const PagePool pool, const PageRows R, const int budget, const int recent, int* __restrict__ picked,
                       const PrefixPart part, const int front, const int wpad)
{
    extern __shared__ __align__(128) unsigned char raw[];
    using S_t = AttendSmem<D, Core>;
    constexpr int NS = kStages<T>, TB = kTileBytes<T, D>, kWarps = Core::kWarps, kNT = kWarps * 32;
    S_t& S = *reinterpret_cast<S_t*>(raw + front);
    float* scores = reinterpret_cast<float*>(raw + front + sizeof(S_t));
    int* list = reinterpret_cast<int*>(scores + wpad);
    unsigned long long* big = reinterpret_cast<unsigned long long*>(raw);
    unsigned char* ring = raw + (threadIdx.x >> 5) * kRingBytes<T, D>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
    const int u = blockIdx.x / C, row = u / pool.heads, h = u - row * pool.heads;
    const int seq = R.seq[row], pos = R.pos[row];
    if (seq < 0) {                                         // a row that is not there, for the whole cluster
        if (part.splits) grid_dependency_wait();           // (this grid ends after the one it started beside)
        return;
    }
    const int sh = __ffs(pool.ps) - 1;
    const int G = R.G;
    int npages = pos < 0 ? 0 : (pos >> sh) + 1;
    bool bad = seq >= R.requests || npages > R.width;
    if (bad) npages = 0;
    const int* table = R.table + (size_t)(bad ? 0 : seq) * R.width;
    const T* qrow = static_cast<const T*>(R.q) + (size_t)row * R.q_stride + (size_t)h * G * D;

    int nlist = npages;
    const int* src = table;                                // physical page of each entry
    const int ncand = npages - recent, take = budget - recent;
    if (budget > 0 && npages > budget) {
        int* pick_out = picked && rank == 0 ? picked + (size_t)u * budget : nullptr;
        if (take > 0) {                                    // (else the newest pages are all)
            // Bounds come through the warp's ring, kScan pages a lane group and stage, each lane reading back what it asked
            // for (registers alone kept 8 KB a warp in flight, and the ring is idle now).
            constexpr int N = 16 / sizeof(T), NV = 2 * D / 8 / N, kScan = 4;
            static_assert(kScan * NV * 512 <= 2 * TB, "a stage of bounds fits a stage of the ring");
            const T* bounds = static_cast<const T*>(pool.bounds);
            const int sub = lane & 7;                      // eight lanes a page
            // each CTA scores a range of the pages
            const int chunk = ((ncand + C - 1) / C + 3) & ~3, jend = min(ncand, (rank + 1) * chunk);
            const int step = kWarps * 4 * kScan;
            int j0 = rank * chunk + warp * 4 * kScan;
            // (an arrival waits for all copies under way, 4000 cycles, so it comes before them)
            if (tid == 0) S.pick.amax = 0u;
            cluster_arrive();
            // the queries first, into a stage that the bounds reach later: behind what bounds all CTAs ask for they came 4000
            // cycles after these
            static_assert(kMaxPageGroups * D * (int)sizeof(T) <= 2 * TB, "a stage of the ring holds the queries");
            unsigned char* qs = raw + (NS - 1) * 2 * TB;
            for (int i = tid; i < G * (D / N); i += kNT) cp_async16(smem_u32(qs + i * 16), qrow + i * N, true);
            cp_commit();
            // each page's id waits in the place of its score
            for (int j = rank * chunk + tid; j < jend; j += kNT) scores[j] = __int_as_float(table[j]);
            __syncthreads();
            auto scan = [&](int j, int stage) {
                if (j < jend)
#pragma unroll
                    for (int x = 0; x < kScan; ++x) {
                        const int p = j + x * 4 + (lane >> 3), id = p < jend ? __float_as_int(scores[p]) : 0;
                        const bool ok = (unsigned)id < (unsigned)pool.pages;
                        const T* from = bounds + ((size_t)(ok ? id : 0) * pool.heads + h) * 2 * D + sub * N;
#pragma unroll
                        for (int i = 0; i < NV; ++i)
                            cp_async16(smem_u32(ring + stage * 2 * TB + ((x * NV + i) * 32 + lane) * 16), from + i * 8 * N, true);
                    }
                cp_commit();
            };
#pragma unroll 1
            for (int k = 0; k < NS - 1; ++k) scan(j0 + k * step, k);
            cp_wait<NS - 1>();
            __syncthreads();
            // (fp32 parts, since the fp64 pipe is so narrow that its conversions took 3 us here)
            for (int i = tid; i < 2 * D; i += kNT) {
                Sum3 s;
                const bool lo = i < D;
                for (int g = 0; g < G; ++g) {
                    const float x = Elem<T>::to_f(reinterpret_cast<const T*>(qs)[g * D + (lo ? i : i - D)]);
                    s.add(lo ? (x > 0.f ? 0.f : x) : (x < 0.f ? 0.f : x));
                }
                S.w[i] = s.rounded();
                S.w_lo()[i] = s.lo;
            }
            __syncthreads();
            float w[NV][N];
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < N; ++e) w[i][e] = S.w[(i * 8 + sub) * N + e].x;
            float w1 = 0.f;                                // sum |w|
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < N; ++e) w1 += fabsf(w[i][e]);
#pragma unroll
            for (int d = 4; d > 0; d >>= 1) w1 += __shfl_xor_sync(0xffffffffu, w1, d);
            AbsMax<T> most;
            cluster_wait();                                // every CTA has set its maximum
            int stage = 0;
#pragma unroll 1
            for (; j0 < jend; j0 += step) {
                scan(j0 + (NS - 1) * step, stage == 0 ? NS - 1 : stage - 1);
                cp_wait<NS - 1>();
#pragma unroll
                for (int x = 0; x < kScan; ++x) {
                    float2 s2 = make_float2(0.f, 0.f);
                    const int j = j0 + x * 4 + (lane >> 3);
                    const bool in = j < jend;
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const uint4 v = *reinterpret_cast<const uint4*>(ring + stage * 2 * TB + ((x * NV + i) * 32 + lane) * 16);
                        most.take(v, in);
                        float f[N];
                        load_vec<T, N>(reinterpret_cast<const T*>(&v), f);
#pragma unroll
                        for (int e = 0; e < N; e += 2)
                            s2 = __ffma2_rn(make_float2(w[i][e], w[i][e + 1]), make_float2(f[e], f[e + 1]), s2);
                    }
                    float s = s2.x + s2.y;
#pragma unroll
                    for (int d = 4; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                    if (in && sub == 0) {
                        if (__float_as_uint(scores[j]) >= (unsigned)pool.pages) {   // no such page: picked, and its row is NaN
                            s = NAN;
                            most.take(make_uint4(~0u, 0u, 0u, 0u), true);
                        }
                        scores[j] = s;
                    }
                }
                stage = stage + 1 == NS ? 0 : stage + 1;
            }
            cp_wait<0>();
            const unsigned amax = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(__fmul_ru(w1, most.value()))));
            if (lane < C) cluster_max_u32(map_to_rank(&S.pick.amax, lane), amax);
            cluster_arrive();
            cluster_wait();
            // the other CTAs' scores, 16 bytes a lane (a store to every CTA as each score was made took four times as long)
#pragma unroll 4
            for (int j = tid * 4; j < ncand; j += kNT * 4) {
                const int owner = j / chunk;
                if (owner != rank) *reinterpret_cast<float4*>(scores + j) = ld_cluster_f4(map_to_rank(scores + j, owner));
            }
            __syncthreads();
            cluster_arrive();                              // (its wait: before scores are overwritten)
            const float bound = pick_bound(S.pick, scores, ncand, take, big, [] { cluster_wait(); }, [&] {
                // (in their place: the fp32 scores are made)
                for (int i = tid; i < 2 * D; i += kNT)
                    reinterpret_cast<double*>(S.w)[i] = (double)S.w[i].x + ((double)S.w[i].y + (double)S.w_lo()[i]);
            }, [&](int j) {
                const int p = table[j];
                if ((unsigned)p >= (unsigned)pool.pages) return (double)NAN;
                const T* b = bounds + ((size_t)p * pool.heads + h) * 2 * D;
                double s = 0.0;
                if (__uint_as_float(S.pick.amax) < FLT_MAX) {      // (finite factors; fp64 holds their sum)
                    for (int e = lane; e < 2 * D; e += 32) s += reinterpret_cast<const double*>(S.w)[e] * (double)Elem<T>::to_f(b[e]);
                } else {
                    // an infinite bound on the side that no query takes counts for nothing: the maxima themselves
                    for (int e = lane; e < D; e += 32)
                        for (int g = 0; g < G; ++g) {
                            const double x = Elem<T>::to_f(qrow[g * D + e]);
                            const double y0 = x * (double)Elem<T>::to_f(b[e]), y1 = x * (double)Elem<T>::to_f(b[D + e]);
                            s += y0 != y0 || y1 != y1 ? (double)NAN : fmax(y0, y1);
                        }
                }
                for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                return s;
            });
            // the picked pages in order: each warp takes a range, each lane the marks of 32 pages at a time
            const int n32 = (ncand + 31) >> 5, w32 = (n32 + kWarps - 1) / kWarps, g0 = min(n32, warp * w32), g1 = min(n32, g0 + w32);
            int count = 0;
#pragma unroll 4
            for (int g = g0; g < g1; ++g) {
                const int j = g * 32 + lane;
                const unsigned in = __ballot_sync(0xffffffffu, j < ncand && scores[j] >= bound);
                if (lane == 0) S.pick.mark[g] = in;
                count += __popc(in);
            }
            if (lane == 0) S.pick.taken[warp] = count;
            __syncthreads();
            int at = 0;
            for (int k = 0; k < warp; ++k) at += S.pick.taken[k];
#pragma unroll 1
            for (int g = g0; g < g1; g += 32) {
                unsigned in = g + lane < g1 ? S.pick.mark[g + lane] : 0u;
                const int c = __popc(in);
                int x = c;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, d);
                    if (lane >= d) x += y;
                }
                int to = at + x - c;
                for (; in; in &= in - 1) list[to++] = (g + lane) * 32 + __ffs(in) - 1;
                at += __shfl_sync(0xffffffffu, x, 31);
            }
            __syncthreads();
        }
        for (int i = tid; i < budget; i += kNT) {
            const int j = i < take ? list[i] : ncand + i - take;
            list[i] = table[j];
            if (pick_out) pick_out[i] = j;
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
                const size_t o = off + (fill ? r * D + c * (16 / (int)sizeof(T)) : 0);
                cp_async16(kd + tile_at<T, D>(r, c * 16), K + o, fill);
                cp_async16(vd + tile_at<T, D>(r, c * 16), V + o, fill);
            }
            if (t + stride < ntiles) pg_next = src[(t + stride) >> tsh];
        }
        cp_commit();
    };
#pragma unroll 1
    for (int s = 0; s < NS - 1; ++s) ask(t0 + s * stride, s);
    Core core;
    core.init(S.core, qrow, G);
    int stage = 0;
#pragma unroll 1
    for (int t = t0; t < ntiles; t += stride) {
        ask(t + (NS - 1) * stride, stage == 0 ? NS - 1 : stage - 1);
        cp_wait<NS - 1>();
        __syncwarp();
        core.tile(ring + 2 * stage * TB, ring + 2 * stage * TB + TB, valid_of(t), S.core, R.qscale, lane, G);
        stage = stage + 1 == NS ? 0 : stage + 1;
    }
    cp_wait<0>();
    __syncwarp();

    // the warps' sums, then the CTAs', then the prefix's
    constexpr int kSums = (int)sizeof(float) * kMaxPageGroups * D;
    static_assert(kRingBytes<T, D> >= 2 * kSums, "a warp's sums and the CTA's lie in a ring");
    core.finish(reinterpret_cast<float*>(ring), S.wml[warp], lane, G, bad);
    __syncthreads();
    float* sums = reinterpret_cast<float*>(raw + kSums);
    constexpr int V4 = D / 32;                             // a lane's channels of a head
    for (int g = warp; g < G; g += kWarps) {
        float m = -INFINITY, l = 0.f, o[V4] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, S.wml[w][g].x);
        const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float a = ex2_approx(S.wml[w][g].x - base);
            l = fmaf(a, S.wml[w][g].y, l);
            float x[V4];
            load_f<V4>(reinterpret_cast<const float*>(raw + w * kRingBytes<T, D>) + g * D + lane * V4, x);
#pragma unroll
            for (int e = 0; e < V4; ++e) o[e] = fmaf(a, x[e], o[e]);
        }
        store_f<V4>(sums + g * D + lane * V4, o);
        if (lane == 0) S.ml[g] = make_float2(m, l);
    }
    if (part.splits) grid_dependency_wait();               // the prefix pass is through
    cluster_arrive();
    cluster_wait();
    // A warp joins a head's sums of all sources, the cluster's CTAs and the prefix's ranges: eight sources' values are
    // asked for at a time, the first beside the sources' maxima.
    T* orow = static_cast<T*>(R.out) + (size_t)row * R.out_stride + (size_t)h * G * D;
    const int ns = C + part.splits;
    const size_t qrows = (size_t)R.rows * pool.heads * G, qr = (size_t)u * G;
#pragma unroll 1
    for (int g = rank * kWarps + warp; g < G; g += C * kWarps) {
        constexpr int NX = (kMaxSources + 31) / 32, kAtOnce = 8;
        float v[kAtOnce][V4];
        auto ask = [&](int s0) {
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int s = s0 + k;
                if (s < C) ld_cluster_f<V4>(map_to_rank(sums + g * D + lane * V4, s), v[k]);
                else if (s < ns) load_f<V4>(part.o + ((s - C) * qrows + qr + g) * D + lane * V4, v[k]);
            }
        };
        ask(0);
        float2 x[NX];
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int k = lane + 32 * i;
            x[i] = make_float2(-INFINITY, 0.f);
            if (k < C) x[i] = ld_cluster_f2(map_to_rank(&S.ml[g], k));
            else if (k < ns) x[i] = part.ml[(k - C) * qrows + qr + g];
            m = fmaxf(m, x[i].x);
        }
        m = warp_max(m);
        const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            x[i].x = ex2_approx(x[i].x - base);            // the source's weight
            l = fmaf(x[i].x, x[i].y, l);
        }
        l = warp_sum(l);
        float o[V4] = {};
#pragma unroll 1
        for (int s0 = 0; s0 < ns; s0 += kAtOnce) {
            const float mine = s0 < 32 ? x[0].x : s0 < 64 ? x[1].x : x[NX - 1].x;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const float a = __shfl_sync(0xffffffffu, mine, (s0 + k) & 31);
                if (s0 + k < ns)
#pragma unroll
                    for (int e = 0; e < V4; ++e) o[e] = fmaf(a, v[k][e], o[e]);
            }
            if (s0 + kAtOnce < ns) ask(s0 + kAtOnce);
        }
        // no key at all, or none of weight: zero, whatever the values are; a bad table entry has made l NaN
        const float f = 1.f / l;
#pragma unroll
        for (int e = 0; e < V4; ++e) o[e] = l == 0.f ? 0.f : o[e] * f;
        store_out<V4>(orow + g * D + lane * V4, o);
    }
    cluster_arrive();
    cluster_wait();                                        // no CTA leaves while another reads its sums
}

// Warps of a CTA.  bf16: two where there are more units than CTAs fit and each
// has few tiles, so that more units are under way (6400 units of 12 tiles: 201
// us with four, 153 with two; 512 of 24: 81, 80; 512 of 96: 83, 89).  fp32,
// whose ring of four leaves an SM one CTA: two (832 units of 3 tiles and a
// prefix: 40 us, 23 with two) unless the units are few.
int attend_warps(long long units, int tiles, bool bf16)
{
    if (bf16) return units > 4 * kSMs && tiles <= 32 ? 2 : 4;
    return units > kSMs / 8 ? 2 : 4;
}

// Clusters of c CTAs (2 to 16) that the GPU holds at once, about: what is left
// over of each group of SMs makes larger ones fit worse (at two CTAs an SM 152,
// 74, 36 and 14 of 2, 4, 8 and 16; at one 76, 36, 15 and 7).  per_sm goes by
// shared memory alone; at head_dim 64 in bf16, registers leave an SM three CTAs
// of four warps where it says four.
int clusters_that_fit(int c, int per_sm)
{
    return c == 2 ? 76 * per_sm : c == 4 ? 36 * per_sm : c == 8 ? (per_sm == 1 ? 15 : 17 * per_sm) : 7 * per_sm;
}

// CTAs of a unit: as many, up to 16, as leave all clusters at once on the GPU
// and every warp three tiles (16 units of 96 tiles: 23 us with one, 12 with
// four; 70 of 68: 18, 15 with four, 18 with eight; 8 of 256: 19 with eight, 18
// with sixteen; 16 of 256: 21 with eight, 32 with sixteen, which take turns).
int cluster_of(long long units, int tiles, int per_sm, int warps)
{
    int c = 1;
    while (c < kMaxCluster && units <= clusters_that_fit(2 * c, per_sm) && tiles >= 3 * c * 2 * warps) c *= 2;
    return c;
}

template <typename T, int D, class Core>
cudaError_t go(const PagePool& p, const PageRows& r, int budget, int recent, int* picked, const PrefixPart& part, cudaStream_t st)
{
    constexpr int NW = Core::kWarps;
    const bool picks = budget > 0 && budget < r.width;
    const int wpad = picks ? (r.width + 3) & ~3 : 0;
    const int front = std::max(NW * kRingBytes<T, D>, 8 * wpad);
    const size_t smem = front + sizeof(AttendSmem<D, Core>) + 4 * ((size_t)wpad + (picks ? budget : 0));
    const auto kernel = page_attend_kernel<T, D, Core>;
    static SmemOnce once;
    const cudaError_t e = once.allow(kernel, true);
    if (e != cudaSuccess) return e;
    const long long units = (long long)r.rows * p.heads;
    const int C = cluster_of(units, (budget > 0 ? std::min(budget, r.width) : r.width) * (p.ps / kKeys), (int)(227 * 1024 / (smem + 1024)), NW);
    cudaLaunchAttribute at[2];
    int na = 0;
    if (C > 1) {
        at[na].id = cudaLaunchAttributeClusterDimension;
        at[na].val.clusterDim.x = (unsigned)C;
        at[na].val.clusterDim.y = at[na].val.clusterDim.z = 1;
        ++na;
    }
    if (part.splits) {                                     // behind a prefix pass: its own keys are read meanwhile
        at[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * C));
    cfg.blockDim = dim3(NW * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = (unsigned)na;
    return cudaLaunchKernelEx(&cfg, kernel, p, r, budget, recent, picked, part, front, wpad);
}

template <int D, int NW>
cudaError_t by_groups(const PagePool& p, const PageRows& r, int budget, int recent, int* picked, const PrefixPart& part, cudaStream_t st)
{
    if (p.dtype) return go<__nv_bfloat16, D, CoreMma<D, NW>>(p, r, budget, recent, picked, part, st);
    if (r.G == 1) return go<float, D, CoreSimt<float, D, 1, NW>>(p, r, budget, recent, picked, part, st);
    if (r.G <= 4) return go<float, D, CoreSimt<float, D, 4, NW>>(p, r, budget, recent, picked, part, st);
    if (r.G <= 8) return go<float, D, CoreSimt<float, D, 8, NW>>(p, r, budget, recent, picked, part, st);
    return go<float, D, CoreSimt<float, D, 16, NW>>(p, r, budget, recent, picked, part, st);
}

template <int D>
cudaError_t by_warps(const PagePool& p, const PageRows& r, int budget, int recent, int* picked, const PrefixPart& part, cudaStream_t st)
{
    const int tiles = (budget > 0 ? std::min(budget, r.width) : r.width) * (p.ps / kKeys);
    if (attend_warps((long long)r.rows * p.heads, tiles, p.dtype != 0) == 2) return by_groups<D, 2>(p, r, budget, recent, picked, part, st);
    return by_groups<D, 4>(p, r, budget, recent, picked, part, st);
}

}  // namespace

cudaError_t launch_page_attend(const PagePool& p, const PageRows& r, int budget, int recent, int* picked,
                               const PrefixPart& part, cudaStream_t st)
{
    return p.D == 64 ? by_warps<64>(p, r, budget, recent, picked, part, st) : by_warps<128>(p, r, budget, recent, picked, part, st);
}

}  // namespace h2o
