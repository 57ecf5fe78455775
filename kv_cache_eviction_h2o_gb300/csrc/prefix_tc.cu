// prefix_tc.cu -- the shared prefix's part of h2o_prefix_attend on the
// 5th-generation tensor cores (bf16).
//
// Query rows of one cache head (row r's G query heads are rows r G .. r G + G - 1)
// go in tiles of 128, keys in tiles of 128, and a CTA sweeps a range of the
// prefix with two score streams:
//   S = Q K^T        (SMEM x SMEM -> TMEM, M = 128, K = D)
//   P = 2^(c S - m)  (128 threads a stream, thread = TMEM lane = query row)
//   O += P V         (TMEM x SMEM -> TMEM, M = 128, N = D)
// so that one stream's exponentials run under the other's products.  With more
// than 128 query rows left the streams are two query tiles over the same keys
// (each key tile is read once for 256 rows); with fewer they are the even and
// the odd key tiles of one query tile, joined at the end.  S and P go by halves
// of 64 keys: while the threads work on one half, the product of the other's P
// and the next tile's scores in its place are made, so neither waits for the
// other's latency.
//
// One CTA per SM: TMEM holds S and O of both streams (P overwrites S: the
// tensor pipe works in the order of issue, and S of the next tile is issued
// after the product that reads P).  Warp 0 loads key and value tiles with TMA
// (a box per page and 64 channels, so pages lie anywhere), warps 1 and 2 issue
// their stream's products, warps 4..7 and 8..11 are the streams' threads.  A
// row's maximum m is raised, and O scaled, only when a logit passes it by more
// than 2^8: the weights are relative to m in any case, and l stays in fp32.  P
// is rounded to bf16 for the product (2^-8 relative a weight, as the output is;
// a second product of what that leaves took 13 us more), the sums l are
// of the unrounded weights.  Waits are bounded; one that runs out leaves NaN
// sums.
//
// Measured, 64 requests of 8 x 8 heads behind 32768 tokens (68.7 GFLOP): 52 us,
// 1.31 PFLOP/s, 0.67 of the bf16 peak measured with a library product.  A tile
// of both streams takes 2900 cycles, of which its products are 2050.  What
// bounds it is the products and the shared memory that feeds them: those of
// Q K^T read both operands from it (by halves of 64 keys the queries twice),
// those of P V one, and the loads write into it, which makes 2300 to 2560 of
// its 128-byte cycles.  Without the loads, the exponentials or both it takes as
// long; with the scores of 128 keys made at once the queries are read once, but
// the threads wait for them (66 us).  Of the rest 3 us pass until the first
// scores and 3 us in writing the sums.
#include <algorithm>

#include "paged.h"
#include "tc.cuh"

namespace h2o {

namespace {

constexpr int kT = 128;
constexpr int kThreads = 384;
constexpr uint32_t kBox = kT * 64 * 2;             // 128 rows x 64 channels: 16 KB
constexpr float kRaise = 8.f;
constexpr int kSteps = 2, kStep = kT / kSteps;     // S and P go by parts of a tile

template <int D> struct Cfg {
    static constexpr int kBoxes = D / 64;
    static constexpr uint32_t kTile = kBoxes * kBox;
    static constexpr int kSlots = D == 128 ? 5 : 8;    // K and V tiles in flight
    static constexpr int kPitch = D * 4 + 16;          // of a row of sums on its way out (16 bytes more: no bank conflicts)
    static_assert(2 * kT * kPitch <= kSlots * (int)kTile, "the ring holds them");
};

template <int D>
struct alignas(1024) Smem {
    uint8_t q[2][Cfg<D>::kTile];
    uint8_t ring[Cfg<D>::kSlots][Cfg<D>::kTile];
    uint64_t full[2][Cfg<D>::kSlots], empty[Cfg<D>::kSlots];
    uint64_t q_ready, s_ready[2][kSteps], p_ready[2][kSteps], pv_done[2][kSteps], last;   // [stream][part of the tile]
    uint64_t landed;                   // all loads are there
    uint32_t tmem;
    int abort, bad;
};
static_assert(sizeof(Smem<128>) + 1024 <= 227 * 1024, "one CTA's shared memory");

// accumulator fp32, bf16 A and B, A K-major, B K-major or (bit 16) N-major
template <int N, bool BMN>
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((BMN ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kT >> 4) << 24);

// The issuing warp runs its loop as a whole, so that descriptors stay in
// uniform registers, and one lane (`on`) issues: a loop inside one lane's
// branch issued a product every 100 to 115 cycles, whatever its size, and one
// warp for both streams left 4000 cycles a tile.
__device__ __forceinline__ uint32_t elect_lane()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
__device__ __forceinline__ void mma_ss(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"(acc), "r"(on)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t on, uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(id), "r"(acc), "r"(on)
                 : "memory");
}
__device__ __forceinline__ void commit(uint32_t on, uint64_t* bar)
{
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(on)
                 : "memory");
}

// a copy of `bytes` (a multiple of 16) out of shared memory by this thread, and the end of all it started
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_store_wait()
{
    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
}

// descriptor of the value tile as the K x N operand, N (channels) contiguous:
// 64-channel boxes 16 KB apart (leading offset), 8 keys every 1024 B
__device__ __forceinline__ uint64_t value_desc(const void* p)
{
    return (uint64_t)((smem_u32(p) & 0x3FFFFu) >> 4) | ((uint64_t)(kBox >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// The ring's order of use: K(0) .. K(L - 1), then V(t), K(t + L) for t = 0, 1, ..
// (L = 1: both streams read each tile; 2: the streams take turns).  A wait
// tells a barrier's phase from its neighbour only, so each barrier's waiters
// see all its phases: where the streams take turns each has full barriers of
// its own (with one set a stream could take the landing of the other's tile,
// two turns of the slot before, for that of its own), and counts their phases
// by what it has waited for.  V(t)'s place:
__device__ __forceinline__ int v_at(int t, int n, int L) { return t + min(n, t + L); }

template <int D>
__device__ __forceinline__ bool wait(Smem<D>& S, uint64_t* bar, int count)
{
    // the barrier's phase number `count` (from 0); once one wait has run out the others do, each for itself
    if (mbar_wait(bar, (uint32_t)count & 1u)) return true;
    *(volatile int*)&S.abort = 1;
    return false;
}

// grid: (pair of query tiles, range of the prefix, cache head)
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV, const PagePool pool,
                     const PageRows R, const int* __restrict__ table, const int prefix_len, const int per, const PrefixPart part, const unsigned long long inv)
{
    using C = Cfg<D>;
    constexpr int NS = C::kSlots;
    extern __shared__ unsigned char raw[];
    Smem<D>& S = *reinterpret_cast<Smem<D>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // (known to be uniform)
    const int G = R.G, nx = R.rows * G, h = blockIdx.z, x0 = blockIdx.x * 2 * kT;
    const bool two = x0 + kT < nx;                   // two query tiles
    const int L = two ? 1 : 2;
    const int j0 = blockIdx.y * per, j1 = min(prefix_len, j0 + per);
    const int n = (j1 - j0 + kT - 1) / kT;           // key tiles, at least one
    auto over_G = [&](int x) { return (long long)((unsigned long long)(unsigned)x * inv >> 32); };   // x / G (x < 2^28)
    auto valid_of = [&](int t) { return min(kT, j1 - j0 - t * kT); };

    grid_launch_dependents();                        // the rows' own pass may start on what SMs are left; it waits before it reads sums
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&S.full[0][s], 1);
            mbar_init(&S.full[1][s], 1);
            mbar_init(&S.empty[s], two ? 2 : 1);
        }
        mbar_init(&S.q_ready, two ? 8 : 4);
        for (int s = 0; s < 2; ++s) {
            for (int b = 0; b < kSteps; ++b) {
                mbar_init(&S.s_ready[s][b], 1);
                mbar_init(&S.p_ready[s][b], 4);
                mbar_init(&S.pv_done[s][b], 1);
            }
        }
        mbar_init(&S.last, 2);
        mbar_init(&S.landed, 1);
        S.abort = S.bad = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&S.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    auto tS = [&](int s) { return tmem + (uint32_t)(s * kT); };
    auto tO = [&](int s) { return tmem + (uint32_t)(2 * kT + s * D); };

    if (warp == 0) {
        // ------------------------------------------------ loads
        const int ps = pool.ps;
        const uint32_t page_bytes = (uint32_t)ps * 128u;   // of one box
        int at = 0;
        uint32_t turns = 0u, owner = 0u;             // by slot: loads on each set of full barriers (mod 2), set of the last
        bool ok = true;
        auto load = [&](const CUtensorMap* map, int t) {
            if (!ok) return;
            const int s = at % NS, f = two ? 0 : t & 1, pages = (valid_of(t) + ps - 1) / ps, i = lane / C::kBoxes, b = lane % C::kBoxes;
            const bool mine = i < pages;             // this lane's box
            int pg = mine ? table[(j0 + t * kT) / ps + i] : 0;
            if ((unsigned)pg >= (unsigned)pool.pages) { pg = 0; *(volatile int*)&S.bad = 1; }
            if (at >= NS) ok = __all_sync(0xffffffffu, wait(S, &S.empty[s], at / NS - 1));
            if (!ok) return;
            if (lane == 0) mbar_arrive_expect_tx(&S.full[f][s], (uint32_t)pages * page_bytes * C::kBoxes);
            __syncwarp();
            if (mine) tma_load_2d(S.ring[s] + b * kBox + i * page_bytes, map, b * 64, (pg * pool.heads + h) * ps, &S.full[f][s]);
            __syncwarp();
            turns ^= 1u << (16 * f + s);
            owner = (owner & ~(1u << s)) | (uint32_t)f << s;
            ++at;
        };
        for (int t = 0; t < min(L, n); ++t) load(&mapK, t);
        for (int t = 0; t < n; ++t) {
            load(&mapV, t);
            if (t + L < n) load(&mapK, t + L);
        }
        // every load has landed before the shared memory is given up, those of an abandoned sweep too
        for (int s = 0; s < min(NS, at); ++s) {
            const uint32_t f = owner >> s & 1u;
            mbar_wait(&S.full[f][s], (turns >> (16 * f + s) & 1u) ^ 1u);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.landed);
    } else if (warp <= 2) {
        // ------------------------------------------------ products of stream s
        const int s = warp - 1;
        const uint32_t on = elect_lane();
        const uint64_t q0 = sw128_desc(S.q[two ? s : 0]), k0 = sw128_desc(S.ring[0]), v0 = value_desc(S.ring[0]);
        const uint32_t sS = tS(s), sO = tO(s);
        bool ok = __all_sync(0xffffffffu, wait(S, &S.q_ready, 0));
        uint64_t* const full = S.full[two ? 0 : s];
        uint32_t seen = 0u;                          // by slot: this stream's waits on it (mod 2)
        auto slot_full = [&](int i) {
            if (ok) ok = __all_sync(0xffffffffu, wait(S, full + i % NS, (int)(seen >> i % NS & 1u)));
            seen ^= 1u << i % NS;
        };
        // scores of step b of the tile in place i
        auto score = [&](int b, int i) {
            if (!ok) return;
            tc_fence_after();
            const uint64_t k = k0 + (uint64_t)((uint32_t)(i % NS) * (C::kTile >> 4) + (uint32_t)b * (kStep * 128u >> 4));
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
                const uint64_t off = (uint64_t)(((uint32_t)(x / 4) * kBox + (uint32_t)(x % 4) * 32u) >> 4);
                mma_ss(on, sS + (uint32_t)(kStep * b), q0 + off, k + off, kIdesc<kStep, false>, x > 0);
            }
            commit(on, &S.s_ready[s][b]);
        };
        // nth: tiles of this stream before; valid: keys of the tile, which is there
        auto values = [&](int b, int nth, int i, int valid) {
            if (ok) ok = __all_sync(0xffffffffu, wait(S, &S.p_ready[s][b], nth));
            if (!ok) return;
            tc_fence_after();
            const uint64_t v = v0 + (uint64_t)((uint32_t)(i % NS) * (C::kTile >> 4) + (uint32_t)b * (kStep * 128u >> 4));
            const int nk = (min(kStep, valid - kStep * b) + 15) / 16;
            auto one = [&](int x) {
                mma_ts(on, sO, sS + (uint32_t)(kStep * b + 8 * x), v + (uint64_t)((uint32_t)x * 2048u >> 4), kIdesc<D, true>,
                       nth > 0 || b > 0 || x > 0);
            };
            if (nk == kStep / 16) {
#pragma unroll
                for (int x = 0; x < kStep / 16; ++x) one(x);
            } else {
                for (int x = 0; x < nk; ++x) one(x);
            }
            commit(on, &S.pv_done[s][b]);
        };
        auto release = [&](int i) {                  // (two query tiles: when both streams have)
            if (ok) commit(on, &S.empty[i % NS]);
        };
        const int stride = two ? 1 : 2, t0 = two ? 0 : s;
        if (t0 < n) {
            slot_full(t0);
            for (int b = 0; b < kSteps; ++b) score(b, t0);
            release(t0);
        }
        for (int t = t0, nth = 0; t < n; t += stride, ++nth) {
            const int v = v_at(t, n, L), k = v + 1;
            const bool more = t + stride < n;
            slot_full(v);                            // (both before the weights: between them and the products every look at a
            if (more) slot_full(k);                  // barrier is waited for, and with four of them the loop took a tenth longer)
            for (int b = 0; b < kSteps; ++b) {
                values(b, nth, v, valid_of(t));
                if (b == kSteps - 1) release(v);
                if (more) {
                    score(b, k);
                    if (b == kSteps - 1) release(k);
                }
            }
        }
        // everything issued is done before TMEM is given back
        commit(on, &S.last);
        mbar_wait(&S.last, 0);
    } else if (warp >= 4) {
        // ------------------------------------------------ softmax
        const int s = (warp - 4) >> 2, w = warp & 3, row = w * 32 + lane;
        const uint32_t lanes = (uint32_t)(w * 32) << 16;
        if (two || s == 0) {
            // the warp's 32 query rows into the swizzled tile, whole rows at a time (they are there 4000 cycles after the
            // start, whether asked for by this loop, an unrolled one, through registers or before the first barrier)
            constexpr int LPR = D / 8, RPI = 32 / LPR;   // lanes of a row, rows a step
            const int c = lane % LPR;
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(R.q) + (size_t)h * G * D + c * 8;
            const long long gap = R.q_stride - G * D;    // row x of the cache head is at (x / G) q_stride + (x % G) D
            const uint32_t dst = smem_u32(S.q[s] + (c / 8) * kBox);
#pragma unroll 1
            for (int r = w * 32 + lane / LPR; r < w * 32 + 32; r += RPI) {
                const int x = x0 + s * kT + r;
                const bool fill = x < nx;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                             "l"(fill ? src + over_G(x) * gap + (long long)x * D : src), "r"(fill ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.q_ready);
        }
        const int x = x0 + s * kT + row, xr = (int)over_G(x);
        const unsigned qr = ((unsigned)(blockIdx.y * R.rows + xr) * pool.heads + h) * G + (x - xr * G);   // its row of sums (below 2^30)
        const float c2 = R.qscale;
        const int steps = kSteps * (two ? n : (n + 1 - s) / 2);   // parts of this stream's tiles
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int i = 0; i < steps; ++i) {
            const int nth = i / kSteps, b = i % kSteps, t = two ? nth : 2 * nth + s, valid = valid_of(t) - kStep * b;
            const uint32_t at = tS(s) + lanes + (uint32_t)(kStep * b);
            // (a part's last product is done before its new scores are made, so the second look never waits; it is there to
            // see every phase: one that was not looked for in time cannot be told from the next but one)
            ok = __all_sync(0xffffffffu, wait(S, &S.s_ready[s][b], nth) && (nth == 0 || wait(S, &S.pv_done[s][b], nth - 1)));
            if (!ok) break;
            tc_fence_after();
            constexpr int NC = kStep / 32;
            uint32_t z[NC][32];
#pragma unroll
            for (int c = 0; c < NC; ++c) tc_ld32_issue(at + 32u * c, z[c]);
#pragma unroll
            for (int c = 0; c < NC; ++c) tc_ld32_wait(z[c]);
            if (valid < kStep) {
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (c * 32 + k >= valid) z[c][k] = 0xff800000u;
            }
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                float mx[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t* y = z[c] + 16 * e;
                    mx[e] = __uint_as_float(y[0]);
#pragma unroll
                    for (int k = 1; k < 15; k += 2) mx[e] = max3f(mx[e], __uint_as_float(y[k]), __uint_as_float(y[k + 1]));
                    mx[e] = fmaxf(mx[e], __uint_as_float(y[15]));
                }
                top = max3f(top, mx[0], mx[1]);
            }
            top *= c2;
            const bool raise = top > m + kRaise;                 // (m = -inf: any finite logit)
            if (__any_sync(0xffffffffu, raise)) {
                const float a = raise ? ex2_fast(m - top) : 1.f;
                if (raise) {
                    m = top;
                    l *= a;
                }
                if (i > 0) {
                    // (all products but, with two parts, the last are done)
                    ok = __all_sync(0xffffffffu, wait(S, &S.pv_done[s][(i - 1) % kSteps], (i - 1) / kSteps));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tc_ld16_issue(tO(s) + lanes + (uint32_t)c, o);
                        tc_ld16_wait(o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                        tc_st16(tO(s) + lanes + (uint32_t)c, o);
                    }
                }
            }
            const float base = m == -INFINITY ? 0.f : m;
            const float2 cc = make_float2(c2, c2), nb = make_float2(-base, -base);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                uint32_t p[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float2 e = __ffma2_rn(make_float2(__uint_as_float(z[c][2 * k]), __uint_as_float(z[c][2 * k + 1])), cc, nb);
                    const float2 x = make_float2(ex2_fast(e.x), ex2_fast(e.y));
                    sum[k & 1] = __fadd2_rn(sum[k & 1], x);
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[k]) : "f"(x.y), "f"(x.x));
                }
                tc_st16(at + 16u * c, p);
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            if (t == n - 1 && valid > 0 && valid < kStep) {
                // the value rows behind the range's last key in its group of 16: their weights are 0, but what lies there may be
                // NaN (two query tiles: both streams write the zeros, each before its own product)
                const int v = v_at(t, n, L), end = (valid + 15) & ~15;
                ok = __all_sync(0xffffffffu, wait(S, &S.landed, 0));
                if (!ok) break;
                for (int x = row; x < (end - valid) * C::kBoxes * 8; x += kT)
                    *reinterpret_cast<uint4*>(S.ring[v % NS] + (x >> 3) % C::kBoxes * kBox + (kStep * b + valid + (x >> 3) / C::kBoxes) * 128 +
                                              (x & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            tc_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.p_ready[s][b]);
        }
        for (int b = 0; b < kSteps; ++b)
            if (ok && steps > 0) ok = __all_sync(0xffffffffu, wait(S, &S.pv_done[s][b], steps / kSteps - 1));
        tc_fence_after();

        // ------------------------------------------------ results
        // Both streams are through, so nothing reads the ring or is in flight to it: rows are put together there and leave
        // as one bulk copy each.  One query tile: stream 1 leaves its part of the rows first, stream 0 adds its own.
        // (The 128 KB of two query tiles leave an SM in about 4000 cycles, as whole-row stores of a warp too; half the
        // channels at a time through the query tiles it was 7000.)
        float2* other = reinterpret_cast<float2*>(S.q[1]);       // both streams' (m, l); one query tile leaves the second's place
        if (!two) other[s * kT + row] = make_float2(m, l);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const bool fine = __all_sync(0xffffffffu, ok && *(volatile int*)&S.abort == 0), join = !two && n > 1;
        float a = 1.f;
        if (join) {
            const float2 y = other[(s ^ 1) * kT + row];
            const float mm = fmaxf(m, y.x), base = mm == -INFINITY ? 0.f : mm;
            a = ex2_fast(m - base);
            l = fmaf(l, a, y.y * ex2_fast(y.x - base));
            m = mm;
        }
        const bool adds = join && s == 0, leaves = two || s == 0;
        if (adds) asm volatile("bar.sync 2, 256;" ::: "memory");
        if (fine && (leaves || join)) {
            float* mine = reinterpret_cast<float*>(S.ring[0] + ((two ? s * kT : 0) + row) * C::kPitch);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tc_ld32_issue(tO(s) + lanes + (uint32_t)c, o);
                tc_ld32_wait(o);
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    float4* to = reinterpret_cast<float4*>(mine + c + k);
                    float4 f = adds ? *to : make_float4(0.f, 0.f, 0.f, 0.f);
                    f.x = fmaf(__uint_as_float(o[k]), a, f.x);
                    f.y = fmaf(__uint_as_float(o[k + 1]), a, f.y);
                    f.z = fmaf(__uint_as_float(o[k + 2]), a, f.z);
                    f.w = fmaf(__uint_as_float(o[k + 3]), a, f.w);
                    *to = f;
                }
            }
            if (leaves && x < nx) {
                fence_proxy_async_smem();
                bulk_store(part.o + (size_t)qr * D, mine, D * 4);
            }
        }
        if (join && s == 1) asm volatile("bar.arrive 2, 256;" ::: "memory");
        if (leaves && x < nx) part.ml[qr] = make_float2(m, fine && *(volatile int*)&S.bad == 0 ? l : NAN);
        bulk_store_wait();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(S.tmem, 512);
}

// [pages * heads * ps][D] bf16, boxes of a page's rows x 64 channels, 128-byte swizzle
bool page_map(CUtensorMap* m, const void* base, const PagePool& p)
{
    EncodeTiledFn enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)p.D, (cuuint64_t)p.pages * p.heads * p.ps};
    const cuuint64_t strides[1] = {(cuuint64_t)p.D * 2};
    const cuuint32_t box[2] = {64u, (cuuint32_t)p.ps};
    const cuuint32_t estr[2] = {1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t go(const PagePool& p, const PageRows& r, const int* table, int prefix_len, const PrefixPart& part, cudaStream_t st)
{
    CUtensorMap mk, mv;
    if (!page_map(&mk, p.K, p) || !page_map(&mv, p.V, p)) return cudaErrorInvalidValue;
    const int per = prefix_tc_range(r.rows, p.heads, r.G, prefix_len);
    const dim3 grid((unsigned)(((long long)r.rows * r.G + 2 * kT - 1) / (2 * kT)), (unsigned)part.splits, (unsigned)p.heads);
    const int smem = (int)sizeof(Smem<D>) + 1024;
    static SmemOnce once;
    const cudaError_t e = once.allow(prefix_tc_kernel<D>);
    if (e != cudaSuccess) return e;
    const unsigned long long inv = ((1ull << 32) + r.G - 1) / r.G;
    prefix_tc_kernel<D><<<grid, kThreads, smem, st>>>(mk, mv, p, r, table, prefix_len, per, part, inv);
    return cudaGetLastError();
}

}  // namespace

// Keys of each CTA's range, a multiple of 128: the number of ranges for the
// shortest time.  In key tiles (1.5 us), a CTA costs those of its range and
// about two for its start, its query tiles and its sums; the rows' own pass
// about three when it finds no SMs left beside this one (8 requests of 8 heads
// behind 2048 tokens: 16.0 us with 16 ranges, 13.2 with 8); and joining the
// ranges 0.4 for every eight of them and four heads.
int prefix_tc_range(int rows, int heads, int G, int prefix_len)
{
    const int units = (int)(((long long)rows * G + 2 * kT - 1) / (2 * kT) * heads);
    const int tiles = (prefix_len + kT - 1) / kT;
    const int most = std::min({tiles, kMaxPrefixSplits, 3 * kSMs / units + 1});   // (beyond three waves nothing is gained)
    const int own = (int)std::min<long long>((long long)rows * heads, kSMs);   // (two CTAs an SM, two a unit where there are few)
    int best = tiles;
    long long cost = -1;
    for (int s = 1; s <= most; ++s) {
        const int each = (tiles + s - 1) / s, n = (tiles + each - 1) / each;
        const long long ctas = (long long)units * n;
        const long long c = 10 * ((ctas + kSMs - 1) / kSMs * (each + 2) + (ctas + own > kSMs ? 3 : 0)) + 4 * ((n + 7) / 8) * ((G + 3) / 4);
        if (cost < 0 || c < cost) { cost = c; best = each; }
    }
    return best * kT;
}

cudaError_t launch_prefix_tc(const PagePool& p, const PageRows& r, const int* table, int prefix_len, const PrefixPart& part,
                             cudaStream_t st)
{
    return p.D == 64 ? go<64>(p, r, table, prefix_len, part, st) : go<128>(p, r, table, prefix_len, part, st);
}

}  // namespace h2o
