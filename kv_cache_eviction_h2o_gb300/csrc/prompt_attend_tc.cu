// prompt_attend_tc.cu -- causal attention over packed prompts on the
// 5th-generation tensor cores (bf16).
//
// A work item is a pair of query tiles of one key head: np = 128 / groups
// positions a tile, whose query heads lie side by side as np * groups rows.
// Keys go in tiles of 128, and a CTA runs two score streams:
//   S = Q K^T        (SMEM x SMEM -> TMEM, M = 128, K = D)
//   P = 2^(c S - m)  (128 threads a stream, thread = TMEM lane = query row)
//   O += P V         (TMEM x SMEM -> TMEM, M = 128, N = D)
// one for each query tile over the same keys; where a request has queries for one
// tile only, for the even and the odd key tiles of that one, joined at the end.  S
// and P go by parts of 64 keys: S has one place, given back as soon as the threads
// have it in registers, and P two, so that the next part's scores are made while
// the threads are at this one's weights.
//
// CTAs are persistent, one an SM: warp 3 finds the items (a request's longest
// rows first), warp 0 loads queries, keys and values with TMA, warps 1 and 2
// issue their stream's products, warps 4..7 and 8..11 are the streams' threads.
// The next item's queries, keys and scores are under way while the last one's
// rows leave.  A row's maximum m is raised, and O scaled, only when a logit
// passes it by more than 2^8.  P is rounded to bf16 for the product, the sums
// l are of the unrounded weights: outputs are 0.0021 off (8 x 2048 tokens) to 0.0023
// (behind 15500), where their own rounding is 0.0016.  Two parts of P and two
// products bring that down to the rounding, and take 206 -> 261 us for 8 x 2048 tokens
// of 8 x 4 heads, 768 -> 1013 for 2048 behind 30000 of 32.
//
// Keys that a row does not see have the weight 0, which leaves a row as it is
// unless their values are infinite or NaN: a row whose weights are numbers, whose
// result is none, and not by its own values' doing (row_stands), is made again
// from the keys it sees alone (prompt_row), once the CTA is through its items (no
// wait stands behind such rows, and the call keeps registers from the loop: in
// there 8 x 2048 tokens take 6 % longer).  Value rows behind a request's last,
// which may be anything, are zeroed in shared memory.  Waits are bounded; one that
// runs out leaves NaN.
//
// Bound: the softmax threads' way from scores to weights, 1500 cycles for 64 keys of
// 128 rows a stream, 640 of them the exponentials; the tensor pipe is busy for 58 %
// and the exponentials' for 29 % of the time.  8192 tokens of 8 x 4 heads of 128: 350
// us, 1.57 PFLOP/s of the products that the mask leaves, 8 prompts of up to 2048: 142 us,
// 1.22 (4400 cycles an item before its first weights and after its last).  (Two places
// for a part's scores and one for its weights: 144 us.)
#include <algorithm>

#include "paged.h"
#include "prompt_rows.cuh"
#include "tc.cuh"

namespace h2o {

namespace {

constexpr int kT = 128;
constexpr int kThreads = 384;
constexpr uint32_t kBox = kT * 64 * 2;             // 128 rows x 64 channels: 16 KB
constexpr float kRaise = 8.f;
constexpr int kSteps = 2, kStep = kT / kSteps;     // S and P go by two parts of a tile

template <int D, bool SPLIT> struct Cfg {
    static constexpr int kBoxes = D / 64;
    static constexpr uint32_t kTile = kBoxes * kBox;
    static constexpr int kSlots = SPLIT ? (D == 128 ? 5 : 8) : D == 128 ? 4 : 6;    // K and V tiles in flight
    static constexpr int kStage = SPLIT ? 16 : 32 * 128;   // bytes of a softmax warp's rows on their way out: 64 channels of each
    static constexpr int kPitch = D * 4 + 16;          // of a row of sums (16 bytes more: no bank conflicts)
    static_assert(2 * kT * kPitch <= (2 + kSlots) * (int)kTile, "the queries' and keys' place holds them");
};

// A pair of query tiles: the request's first query row, its queries, the pair's first position; the first key row of
// this CTA's range, the request's keys before it and those of it; n: key tiles of the range; ring: tiles the ring has
// taken before; all: the request's keys.
struct Item {
    int q0, nq, p, k0, before, nk, h, n, ring, all, stop;
};

template <int D, bool SPLIT>
struct alignas(1024) Smem {
    using C = Cfg<D, SPLIT>;
    uint8_t q[2][C::kTile];
    uint8_t ring[C::kSlots][C::kTile];
    uint8_t out[8][C::kStage];
    uint64_t full[C::kSlots], empty[C::kSlots];
    uint64_t q_full, q_empty, s_ready[2], s_free[2], p_ready[2][2], pv_done[2][2], o_free[2], last;   // [stream][place of P]
    uint64_t item_full[2], item_empty[2], joined, taken;
    alignas(16) uint4 taken_at;
    float2 ml[2][kT];
    Item item[2];
    uint32_t tmem;
    int abort, any;                    // any: there was an item
    int odd;                           // there are rows to be looked at again:
    uint32_t again[2][8];              // those of the last two items' softmax warps
};
static_assert(sizeof(Smem<128, false>) <= 227 * 1024 && sizeof(Smem<128, true>) <= 227 * 1024, "one CTA's shared memory");

// accumulator fp32, bf16 A and B, A K-major, B K-major or (bit 16) N-major
template <int N, bool BMN>
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((BMN ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kT >> 4) << 24);

// The issuing warp runs its loop as a whole, so that descriptors stay in uniform registers, and one lane (`on`) issues.
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
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
template <int N> __device__ __forceinline__ void ld_cluster_f(uint32_t addr, float* x)
{
    if constexpr (N == 4) {
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(addr) : "memory");
    } else {
        const float2 w = ld_cluster_f2(addr);
        x[0] = w.x; x[1] = w.y;
    }
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(src)) : "memory");
}
// Ask for the block index of a CTA of this grid that has not started, which then never does; 16 bytes to dst.
__device__ __forceinline__ void take_cta(void* dst, uint64_t* bar)
{
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(smem_u32(dst)), "r"(smem_u32(bar)) : "memory");
}
// What take_cta left: its index (x), or -1 when none was left.
__device__ __forceinline__ int taken_cta(const void* src)
{
    unsigned long long lo, hi;
    uint32_t ok, x;
    asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(lo), "=l"(hi) : "r"(smem_u32(src)) : "memory");
    asm volatile("{\n\t.reg .b128 r;\n\t.reg .pred p;\n\tmov.b128 r, {%2, %3};\n\tmov.u32 %1, 0;\n\t"
                 "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\t"
                 "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
                 : "=r"(ok), "=r"(x)
                 : "l"(lo), "l"(hi)
                 : "memory");
    return ok ? (int)x : -1;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// descriptor of the value tile as the K x N operand, N (channels) contiguous:
// 64-channel boxes 16 KB apart (leading offset), 8 keys every 1024 B
__device__ __forceinline__ uint64_t value_desc(const void* p)
{
    return (uint64_t)((smem_u32(p) & 0x3FFFFu) >> 4) | ((uint64_t)(kBox >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// An item's tiles in the ring's order of use: K(0) .. K(L - 1), then V(t), K(t + L) for t = 0, 1, ..
// (L = 1: both streams use each tile; 2: they take turns).  Both streams wait for each tile and give each back, so that
// every barrier's phases are seen.  V(t)'s place:
__device__ __forceinline__ int v_at(int t, int n, int L) { return t + min(n, t + L); }

// At most a second or so, 2^31 cycles.
template <class Shared>
__device__ __forceinline__ bool wait(Shared& S, uint64_t* bar, int count)
{
    // the barrier's phase number `count` (from 0)
    const uint32_t parity = (uint32_t)count & 1u;
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    do {
        if (mbar_try_wait(bar, parity)) return true;
    } while (clock64() - t0 < 1ll << 31);
    *(volatile int*)&S.abort = 1;
    return false;
}

// Rows `redo` of a warp's 32 of an item, whose results are no number though the sums of their weights are (pos and g: this
// lane's row's position and head of the group).  Values that such a row does not see may have made it so, or the sum of
// finite ones, whose weights here are up to 2^8, passed fp32's range: it is made again.  Where its own infinities and NaN did, it stands.
template <int D>
__device__ __noinline__ void look_again(const PackedArgs& A, unsigned redo, const Item& it, int pos, int g, int end)
{
    using T = __nv_bfloat16;
    const T* const K = static_cast<const T*>(A.k) + it.k0 * A.k_stride + it.h * D;
    const T* const V = static_cast<const T*>(A.v) + it.k0 * A.v_stride + it.h * D;
    const int head = it.h * A.G + g, sees = min(it.all, it.all - it.nq + pos + 1);
    T* const out = static_cast<T*>(A.out) + (it.q0 + (long long)pos) * A.out_stride + head * D;
    auto row = [&](int r) { return reinterpret_cast<T*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out), r)); };
    OddRows<D> looked;
    // all of them at once: the channels that are no number in any of them, and what the first of them sees
    constexpr int U = 8;
    unsigned odd = 0, rest = redo;
#pragma unroll 1
    while (rest) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = __ffs(rest ? rest : redo) - 1;   // (the first once more where fewer than U are left)
            rest &= rest - 1;
            odd |= odd_channels<T, D>(row(r));
        }
    }
    if (row_stands(looked, odd, V, A.v_stride, __shfl_sync(0xffffffffu, sees, __ffs(redo) - 1), end)) return;
#pragma unroll 1
    for (; redo; redo &= redo - 1) {
        const int r = __ffs(redo) - 1, n = __shfl_sync(0xffffffffu, sees, r);
        T* const o = row(r);
        const T* const q = static_cast<const T*>(A.q) + (it.q0 + (long long)__shfl_sync(0xffffffffu, pos, r)) * A.q_stride + __shfl_sync(0xffffffffu, head, r) * D;
        if (!row_stands(looked, odd_channels<T, D>(o), V, A.v_stride, n, end)) prompt_row<T, D>(q, K, A.k_stride, V, A.v_stride, n, A.qscale, o);
    }
}

// SPLIT: a cluster takes one item, its CTAs ranges of the item's keys, and their sums are joined at the end.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                     const __grid_constant__ CUtensorMap mapO, const __grid_constant__ PackedArgs A, const int np, const int boxes, const int works)
{
    using C_ = Cfg<D, SPLIT>;
    constexpr int NS = C_::kSlots;
    extern __shared__ __align__(1024) unsigned char raw[];
    Smem<D, SPLIT>& S = *reinterpret_cast<Smem<D, SPLIT>*>(raw);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // (known to be uniform)
    const int G = A.G;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], 2);
        }
        mbar_init(&S.q_full, 1);
        mbar_init(&S.q_empty, 2);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&S.s_ready[s], 1);
            mbar_init(&S.s_free[s], 4);
            for (int b = 0; b < 2; ++b) {
                mbar_init(&S.p_ready[s][b], 4);
                mbar_init(&S.pv_done[s][b], 1);
            }
            mbar_init(&S.o_free[s], 4);
            mbar_init(&S.item_full[s], 1);
            mbar_init(&S.item_empty[s], 11);
        }
        mbar_init(&S.last, 2);
        mbar_init(&S.joined, 8);
        mbar_init(&S.taken, 1);
        S.odd = 0;
        for (int w = 0; w < 8; ++w) S.again[0][w] = S.again[1][w] = 0u;
        S.abort = (smem_u32(raw) & 1023u) != 0;          // (the swizzle goes by address bits; there is no other shared memory, so it is 0)
        fence_mbar_init();
    }
    if (warp == 0 && lane < 4) {
        const CUtensorMap* map = lane == 0 ? &mapQ : lane == 1 ? &mapK : lane == 2 ? &mapV : &mapO;
        asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
    }
    if (warp == 1) {
        tmem_alloc(&S.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    // a stream's scores of one part, its weights of two, its sums
    auto tS = [&](int s) { return tmem + (uint32_t)(s * kT); };
    auto tP = [&](int s, int i) { return tmem + (uint32_t)(s * kT + kStep + (i & 1) * (kStep / 2)); };
    auto tO = [&](int s) { return tmem + (uint32_t)(2 * kT + s * D); };

    // each role's walk through the items; false: no more
    int nth_item = 0;
    Item it;
    auto next = [&]() {
        const int k = nth_item++;
        const bool ok = __all_sync(0xffffffffu, wait(S, &S.item_full[k & 1], k >> 1));
        if (!ok) return false;
        it = S.item[k & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.item_empty[k & 1]);
        return it.stop == 0;
    };
    auto aborted = [&]() { return __any_sync(0xffffffffu, *(volatile int*)&S.abort != 0); };
    // key tiles of stream s's rows, and how many keys those see
    auto keys_of = [&](int s) {
        const int end = min(it.nq, it.p + (it.p + np < it.nq ? s + 1 : 1) * np);
        return max(0, min(it.nk, it.all - it.nq + end - it.before));
    };
    // parts of the tiles first, first + stride, .. that hold keys
    auto parts_of = [&](int keys, int first, int stride) {
        const int n = (keys + kT - 1) / kT, nt = n > first ? (n - first + stride - 1) / stride : 0;
        return kSteps * nt - (nt > 0 && keys - (first + (nt - 1) * stride) * kT <= kStep ? 1 : 0);
    };
    const int C = SPLIT ? (int)cluster_nctarank() : 1, rank = SPLIT ? (int)cluster_ctarank() : 0;

    if (warp == 3) {
        // ------------------------------------------------ items
        // This CTA's own, then those of CTAs that have not started, one ahead of what the others work on, so that each CTA takes
        // what its time allows (8 x 2048 tokens of 8 x 4 heads: dealt out in turn and back, the longest share was a fifth above the mean).
        int ring = 0, put = 0;
        const int pair = 2 * np;
        bool ok = true;
        int w = SPLIT ? blockIdx.x / C : blockIdx.x;
        for (int k = 0; ok && w >= 0; ++k) {
            if (k > 0) {
                if (SPLIT) break;
                if (put > 0) ok = __all_sync(0xffffffffu, wait(S, &S.item_empty[(put - 1) & 1], (put - 1) / 2));
                if (!ok || __any_sync(0xffffffffu, *(volatile int*)&S.odd)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&S.taken, 16);
                    take_cta(&S.taken_at, &S.taken);
                }
                __syncwarp();
                ok = __all_sync(0xffffffffu, wait(S, &S.taken, k - 1));
                if (!ok) break;
                w = taken_cta(&S.taken_at);
                fence_proxy_async_smem();                  // (read before it is written again)
                __syncwarp();
                if (w < 0) break;
            }
            const int x = works / A.heads - 1 - w / A.heads, i = request_at(A, x, pair);
            if (i < 0) continue;
            Item m;
            m.q0 = A.q_start[i];
            m.k0 = A.k_start[i];
            const int q1 = A.q_start[i + 1], k1 = A.k_start[i + 1];
            if (m.q0 < 0 || q1 <= m.q0 || q1 > A.rows || m.k0 < 0 || k1 < m.k0 || k1 > A.k_rows) continue;
            m.nq = q1 - m.q0;
            m.all = k1 - m.k0;
            const long long p = (long long)(x - (m.q0 / pair + i)) * pair;
            if (p < 0 || p >= m.nq) continue;
            m.p = (int)p;
            m.h = w % A.heads;
            const int seen = max(0, min(m.all, m.all - m.nq + min(m.nq, m.p + pair))), tiles = (seen + kT - 1) / kT;
            const int t0 = SPLIT ? (int)((long long)tiles * rank / C) : 0;
            m.n = (SPLIT ? (int)((long long)tiles * (rank + 1) / C) : tiles) - t0;
            m.before = t0 * kT;
            m.k0 += m.before;
            m.nk = max(0, min(m.all - m.before, m.n * kT));
            m.ring = ring;
            m.stop = 0;
            if (lane == 0) {                               // (the one before the last in this place has been taken by all)
                S.item[put & 1] = m;
                mbar_arrive(&S.item_full[put & 1]);
            }
            __syncwarp();
            ++put;
            ring += 2 * m.n;
        }
        if (put > 0) wait(S, &S.item_empty[(put - 1) & 1], (put - 1) / 2);
        if (lane == 0) {
            S.any = put > 0;
            S.item[put & 1].stop = 1;
            mbar_arrive(&S.item_full[put & 1]);
        }
    } else if (warp == 0) {
        // ------------------------------------------------ loads
        int at = 0, queries = 0;
        bool ok = true;
        const uint32_t q_bytes = (uint32_t)(np * G) * 128u * C_::kBoxes;
        while (next()) {
            if (!ok || aborted() || it.n == 0) continue;
            const bool two = it.p + np < it.nq;
            const int L = two ? 1 : 2;
            auto load = [&](const CUtensorMap* map, int t) {
                if (!ok) return;
                const int s = at % NS;
                if (at >= NS) ok = __all_sync(0xffffffffu, wait(S, &S.empty[s], at / NS - 1));
                if (!ok) return;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&S.full[s], C_::kTile);
#pragma unroll
                    for (int b = 0; b < C_::kBoxes; ++b) tma_load_3d(S.ring[s] + b * kBox, map, b * 64, it.h, it.k0 + t * kT, &S.full[s]);
                }
                __syncwarp();
                ++at;
            };
            if (queries) ok = __all_sync(0xffffffffu, wait(S, &S.q_empty, queries - 1));
            if (!ok) continue;
            ++queries;
            if (lane == 0) {
                mbar_arrive_expect_tx(&S.q_full, two ? 2 * q_bytes : q_bytes);
                for (int s = 0; s < (two ? 2 : 1); ++s)
#pragma unroll
                    for (int b = 0; b < C_::kBoxes; ++b)
                        tma_load_3d(S.q[s] + b * kBox, &mapQ, b * 64, it.h * G, it.q0 + it.p + s * np, &S.q_full);
            }
            __syncwarp();
            for (int t = 0; t < min(L, it.n); ++t) load(&mapK, t);
            for (int t = 0; t < it.n; ++t) {
                load(&mapV, t);
                if (t + L < it.n) load(&mapK, t + L);
            }
        }
        // every load has landed before the shared memory is given up, those of an abandoned sweep too
        if (queries) mbar_wait(&S.q_full, (uint32_t)(queries - 1) & 1u);
        for (int s = 0; s < min(NS, at); ++s) mbar_wait(&S.full[s], (uint32_t)((at - 1 - s) / NS) & 1u);
    } else if (warp <= 2) {
        // ------------------------------------------------ products of stream s
        const int s = warp - 1;
        const uint32_t on = elect_lane();
        const uint64_t k0 = sw128_desc(S.ring[0]), v0 = value_desc(S.ring[0]);
        const uint32_t sS = tS(s), sO = tO(s);
        bool ok = true;
        int at = 0, queries = 0, outs = 0, done = 0;     // ring tiles, items, results and parts of this stream so far
        while (next()) {
            if (!ok || aborted() || it.n == 0) continue;
            const bool two = it.p + np < it.nq;
            const uint64_t q0 = sw128_desc(S.q[two ? s : 0]);
            const int L = two ? 1 : 2, first = two ? 0 : s, stride = two ? 1 : 2, keys = keys_of(s), ni = parts_of(keys, first, stride);
            const int base = at;
            at += 2 * it.n;
            ok = __all_sync(0xffffffffu, wait(S, &S.q_full, queries));
            ++queries;
            auto release = [&](int i) {                  // when all products so far are done
                if (ok) commit(on, &S.empty[i % NS]);
            };
            // The ring's tiles in their order: those before x that are the other stream's, or whose keys no row of this one sees, go back.
            int r = base;
            auto reach = [&](int x) {
                for (; ok && r <= x; ++r) {
                    ok = __all_sync(0xffffffffu, wait(S, &S.full[r % NS], r / NS));
                    if (r < x) release(r);
                }
            };
            // where in the ring: K(t) and V(t)
            auto k_place = [&](int t) { return base + (t < L ? t : v_at(t - L, it.n, L) + 1); };
            auto v_place = [&](int t) { return base + v_at(t, it.n, L); };
            // scores of part i, in the place of those of part i - 1
            auto score = [&](int i) {
                const int b = i % kSteps, k_at = k_place(first + i / kSteps * stride);
                reach(k_at);
                if (ok && done + i > 0) ok = __all_sync(0xffffffffu, wait(S, &S.s_free[s], done + i - 1));
                if (!ok) return;
                tc_fence_after();
                const uint64_t k = k0 + (uint64_t)((uint32_t)(k_at % NS) * (C_::kTile >> 4) + (uint32_t)b * (kStep * 128u >> 4));
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    const uint64_t off = (uint64_t)(((uint32_t)(x / 4) * kBox + (uint32_t)(x % 4) * 32u) >> 4);
                    mma_ss(on, sS, q0 + off, k + off, kIdesc<kStep, false>, x > 0);
                }
                commit(on, &S.s_ready[s]);
                if (b == kSteps - 1 || i + 1 == ni) release(k_at);
                if (i + 1 == ni) commit(on, &S.q_empty);
            };
            auto values = [&](int i) {
                const int b = i % kSteps, t = first + i / kSteps * stride, v_at_ = v_place(t), gi = done + i;
                reach(v_at_);
                if (ok) ok = __all_sync(0xffffffffu, wait(S, &S.p_ready[s][gi & 1], gi >> 1));
                if (!ok) return;
                tc_fence_after();
                const uint64_t v = v0 + (uint64_t)((uint32_t)(v_at_ % NS) * (C_::kTile >> 4) + (uint32_t)b * (kStep * 128u >> 4));
                const uint32_t p = tP(s, gi);
                const int nk = (min(kStep, keys - t * kT - kStep * b) + 15) / 16;
                auto one = [&](int x) {
                    mma_ts(on, sO, p + (uint32_t)(8 * x), v + (uint64_t)((uint32_t)x * 2048u >> 4), kIdesc<D, true>, i > 0 || x > 0);
                };
                if (nk == kStep / 16) {
#pragma unroll
                    for (int x = 0; x < kStep / 16; ++x) one(x);
                } else {
                    for (int x = 0; x < nk; ++x) one(x);
                }
                commit(on, &S.pv_done[s][gi & 1]);
                if (b == kSteps - 1 || i + 1 == ni) release(v_at_);
            };
            if (ni > 0) score(0);
            for (int i = 0; i < ni; ++i) {
                if (i + 1 < ni) score(i + 1);
                if (i == 0) {                            // the last result has left O
                    if (ok && outs) ok = __all_sync(0xffffffffu, wait(S, &S.o_free[s], outs - 1));
                    ++outs;
                }
                values(i);
            }
            done += ni;
            reach(base + 2 * it.n - 1);
            // (reach leaves the last tile to its caller; it is V's last, this stream's or not)
            if (ok && (ni == 0 || v_place(first + (ni - 1) / kSteps * stride) != base + 2 * it.n - 1)) release(base + 2 * it.n - 1);
            if (ni == 0 && ok) commit(on, &S.q_empty);
        }
        // everything issued is done before TMEM is given back
        commit(on, &S.last);
        mbar_wait(&S.last, 0);
    } else {
        // ------------------------------------------------ softmax
        const int s = (warp - 4) >> 2, w = warp & 3, row = w * 32 + lane;
        const uint32_t lanes = (uint32_t)(w * 32) << 16;
        const float c2 = A.qscale;
        const int prow = row / G, g = row - prow * G;    // position and head of the row within its tile
        int done = 0, meets = 0;                         // parts of this stream so far
        bool ok = true;
        // all softmax warps, and what they have written
        auto meet = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.joined);
            if (ok) ok = __all_sync(0xffffffffu, wait(S, &S.joined, meets));
            ++meets;
            tc_fence_after();
        };
        while (next()) {
            const bool two = it.p + np < it.nq;
            const int pos = it.p + (two ? s * np : 0) + prow;
            const bool live = row < np * G && pos < it.nq;
            const int sees = min(it.nk, it.all - it.nq + pos + 1 - it.before);    // keys of this row in the range (not live: of no matter)
            const int keys = keys_of(s), first = two ? 0 : s, stride = two ? 1 : 2, nt = parts_of(keys, first, stride);
            float m = -INFINITY, l = 0.f;
            if (ok && aborted()) ok = false;
            for (int i = 0; i < nt && ok; ++i) {
                const int b = i % kSteps, t = first + i / kSteps * stride, j0 = t * kT + kStep * b, gi = done + i;
                ok = __all_sync(0xffffffffu, wait(S, &S.s_ready[s], gi));
                if (!ok) break;
                tc_fence_after();
                constexpr int NC = kStep / 32;
                uint32_t z[NC][32];
#pragma unroll
                for (int c = 0; c < NC; ++c) tc_ld32_issue(tS(s) + lanes + 32u * c, z[c]);
#pragma unroll
                for (int c = 0; c < NC; ++c) tc_ld32_wait(z[c]);
                // the next part's scores may take their place
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.s_free[s]);
                const int valid = sees - j0;
                if (__any_sync(0xffffffffu, valid < kStep)) {
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
                // the weights' place: those of the part before the last have been multiplied
                if (i > 1) ok = __all_sync(0xffffffffu, wait(S, &S.pv_done[s][gi & 1], (gi >> 1) - 1));
                if (!ok) break;
                top *= c2;
                const bool raise = top > m + kRaise;                 // (m = -inf: any finite logit)
                if (__any_sync(0xffffffffu, raise)) {
                    const float a = raise ? ex2_fast(m - top) : 1.f;
                    if (raise) {
                        m = top;
                        l *= a;
                    }
                    if (i > 0) {
                        ok = __all_sync(0xffffffffu, wait(S, &S.pv_done[s][(gi - 1) & 1], (gi - 1) >> 1));   // (all before it are done)
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
                    tc_st16(tP(s, gi) + lanes + 16u * c, p);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                // value rows behind the request's last key in its group of 16: zeros (both streams may write them, each before
                // its own product)
                const int left = it.all - it.before - j0, end = (min(keys - j0, kStep) + 15) & ~15;
                if (left < end && left > 0 && keys > j0) {
                    const int v = it.ring + v_at(t, it.n, two ? 1 : 2);
                    ok = __all_sync(0xffffffffu, wait(S, &S.full[v % NS], v / NS));
                    if (!ok) break;
                    for (int x = row; x < (end - left) * C_::kBoxes * 8; x += kT)
                        *reinterpret_cast<uint4*>(S.ring[v % NS] + (x >> 3) % C_::kBoxes * kBox + (kStep * b + left + (x >> 3) / C_::kBoxes) * 128 +
                                                  (x & 7) * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                tc_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.p_ready[s][gi & 1]);
            }
            // all products are done (each phase is looked at)
            for (int i = max(0, nt - 2); i < nt; ++i)
                if (ok) ok = __all_sync(0xffffffffu, wait(S, &S.pv_done[s][(done + i) & 1], (done + i) >> 1));
            tc_fence_after();
            done += nt;

            // ------------------------------------------------ results
            // One query tile: both streams' sums, half of the channels each.
            float a0 = 1.f, a1 = 0.f;
            if constexpr (SPLIT) {
                // both streams are through (each has seen its last product's end, and all tiles have been waited for), so the
                // queries' and keys' place is free
                meet();
                S.ml[s][row] = make_float2(m, !ok || aborted() ? NAN : nt > 0 ? l : -1.f);
                float* mine = reinterpret_cast<float*>(S.q[0] + (s * kT + row) * C_::kPitch);
                if (nt > 0) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tc_ld32_issue(tO(s) + lanes + (uint32_t)c, o);
                        tc_ld32_wait(o);
#pragma unroll
                        for (int k = 0; k < 32; k += 4) *reinterpret_cast<uint4*>(mine + c + k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                    }
                }
                tc_fence_before();
                continue;
            }
            if (!two) {
                S.ml[s][row] = make_float2(m, l);
                meet();
                const float2 x = S.ml[0][row], y = S.ml[1][row];
                const float mm = fmaxf(x.x, y.x), base = mm == -INFINITY ? 0.f : mm;
                a0 = ex2_fast(x.x - base);
                a1 = ex2_fast(y.x - base);
                l = fmaf(x.y, a0, y.y * a1);
                if (it.n == 1) a1 = 0.f;                 // (the odd stream's O is none of this item)
            }
            const bool fine = ok && !aborted();
            const float f = l == 0.f ? 0.f : 1.f / l;
            // A warp's rows go through shared memory, 64 channels at a time, and leave as one box of all their positions
            // and heads where all are there and fill it (the threads do not wait for it: an SM writes about 32 bytes a cycle,
            // and storing 16 bytes of each row took 6000 cycles an item), else 128 bytes of four rows a store.
            const unsigned lives = __ballot_sync(0xffffffffu, live);
            const bool box = boxes && lives == 0xffffffffu;
            const long long at = (long long)(it.q0 + pos) * A.out_stride + (it.h * G + g) * D;
            uint8_t* stage = S.out[warp - 4];
            float2 odd2 = make_float2(0.f, 0.f);                                // 0 times every result
            const uint32_t keep = l == 0.f || !fine ? 0u : ~0u, fill = fine ? 0u : 0x7fff7fffu;   // (no weight: zero; a wait that ran out: NaN)
            const int c0 = two ? 0 : s * 64, c1 = two ? D : min(D, c0 + 64);    // (one tile: both streams' sums, 64 channels each)
#pragma unroll 1
            for (int c = c0; c < c1; c += 64) {
                uint32_t r[32];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t o[32];
                    tc_ld32_issue(tO(two ? s : 0) + lanes + (uint32_t)(c + 32 * h), o);
                    tc_ld32_wait(o);
                    if (!two && it.n > 1) {
                        uint32_t y[32];
                        tc_ld32_issue(tO(1) + lanes + (uint32_t)(c + 32 * h), y);
                        tc_ld32_wait(y);
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(fmaf(__uint_as_float(o[k]), a0, __uint_as_float(y[k]) * a1));
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 x = __fmul2_rn(make_float2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])), make_float2(f, f));
                        odd2 = __ffma2_rn(x, make_float2(0.f, 0.f), odd2);
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r[16 * h + k]) : "f"(x.y), "f"(x.x));
                        r[16 * h + k] = (r[16 * h + k] & keep) | fill;
                    }
                }
                if (two && c + 64 == c1) {                 // the sums have been read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0 && nt > 0) mbar_arrive(&S.o_free[s]);
                }
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // what left the stage before has been read
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<uint4*>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) = make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
                if (box) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&mapO, stage, c, it.h * G, it.q0 + pos);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                } else {
                    __syncwarp();
#pragma unroll 1
                    for (int k = 0; k < 8; ++k) {
                        const int x = 4 * k + (lane >> 3), i = lane & 7;
                        const long long to = __shfl_sync(0xffffffffu, at, x);
                        const uint4 y = *reinterpret_cast<const uint4*>(stage + x * 128 + ((i ^ (x & 7)) << 4));
                        if (lives >> x & 1u) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(A.out) + to + c + i * 8) = y;
                    }
                    __syncwarp();
                }
            }
            // rows whose result is no number though the sum of their weights is one
            const unsigned again = __ballot_sync(0xffffffffu, live && fine && !(odd2.x == 0.f && odd2.y == 0.f) && l != 0.f && l == l);
            if (lane == 0) {
                S.again[(nth_item - 1) & 1][warp - 4] = again;
                if (again) S.odd = 1;
            }
            if (!two) {
                meet();                                    // (the sums have been read by the other stream's threads too)
                if (lane == 0 && nt > 0) mbar_arrive(&S.o_free[s]);
            }
            __syncwarp();
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(S.tmem, 512);
    if constexpr (!SPLIT) {
        // (items that both streams worked on are looked at by the even one's warps; the item warp has taken none after the next)
        if (S.odd && warp >= 4) {
            const int s = (warp - 4) >> 2, w = warp & 3, row = w * 32 + lane, prow = row / G;
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                const Item& it = S.item[i];
                const bool two = it.p + np < it.nq;
                const unsigned again = two ? S.again[i][warp - 4] : s == 0 ? S.again[i][w] | S.again[i][w + 4] : 0u;
                const int seen = min(it.all, it.all - it.nq + min(it.nq, it.p + (two ? s + 1 : 1) * np));
                if (again) look_again<D>(A, again, it, it.p + (two ? s * np : 0) + prow, row - prow * G, min(it.all, (seen + 15) & ~15));
            }
        }
    }
    if constexpr (SPLIT) {
        // the cluster's sums, a warp a row: of both streams where they had one tile's keys in turn
        cluster_arrive();
        cluster_wait();
        if (S.any) {
            const Item it = S.item[0];
            const bool two = it.p + np < it.nq;
            const int rows = min(it.nq - it.p, 2 * np) * G;
            constexpr int V4 = D / 32;
            unsigned again = 0;                                  // (rows <= 256, so there are at most 11 turns)
            int turn = 0;
#pragma unroll 1
            for (int x = rank * (kThreads / 32) + warp; x < rows; x += C * (kThreads / 32), ++turn) {
                const int s = x / (np * G), r = x - s * np * G, pos = it.p + x / G, g = x % G;
                float m = -INFINITY, l = 0.f, o[V4] = {};
#pragma unroll 1
                for (int c = 0; c < (two ? 1 : 2) * C; ++c) {
                    const int from = two ? c : c >> 1, st = two ? s : c & 1;
                    const float2 y = ld_cluster_f2(map_to_rank(&S.ml[st][r], from));
                    if (y.y < 0.f) continue;                     // no keys, and no sums
                    float v[V4];
                    ld_cluster_f<V4>(map_to_rank(S.q[0] + (st * kT + r) * C_::kPitch, from) + lane * V4 * 4, v);
                    const float mn = fmaxf(m, y.x), base = mn == -INFINITY ? 0.f : mn, a = ex2_fast(m - base), b = ex2_fast(y.x - base);
                    m = mn;
                    l = fmaf(l, a, y.y * b);
#pragma unroll
                    for (int e = 0; e < V4; ++e) o[e] = fmaf(o[e], a, v[e] * b);
                }
                const float f = 1.f / l;
                bool odd = false;
#pragma unroll
                for (int e = 0; e < V4; ++e) {
                    o[e] = l == 0.f ? 0.f : o[e] * f;
                    odd |= !(fabsf(o[e]) < INFINITY);
                }
                if (__any_sync(0xffffffffu, odd) && l == l) again |= 1u << turn;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(A.out) + (it.q0 + (long long)pos) * A.out_stride + (it.h * G + g) * D;
                uint32_t w[V4 / 2];
#pragma unroll
                for (int i = 0; i < V4 / 2; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(o[2 * i + 1]), "f"(o[2 * i]));
                if constexpr (V4 == 4) *reinterpret_cast<uint2*>(out + lane * 4) = make_uint2(w[0], w[1]);
                else *reinterpret_cast<uint32_t*>(out + lane * 2) = w[0];
            }
            // no number, though the weights are: as look_again
            if (again) {
                const long long k0 = it.k0 - it.before;
                const __nv_bfloat16* const K = static_cast<const __nv_bfloat16*>(A.k) + k0 * A.k_stride + it.h * D;
                const __nv_bfloat16* const V = static_cast<const __nv_bfloat16*>(A.v) + k0 * A.v_stride + it.h * D;
                const int end = min(it.all, (it.all - it.nq + min(it.nq, it.p + 2 * np) + 15) & ~15);
                OddRows<D> looked;
#pragma unroll 1
                for (; again; again &= again - 1) {
                    const int x = rank * (kThreads / 32) + warp + (__ffs(again) - 1) * C * (kThreads / 32), pos = it.p + x / G, head = it.h * G + x % G;
                    const int seen = min(it.all, it.all - it.nq + pos + 1);
                    __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(A.out) + (it.q0 + (long long)pos) * A.out_stride + head * D;
                    if (!row_stands(looked, odd_channels<__nv_bfloat16, D>(out), V, A.v_stride, seen, end))
                        prompt_row<__nv_bfloat16, D>(static_cast<const __nv_bfloat16*>(A.q) + (it.q0 + (long long)pos) * A.q_stride + head * D, K, A.k_stride, V,
                                                     A.v_stride, seen, A.qscale, out);
                }
            }
        }
        cluster_arrive();
        cluster_wait();                                    // no CTA leaves while another reads its sums
    }
}

// rows [n][heads][D] bf16, `stride` elements apart; boxes of 64 channels x bh heads x bn rows, 128-byte swizzle
bool rows_map(CUtensorMap* m, const void* base, int D, int heads, int n, long long stride, int bh, int bn)
{
    EncodeTiledFn enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)n};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)bh, (cuuint32_t)bn};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t go(const PackedArgs& a, cudaStream_t st)
{
    const int np = kT / a.G;
    CUtensorMap mq, mk, mv, mo;
    const int boxes = (a.G & (a.G - 1)) == 0;              // a warp's 32 rows are whole positions
    if (!rows_map(&mo, a.out, D, a.heads * a.G, a.rows, a.out_stride, a.G, 32 / a.G) || !rows_map(&mq, a.q, D, a.heads * a.G, a.rows, a.q_stride, a.G, np) || !rows_map(&mk, a.k, D, a.heads, a.k_rows, a.k_stride, 1, kT) ||
        !rows_map(&mv, a.v, D, a.heads, a.k_rows, a.v_stride, 1, kT))
        return cudaErrorInvalidValue;
    const long long works = ((long long)a.rows / (2 * np) + a.requests) * a.heads;
    // where there are fewer items than SMs, a cluster of CTAs for each
    const long long items = (long long)a.heads * a.requests * (((long long)a.rows / a.requests + 2 * np - 1) / (2 * np) + (a.rows < a.requests));
    const int C = key_cluster(items, (long long)a.k_rows / a.requests, 1, 2 * kT);
    if (works * C > INT32_MAX) return cudaErrorInvalidValue;
    if (C > 1) {
        const auto kernel = prompt_tc_kernel<D, true>;
        static SmemOnce once;
        const cudaError_t e = once.allow(kernel, true);
        if (e != cudaSuccess) return e;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)C;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(works * C));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = sizeof(Smem<D, true>);
        cfg.stream = st;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kernel, mq, mk, mv, mo, a, np, boxes, (int)works);
    }
    const auto kernel = prompt_tc_kernel<D, false>;
    static SmemOnce once;
    const cudaError_t e = once.allow(kernel);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)works, kThreads, sizeof(Smem<D, false>), st>>>(mq, mk, mv, mo, a, np, boxes, (int)works);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_tc(const PackedArgs& a, int D, cudaStream_t st) { return D == 64 ? go<64>(a, st) : go<128>(a, st); }

}  // namespace h2o
