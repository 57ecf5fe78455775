// prompt_attend.cu -- causal attention over packed prompts in fp32, on the
// tensor cores' bf16 products, six to one.
//
// x = h + m + l, each the bf16 nearest to what is left, holds all 24 bits of x from
// 2^-110 on (below, what is left is half of bf16's last step, 2^-134).  Of the nine products of two such sums the six from h h' to 2^-16
// of it (h h', h m', m h', h l', m m', l h') are made, and the others are below
// 2^-23 of the product; sums of 16 products are added up in fp32.  (Three products
// of tf32 halves took as long: 8 x 2048 tokens of 8 x 4 heads of 128, 3.4 ms, of 3.3
// before sums of 16 and 3.8 with them.)
//
// A CTA of four warps takes tiles of 16 query rows (a request's positions, the
// heads of a group side by side) and key tiles of 32 through a ring of two in
// shared memory.  Warps share the rows or, where requests have few, the keys of
// each tile (WK of them); a cluster's CTAs share the key tiles where there are
// few tiles of rows, and their sums are joined at the end.  Channels and keys are
// paired with product indexes so that every operand is read 16 bytes at a time
// from rows whose length lets 8 lanes meet no bank twice.
//
// Bound: issue, of the products and of the splits: 8 prompts of up to 2048 tokens of 8 x 4 heads of
// 128 take 3.82 ms, 45 TFLOP/s of the formula's products and six times that made.
// Each warp splits the keys it reads, four times a CTA.  128 tokens of 4 heads of 64
// take 9.1 us, the latency of four key tiles a warp and of the launch.
#include <algorithm>

#include "prompt_rows.cuh"

namespace h2o {

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kKeys = 32;                              // of a tile

template <int D, int WK> struct alignas(16) Smem {
    static constexpr int kRows = 16 * kWarps / WK, kStages = 2;
    float q[kRows][D + 16];
    float k[kStages][kKeys][D + 16];
    float v[kStages][kKeys][D + 4];
    float2 ml[kWarps][16];                             // of each warp's rows
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool fill)
{
    // bytes not read are written as zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(fill ? 16 : 0) : "memory");
}

__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// x and y as three pairs of bf16.  (An infinity or NaN, or what rounds to one, leaves a NaN: the sum is no number.)
__device__ __forceinline__ void split(float x, float y, uint32_t& h, uint32_t& m, uint32_t& l)
{
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(y), "f"(x));
    x -= __uint_as_float(h << 16);
    y -= __uint_as_float(h & 0xffff0000u);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(m) : "f"(y), "f"(x));
    x -= __uint_as_float(m << 16);
    y -= __uint_as_float(m & 0xffff0000u);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(l) : "f"(y), "f"(x));
}
// c[i] += a b[i] for a and b in three parts.  The tensor cores cut a sum's bits off where an addition rounds, which adds up
// over long sums (20000 keys: 8e-6 off), so sums of 16 terms are added up by the FMA pipe; the small products come first
// and those of one sum apart from one another.
template <int N>
__device__ __forceinline__ void mma_six(float (*c)[4], const uint32_t (&a)[3][4], const uint32_t (&b)[N][3][2])
{
    constexpr int pa[6] = {2, 1, 0, 1, 0, 0}, pb[6] = {0, 1, 2, 0, 1, 0};
    float s[N][4] = {};
#pragma unroll
    for (int p = 0; p < 6; ++p)
#pragma unroll
        for (int i = 0; i < N; ++i) mma16(s[i], a[pa[p]], b[i][pb[p]]);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[i][e] += s[i][e];
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// A cluster takes one tile of query rows of one key head, its CTAs ranges of the keys.
template <int D, int WK>
__global__ void __launch_bounds__(kThreads) prompt_f32_kernel(const PackedArgs A, const int np, const int works)
{
    using M = Smem<D, WK>;
    constexpr int R = M::kRows, NS = M::kStages, NT = kKeys / 8 / WK;       // NT: steps of eight keys of a warp's part of a tile
    extern __shared__ __align__(16) unsigned char raw[];
    M& S = *reinterpret_cast<M*>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank(), G = A.G;
    const int w = blockIdx.x / C, x = works / A.heads - 1 - w / A.heads, h = w % A.heads;   // (a request's longest rows first)
    // (what follows is the same for the whole cluster)
    const int i = request_at(A, x, np);
    if (i < 0) return;
    const int q0 = A.q_start[i], q1 = A.q_start[i + 1], k0 = A.k_start[i], k1 = A.k_start[i + 1];
    if (q0 < 0 || q1 <= q0 || q1 > A.rows || k0 < 0 || k1 < k0 || k1 > A.k_rows) return;
    const int nq = q1 - q0, nk = k1 - k0;
    const long long first = (long long)(x - (q0 / np + i)) * np;
    if (first < 0 || first >= nq) return;
    const int p = (int)first, end = max(0, min(nk, nk - nq + min(nq, p + np)));   // keys that any of its rows sees
    const int tiles = (end + kKeys - 1) / kKeys, t_0 = (int)((long long)tiles * rank / C), t_1 = (int)((long long)tiles * (rank + 1) / C);
    const float* const Q = static_cast<const float*>(A.q);
    const float* const K = static_cast<const float*>(A.k) + (long long)k0 * A.k_stride + h * D;
    const float* const V = static_cast<const float*>(A.v) + (long long)k0 * A.v_stride + h * D;

    // row r of the tile: position p + r / G, head r % G
    constexpr int CH = D / 4;
    for (int c = tid; c < R * CH; c += kThreads) {
        const int r = c / CH, e = (c % CH) * 4, pos = p + r / G;
        const bool in = r < np * G && pos < nq;
        cp_async16(&S.q[r][e], in ? Q + (long long)(q0 + pos) * A.q_stride + (h * G + r % G) * D + e : Q, in);
    }
    auto ask = [&](int tile, int stage) {
        if (tile < t_1)
            for (int c = tid; c < kKeys * CH; c += kThreads) {
                const int r = c / CH, e = (c % CH) * 4, key = tile * kKeys + r;
                const bool in = key < nk;                  // keys behind the request's last are zeros
                cp_async16(&S.k[stage][r][e], in ? K + key * A.k_stride + e : K, in);
                cp_async16(&S.v[stage][r][e], in ? V + key * A.v_stride + e : V, in);
            }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int s = 0; s < NS - 1; ++s) ask(t_0 + s, s);

    const int wr = warp / WK, wk = warp % WK;              // which rows, which keys of a tile
    // keys that rows g and g + 8 of this warp see
    int sees[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int pos = p + (wr * 16 + g + 8 * e) / G;
        sees[e] = max(0, min(end, nk - nq + pos + 1));
    }
    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    for (int tile = t_0; tile < t_1; ++tile) {
        const int stage = (tile - t_0) % NS;
        ask(tile + NS - 1, (tile - t_0 + NS - 1) % NS);
        asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
        __syncthreads();
        float z[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) z[n][0] = z[n][1] = z[n][2] = z[n][3] = 0.f;
#pragma unroll (NT == 1 ? 4 : 1)
        for (int j = 0; j < D / 16; ++j) {                 // channels 16 j + 4 t + (0, 1) and (2, 3): product indexes 2 t, + 1 and + 8, + 9
            const float4 x0 = *reinterpret_cast<const float4*>(&S.q[wr * 16 + g][16 * j + 4 * t]);
            const float4 x1 = *reinterpret_cast<const float4*>(&S.q[wr * 16 + g + 8][16 * j + 4 * t]);
            uint32_t a[3][4];
            split(x0.x, x0.y, a[0][0], a[1][0], a[2][0]);
            split(x1.x, x1.y, a[0][1], a[1][1], a[2][1]);
            split(x0.z, x0.w, a[0][2], a[1][2], a[2][2]);
            split(x1.z, x1.w, a[0][3], a[1][3], a[2][3]);
            uint32_t b[NT][3][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float4 y = *reinterpret_cast<const float4*>(&S.k[stage][(wk * NT + n) * 8 + g][16 * j + 4 * t]);
                split(y.x, y.y, b[n][0][0], b[n][1][0], b[n][2][0]);
                split(y.z, y.w, b[n][0][1], b[n][1][1], b[n][2][1]);
            }
            mma_six<NT>(z, a, b);
        }
        // columns 2 t, 2 t + 1 of step n are its keys; rows g (0, 1) and g + 8 (2, 3)
        float a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float top = -INFINITY;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float& y = z[n][2 * e + c];
                    y = tile * kKeys + (wk * NT + n) * 8 + 2 * t + c < sees[e] ? y * A.qscale : -INFINITY;
                    top = fmaxf(top, y);
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float mn = fmaxf(m[e], top), base = mn == -INFINITY ? 0.f : mn;
            a[e] = ex2_approx(m[e] - base);
            m[e] = mn;
            l[e] *= a[e];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float& y = z[n][2 * e + c];
                    y = ex2_approx(y - base);
                    l[e] += y;
                }
        }
        if (__any_sync(0xffffffffu, a[0] != 1.f || a[1] != 1.f)) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n) { o[n][0] *= a[0]; o[n][1] *= a[0]; o[n][2] *= a[1]; o[n][3] *= a[1]; }
        }
        constexpr int NP = (NT + 1) / 2;                   // steps of 16 keys (of 8 and nothing where a warp has 8)
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const bool both = 2 * n + 1 < NT;
            uint32_t w[3][4] = {};
            split(z[2 * n][0], z[2 * n][1], w[0][0], w[1][0], w[2][0]);
            split(z[2 * n][2], z[2 * n][3], w[0][1], w[1][1], w[2][1]);
            if (both) {
                split(z[(2 * n + 1) % NT][0], z[(2 * n + 1) % NT][1], w[0][2], w[1][2], w[2][2]);
                split(z[(2 * n + 1) % NT][2], z[(2 * n + 1) % NT][3], w[0][3], w[1][3], w[2][3]);
            }
            const float* v = S.v[stage][(wk * NT + 2 * n) * 8 + 2 * t];
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {             // channels 32 c + 4 g + (0 .. 3): column g of four steps
                float x[4][4] = {};                        // of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
                for (int r = 0; r < (both ? 4 : 2); ++r) {
                    const float4 y = *reinterpret_cast<const float4*>(v + ((r & 1) + (r >> 1) * 8) * (D + 4) + 32 * c + 4 * g);
                    x[r][0] = y.x; x[r][1] = y.y; x[r][2] = y.z; x[r][3] = y.w;
                }
                uint32_t b[4][3][2] = {};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    split(x[0][s], x[1][s], b[s][0][0], b[s][1][0], b[s][2][0]);
                    if (both) split(x[2][s], x[3][s], b[s][0][1], b[s][1][1], b[s][2][1]);
                }
                mma_six<4>(o + 4 * c, w, b);
            }
        }
        __syncthreads();                                   // the stage may be written again
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    // the warps' sums, in the place of the keys and values: [warp][16][D], then the CTA's, then the cluster's
    float* part = &S.k[0][0][0];
    static_assert(sizeof(M::k) + sizeof(M::v) >= sizeof(float) * kWarps * 16 * D, "they fit");
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        float* to = part + (warp * 16 + g + 8 * e) * D + 8 * t;
        // columns 2 t, 2 t + 1 of steps 4 c + s: channels 32 c + 8 t + s and + 4
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            *reinterpret_cast<float4*>(to + 32 * c) = make_float4(o[4 * c][2 * e], o[4 * c + 1][2 * e], o[4 * c + 2][2 * e], o[4 * c + 3][2 * e]);
            *reinterpret_cast<float4*>(to + 32 * c + 4) = make_float4(o[4 * c][2 * e + 1], o[4 * c + 1][2 * e + 1], o[4 * c + 2][2 * e + 1], o[4 * c + 3][2 * e + 1]);
        }
        if (t == 0) S.ml[warp][g + 8 * e] = make_float2(m[e], l[e]);
    }
    cluster_arrive();
    cluster_wait();
    // each row by D / 4 lanes: the parts of WK warps of every CTA
    constexpr int LR = D / 4;
    OddRows<D> looked;
#pragma unroll 1
    for (int r0 = (rank * kThreads + tid) / LR; r0 < (R + 31) / 32 * 32; r0 += C * kThreads / LR) {   // (whole warps)
        const int r = min(r0, R - 1), e = (tid % LR) * 4, pos = p + r / G;
        const bool in = r0 < R && r < np * G && pos < nq;
        float mm = -INFINITY, ll = 0.f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < C; ++c)
            for (int k = 0; k < WK; ++k) {
                const int u = r / 16 * WK + k;             // the warp
                const float2 x2 = ld_cluster_f2(map_to_rank(&S.ml[u][r % 16], c));
                const float4 v = ld_cluster_f4(map_to_rank(part + (u * 16 + r % 16) * D + e, c));
                const float mn = fmaxf(mm, x2.x), base = mn == -INFINITY ? 0.f : mn, a = ex2_approx(mm - base), b = ex2_approx(x2.x - base);
                mm = mn;
                ll = fmaf(ll, a, x2.y * b);
                y = make_float4(fmaf(y.x, a, v.x * b), fmaf(y.y, a, v.y * b), fmaf(y.z, a, v.z * b), fmaf(y.w, a, v.w * b));
            }
        const float f = 1.f / ll;
        y = ll == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
        float* out = static_cast<float*>(A.out) + (long long)(q0 + pos) * A.out_stride + (h * G + r % G) * D;
        if (in) *reinterpret_cast<float4*>(out + e) = y;
        // Rows whose result is no number: what they do not see may have made it so, or values of theirs whose bf16 parts are
        // none.  They are made again unless a NaN among what they see has.
        const bool odd = in && !(fabsf(y.x) < INFINITY && fabsf(y.y) < INFINITY && fabsf(y.z) < INFINITY && fabsf(y.w) < INFINITY);
        unsigned redo = __ballot_sync(0xffffffffu, odd);
        __syncwarp();
        while (redo) {
            const int from = (__ffs(redo) - 1) / LR * LR;
            redo &= LR == 32 ? 0u : ~(((1u << LR % 32) - 1u) << from);
            const int rr = __shfl_sync(0xffffffffu, r, from), rpos = p + rr / G, seen = min(nk, nk - nq + rpos + 1);
            const float rl = __shfl_sync(0xffffffffu, ll, from);
            const float* q = Q + (long long)(q0 + rpos) * A.q_stride + (h * G + rr % G) * D;
            float* to = static_cast<float*>(A.out) + (long long)(q0 + rpos) * A.out_stride + (h * G + rr % G) * D;
            if (rl != rl ? nan_logit(looked, q, K, A.k_stride, seen) : row_stands(looked, odd_channels<float, D>(to), V, A.v_stride, seen, nk)) continue;
            prompt_row<float, D>(q, K, A.k_stride, V, A.v_stride, seen, A.qscale, to);
        }
    }
    cluster_arrive();
    cluster_wait();                                        // no CTA leaves while another reads its sums
}

template <int D, int WK>
cudaError_t go(const PackedArgs& a, cudaStream_t st)
{
    using M = Smem<D, WK>;
    const auto kernel = prompt_f32_kernel<D, WK>;
    static SmemOnce once;
    const cudaError_t e = once.allow(kernel, true);
    if (e != cudaSuccess) return e;
    const int np = M::kRows / a.G;
    const long long works = ((long long)a.rows / np + a.requests) * a.heads;
    const long long tiles = (long long)a.heads * a.requests * (((long long)a.rows / a.requests + np - 1) / np + (a.rows < a.requests));
    const int C = key_cluster(tiles, (long long)a.k_rows / a.requests, 2, 4 * kKeys);
    if (works * C > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(works * C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(M);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = C > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a, np, (int)works);
}

// no keys at all: rows of zeros, by a warp a row and head
template <typename T, int D>
__global__ void __launch_bounds__(256) prompt_empty_kernel(const PackedArgs A)
{
    const long long u = (long long)blockIdx.x * 8 + (threadIdx.x >> 5), hq = (long long)A.heads * A.G;
    const int row = (int)(u / hq), h = (int)(u % hq);
    if (row >= A.rows) return;
    int lo = 0, hi = A.requests;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (A.q_start[mid] <= row) lo = mid; else hi = mid;
    }
    if (row < A.q_start[lo] || row >= A.q_start[lo + 1] || A.q_start[lo] < 0 || A.q_start[lo + 1] > A.rows || A.k_start[lo] != 0 || A.k_start[lo + 1] != 0) return;
    prompt_row<T, D>(static_cast<const T*>(A.q) + row * A.q_stride + h * D, nullptr, 0, nullptr, 0, 0, 1.f,
                     static_cast<T*>(A.out) + row * A.out_stride + h * D);
}

}  // namespace

cudaError_t launch_prompt_attend(const PackedArgs& a, int D, int dtype, cudaStream_t st)
{
    if (!a.k_rows) {
        const unsigned grid = (unsigned)(((long long)a.rows * a.heads * a.G + 7) / 8);
        if (dtype) D == 64 ? prompt_empty_kernel<__nv_bfloat16, 64><<<grid, 256, 0, st>>>(a) : prompt_empty_kernel<__nv_bfloat16, 128><<<grid, 256, 0, st>>>(a);
        else D == 64 ? prompt_empty_kernel<float, 64><<<grid, 256, 0, st>>>(a) : prompt_empty_kernel<float, 128><<<grid, 256, 0, st>>>(a);
        return cudaGetLastError();
    }
    if (dtype) return launch_prompt_tc(a, D, st);
    // Few rows a request, or so few tiles of 64 that tiles of 16 rows do not fill the GPU either: the warps share keys (128
    // tokens of 4 heads: 16.6 us by rows, 10.4 so).
    const long long most = (a.rows + a.requests - 1) / a.requests * (long long)a.G, tiles = (most + 63) / 64 * a.requests * a.heads;
    if (most <= 24 || tiles * 4 <= kSMs) return D == 64 ? go<64, 4>(a, st) : go<128, 4>(a, st);
    return D == 64 ? go<64, 1>(a, st) : go<128, 1>(a, st);
}

}  // namespace h2o
