// prefix.cu -- the shared prefix's part of h2o_prefix_attend: every query row
// against the same keys, so the keys are read once for a tile of rows and the
// products are matrix products over all rows of a cache head.  The prefix is
// split into ranges of keys; each leaves its running maximum, sum and values
// per query row for the rows' own pass to join.
#include <algorithm>

#include "common.cuh"
#include "paged.h"

namespace h2o {

namespace {

// fp32 on the CUDA cores (bf16: prefix_tc.cu).  64 query rows x 64 keys a step: 16 x 16
// threads, 4 x 4 logits and 4 x D / 16 output channels each.

constexpr int kRows = 64, kCols = 64;

template <int D>
struct SimtSmem {
    float q[kRows][D + 4];
    float kv[kCols][D + 4];            // keys, then the values of the same positions
    float p[kRows][kCols + 4];
};

// prefix positions [j0, j0 + 64) of one cache head, zeros from j1 on: asked for
// into registers, and put into S.kv when that is free
template <int D>
struct Rows64 {
    static constexpr int VPR = D / 4, N = kCols * VPR / 256;
    float4 v[N];
    __device__ __forceinline__ void ask(const float* src, const PagePool& pool, const int* table, int h, int j0, int j1, bool& bad)
    {
        const int sh = __ffs(pool.ps) - 1;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int k = threadIdx.x + i * 256, j = j0 + k / VPR, e = (k % VPR) * 4;
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j < j1) {
                const int pg = table[j >> sh];
                if ((unsigned)pg < (unsigned)pool.pages)
                    v[i] = *reinterpret_cast<const float4*>(src + (((size_t)pg * pool.heads + h) * pool.ps + (j & (pool.ps - 1))) * D + e);
                else
                    bad = true;
            }
        }
    }
    __device__ __forceinline__ void put(float (*dst)[D + 4]) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int k = threadIdx.x + i * 256;
            *reinterpret_cast<float4*>(&dst[k / VPR][(k % VPR) * 4]) = v[i];
        }
    }
};

// grid: (query tile, split, cache head)
template <int D>
__global__ void __launch_bounds__(256, 2) prefix_simt_kernel(const PagePool pool, const PageRows R, const int* __restrict__ table,
                                                          const int prefix_len, const int per, const PrefixPart part)
{
    extern __shared__ __align__(16) unsigned char raw[];
    SimtSmem<D>& S = *reinterpret_cast<SimtSmem<D>*>(raw);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int h = blockIdx.z, x0 = blockIdx.x * kRows, G = R.G, nx = R.rows * G;
    const int j0 = blockIdx.y * per, j1 = min(prefix_len, j0 + per);
    grid_launch_dependents();          // the rows' own pass may start on what SMs are left; it waits before it reads sums
    const bool live = x0 + ty * 4 < nx;    // (of the last tile, warps without rows only help loading)
    bool bad = false;
    const float* K = static_cast<const float*>(pool.K);
    const float* V = static_cast<const float*>(pool.V);
    Rows64<D> next;                    // keys while values are in use, and the other way round
    next.ask(K, pool, table, h, j0, j1, bad);
    for (int i = tid; i < kRows * D / 4; i += 256) {
        const int r = i / (D / 4), e = i % (D / 4) * 4, x = x0 + r;
        *reinterpret_cast<float4*>(&S.q[r][e]) =
            x < nx ? *reinterpret_cast<const float4*>(static_cast<const float*>(R.q) + (size_t)(x / G) * R.q_stride + (size_t)(h * G + x % G) * D + e)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    constexpr int NJ = D / 64;
    float m[4], l[4], o[4][NJ][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][j][k] = 0.f;
    }
    for (int j = j0; j < j1; j += kCols) {
        __syncthreads();
        next.put(S.kv);
        next.ask(V, pool, table, h, j, j1, bad);
        __syncthreads();
        float z[4][4] = {};
        if (live)
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = *reinterpret_cast<const float4*>(&S.q[ty * 4 + i][d]);
                    b[i] = *reinterpret_cast<const float4*>(&S.kv[tx + 16 * i][d]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        z[i][k] = fmaf(a[i].x, b[k].x, z[i][k]);
                        z[i][k] = fmaf(a[i].y, b[k].y, z[i][k]);
                        z[i][k] = fmaf(a[i].z, b[k].z, z[i][k]);
                        z[i][k] = fmaf(a[i].w, b[k].w, z[i][k]);
                    }
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float t = -INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                z[i][k] = j + tx + 16 * k < j1 ? z[i][k] * R.qscale : -INFINITY;
                t = fmaxf(t, z[i][k]);
            }
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
            const float mn = fmaxf(m[i], t), base = mn == -INFINITY ? 0.f : mn, a = ex2_approx(m[i] - base);
            m[i] = mn;
            l[i] *= a;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float p = ex2_approx(z[i][k] - base);
                l[i] += p;
                S.p[ty * 4 + i][tx + 16 * k] = p;
            }
#pragma unroll
            for (int n = 0; n < NJ; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[i][n][k] *= a;
        }
        __syncthreads();
        next.put(S.kv);
        if (j + kCols < j1) next.ask(K, pool, table, h, j + kCols, j1, bad);
        __syncthreads();
        if (live)
#pragma unroll 2
            for (int c = 0; c < kCols; c += 4) {
                float4 p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(&S.p[ty * 4 + i][c]);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int n = 0; n < NJ; ++n) {
                        const float4 v = *reinterpret_cast<const float4*>(&S.kv[c + k][n * 64 + tx * 4]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float w = k == 0 ? p[i].x : k == 1 ? p[i].y : k == 2 ? p[i].z : p[i].w;
                            o[i][n][0] = fmaf(w, v.x, o[i][n][0]);
                            o[i][n][1] = fmaf(w, v.y, o[i][n][1]);
                            o[i][n][2] = fmaf(w, v.z, o[i][n][2]);
                            o[i][n][3] = fmaf(w, v.w, o[i][n][3]);
                        }
                    }
            }
    }
    // a page that is not there: every row of this range is NaN
    if (__syncthreads_or(bad)) l[0] = l[1] = l[2] = l[3] = NAN;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int x = x0 + ty * 4 + i;
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
        if (x >= nx) continue;
        const size_t qr = ((size_t)blockIdx.y * R.rows * pool.heads + (size_t)(x / G) * pool.heads + h) * G + x % G;
        if (tx == 0) part.ml[qr] = make_float2(m[i], l[i]);
#pragma unroll
        for (int n = 0; n < NJ; ++n)
            *reinterpret_cast<float4*>(part.o + qr * D + n * 64 + tx * 4) = make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
    }
}

// Keys of each range, a multiple of 64: the number of ranges that makes the
// shortest sequence of waves (two CTAs an SM), a CTA costing its steps and
// about one more for its start and its sums.
int range_keys(int rows, int heads, int G, int prefix_len)
{
    const long long tiles = ((long long)rows * G + kRows - 1) / kRows * heads;
    const int steps = (prefix_len + kCols - 1) / kCols, resident = 2 * kSMs;
    const int most = (int)std::min<long long>(std::min(steps, kMaxPrefixSplits), 3 * resident / tiles + 1);
    int best = steps;
    long long cost = -1;
    for (int s = 1; s <= most; ++s) {
        const int each = (steps + s - 1) / s;
        const long long ctas = tiles * ((steps + each - 1) / each), c = (ctas + resident - 1) / resident * (each + 1);
        if (cost < 0 || c < cost) { cost = c; best = each; }
    }
    return best * kCols;
}

}  // namespace

int prefix_splits(int rows, int heads, int G, int D, int prefix_len, int dtype)
{
    if (rows < 1 || prefix_len < 1) return 0;
    const int per = dtype ? prefix_tc_range(rows, heads, G, prefix_len) : range_keys(rows, heads, G, prefix_len);
    return (prefix_len + per - 1) / per;
}

cudaError_t launch_prefix(const PagePool& p, const PageRows& r, const int* prefix_table, int prefix_len,
                          const PrefixPart& part, cudaStream_t st)
{
    if (p.dtype) return launch_prefix_tc(p, r, prefix_table, prefix_len, part, st);
    const int per = range_keys(r.rows, p.heads, r.G, prefix_len);
    const dim3 grid((unsigned)((r.rows * (long long)r.G + kRows - 1) / kRows), (unsigned)part.splits, (unsigned)p.heads);
    auto go = [&](auto d) {
        constexpr int D = decltype(d)::value;
        const int smem = (int)sizeof(SimtSmem<D>);
        static SmemOnce once;
        const cudaError_t e = once.allow(prefix_simt_kernel<D>);
        if (e != cudaSuccess) return e;
        prefix_simt_kernel<D><<<grid, 256, smem, st>>>(p, r, prefix_table, prefix_len, per, part);
        return cudaGetLastError();
    };
    return p.D == 64 ? go(std::integral_constant<int, 64>()) : go(std::integral_constant<int, 128>());
}

}  // namespace h2o
