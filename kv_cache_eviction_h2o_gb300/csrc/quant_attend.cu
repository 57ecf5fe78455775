// quant_attend.cu -- attention of single tokens over quantised paged caches
// (h2o_page_quant_attend), on the CUDA cores.
//
// A warp a query row of one head: logits scale ks q.ck, weights 2^(z - m) vs on
// the value codes, keys one after another.
#include "common.cuh"
#include "prompts.h"

namespace h2o {

namespace {

constexpr int kWarps = 8;

template <int E, int BITS>
__device__ __forceinline__ void codes_of(const unsigned char* row, int lane, float* x)
{
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = lane * E + e;
        if constexpr (BITS == 8) x[e] = (float)reinterpret_cast<const signed char*>(row)[c];
        else x[e] = (float)((row[c >> 1] >> ((c & 1) * 4) & 15) - 8);
    }
}

template <typename T, int D, int BITS>
__global__ void __launch_bounds__(kWarps * 32) quant_rows_kernel(const QuantPool P, const PageRows R)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, hq = P.heads * R.G, sh = __ffs(P.ps) - 1;
    const long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int row = (int)(u / hq), h = (int)(u % hq);
    if (row >= R.rows) return;
    const int seq = R.seq[row], pos = R.pos[row];
    if (seq < 0) return;
    bool bad = seq >= R.requests || (pos >= 0 && (pos >> sh) >= R.width);
    const int n = bad || pos < 0 ? 0 : pos + 1;
    float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
    load_vec<T, E>(static_cast<const T*>(R.q) + row * R.q_stride + h * D + lane * E, q);
    for (int j = 0; j < n; ++j) {
        const int pg = R.table[(size_t)seq * R.width + (j >> sh)];
        if ((unsigned)pg >= (unsigned)P.pages) { bad = true; break; }
        const size_t at = ((size_t)pg * P.heads + h / R.G) * P.ps + (j & (P.ps - 1));
        float x[E], y[E], z = 0.f;
        codes_of<E, BITS>(static_cast<const unsigned char*>(P.K) + at * D * BITS / 8, lane, x);
        codes_of<E, BITS>(static_cast<const unsigned char*>(P.V) + at * D * BITS / 8, lane, y);
#pragma unroll
        for (int e = 0; e < E; ++e) z = fmaf(q[e], x[e], z);
        z = warp_sum(z) * P.ks[at] * R.qscale;
        const float mn = z > m || z != z ? z : m, base = mn == -INFINITY ? 0.f : mn;
        const float a = ex2_approx(m - base), p = ex2_approx(z - base), pv = p * P.vs[at];
        m = mn;
        l = fmaf(l, a, p);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(pv, y[e], o[e] * a);
    }
    const float f = 1.f / l;
    T* out = static_cast<T*>(R.out) + row * R.out_stride + h * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float x = bad ? NAN : l == 0.f ? 0.f : o[e] * f;
        if constexpr (sizeof(T) == 2) out[e] = __float2bfloat16_rn(x);
        else out[e] = x;
    }
}

template <typename T, int D>
void go(const QuantPool& p, const PageRows& r, cudaStream_t st)
{
    const long long warps = (long long)r.rows * p.heads * r.G;
    const unsigned grid = (unsigned)((warps + kWarps - 1) / kWarps);
    if (p.bits == 8) quant_rows_kernel<T, D, 8><<<grid, kWarps * 32, 0, st>>>(p, r);
    else quant_rows_kernel<T, D, 4><<<grid, kWarps * 32, 0, st>>>(p, r);
}

}  // namespace

cudaError_t launch_page_quant_attend(const QuantPool& p, const PageRows& r, cudaStream_t st)
{
    if (p.dtype) p.D == 64 ? go<__nv_bfloat16, 64>(p, r, st) : go<__nv_bfloat16, 128>(p, r, st);
    else p.D == 64 ? go<float, 64>(p, r, st) : go<float, 128>(p, r, st);
    return cudaGetLastError();
}

}  // namespace h2o
