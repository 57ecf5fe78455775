// prompt_attend.cu -- causal attention over the packed rows of requests, on
// the CUDA cores.
//
// A warp a query row of one head: a running maximum m (base 2) and sum l, keys
// one after another.
#include "prompt_rows.cuh"

namespace h2o {

namespace {

constexpr int kWarps = 8;

// The request that row r is of, or -1: the last one that starts at r or before, if r is in it.
__device__ __forceinline__ int request_of(const int* start, int n, int r)
{
    int lo = 0, hi = n;                                    // start[lo] <= r < start[hi], should both be
    if (r < start[0] || r >= start[n]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (start[mid] <= r) lo = mid; else hi = mid;
    }
    return lo;
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) prompt_rows_kernel(const PackedArgs A)
{
    const int hq = A.heads * A.G;
    const long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int row = (int)(u / hq), h = (int)(u % hq);
    if (row >= A.rows) return;
    const int i = request_of(A.q_start, A.requests, row);
    if (i < 0) return;
    const int q0 = A.q_start[i], q1 = A.q_start[i + 1], k0 = A.k_start[i], k1 = A.k_start[i + 1];
    if (q0 < 0 || q1 > A.rows || row < q0 || row >= q1 || k0 < 0 || k1 < k0 || k1 > A.k_rows) return;
    const int n = min(k1 - k0, k1 - k0 - (q1 - q0) + (row - q0) + 1);    // keys it sees
    prompt_row<T, D>(static_cast<const T*>(A.q) + row * A.q_stride + h * D, static_cast<const T*>(A.k) + k0 * A.k_stride + h / A.G * D, A.k_stride,
                     static_cast<const T*>(A.v) + k0 * A.v_stride + h / A.G * D, A.v_stride, n, A.qscale,
                     static_cast<T*>(A.out) + row * A.out_stride + h * D);
}

}  // namespace

cudaError_t launch_prompt_attend(const PackedArgs& a, int D, int dtype, cudaStream_t st)
{
    const long long warps = (long long)a.rows * a.heads * a.G;
    const unsigned grid = (unsigned)((warps + kWarps - 1) / kWarps);
    if (dtype && a.k_rows) return launch_prompt_tc(a, D, st);
    if (dtype) {
        if (D == 64) prompt_rows_kernel<__nv_bfloat16, 64><<<grid, kWarps * 32, 0, st>>>(a);
        else prompt_rows_kernel<__nv_bfloat16, 128><<<grid, kWarps * 32, 0, st>>>(a);
    } else {
        if (D == 64) prompt_rows_kernel<float, 64><<<grid, kWarps * 32, 0, st>>>(a);
        else prompt_rows_kernel<float, 128><<<grid, kWarps * 32, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace h2o
