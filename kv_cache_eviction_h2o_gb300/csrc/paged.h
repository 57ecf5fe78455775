// paged.h -- launchers of the paged-cache operators (page_api.cu checks the
// arguments; paged.cu, page_attend.cu and prefix.cu hold the kernels).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace h2o {

constexpr int kSMs = 152;
constexpr int kMaxPageRequests = 16384;   // requests of one h2o_page_tables call
constexpr int kMaxTableWidth = 16384;     // pages of one request
constexpr int kMaxPickedPages = 4096;     // budget of a call that has to choose
constexpr int kMaxPageGroups = 16;        // query heads per cache head
constexpr int kMaxPrefixSplits = 64;      // ranges of a shared prefix
constexpr int kMaxPrefix = 1 << 30;       // tokens of a shared prefix (positions rounded up to a tile fit an int)

// Lets a kernel use all shared memory a CTA can have, once per device (a
// kernel's own static object, so a race between threads sets the same twice).
struct SmemOnce {
    bool done[64] = {};
    template <class Kernel> cudaError_t allow(Kernel* kernel, bool large_clusters = false)
    {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        if (done[dev]) return cudaSuccess;
        cudaFuncAttributes a;
        e = cudaFuncGetAttributes(&a, kernel);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - (int)a.sharedSizeBytes);
        if (e == cudaSuccess && large_clusters) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) done[dev] = true;
        return e;
    }
};

// The page pool: K, V [pages][heads][ps][D], bounds [pages][heads][2][D].
struct PagePool {
    void* K;
    void* V;
    void* bounds;
    int pages, heads, ps, D, dtype;
};

struct TablesArgs {
    const int* before;
    const int* fresh;      // new tokens
    const int* free_pages;
    int* table;
    int* after;
    int* row_start;
    int* row_seq;
    int* row_pos;
    int* slot;
    int* status;
    int n, n_free, ps, width, cap;
};

struct PageRows {
    const void* q;         // [rows][heads * G][D], rows q_stride elements apart
    void* out;
    long long q_stride, out_stride;
    const int* seq;        // [rows] request, < 0: the row is left out
    const int* pos;        // [rows] newest position the row sees (< 0: none)
    const int* table;      // [requests][width]
    int rows, G, requests, width;
    float qscale;          // softmax scale * log2(e)
};

// What the prefix pass leaves for the rows' own pass, for `splits` ranges of
// the prefix and rows * heads * G query rows each: m (base-2 maximum), l
// (sum of 2^(z - m)) and o (the weighted values, not divided by l).
struct PrefixPart {
    float* o;              // [splits][query rows][D]
    float2* ml;            // [splits][query rows]
    int splits;
};

// the same on the tensor cores (bf16); keys of each range
int prefix_tc_range(int rows, int heads, int G, int prefix_len);
cudaError_t launch_prefix_tc(const PagePool& p, const PageRows& r, const int* prefix_table, int prefix_len,
                             const PrefixPart& part, cudaStream_t st);
cudaError_t launch_page_tables(const TablesArgs& a, cudaStream_t st);
cudaError_t launch_page_write(const PagePool& p, const void* k, const void* v, long long k_stride, long long v_stride,
                              const int* slot, int rows, cudaStream_t st);
// budget > 0: the pages chosen by their bounds; 0: all pages, joined with `part`
cudaError_t launch_page_attend(const PagePool& p, const PageRows& r, int budget, int recent, int* picked,
                               const PrefixPart& part, cudaStream_t st);
// ranges the prefix is split into (a part of the workspace each)
int prefix_splits(int rows, int heads, int G, int D, int prefix_len, int dtype);
cudaError_t launch_prefix(const PagePool& p, const PageRows& r, const int* prefix_table, int prefix_len,
                          const PrefixPart& part, cudaStream_t st);

}  // namespace h2o
