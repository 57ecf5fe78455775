// prompts.h -- launchers of the rotary positions, prompt attention and
// quantised paged caches (prompt_api.cu checks the arguments).
#pragma once

#include "paged.h"

namespace h2o {

constexpr int kMaxPromptRequests = 16384;   // requests of one h2o_prompt_attend call
constexpr int kMaxPromptRows = 1 << 24;     // its query rows and its key rows (one query tile's keys take less than a wait's limit)

struct RopeArgs {
    const void* in[2];             // q, k: [rows][heads][D], rows `stride` elements apart
    void* out[2];
    long long in_stride[2], out_stride[2];
    int heads[2];
    const int* pos;                // [rows]
    const long long* table;        // [rot / 2] 2^-64 turns a position
    int rows, rot;
    float amplitude;
};

struct PackedArgs {
    const void* q;                 // [rows][heads * G][D]
    const void* k;                 // [k_rows][heads][D]
    const void* v;
    void* out;
    long long q_stride, k_stride, v_stride, out_stride;
    const int* q_start;            // [requests + 1]
    const int* k_start;
    int rows, k_rows, heads, G, requests;
    float qscale;                  // softmax scale * log2(e)
};

// K, V [pages][heads][ps][D] codes of `bits`, ks, vs [pages][heads][ps]; dtype that of the rows outside
struct QuantPool {
    void* K;
    void* V;
    float* ks;
    float* vs;
    int pages, heads, ps, D, bits, dtype;
};

cudaError_t launch_rope(const RopeArgs& a, int form, int D, int dtype, cudaStream_t st);
cudaError_t launch_prompt_attend(const PackedArgs& a, int D, int dtype, cudaStream_t st);
cudaError_t launch_prompt_tc(const PackedArgs& a, int D, cudaStream_t st);   // bf16, at least one key row
cudaError_t launch_page_quant_write(const QuantPool& p, const void* k, const void* v, long long k_stride, long long v_stride,
                                    const int* slot, int rows, cudaStream_t st);
cudaError_t launch_page_quant_read(const QuantPool& p, const int* slot, int rows, void* k, long long k_stride, void* v,
                                   long long v_stride, cudaStream_t st);
cudaError_t launch_page_quant_attend(const QuantPool& p, const PageRows& r, cudaStream_t st);

}  // namespace h2o
