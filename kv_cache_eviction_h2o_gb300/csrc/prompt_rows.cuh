// prompt_rows.cuh -- one query row of a prompt's attention by one warp on the
// CUDA cores: what the tiled kernels leave to it, and what they are not for.
#pragma once

#include "common.cuh"
#include "prompts.h"

namespace h2o {

// out = softmax(scale q.k) v over the n keys from k and v on (rows of one
// head, kstride and vstride elements apart): a running maximum m (base 2) and sum l,
// keys one after another, and no key beyond them is looked at.
template <typename T, int D>
__device__ __noinline__ void prompt_row(const T* q, const T* k, long long kstride, const T* v, long long vstride, int n, float qscale, T* out)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    float x[E], o[E] = {}, m = -INFINITY, l = 0.f;
    load_vec<T, E>(q + lane * E, x);
    for (int j = 0; j < n; ++j) {
        float y[E], w[E], z = 0.f;
        load_vec<T, E>(k + j * kstride + lane * E, y);
        load_vec<T, E>(v + j * vstride + lane * E, w);
#pragma unroll
        for (int e = 0; e < E; ++e) z = fmaf(x[e], y[e], z);
        z = warp_sum(z) * qscale;
        const float mn = z > m || z != z ? z : m, base = mn == -INFINITY ? 0.f : mn;
        const float a = ex2_approx(m - base), p = ex2_approx(z - base);
        m = mn;
        l = fmaf(l, a, p);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(p, w[e], o[e] * a);
    }
    const float f = 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float r = l == 0.f ? 0.f : o[e] * f;
        if constexpr (sizeof(T) == 2) out[lane * E + e] = __float2bfloat16_rn(r);
        else out[lane * E + e] = r;
    }
}

}  // namespace h2o
