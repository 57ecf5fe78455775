// page_quant.cu -- rows into a paged cache of 8- or 4-bit codes, and back.
//
// A row x of a head becomes codes rint(x_e inv), inv = 127 / amax or 7 / amax,
// and the scale amax / 127 or amax / 7, amax = max |x_e|, all in fp32 as
// q8_* and q4_* (common.cuh) have it.  The largest |x| is found on the bits
// without their sign, whose order as integers is that of the values with
// infinities and then NaN above all: one comparison tells rows that have
// either, which get the scale NaN.
//
// Bound: HBM.  A lane holds 16 bytes of a row of K and of the same row of V, so
// a row's head is 8 to 32 lanes.
#include "common.cuh"
#include "prompts.h"

namespace h2o {

namespace {

constexpr int kThreads = 256;

// 16 bytes of a row: fp32 values
template <typename T> struct Lane {
    static constexpr int E = 16 / sizeof(T);
    float x[E];
    __device__ __forceinline__ void load(const T* p) { load_vec<T, E>(p, x); }
    __device__ __forceinline__ uint32_t amax_bits() const
    {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < E; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ void store(T* p) const
    {
        if constexpr (sizeof(T) == 2) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        }
    }
};

// E codes at p
template <int BITS, int E>
__device__ __forceinline__ void put_codes(unsigned char* p, const float* x, float inv)
{
    if constexpr (BITS == 8) {
        if constexpr (E == 8) *reinterpret_cast<uint2*>(p) = make_uint2(q8_pack4(x, inv), q8_pack4(x + 4, inv));
        else *reinterpret_cast<uint32_t*>(p) = q8_pack4(x, inv);
    } else {
        if constexpr (E == 8) *reinterpret_cast<uint32_t*>(p) = q4_pack<4>(x, inv);
        else *reinterpret_cast<unsigned short*>(p) = (unsigned short)q4_pack<2>(x, inv);
    }
}
template <int BITS, int E>
__device__ __forceinline__ void get_codes(const unsigned char* p, float* x)
{
    if constexpr (BITS == 8) {
        if constexpr (E == 8) {
            const uint2 w = *reinterpret_cast<const uint2*>(p);
            q8_unpack4(w.x, x);
            q8_unpack4(w.y, x + 4);
        } else {
            q8_unpack4(*reinterpret_cast<const uint32_t*>(p), x);
        }
    } else {
        if constexpr (E == 8) {
            float y[8];
            q4_unpack8(*reinterpret_cast<const uint32_t*>(p), y);
#pragma unroll
            for (int i = 0; i < 4; ++i) { x[2 * i] = y[i]; x[2 * i + 1] = y[4 + i]; }
        } else {
            q4_unpack4(*reinterpret_cast<const unsigned short*>(p), x);
        }
    }
}

// This thread's row, head and place in the pool; false: none.
template <typename T, int D>
struct Place {
    static constexpr int E = 16 / sizeof(T), L = D / E;    // lanes of a row's head
    int row, h, c;                                         // c: lane of the row's head
    size_t at;                                             // its row of codes, and its scale
    __device__ __forceinline__ bool find(const QuantPool& p, const int* slot, int rows)
    {
        const long long x = (long long)blockIdx.x * kThreads + threadIdx.x;
        const unsigned u = (unsigned)(x / L);
        c = (int)(x % L);
        row = (int)(u / (unsigned)p.heads);
        h = (int)(u - (unsigned)row * p.heads);
        const int s = row < rows ? slot[row] : -1, sh = __ffs(p.ps) - 1;
        if (s < 0 || s >= (long long)p.pages * p.ps) return false;
        at = ((size_t)(s >> sh) * p.heads + h) * p.ps + (s & (p.ps - 1));
        return true;
    }
};

template <typename T, int D, int BITS>
__global__ void __launch_bounds__(kThreads) page_quant_write_kernel(const QuantPool p, const T* __restrict__ k, const T* __restrict__ v,
                                                                    const long long k_stride, const long long v_stride,
                                                                    const int* __restrict__ slot, const int rows)
{
    using P = Place<T, D>;
    constexpr int E = P::E, L = P::L;
    P w;
    const bool in = w.find(p, slot, rows);
    Lane<T> x[2] = {};
    if (in) {
        x[0].load(k + w.row * k_stride + w.h * D + w.c * E);
        x[1].load(v + w.row * v_stride + w.h * D + w.c * E);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t m = x[i].amax_bits();
#pragma unroll
        for (int d = L / 2; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        const bool finite = m < 0x7f800000u;
        const float amax = finite ? __uint_as_float(m) : 0.f;
        const float inv = BITS == 8 ? q8_inv(amax) : q4_inv(amax), scale = finite ? (BITS == 8 ? q8_scale(amax) : q4_scale(amax)) : NAN;
        if (!finite)
#pragma unroll
            for (int e = 0; e < E; ++e) x[i].x[e] = 0.f;
        if (in) {
            put_codes<BITS, E>(static_cast<unsigned char*>(i ? p.V : p.K) + (w.at * D + w.c * E) * BITS / 8, x[i].x, inv);
            if (w.c == i) (i ? p.vs : p.ks)[w.at] = scale;
        }
    }
}

template <typename T, int D, int BITS>
__global__ void __launch_bounds__(kThreads) page_quant_read_kernel(const QuantPool p, const int* __restrict__ slot, const int rows,
                                                                   T* __restrict__ k, const long long k_stride, T* __restrict__ v,
                                                                   const long long v_stride)
{
    using P = Place<T, D>;
    constexpr int E = P::E;
    P w;
    if (!w.find(p, slot, rows)) return;
    Lane<T> x[2];
    const float s[2] = {p.ks[w.at], p.vs[w.at]};
#pragma unroll
    for (int i = 0; i < 2; ++i)
        get_codes<BITS, E>(static_cast<const unsigned char*>(i ? p.V : p.K) + (w.at * D + w.c * E) * BITS / 8, x[i].x);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int e = 0; e < E; ++e) x[i].x[e] *= s[i];
        x[i].store((i ? v + w.row * v_stride : k + w.row * k_stride) + w.h * D + w.c * E);
    }
}

// f(element type, head_dim, bits of a code), as types
template <class F>
cudaError_t by_type(const QuantPool& p, F f)
{
    auto bits = [&](auto t, auto d) {
        if (p.bits == 8) f(t, d, std::integral_constant<int, 8>());
        else f(t, d, std::integral_constant<int, 4>());
    };
    auto dim = [&](auto t) {
        if (p.D == 64) bits(t, std::integral_constant<int, 64>());
        else bits(t, std::integral_constant<int, 128>());
    };
    if (p.dtype) dim(__nv_bfloat16());
    else dim(float());
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_page_quant_write(const QuantPool& p, const void* k, const void* v, long long k_stride, long long v_stride,
                                    const int* slot, int rows, cudaStream_t st)
{
    return by_type(p, [&](auto t, auto d, auto bits) {
        using T = decltype(t);
        constexpr int D = decltype(d)::value;
        const long long threads = (long long)rows * p.heads * Place<T, D>::L;
        page_quant_write_kernel<T, D, decltype(bits)::value><<<(unsigned)((threads + kThreads - 1) / kThreads), kThreads, 0, st>>>(
            p, static_cast<const T*>(k), static_cast<const T*>(v), k_stride, v_stride, slot, rows);
    });
}

cudaError_t launch_page_quant_read(const QuantPool& p, const int* slot, int rows, void* k, long long k_stride, void* v,
                                   long long v_stride, cudaStream_t st)
{
    return by_type(p, [&](auto t, auto d, auto bits) {
        using T = decltype(t);
        constexpr int D = decltype(d)::value;
        const long long threads = (long long)rows * p.heads * Place<T, D>::L;
        page_quant_read_kernel<T, D, decltype(bits)::value><<<(unsigned)((threads + kThreads - 1) / kThreads), kThreads, 0, st>>>(
            p, slot, rows, static_cast<T*>(k), k_stride, static_cast<T*>(v), v_stride);
    });
}

}  // namespace h2o
