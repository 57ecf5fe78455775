// page_quant.cu -- rows into a paged cache of 8- or 4-bit codes, and back.
//
// A row x of a head becomes codes rint(x_e inv), inv = 127 / amax or 7 / amax,
// and the scale amax / 127 or amax / 7, amax = max |x_e|, all in fp32 as
// q8_* and q4_* (common.cuh) have it.  The largest |x| is found on the bits
// without their sign, whose order as integers is that of the values with
// infinities and then NaN above all: one comparison tells rows that have
// either, which get the scale NaN.
//
// Bound: HBM, and issue when writing.  A lane holds 16 bytes of a row of K and of the
// same row of V, so a row's head is 8 to 32 lanes.  32768 rows of 8 heads of 128, bf16,
// to 4-bit codes: 35 us, 4.9 TB/s (the pipe that compares and packs is busy for 64 %);
// rows of 32 heads back from 4-bit codes: 109 us, 6.2 TB/s.
#include <type_traits>

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

// The largest |x| of a row's L lanes of 16 bytes, of keys and of values, as fp32's bits.  (bf16: both in one word.)
template <typename T, int L>
__device__ __forceinline__ void amax_bits(const uint4 (&v)[2], uint32_t (&m)[2])
{
    if constexpr (sizeof(T) == 2) {
        uint32_t a[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            a[i] = v[i].x & 0x7fff7fffu;
            asm("max.u16x2 %0, %0, %1;" : "+r"(a[i]) : "r"(v[i].y & 0x7fff7fffu));
            asm("max.u16x2 %0, %0, %1;" : "+r"(a[i]) : "r"(v[i].z & 0x7fff7fffu));
            asm("max.u16x2 %0, %0, %1;" : "+r"(a[i]) : "r"(v[i].w & 0x7fff7fffu));
        }
        uint32_t both = __byte_perm(a[0], a[1], 0x5410);
        asm("max.u16x2 %0, %0, %1;" : "+r"(both) : "r"(__byte_perm(a[0], a[1], 0x7632)));
#pragma unroll
        for (int d = L / 2; d > 0; d >>= 1) asm("max.u16x2 %0, %0, %1;" : "+r"(both) : "r"(__shfl_xor_sync(0xffffffffu, both, d)));
        m[0] = both << 16;
        m[1] = both & 0xffff0000u;
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[i] = max(max(v[i].x & 0x7fffffffu, v[i].y & 0x7fffffffu), max(v[i].z & 0x7fffffffu, v[i].w & 0x7fffffffu));
#pragma unroll
            for (int d = L / 2; d > 0; d >>= 1) m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], d));
        }
    }
}
// four bytes, the lowest of each
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// E codes as q8_pack4 and q4_pack make them, for a finite inv: |x inv| is below 2^22, so adding 1.5 2^23 (and the 4-bit
// offset, which is even) rounds it to the nearest whole number, half to even, and leaves it in the low bits; and it is
// within the codes' range, since the largest |x| inv is 127 or 7 but for two roundings.
template <int BITS, int E>
__device__ __forceinline__ uint2 make_codes(const float* x, float inv)
{
    uint32_t u[E];
#pragma unroll
    for (int i = 0; i < E; ++i) u[i] = __float_as_uint(__fadd_rn(__fmul_rn(x[i], inv), BITS == 8 ? 12582912.f : 12582920.f));
    if constexpr (BITS == 8) {
        return make_uint2(low_bytes(u[0], u[1], u[2], u[3]), E == 8 ? low_bytes(u[E - 4], u[E - 3], u[E - 2], u[E - 1]) : 0u);
    } else if constexpr (E == 8) {
        return make_uint2(low_bytes(u[0], u[2], u[4], u[6]) + 16u * low_bytes(u[1], u[3], u[5], u[7]), 0u);
    } else {
        return make_uint2((u[0] & 15u) | (u[1] & 15u) << 4 | (u[2] & 15u) << 8 | (u[3] & 15u) << 12, 0u);
    }
}
// the same whatever inv is
template <int BITS, int E>
__device__ __forceinline__ uint2 make_codes_any(const float* x, float inv)
{
    if constexpr (BITS == 8) return make_uint2(q8_pack4(x, inv), E == 8 ? q8_pack4(x + E - 4, inv) : 0u);
    else return make_uint2(q4_pack<E / 2>(x, inv), 0u);
}
template <int BITS, int E>
__device__ __forceinline__ void put_codes(unsigned char* p, uint2 w)
{
    if constexpr (BITS * E == 64) *reinterpret_cast<uint2*>(p) = w;
    else if constexpr (BITS * E == 32) *reinterpret_cast<uint32_t*>(p) = w.x;
    else *reinterpret_cast<unsigned short*>(p) = (unsigned short)w.x;
}
// B bytes of codes into registers
template <int B>
__device__ __forceinline__ void get_raw(const unsigned char* p, uint32_t (&r)[2])
{
    if constexpr (B == 8) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        r[0] = w.x; r[1] = w.y;
    } else if constexpr (B == 4) {
        r[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
        r[0] = *reinterpret_cast<const unsigned short*>(p);
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

// A thread's i-th row of head h among RPT, and its place in the pool.  Units (row, head) lie one after another, a CTA has
// RPT * 256 / L of them.
template <typename T, int D>
struct Place {
    static constexpr int E = 16 / sizeof(T), L = D / E, kUnits = kThreads / L;    // L: lanes of a row's head
    int row, h;
    bool in;
    size_t at;                                             // its row of codes, and its scale
};
template <typename T, int D, int RPT>
__device__ __forceinline__ void find(Place<T, D> (&w)[RPT], const QuantPool& p, const int* slot, int rows)
{
    using P = Place<T, D>;
    const unsigned u = blockIdx.x * (unsigned)(RPT * P::kUnits) + threadIdx.x / P::L, heads = (unsigned)p.heads;
    const unsigned by = P::kUnits / heads, over = P::kUnits - by * heads;   // a step of kUnits: rows, heads
    unsigned row = u / heads, h = u - row * heads;
    const int sh = __ffs(p.ps) - 1;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        w[i].row = (int)row;
        w[i].h = (int)h;
        const int s = row < (unsigned)rows ? slot[row] : -1;
        w[i].in = s >= 0 && s < (long long)p.pages * p.ps;
        w[i].at = w[i].in ? ((size_t)(s >> sh) * heads + h) * p.ps + (s & (p.ps - 1)) : 0;
        row += by;
        h += over;
        if (h >= heads) { h -= heads; ++row; }
    }
}

template <typename T, int D, int BITS, int RPT>
__global__ void __launch_bounds__(kThreads) page_quant_write_kernel(const QuantPool p, const T* __restrict__ k, const T* __restrict__ v,
                                                                    const long long k_stride, const long long v_stride,
                                                                    const int* __restrict__ slot, const int rows)
{
    using P = Place<T, D>;
    constexpr int E = P::E, L = P::L;
    const int c = threadIdx.x % L;
    P w[RPT];
    uint4 raw[RPT][2];
    find(w, p, slot, rows);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
        if (w[i].in) {
            raw[i][0] = *reinterpret_cast<const uint4*>(k + w[i].row * k_stride + w[i].h * D + c * E);
            raw[i][1] = *reinterpret_cast<const uint4*>(v + w[i].row * v_stride + w[i].h * D + c * E);
        }
    }
    // The quotients of a row's lanes' 2 RPT items (keys and values of RPT rows), inv then scale, are made a lane each.
    constexpr int N = 2 * RPT;
    const float top = BITS == 8 ? 127.f : 7.f;
    uint32_t m[N];
    bool odd = false;                                      // a row that holds no number, or whose inv is out of range
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        uint32_t x[2];
        amax_bits<T, L>(raw[i], x);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            m[2 * i + j] = x[j];
            odd |= x[j] - 1u < 0x03ffffffu || x[j] >= 0x7f800000u;   // (0 < largest < 2^-119)
        }
    }
    odd = __any_sync(0xffffffffu, odd);
    float quotient[(2 * N + L - 1) / L];
#pragma unroll
    for (int j = 0; j < (2 * N + L - 1) / L; ++j) {
        const int task = c + j * L, item = task % N;
        uint32_t mine = m[0];
#pragma unroll
        for (int i = 1; i < N; ++i) mine = item == i ? m[i] : mine;
        const bool finite = mine < 0x7f800000u, scale = task >= N;
        const float amax = finite ? __uint_as_float(mine) : 0.f;
        quotient[j] = __fdiv_rn(scale ? amax : top, scale ? top : amax);
        if (!scale && amax == 0.f) quotient[j] = 0.f;
        if (scale && task < 2 * N) {
            const int row = item >> 1;
            P x = w[0];
#pragma unroll
            for (int i = 1; i < RPT; ++i)
                if (row == i) x = w[i];
            if (x.in) (item & 1 ? p.vs : p.ks)[x.at] = finite ? quotient[j] : NAN;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const P& x = w[i / 2];
        const float inv = __shfl_sync(0xffffffffu, quotient[i / L], i % L, L);
        Lane<T> y;
        y.load(reinterpret_cast<const T*>(&raw[i / 2][i & 1]));
        uint2 code;
        if (!odd) {
            code = make_codes<BITS, E>(y.x, inv);
        } else {
            if (m[i] >= 0x7f800000u)
#pragma unroll
                for (int e = 0; e < E; ++e) y.x[e] = 0.f;
            code = make_codes_any<BITS, E>(y.x, inv);
        }
        if (x.in) put_codes<BITS, E>(static_cast<unsigned char*>(i & 1 ? p.V : p.K) + (x.at * D + c * E) * BITS / 8, code);
    }
}

template <typename T, int D, int BITS, int RPT>
__global__ void __launch_bounds__(kThreads) page_quant_read_kernel(const QuantPool p, const int* __restrict__ slot, const int rows,
                                                                   T* __restrict__ k, const long long k_stride, T* __restrict__ v,
                                                                   const long long v_stride)
{
    using P = Place<T, D>;
    constexpr int E = P::E, B = E * BITS / 8;              // B: bytes of this lane's codes
    const int c = threadIdx.x % P::L;
    P w[RPT];
    uint32_t raw[RPT][2][2];
    float s[RPT][2];
    find(w, p, slot, rows);
#pragma unroll
    for (int i = 0; i < 2 * RPT; ++i) {
        const P& x = w[i / 2];
        const bool values = i & 1;
        if (x.in) {
            get_raw<B>(static_cast<const unsigned char*>(values ? p.V : p.K) + x.at * (D * BITS / 8) + c * B, raw[i / 2][i & 1]);
            s[i / 2][i & 1] = (values ? p.vs : p.ks)[x.at];
        }
    }
#pragma unroll
    for (int i = 0; i < 2 * RPT; ++i) {
        const P& x = w[i / 2];
        if (!x.in) continue;
        Lane<T> y;
        get_codes<BITS, E>(reinterpret_cast<const unsigned char*>(raw[i / 2][i & 1]), y.x);
#pragma unroll
        for (int e = 0; e < E; ++e) y.x[e] *= s[i / 2][i & 1];
        y.store((i & 1 ? v + x.row * v_stride : k + x.row * k_stride) + x.h * D + c * E);
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

// f(rows a thread, CTAs): four where that still makes eight CTAs an SM
template <class F>
void by_rows(long long units, int each, F f)
{
    const long long four = (units + 4 * each - 1) / (4 * each);
    if (four >= 8 * kSMs) f(std::integral_constant<int, 4>(), (unsigned)four);
    else f(std::integral_constant<int, 1>(), (unsigned)((units + each - 1) / each));
}

}  // namespace

cudaError_t launch_page_quant_write(const QuantPool& p, const void* k, const void* v, long long k_stride, long long v_stride,
                                    const int* slot, int rows, cudaStream_t st)
{
    return by_type(p, [&](auto t, auto d, auto bits) {
        using T = decltype(t);
        constexpr int D = decltype(d)::value, B = decltype(bits)::value;
        by_rows((long long)rows * p.heads, Place<T, D>::kUnits, [&](auto rpt, unsigned grid) {
            page_quant_write_kernel<T, D, B, decltype(rpt)::value><<<grid, kThreads, 0, st>>>(
                p, static_cast<const T*>(k), static_cast<const T*>(v), k_stride, v_stride, slot, rows);
        });
    });
}

cudaError_t launch_page_quant_read(const QuantPool& p, const int* slot, int rows, void* k, long long k_stride, void* v,
                                   long long v_stride, cudaStream_t st)
{
    return by_type(p, [&](auto t, auto d, auto bits) {
        using T = decltype(t);
        constexpr int D = decltype(d)::value, B = decltype(bits)::value;
        by_rows((long long)rows * p.heads, Place<T, D>::kUnits, [&](auto rpt, unsigned grid) {
            page_quant_read_kernel<T, D, B, decltype(rpt)::value><<<grid, kThreads, 0, st>>>(
                p, slot, rows, static_cast<T*>(k), k_stride, static_cast<T*>(v), v_stride);
        });
    });
}

}  // namespace h2o
