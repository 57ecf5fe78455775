// rope.cu -- rotary positions of query and key rows.
//
// Pair i of a head, channels (i, rot / 2 + i) or (2i, 2i + 1), is turned by
// t = 2 pi pos F_i 2^-64.  The table's F_i are 64-bit fractions of a turn, so
// pos F_i modulo 2^64 is exact whatever the position, in two integer products
// (an fp32 angle is off by 2^-25 of itself, 0.03 radians at 10^6; the fp64 pipe
// is too narrow for one angle a channel pair).  Of the fraction the nearest
// quarter turn goes into signs and the order of the two, and within an eighth
// of a turn either side sine and cosine are their Taylor sums to x^9 and x^10,
// whose next terms are below 2^-29.
//
// Bound: HBM, each channel read and written once.  A thread turns V pairs of
// the same angles in several heads, so that the angles cost little beside
// the 4 V channels a head it moves.  16384 rows of 32 + 8 heads of 128, bf16: 53.7 us,
// 6.25 TB/s; 64 rows: 2.7 us, a launch.  Where rot / 2 is odd, a thread moves one
// channel of either half: 8000 rows take 45 us, with rot 24 28.
#include <algorithm>

#include "common.cuh"
#include "prompts.h"

namespace h2o {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;              // heads whose loads are under way together

template <typename T, int V> struct Chunk;
template <int V> struct Chunk<float, V> {
    float x[V];
    __device__ __forceinline__ void load(const float* p)
    {
        if constexpr (V == 4) { const float4 w = *reinterpret_cast<const float4*>(p); x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w; }
        else if constexpr (V == 2) { const float2 w = *reinterpret_cast<const float2*>(p); x[0] = w.x; x[1] = w.y; }
        else x[0] = *p;
    }
    __device__ __forceinline__ void store(float* p) const
    {
        if constexpr (V == 4) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        else if constexpr (V == 2) *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
        else *p = x[0];
    }
    __device__ __forceinline__ float get(int i) const { return x[i]; }
    __device__ __forceinline__ void set2(int i, float a, float b) { x[i] = a; x[i + 1] = b; }
    __device__ __forceinline__ void set1(float a) { x[0] = a; }
};
template <int V> struct Chunk<__nv_bfloat16, V> {
    uint32_t x[V < 2 ? 1 : V / 2];
    __device__ __forceinline__ void load(const __nv_bfloat16* p)
    {
        if constexpr (V == 8) { const uint4 w = *reinterpret_cast<const uint4*>(p); x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w; }
        else if constexpr (V == 4) { const uint2 w = *reinterpret_cast<const uint2*>(p); x[0] = w.x; x[1] = w.y; }
        else if constexpr (V == 2) x[0] = *reinterpret_cast<const uint32_t*>(p);
        else x[0] = *reinterpret_cast<const unsigned short*>(p);
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const
    {
        if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(x[0], x[1], x[2], x[3]);
        else if constexpr (V == 4) *reinterpret_cast<uint2*>(p) = make_uint2(x[0], x[1]);
        else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(p) = x[0];
        else *reinterpret_cast<unsigned short*>(p) = (unsigned short)x[0];
    }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(i & 1 ? x[i / 2] & 0xffff0000u : x[i / 2] << 16); }
    __device__ __forceinline__ void set2(int i, float a, float b) { asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(x[i / 2]) : "f"(b), "f"(a)); }
    __device__ __forceinline__ void set1(float a) { x[0] = __bfloat16_as_ushort(__float2bfloat16_rn(a)); }
};

// (cos, sin) of u 2^-32 turns
__device__ __forceinline__ float2 turn(uint32_t u)
{
    const uint32_t quarter = (u + 0x20000000u) >> 30;
    const float x = (float)(int)(u - (quarter << 30)) * 1.4629180792671596e-9f, y = x * x;   // 2 pi 2^-32
    float s = fmaf(y, 2.7557319e-6f, -1.9841270e-4f);                  // 1/9!, 1/7!
    s = fmaf(y, s, 8.3333333e-3f);
    s = fmaf(y, s, -1.6666667e-1f);
    s = fmaf(x * y, s, x);
    float c = fmaf(y, -2.7557319e-7f, 2.4801587e-5f);                  // 1/10!, 1/8!
    c = fmaf(y, c, -1.3888889e-3f);
    c = fmaf(y, c, 4.1666667e-2f);
    c = fmaf(y, c, -0.5f);
    c = fmaf(y, c, 1.f);
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
    return make_float2(quarter == 1 || quarter == 2 ? -a : a, quarter >= 2 ? -b : b);
}

// A thread's item of a head: two chunks of V channels.  Half layout: V pairs,
// chunks i V and rot / 2 + i V, or 2 V channels behind rot that stay as they
// are.  Pairs: V pairs in 2 V channels side by side, some of which may stay.
template <typename T, int V, bool PAIRS>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs A, const int D, const int groups)
{
    const int items = D / (2 * V), all = A.heads[0] + A.heads[1], half = A.rot / 2;
    const long long at = (long long)blockIdx.x * kThreads + threadIdx.x;
    const unsigned t = (unsigned)(at >> (__ffs(items) - 1)), row = t / (unsigned)groups;
    const int item = (int)(at & (items - 1)), g = (int)(t - row * groups);
    if (row >= (unsigned)A.rows) return;
    const int pos = A.pos[row];
    if (pos < 0) return;
    const int p0 = item * V;                               // the first pair
    const bool turned = p0 < half;
    const int c0 = PAIRS || !turned ? 2 * p0 : p0, c1 = c0 + (PAIRS || !turned ? V : half);
    float2 cs[V];
    if (turned) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const unsigned long long f = p0 + i < half ? (unsigned long long)A.table[p0 + i] : 0ull;
            cs[i] = turn((uint32_t)((unsigned long long)(unsigned)pos * f >> 32));
            cs[i].x *= A.amplitude;
            cs[i].y *= A.amplitude;
        }
    }
    const T* in[2];
    T* out[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        in[x] = static_cast<const T*>(A.in[x]) + (long long)row * A.in_stride[x];
        out[x] = static_cast<T*>(A.out[x]) + (long long)row * A.out_stride[x];
    }
#pragma unroll 1
    for (int h0 = g; h0 < all; h0 += kBatch * groups) {
        Chunk<T, V> a[kBatch], b[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int h = h0 + j * groups;
            if (h >= all) break;
            const T* p = h < A.heads[0] ? in[0] + (long long)h * D : in[1] + (long long)(h - A.heads[0]) * D;
            a[j].load(p + c0);
            b[j].load(p + c1);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int h = h0 + j * groups;
            if (h >= all) break;
            if (turned) {
                if constexpr (PAIRS) {
                    // channels 2 p0 .. 2 p0 + V - 1 are in a, the others in b
                    static_assert(V % 2 == 0, "pairs lie in one chunk");
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        Chunk<T, V>& z = i < V / 2 ? a[j] : b[j];
                        const int e = 2 * i % V;
                        const float x = z.get(e), y = z.get(e + 1);
                        if (p0 + i < half) z.set2(e, fmaf(x, cs[i].x, -y * cs[i].y), fmaf(y, cs[i].x, x * cs[i].y));
                    }
                } else if constexpr (V == 1) {
                    const float x = a[j].get(0), y = b[j].get(0);
                    a[j].set1(fmaf(x, cs[0].x, -y * cs[0].y));
                    b[j].set1(fmaf(y, cs[0].x, x * cs[0].y));
                } else {
#pragma unroll
                    for (int i = 0; i < V; i += 2) {
                        const float x0 = a[j].get(i), x1 = a[j].get(i + 1), y0 = b[j].get(i), y1 = b[j].get(i + 1);
                        a[j].set2(i, fmaf(x0, cs[i].x, -y0 * cs[i].y), fmaf(x1, cs[i + 1].x, -y1 * cs[i + 1].y));
                        b[j].set2(i, fmaf(y0, cs[i].x, x0 * cs[i].y), fmaf(y1, cs[i + 1].x, x1 * cs[i + 1].y));
                    }
                }
            }
            T* p = h < A.heads[0] ? out[0] + (long long)h * D : out[1] + (long long)(h - A.heads[0]) * D;
            a[j].store(p + c0);
            b[j].store(p + c1);
        }
    }
}

template <typename T, int V, bool PAIRS>
cudaError_t go(const RopeArgs& a, int D, cudaStream_t st)
{
    const int all = a.heads[0] + a.heads[1], items = D / (2 * V);
    // heads a thread: as many, up to eight, as leave every SM a thousand threads
    int each = 8;
    while (each > 1 && (long long)a.rows * items * ((all + each - 1) / each) < 1024LL * kSMs) each /= 2;
    const int groups = (all + each - 1) / each;
    const long long threads = (long long)a.rows * groups * items;
    rope_kernel<T, V, PAIRS><<<(unsigned)((threads + kThreads - 1) / kThreads), kThreads, 0, st>>>(a, D, groups);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int form, int D, int dtype, cudaStream_t st)
{
    const bool bf16 = dtype != 0;
    // (one pair: the two layouts are the same, and neighbours go 16 bytes at a time: 8000 rows of 40 heads 45 us by halves)
    if (form || a.rot == 2) return bf16 ? go<__nv_bfloat16, 8, true>(a, D, st) : go<float, 4, true>(a, D, st);
    const int half = a.rot / 2, v = half & -half;          // the second half starts on a multiple of v channels
    if (bf16) {
        if (v >= 8) return go<__nv_bfloat16, 8, false>(a, D, st);
        if (v == 4) return go<__nv_bfloat16, 4, false>(a, D, st);
        if (v == 2) return go<__nv_bfloat16, 2, false>(a, D, st);
        return go<__nv_bfloat16, 1, false>(a, D, st);
    }
    if (v >= 4) return go<float, 4, false>(a, D, st);
    if (v == 2) return go<float, 2, false>(a, D, st);
    return go<float, 1, false>(a, D, st);
}

}  // namespace h2o
