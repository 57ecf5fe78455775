// quant_attend.cu -- attention of single tokens over quantised paged caches
// (h2o_page_quant_attend).
//
// Work unit: one query row of one cache head, its G query heads together, so a
// token's codes are read once for all of them.  A unit's tiles of 16 keys are
// dealt to the warps of a cluster of 1 to 16 CTAs, whose sums are joined at the end.
//
// Codes go into fp16 products as they lie: a code with its offset is an unsigned
// number u below 2^8, whose bits are the fp16 subnormal u 2^-24, so widening it is
// a mask (4-bit codes in the upper nibble of a byte are 16 u 2^-24, their query
// channels a sixteenth).  S^T = K Q^T has keys as rows and starts from
// -offset 2^-24 sum_e q_e instead of 0, which takes the offset out.  O^T = V^T W^T
// has channels as rows; here the offset is subtracted from each value, since it
// would cancel in sums over many keys.
//   z = ks (scale q.c),  p = 2^(z - m),  l = sum p,  w = p vs 2^(m - E),
//   O 2^(E - m) / l
// with whole numbers m and E for each query head: m is raised when a logit passes it
// by 8, E, the exponent of the sums' unit, when a weight with its value's scale passes 2^15,
// so that w keeps fp16's bits however far the scales are apart.  Queries are
// fp16 numbers with 2^eq apart (the row's largest is between 2^13 and 2^14); fp32
// rows take two for q and two for w.
//
// Bound: HBM (d bits / 8 + 4 bytes a row, twice a token).
#include <algorithm>

#include "common.cuh"
#include "prompts.h"

namespace h2o {

namespace {

constexpr int kKeys = 16;              // keys of a tile (page sizes are its multiples)
constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kMaxCluster = 16;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 floats_of(uint32_t h)
{
    float2 f;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(h));
    return f;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^e for a whole e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
template <int N> __device__ __forceinline__ void ld_cluster_f(uint32_t addr, float* x)
{
    if constexpr (N == 4) {
        const float4 w = ld_cluster_f4(addr);
        x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
    } else {
        const float2 w = ld_cluster_f2(addr);
        x[0] = w.x; x[1] = w.y;
    }
}
template <int N> __device__ __forceinline__ void load_f(const float* p, float* x)
{
    if constexpr (N == 4) {
        const float4 w = *reinterpret_cast<const float4*>(p);
        x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
    } else {
        const float2 w = *reinterpret_cast<const float2*>(p);
        x[0] = w.x; x[1] = w.y;
    }
}
template <int N> __device__ __forceinline__ void store_out(float* p, const float* x)
{
    if constexpr (N == 4) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
}
template <int N> __device__ __forceinline__ void store_out(__nv_bfloat16* p, const float* x)
{
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    if constexpr (N == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
}

// A tile's rows of RB bytes lie one after another, 16-byte chunks of each 128-byte line exchanged so that the reads of
// 8 rows' chunks, and of one chunk of every other row, meet no bank twice.
template <int RB>
__device__ __forceinline__ uint32_t chunk_at(int chunk)
{
    const int line = chunk >> 3, f = RB == 128 ? ((line >> 1 & 3) << 1) ^ ((line & 1) << 2) : (line & 3) << 1;
    return (uint32_t)(line * 128 + (((chunk & 7) ^ f) << 4));
}
template <int RB>
__device__ __forceinline__ uint32_t byte_at(int row, int byte)
{
    const int lin = row * RB + byte;
    return chunk_at<RB>(lin >> 4) + (lin & 15);
}

template <int D, int BITS> struct Tile {
    static constexpr int kRow = D * BITS / 8;              // bytes of a row of codes
    static constexpr int kCodes = kKeys * kRow;
    static constexpr int kBytes = 2 * kCodes + 2 * kKeys * 4;
    static constexpr int kStages = kRow == 128 ? 3 : kRow == 64 ? 6 : 8;
    static constexpr int kRing = kStages * kBytes;         // a warp's
};

// One warp's running sums.  Lane (g, t) = (lane / 4, lane % 4).  NT: groups of eight query heads; PARTS: fp16 numbers a
// query channel and a weight.
template <int D, int BITS, int NT, int PARTS>
struct Core {
    static constexpr int KS = D / 16;                      // steps of the products over channels, and of 16 channels of O^T
    static constexpr float kOffset = BITS == 8 ? 128.f : 8.f;
    uint32_t q[PARTS][NT][KS][2];
    float o[NT][KS][4];
    float zero[NT][2];                                     // -offset 2^-24 sum_e q_e of heads 2t, 2t + 1
    float za[NT][2], zb[NT][2];                            // 2^(24 + eq) scale log2(e), in two factors
    float m[NT][2], l[NT][2], f[NT][2];                    // f = 2^(m - E), 0 before E is known
    int unit[NT][2];                                       // E - m

    // Channel of code i of word j of a row's part t (the words are one step of K, or two with 4 bits).
    __device__ __forceinline__ static int channel(int t, int j, int i)
    {
        if constexpr (BITS == 8) return D == 128 ? (j >> 2) * 64 + t * 16 + (j & 3) * 4 + i : t * 16 + j * 4 + i;
        else return t * (D / 4) + j * 8 + i;
    }

    template <typename T>
    __device__ __forceinline__ void init(const T* qrow, int G, float qscale)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int head = n * 8 + g;
            const T* row = qrow + (size_t)(head < G ? head : 0) * D;
            uint32_t big = 0u;
            float x[KS][4];                                // of step k: those for b0's halves, then b1's
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                int c[4];
                if constexpr (BITS == 8) { c[0] = channel(t, k, 0); c[1] = channel(t, k, 2); c[2] = channel(t, k, 1); c[3] = channel(t, k, 3); }
                else { const int i = (k & 1) * 2; c[0] = channel(t, k / 2, i); c[1] = channel(t, k / 2, i + 4); c[2] = channel(t, k / 2, i + 1); c[3] = channel(t, k / 2, i + 5); }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[k][e] = head < G ? Elem<T>::to_f(row[c[e]]) : 0.f;
                    big = max(big, __float_as_uint(x[k][e]) & 0x7fffffffu);
                }
            }
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
            // 2^13 <= largest 2^-eq < 2^14 (of numbers below 2^-126, a little less)
            const int eq = big ? max((int)(big >> 23), 1) - 127 - 13 : 0;
            const float down0 = pow2(-(eq / 2)), down1 = pow2(eq / 2 - eq);
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[k][e] = x[k][e] * down0 * down1;
                if constexpr (BITS == 4) { x[k][2] *= 0.0625f; x[k][3] *= 0.0625f; }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float2 y = make_float2(x[k][2 * h], x[k][2 * h + 1]);
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {
                        q[p][n][k][h] = half2_of(y.x, y.y);
                        const float2 z = floats_of(q[p][n][k][h]);
                        sum += (BITS == 4 && h ? 16.f : 1.f) * (z.x + z.y);
                        y = make_float2(y.x - z.x, y.y - z.y);
                    }
                }
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            const int up = 24 + eq;                        // (-116 .. 138)
            const float a = pow2(up / 2), b = big < 0x7f800000u ? pow2(up - up / 2) * qscale : NAN;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int from = (2 * t + i) * 4;          // a lane of head 2t + i
                zero[n][i] = __shfl_sync(0xffffffffu, sum, from) * (-kOffset * 0x1p-24f);
                za[n][i] = __shfl_sync(0xffffffffu, a, from);
                zb[n][i] = __shfl_sync(0xffffffffu, b, from);
                m[n][i] = -INFINITY;
                l[n][i] = f[n][i] = 0.f;
                unit[n][i] = 0;
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
        }
    }

    // the weights of this lane's keys (g and g + 8) for its two heads
    struct Weights { float p[4], w[4]; };
    __device__ __forceinline__ Weights weigh(const float (&z)[4], float v0, float v1, int n) const
    {
        Weights r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float base = m[n][i & 1] == -INFINITY ? 0.f : m[n][i & 1];
            r.p[i] = ex2_approx(z[i] - base);
            r.w[i] = r.p[i] * f[n][i & 1] * (i < 2 ? v0 : v1);
        }
        return r;
    }

    // m to the largest of these logits where they pass it by 8, and the sums' unit to what w asks for
    __device__ __forceinline__ void raise(const float (&z)[4], float v0, float v1, int n)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float top = fmaxf(z[i], z[i + 2]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            if (top > m[n][i] + 8.f && top < INFINITY) {
                const float to = ceilf(top), by = to - m[n][i];
                l[n][i] *= ex2_approx(-by);
                m[n][i] = to;
                if (f[n][i] != 0.f) unit[n][i] -= (int)fminf(by, 1000.f);
            }
            const float base = m[n][i] == -INFINITY ? 0.f : m[n][i];
            float u = fmaxf(z[i] - base + lg2(v0), z[i + 2] - base + lg2(v1));   // (a scale of 0: -inf)
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, d));
            const bool known = f[n][i] != 0.f;
            int e = unit[n][i];
            if (u > -INFINITY && (!known || u > (float)(e + 15))) e = (int)ceilf(fminf(u, 1000.f)) - 6;
            else if (!known) continue;
            e = max(-118, min(126, e));                    // f within fp32, with room for p <= 2^8
            const float a = pow2(max(-126, min(126, unit[n][i] - e)));
            if (known && unit[n][i] != e)
#pragma unroll
                for (int k = 0; k < KS; ++k) { o[n][k][i] *= a; o[n][k][i + 2] *= a; }
            unit[n][i] = e;
            f[n][i] = pow2(-e);
        }
    }

    __device__ __forceinline__ void tile(const unsigned char* stage, int valid)
    {
        using L = Tile<D, BITS>;
        constexpr int RB = L::kRow;
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const unsigned char* vt = stage + L::kCodes;
        const float* ks = reinterpret_cast<const float*>(stage + 2 * L::kCodes);
        const float k0 = ks[g], k1 = ks[g + 8];
        float v0 = ks[kKeys + g], v1 = ks[kKeys + g + 8];
        // scores: rows g and g + 8 are the keys
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) { s[n][0] = s[n][2] = zero[n][0]; s[n][1] = s[n][3] = zero[n][1]; }
        {
            constexpr int W = KS * 4 * BITS / 32;          // words of a row's part
            uint32_t w[2][W];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int key = g + 8 * r;
                if constexpr (W >= 4) {
#pragma unroll
                    for (int c = 0; c < W / 4; ++c) {
                        const uint4 x = *reinterpret_cast<const uint4*>(stage + byte_at<RB>(key, c * 64 + t * 16));
                        w[r][4 * c] = x.x; w[r][4 * c + 1] = x.y; w[r][4 * c + 2] = x.z; w[r][4 * c + 3] = x.w;
                    }
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(stage + byte_at<RB>(key, t * 8));
                    w[r][0] = x.x; w[r][1] = x.y;
                }
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t a[4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if constexpr (BITS == 8) {
                        a[r] = (w[r][k] ^ 0x80808080u) & 0x00ff00ffu;
                        a[r + 2] = ((w[r][k] >> 8) ^ 0x00800080u) & 0x00ff00ffu;
                    } else {
                        const uint32_t x = k & 1 ? w[r][k / 2] >> 8 : w[r][k / 2];
                        a[r] = x & 0x000f000fu;
                        a[r + 2] = x & 0x00f000f0u;
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) mma16(s[n], a[0], a[1], a[2], a[3], q[p][n][k][0], q[p][n][k][1]);
            }
        }
        if (valid < kKeys) {                               // scales behind the newest key may be anything
            if (g >= valid) v0 = 0.f;
            if (g + 8 >= valid) v1 = 0.f;
        }
        uint32_t b[PARTS][NT][2];                          // W^T as the K x N operand
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                z[i] = s[n][i] * za[n][i & 1] * (i < 2 ? k0 : k1) * zb[n][i & 1];
                if (valid < kKeys && g + (i < 2 ? 0 : 8) >= valid) z[i] = -INFINITY;
            }
            Weights x = weigh(z, v0, v1, n);
            bool over = f[n][0] == 0.f || f[n][1] == 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) over |= z[i] > m[n][i & 1] + 8.f || x.w[i] > 32768.f;
            if (__any_sync(0xffffffffu, over)) {
                raise(z, v0, v1, n);
                x = weigh(z, v0, v1, n);
            }
            l[n][0] += x.p[0] + x.p[2];
            l[n][1] += x.p[1] + x.p[3];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float2 y = make_float2(x.w[2 * r], x.w[2 * r + 1]);
#pragma unroll
                for (int p = 0; p < PARTS; ++p) {
                    const uint32_t h = half2_of(y.x, y.y);
                    b[p][n][r] = transposed(h);
                    const float2 u = floats_of(h);
                    y = make_float2(y.x - u.x, y.y - u.y);
                }
            }
        }
        // values: rows g and g + 8 of step k are channels g D / 8 + 2k and + 1, columns the keys
        constexpr int VB = D / 8 * BITS / 8;               // bytes of this lane's channels of a key
        uint32_t w[4][VB < 4 ? 1 : VB / 4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const unsigned char* at = vt + byte_at<RB>(2 * t + (r & 1) + (r >> 1) * 8, g * VB);
            if constexpr (VB == 16) {
                const uint4 x = *reinterpret_cast<const uint4*>(at);
                w[r][0] = x.x; w[r][1] = x.y; w[r][2] = x.z; w[r][3] = x.w;
            } else if constexpr (VB == 8) {
                const uint2 x = *reinterpret_cast<const uint2*>(at);
                w[r][0] = x.x; w[r][1] = x.y;
            } else {
                w[r][0] = *reinterpret_cast<const uint32_t*>(at);
            }
        }
        constexpr int CW = 32 / BITS;                      // codes of a word
#pragma unroll
        for (int j = 0; j < VB / 4; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {                  // half words: two or four channels of two keys
                const uint32_t x = __byte_perm(w[0][j], w[1][j], h ? 0x7632 : 0x5410), y = __byte_perm(w[2][j], w[3][j], h ? 0x7632 : 0x5410);
#pragma unroll
                for (int c = 0; c < CW / 4; ++c) {
                    uint32_t a[4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t z = i ? y : x;
                        if constexpr (BITS == 8) {
                            a[2 * i] = hadd2((z ^ 0x80808080u) & 0x00ff00ffu, 0x80808080u);              // - 128 2^-24
                            a[2 * i + 1] = hadd2(((z >> 8) ^ 0x00800080u) & 0x00ff00ffu, 0x80808080u);
                        } else {
                            const uint32_t u = c ? z >> 8 : z;
                            a[2 * i] = hadd2(u & 0x000f000fu, 0x80088008u);                              // - 8 2^-24
                            a[2 * i + 1] = hfma2(u & 0x00f000f0u, 0x2c002c00u, 0x80088008u);             // / 16
                        }
                    }
                    const int k = j * (CW / 2) + h * (CW / 4) + c;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int p = 0; p < PARTS; ++p) mma16(o[n][k], a[0], a[1], a[2], a[3], b[p][n][0], b[p][n][1]);
                }
            }
    }

    // o to out [8 NT][D], (m, l) to ml [8 NT]
    __device__ __forceinline__ void finish(float* out, float2* ml, int G, bool bad)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float s = l[n][i];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                const int head = n * 8 + 2 * t + i;
                if (head >= G) continue;
                const float up = f[n][i] == 0.f ? 0.f : 1.f / f[n][i];   // 2^(E - m)
#pragma unroll
                for (int k = 0; k < KS; k += 2)
                    *reinterpret_cast<float4*>(out + head * D + g * (D / 8) + 2 * k) =
                        make_float4(o[n][k][i] * 0x1p24f * up, o[n][k][2 + i] * 0x1p24f * up, o[n][k + 1][i] * 0x1p24f * up, o[n][k + 1][2 + i] * 0x1p24f * up);
                if (g == 0) ml[head] = make_float2(m[n][i], bad ? NAN : s);
            }
    }
};

template <int NT> struct alignas(16) Joins {
    float2 wml[kWarps][8 * NT];
    float2 ml[8 * NT];
};

template <typename T, int D, int BITS, int NT>
__global__ void __launch_bounds__(kThreads, NT == 2 && sizeof(T) == 4 ? 2 : NT == 2 || sizeof(T) == 4 ? 3 : 4) quant_attend_kernel(const QuantPool pool, const PageRows R)
{
    using L = Tile<D, BITS>;
    constexpr int NS = L::kStages;
    extern __shared__ __align__(128) unsigned char raw[];
    Joins<NT>& S = *reinterpret_cast<Joins<NT>*>(raw + kWarps * L::kRing);
    unsigned char* ring = raw + (threadIdx.x >> 5) * L::kRing;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
    const int u = blockIdx.x / C, row = u / pool.heads, h = u - row * pool.heads;
    const int seq = R.seq[row], pos = R.pos[row];
    if (seq < 0) return;                                   // a row that is not there, for the whole cluster
    const int sh = __ffs(pool.ps) - 1, G = R.G;
    int npages = pos < 0 ? 0 : (pos >> sh) + 1;
    bool bad = seq >= R.requests || npages > R.width;
    if (bad) npages = 0;
    const int* table = R.table + (size_t)(bad ? 0 : seq) * R.width;

    // tiles of 16 keys, dealt to the warps of the cluster in turn
    const int tsh = sh - 4;                                // log2 of the tiles of a page
    const int ntiles = npages ? (pos >> 4) + 1 : 0;
    const int stride = C * kWarps, t0 = rank * kWarps + warp;
    int pg_next = t0 < ntiles ? table[t0 >> tsh] : 0;      // the page of the next tile to be asked for
    auto ask = [&](int t, int stage) {
        if (t < ntiles) {
            const int pg = pg_next;
            const bool ok = (unsigned)pg < (unsigned)pool.pages;
            if (!ok) bad = true;                           // (its row is NaN: any page's codes do)
            const size_t at = ((size_t)(ok ? pg : 0) * pool.heads + h) * pool.ps + ((size_t)(t & ((1 << tsh) - 1)) << 4);
            const unsigned char* K = static_cast<const unsigned char*>(pool.K) + at * L::kRow;
            const unsigned char* V = static_cast<const unsigned char*>(pool.V) + at * L::kRow;
            const uint32_t to = smem_u32(ring + stage * L::kBytes);
#pragma unroll
            for (int i = 0; i < L::kRow / 32; ++i) {
                const int c = lane + 32 * i;
                cp_async16(to + chunk_at<L::kRow>(c), K + c * 16);
                cp_async16(to + L::kCodes + chunk_at<L::kRow>(c), V + c * 16);
            }
            if (lane < 8) cp_async16(to + 2 * L::kCodes + lane * 16, (lane < 4 ? pool.ks : pool.vs) + at + (lane & 3) * 4);
            if (t + stride < ntiles) pg_next = table[(t + stride) >> tsh];
        }
        cp_commit();
    };
#pragma unroll 1
    for (int s = 0; s < NS - 1; ++s) ask(t0 + s * stride, s);
    Core<D, BITS, NT, sizeof(T) == 2 ? 1 : 2> core;
    core.init(static_cast<const T*>(R.q) + (size_t)row * R.q_stride + (size_t)h * G * D, G, R.qscale);
    int stage = 0;
#pragma unroll 1
    for (int t = t0; t < ntiles; t += stride) {
        ask(t + (NS - 1) * stride, stage == 0 ? NS - 1 : stage - 1);
        cp_wait<NS - 1>();
        __syncwarp();
        core.tile(ring + stage * L::kBytes, t == ntiles - 1 ? (pos & 15) + 1 : kKeys);
        __syncwarp();
        stage = stage + 1 == NS ? 0 : stage + 1;
    }
    cp_wait<0>();
    __syncwarp();

    // the warps' sums, then the CTAs'
    static_assert(L::kRing >= (int)sizeof(float) * 8 * NT * D, "a warp's sums lie in its ring");
    core.finish(reinterpret_cast<float*>(ring), S.wml[warp], G, bad);
    __syncthreads();
    float* sums = reinterpret_cast<float*>(raw);           // in the place of warp 0's
    constexpr int V4 = D / 32;                             // a lane's channels of a head
    for (int g = warp; g < G; g += kWarps) {
        float m = -INFINITY, l = 0.f, o[V4] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, S.wml[w][g].x);
        const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float a = ex2_approx(S.wml[w][g].x - base);
            l = fmaf(a, S.wml[w][g].y, l);
            float x[V4];
            load_f<V4>(reinterpret_cast<const float*>(raw + w * L::kRing) + g * D + lane * V4, x);
#pragma unroll
            for (int e = 0; e < V4; ++e) o[e] = fmaf(a, x[e], o[e]);
        }
        store_out<V4>(sums + g * D + lane * V4, o);
        if (lane == 0) S.ml[g] = make_float2(m, l);
    }
    cluster_arrive();
    cluster_wait();
    // a warp joins a head's sums of all CTAs
    T* orow = static_cast<T*>(R.out) + (size_t)row * R.out_stride + (size_t)h * G * D;
#pragma unroll 1
    for (int g = rank * kWarps + warp; g < G; g += C * kWarps) {
        const float2 x = lane < C ? ld_cluster_f2(map_to_rank(&S.ml[g], lane)) : make_float2(-INFINITY, 0.f);
        const float m = warp_max(x.x), base = m == -INFINITY ? 0.f : m;
        const float mine = ex2_approx(x.x - base), l = warp_sum(mine * x.y);
        float o[V4] = {};
#pragma unroll 4
        for (int s = 0; s < C; ++s) {
            const float a = __shfl_sync(0xffffffffu, mine, s);
            float v[V4];
            ld_cluster_f<V4>(map_to_rank(sums + g * D + lane * V4, s), v);
#pragma unroll
            for (int e = 0; e < V4; ++e) o[e] = fmaf(a, v[e], o[e]);
        }
        // no key at all, or none of weight: zero; a bad table entry has made l NaN
        const float f = 1.f / l;
#pragma unroll
        for (int e = 0; e < V4; ++e) o[e] = l == 0.f ? 0.f : o[e] * f;
        store_out<V4>(orow + g * D + lane * V4, o);
    }
    cluster_arrive();
    cluster_wait();                                        // no CTA leaves while another reads its sums
}

// Clusters of c CTAs that the GPU holds at once, about (per_sm CTAs an SM).
int clusters_that_fit(int c, int per_sm)
{
    return c == 2 ? 76 * per_sm : c == 4 ? 36 * per_sm : c == 8 ? (per_sm == 1 ? 15 : 17 * per_sm) : 7 * per_sm;
}

template <typename T, int D, int BITS, int NT>
cudaError_t go(const QuantPool& p, const PageRows& r, cudaStream_t st)
{
    using L = Tile<D, BITS>;
    const auto kernel = quant_attend_kernel<T, D, BITS, NT>;
    const size_t smem = kWarps * L::kRing + sizeof(Joins<NT>);
    static SmemOnce once;
    const cudaError_t e = once.allow(kernel, true);
    if (e != cudaSuccess) return e;
    const long long units = (long long)r.rows * p.heads;
    const int tiles = r.width * (p.ps / kKeys), per_sm = 4;
    int C = 1;
    while (C < kMaxCluster && units <= clusters_that_fit(2 * C, per_sm) && tiles >= 3 * C * 2 * kWarps) C *= 2;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = C > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p, r);
}

template <typename T, int D, int BITS>
cudaError_t by_groups(const QuantPool& p, const PageRows& r, cudaStream_t st)
{
    return r.G <= 8 ? go<T, D, BITS, 1>(p, r, st) : go<T, D, BITS, 2>(p, r, st);
}
template <typename T, int D>
cudaError_t by_bits(const QuantPool& p, const PageRows& r, cudaStream_t st)
{
    return p.bits == 8 ? by_groups<T, D, 8>(p, r, st) : by_groups<T, D, 4>(p, r, st);
}

}  // namespace

cudaError_t launch_page_quant_attend(const QuantPool& p, const PageRows& r, cudaStream_t st)
{
    if (p.dtype) return p.D == 64 ? by_bits<__nv_bfloat16, 64>(p, r, st) : by_bits<__nv_bfloat16, 128>(p, r, st);
    return p.D == 64 ? by_bits<float, 64>(p, r, st) : by_bits<float, 128>(p, r, st);
}

}  // namespace h2o
