// quant_attend.cu -- attention of single tokens over quantised paged caches
// (h2o_page_quant_attend).
//
// Work unit: one query row of one cache head, its G query heads together, so a
// token's codes are read once for all of them.  A unit's tiles of 16 keys are
// dealt to the warps of a cluster of 1 to 16 CTAs, whose sums are joined at the end.
//
// Codes go into fp16 products: a code with its offset is an unsigned number u
// below 2^8, whose bits are the fp16 subnormal u 2^-24, so widening it is a mask
// (the upper 4-bit code of a byte 16 u 2^-24).  S^T = K Q^T has keys as rows.  With
// bf16 rows it takes the subnormals as they are (queries of upper codes a
// sixteenth) and starts from -offset 2^-24 sum_e q_e, which takes the offset out;
// the tensor cores align a subnormal's products as if it were 2^-14, which leaves
// 2^-24 of the largest q 2^-14 (2^-13 of one product's largest a logit).  fp32 rows, and the
// values of O^T = V^T W^T, whose offset would cancel in sums over many keys, go
// through one fused multiply-add of two halves to c 2^-10.
//   z = ks (scale q.c),  p = 2^(z - m),  l = sum p,  w = p vs 2^(m - E),
//   O 2^(E - m) / l
// with whole numbers m and E for each query head: m is raised, to 8 above the logit,
// when one passes it (so that p is at most 1, and sums are no larger than the
// values'), E, the exponent of the sums' unit, when a weight with its value's scale
// passes 2^15, so that w keeps fp16's bits however far the scales are apart.
// Queries are fp16 numbers with 2^eq apart (the row's largest is between 2^13 and
// 2^14); fp32 rows take two for q and two for w.  (One for w with bf16 rows: up to 2^-11
// of each weight, of either sign, is not to be seen beside the output's own
// rounding: 0.0017 off, as a form with fp32 weights.)
//
// Bound: HBM (d bits / 8 + 4 bytes a row, twice a token), and with 4-bit codes issue,
// of widening them.  64 requests of up to 24576 tokens, 8 x 4 heads of 128, bf16: int8
// 379 us, 6.6 TB/s; 4 bits 239 us, 5.4 TB/s (the integer pipe is busy for 58 %, its
// warps take turns at it).  One request of 32768, 32 heads, int8: 51 us, 5.4 TB/s.
#include <algorithm>
#include <cfloat>

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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t a)
{
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
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
// max(a, b, c) in one instruction
__device__ __forceinline__ float max3f(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
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
// one chunk of 8 rows (ldmatrix), and of neighbouring rows' chunks, meet no bank twice.
template <int RB>
__device__ __forceinline__ uint32_t chunk_at(int chunk)
{
    const int line = chunk >> 3, f = RB == 128 ? (line & 1) << 2 | (line >> 1 & 3) : RB == 64 ? line & 3 : line & 1;
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
    static constexpr int kStages = kRow == 128 ? 4 : kRow == 64 ? 6 : 10;   // tiles in flight, in twos
    static constexpr int kRing = kStages * kBytes;         // a warp's
};

// One warp's running sums.  Lane (g, t) = (lane / 4, lane % 4).  NT: groups of eight query heads; PARTS: fp16 numbers a
// query channel and a weight.
template <int D, int BITS, int NT, int PARTS>
struct Core {
    static constexpr int KS = D / 16;                      // steps of the products over channels, and of 16 channels of O^T
    static constexpr float kOffset = BITS == 8 ? 128.f : 8.f;
    static constexpr bool kRaw = PARTS == 1;               // key codes as subnormals
    static constexpr int kLowest = -126;                   // of E - m: f = 2^(m - E) is within fp32
    uint32_t q[PARTS][NT][KS][2];
    float o[NT][KS][4];
    float zero[NT][2];                                     // what the scores of heads 2t, 2t + 1 start from
    float2 zf[NT];                                         // 2^(24 + eq) scale log2(e)
    float2 m[NT], l[NT], f[NT];                            // f = 2^(m - E)
    int unit[NT][2];                                       // E - m

    __device__ __forceinline__ static float& at(float2& x, int i) { return i ? x.y : x.x; }

    // Codes of a word of two pieces of 16 bits: of each the first (HI 0) or second code, with its offset, as the fp16 subnormals
    // u 2^-24, or 16 u 2^-24 for the second of four bits.
    template <int HI>
    __device__ __forceinline__ static uint32_t code(uint32_t w)
    {
        if constexpr (BITS == 8) return ((HI ? w >> 8 : w) & 0x00ff00ffu) ^ 0x00800080u;
        else return w & (HI ? 0x00f000f0u : 0x000f000fu);
    }
    // the same without the offset, as c 2^-10
    template <int HI>
    __device__ __forceinline__ static uint32_t normal(uint32_t u)
    {
        return hfma2(u, BITS == 4 && HI ? 0x64006400u : 0x74007400u, BITS == 8 ? 0xb000b000u : 0xa000a000u);
    }

    // c += a b[..][n][k].  With two parts sums of 16 products are added up by the FMA pipe, times `unit`: the tensor cores cut a
    // sum's bits off where an addition rounds, which adds up over many keys.
    template <int K>
    __device__ __forceinline__ static void mma_parts(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[PARTS][NT][K][2], int n, int k, float unit = 1.f)
    {
        if constexpr (PARTS == 1) {
            mma16(c, a[0], a[1], a[2], a[3], b[0][n][k][0], b[0][n][k][1]);
        } else {
            float s[4] = {};
#pragma unroll
            for (int p = PARTS - 1; p >= 0; --p) mma16(s, a[0], a[1], a[2], a[3], b[p][n][k][0], b[p][n][k][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = fmaf(s[e], unit, c[e]);
        }
    }

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
            // a word's channels lie side by side: 4 or 8 of them at a time
#pragma unroll
            for (int j = 0; j < KS / (BITS == 8 ? 1 : 2); ++j) {
                constexpr int N = BITS == 8 ? 4 : 8;
                float y[N];
                load_vec<T, 4>(row + channel(t, j, 0), y);
                if constexpr (N == 8) load_vec<T, 4>(row + channel(t, j, 0) + 4, y + 4);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    if (head >= G) y[e] = 0.f;
                    big = max(big, __float_as_uint(y[e]) & 0x7fffffffu);
                }
                if constexpr (BITS == 8) {
                    x[j][0] = y[0]; x[j][1] = y[2]; x[j][2] = y[1]; x[j][3] = y[3];
                } else {
                    x[2 * j][0] = y[0]; x[2 * j][1] = y[4]; x[2 * j][2] = y[1]; x[2 * j][3] = y[5];
                    x[2 * j + 1][0] = y[2]; x[2 * j + 1][1] = y[6]; x[2 * j + 1][2] = y[3]; x[2 * j + 1][3] = y[7];
                }
            }
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
            // 2^13 <= largest 2^-eq < 2^14 (of numbers below 2^-126, a little less)
            const int eq = max((int)(big >> 23), 1) - 127 - 13;
            const float down0 = pow2(-(eq / 2)), down1 = pow2(eq / 2 - eq);
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[k][e] = x[k][e] * down0 * down1;
                if constexpr (kRaw && BITS == 4) { x[k][2] *= 0.0625f; x[k][3] *= 0.0625f; }
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
            const int up = 24 + eq;
            // A row whose largest value times scale passes 2^114, or that holds an infinity or a NaN, is NaN; up to there the factor
            // is below 2^11 2^114 log2(e).
            const float a = __uint_as_float(big) * qscale <= 0x1.715476p114f ? pow2(up / 2) * qscale * pow2(up - up / 2) : NAN;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int from = (2 * t + i) * 4;          // a lane of head 2t + i
                zero[n][i] = kRaw ? __shfl_sync(0xffffffffu, sum, from) * (-kOffset * 0x1p-24f) : 0.f;
                at(zf[n], i) = __shfl_sync(0xffffffffu, a, from);
                at(m[n], i) = -FLT_MAX;                    // (below every logit that counts)
                at(l[n], i) = 0.f;
                unit[n][i] = kLowest;
                at(f[n], i) = pow2(-kLowest);
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
        }
    }

    // weights of this lane's keys, g and g + 8 of a tile, for its two heads: d = z - m
    __device__ __forceinline__ void weigh(const float2 (&d)[2], const float (&v)[2], int n, float2 (&p)[2], float2 (&w)[2]) const
    {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            p[r] = make_float2(ex2_approx(d[r].x), ex2_approx(d[r].y));
            w[r] = __fmul2_rn(__fmul2_rn(p[r], f[n]), make_float2(v[r], v[r]));
        }
    }

    // m to 8 above the largest of these logits z = d + m where they pass it, and the sums' unit to what w asks for; d anew
    template <int TILES>
    __device__ __forceinline__ void raise(const float2 (&z)[TILES][2], const float (&v)[TILES][2], int n)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            auto zi = [&](int x, int r) { return i ? z[x][r].y : z[x][r].x; };
            float top = -INFINITY;
#pragma unroll
            for (int x = 0; x < TILES; ++x) top = max3f(top, zi(x, 0), zi(x, 1));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            float& mi = at(m[n], i);
            if (top > mi && top < INFINITY) {
                const float to = ceilf(top) + 8.f, by = to - mi;
                at(l[n], i) *= ex2_approx(-by);
                mi = to;
                unit[n][i] -= (int)fminf(by, 1000.f);
            }
            float u = -INFINITY;                           // log2 of the largest p vs (a scale of 0: -inf)
#pragma unroll
            for (int x = 0; x < TILES; ++x) u = max3f(u, zi(x, 0) - mi + lg2(v[x][0]), zi(x, 1) - mi + lg2(v[x][1]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, d));
            int e = unit[n][i];
            if (u > (float)(e + 15)) e = (int)ceilf(fminf(u, 1000.f)) - 6;
            e = max(kLowest, min(126, e));
            if (unit[n][i] != e) {
                const float a = pow2(max(-126, min(126, unit[n][i] - e)));
#pragma unroll
                for (int k = 0; k < KS; ++k) { o[n][k][i] *= a; o[n][k][i + 2] *= a; }
            }
            unit[n][i] = e;
            at(f[n], i) = pow2(-e);
        }
    }

    // TILES tiles, of whose keys the first `valid` count
    template <int TILES>
    __device__ __forceinline__ void tiles(const unsigned char* const (&stage)[TILES], int valid)
    {
        using L = Tile<D, BITS>;
        constexpr int RB = L::kRow;
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        // scores: rows g and g + 8 are the keys
        float s[NT][TILES][4];
#pragma unroll
        for (int x = 0; x < TILES; ++x) {
#pragma unroll
            for (int n = 0; n < NT; ++n) { s[n][x][0] = s[n][x][2] = zero[n][0]; s[n][x][1] = s[n][x][3] = zero[n][1]; }
            constexpr int W = KS * 4 * BITS / 32;          // words of a row's part
            uint32_t w[2][W];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int key = g + 8 * r;
                if constexpr (W >= 4) {
#pragma unroll
                    for (int c = 0; c < W / 4; ++c) {
                        const uint4 y = *reinterpret_cast<const uint4*>(stage[x] + byte_at<RB>(key, c * 64 + t * 16));
                        w[r][4 * c] = y.x; w[r][4 * c + 1] = y.y; w[r][4 * c + 2] = y.z; w[r][4 * c + 3] = y.w;
                    }
                } else {
                    const uint2 y = *reinterpret_cast<const uint2*>(stage[x] + byte_at<RB>(key, t * 8));
                    w[r][0] = y.x; w[r][1] = y.y;
                }
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t a[4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t y = BITS == 8 ? w[r][k] : k & 1 ? w[r][k / 2] >> 8 : w[r][k / 2];
                    a[r] = code<0>(y);
                    a[r + 2] = code<1>(y);
                    if constexpr (!kRaw) {
                        a[r] = normal<0>(a[r]);
                        a[r + 2] = normal<1>(a[r + 2]);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_parts(s[n][x], a, q, n, k, 0x1p-14f);   // (q.c 2^-24 2^-eq either way: times any ks that a write makes, a number)
            }
        }
        float kf[TILES][2], v[TILES][2];
#pragma unroll
        for (int x = 0; x < TILES; ++x) {
            const float* ks = reinterpret_cast<const float*>(stage[x] + 2 * L::kCodes);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                kf[x][r] = ks[g + 8 * r];
                v[x][r] = ks[kKeys + g + 8 * r];
                if (valid < TILES * kKeys && x * kKeys + g + 8 * r >= valid) v[x][r] = 0.f;   // (scales behind the newest key may be anything)
            }
        }
        uint32_t b[PARTS][NT][TILES][2];                   // W^T as the K x N operand
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float2 z[TILES][2], d[TILES][2], p[TILES][2], w[TILES][2];
            float over = -INFINITY, most = 0.f;
#pragma unroll
            for (int x = 0; x < TILES; ++x) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    z[x][r] = __fmul2_rn(__fmul2_rn(make_float2(s[n][x][2 * r], s[n][x][2 * r + 1]), make_float2(kf[x][r], kf[x][r])), zf[n]);
                    if (valid < TILES * kKeys && x * kKeys + g + 8 * r >= valid) z[x][r] = make_float2(-INFINITY, -INFINITY);
                    d[x][r] = __fadd2_rn(z[x][r], make_float2(-m[n].x, -m[n].y));
                    over = max3f(over, d[x][r].x, d[x][r].y);
                }
                weigh(d[x], v[x], n, p[x], w[x]);
#pragma unroll
                for (int r = 0; r < 2; ++r) most = max3f(most, w[x][r].x, w[x][r].y);
            }
            if (__any_sync(0xffffffffu, over > 0.f || most > 32768.f)) {
                raise<TILES>(z, v, n);
#pragma unroll
                for (int x = 0; x < TILES; ++x) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) d[x][r] = __fadd2_rn(z[x][r], make_float2(-m[n].x, -m[n].y));
                    weigh(d[x], v[x], n, p[x], w[x]);
                }
            }
#pragma unroll
            for (int x = 0; x < TILES; ++x) {
                l[n] = __fadd2_rn(l[n], __fadd2_rn(p[x][0], p[x][1]));
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float2 y = w[x][r];
#pragma unroll
                    for (int i = 0; i < PARTS; ++i) {
                        const uint32_t h = half2_of(y.x, y.y);
                        b[i][n][x][r] = transposed(h);
                        const float2 u = floats_of(h);
                        y = make_float2(y.x - u.x, y.y - u.y);
                    }
                }
            }
        }
        // values: 8 x 8 matrices of 16-bit pieces of 8 keys, transposed, give a lane the same piece of keys 2t and 2t + 1 side by
        // side: two or four channels, rows g and g + 8 of one or two steps
        constexpr int CP = 16 / BITS;                      // channels of a piece
        const int mat = lane >> 3, r8 = lane & 7;
#pragma unroll
        for (int x = 0; x < TILES; ++x) {
            const uint32_t at = smem_u32(stage[x] + L::kCodes);
#pragma unroll
            for (int c = 0; c < RB / 16; c += 2) {         // two chunks of 16 bytes a row: matrices of keys 0-7 and 8-15 of each
                uint32_t y[4];
                asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                             : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                             : "r"(at + byte_at<RB>((mat & 1) * 8 + r8, (c + (mat >> 1)) * 16))
                             : "memory");
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < CP / 2; ++j) {
                        uint32_t a[4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t u = y[2 * h + i];
                            const uint32_t w = BITS == 4 && j ? u >> 8 : u;
                            a[2 * i] = normal<0>(code<0>(w));
                            a[2 * i + 1] = normal<1>(code<1>(w));
                        }
                        const int k = (c + h) * (CP / 2) + j;
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_parts(o[n][k], a, b, n, x);
                    }
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
                float s = at(l[n], i);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                const int head = n * 8 + 2 * t + i;
                if (head >= G) continue;
                const float up = 1.f / at(f[n], i);        // 2^(E - m)
                // of chunk c of a row of values a lane has the channels of piece g, one after another
#pragma unroll
                for (int k = 0; k < KS; k += 8 / BITS) {
                    float* to = out + head * D + (BITS == 8 ? k * 16 + 2 * g : k * 16 + 4 * g);
                    if constexpr (BITS == 8) *reinterpret_cast<float2*>(to) = make_float2(o[n][k][i] * 0x1p10f * up, o[n][k][2 + i] * 0x1p10f * up);
                    else *reinterpret_cast<float4*>(to) = make_float4(o[n][k][i] * 0x1p10f * up, o[n][k][2 + i] * 0x1p10f * up,
                                                                      o[n][k + 1][i] * 0x1p10f * up, o[n][k + 1][2 + i] * 0x1p10f * up);
                }
                if (g == 0) ml[head] = make_float2(at(m[n], i), bad ? NAN : s);
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
    const unsigned char* const K = static_cast<const unsigned char*>(pool.K) + lane * 16;
    const unsigned char* const V = static_cast<const unsigned char*>(pool.V) + lane * 16;
    const float* const scales = (lane < 4 ? pool.ks : pool.vs) + (lane & 3) * 4;
    auto ask = [&](int t, int stage) {
#pragma unroll
        for (int x = 0; x < 2; ++x, t += stride) {
            if (t >= ntiles) break;
            const bool ok = (unsigned)pg_next < (unsigned)pool.pages;
            if (!ok) bad = true;                           // (its row is NaN: any page's codes do)
            const unsigned at = ((unsigned)((ok ? pg_next : 0) * pool.heads + h) << tsh) + (unsigned)(t & ((1 << tsh) - 1));   // tile of the pool (< 2^27)
            const uint32_t to = smem_u32(ring + (stage + x) * L::kBytes);
#pragma unroll
            for (int i = 0; i < L::kRow / 32; ++i) {
                cp_async16(to + chunk_at<L::kRow>(lane + 32 * i), K + (size_t)at * L::kCodes + i * 512);
                cp_async16(to + L::kCodes + chunk_at<L::kRow>(lane + 32 * i), V + (size_t)at * L::kCodes + i * 512);
            }
            if (lane < 8) cp_async16(to + 2 * L::kCodes + lane * 16, scales + (size_t)at * kKeys);
            if (t + stride < ntiles) pg_next = table[(t + stride) >> tsh];
        }
        cp_commit();
    };
    // a warp's tiles in twos
    static_assert(NS % 2 == 0, "whole twos");
#pragma unroll 1
    for (int s = 0; s < NS - 2; s += 2) ask(t0 + s * stride, s);
    Core<D, BITS, NT, sizeof(T) == 2 ? 1 : 2> core;
    core.init(static_cast<const T*>(R.q) + (size_t)row * R.q_stride + (size_t)h * G * D, G, R.qscale);
    int stage = 0;
#pragma unroll 1
    for (int t = t0; t < ntiles; t += 2 * stride) {
        ask(t + (NS - 2) * stride, stage == 0 ? NS - 2 : stage - 2);
        cp_wait<NS / 2 - 1>();
        __syncwarp();
        const unsigned char* const a = ring + stage * L::kBytes;
        const int mine = t == ntiles - 1 ? (pos & 15) + 1 : kKeys;
        if (t + stride < ntiles) {
            core.template tiles<2>({a, a + L::kBytes}, t + stride == ntiles - 1 ? kKeys + (pos & 15) + 1 : 2 * kKeys);
        } else {
            core.template tiles<1>({a}, mine);
        }
        __syncwarp();
        stage = stage + 2 == NS ? 0 : stage + 2;
    }
    cp_wait<0>();
    __syncwarp();

    // the warps' sums, then the CTAs'
    static_assert(L::kRing >= (int)sizeof(float) * 8 * NT * D, "a warp's sums lie in its ring");
    core.finish(reinterpret_cast<float*>(ring), S.wml[warp], G, bad);
    __syncthreads();
    float* sums = reinterpret_cast<float*>(raw);           // in the place of warp 0's
    constexpr int V4 = D / 32;                             // a lane's channels of a head
    T* orow = static_cast<T*>(R.out) + (size_t)row * R.out_stride + (size_t)h * G * D;
    // no key at all, or none of weight: zero; a bad table entry has made l NaN
    auto leave = [&](int g, float l, float (&o)[V4]) {
        const float f = 1.f / l;
#pragma unroll
        for (int e = 0; e < V4; ++e) o[e] = l == 0.f ? 0.f : o[e] * f;
        store_out<V4>(orow + g * D + lane * V4, o);
    };
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
        if (C == 1) {
            leave(g, l, o);
        } else {
            store_out<V4>(sums + g * D + lane * V4, o);
            if (lane == 0) S.ml[g] = make_float2(m, l);
        }
    }
    if (C == 1) return;
    cluster_arrive();
    cluster_wait();
    // a warp joins a head's sums of all CTAs
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
        leave(g, l, o);
    }
    cluster_arrive();
    cluster_wait();                                        // no CTA leaves while another reads its sums
}

// CTAs of a unit: as many, up to 16, as fill the GPU twice with every warp left a tile (64 units of 256 tiles: 30 us with
// one, 16 with four, 20 with eight; 32 of 2048: 66 with four, 50 with eight, 61 with sixteen), and beyond that, so that units of
// unequal lengths share the SMs evenly, as leave a warp 48 tiles and the GPU 2048 CTAs (512 units of up to 1536 tiles: 280 us
// with one, 243 with four, 253 with eight).
int cluster_of(long long units, int tiles)
{
    int c = 1;
    while (c < kMaxCluster && ((units * 2 * c <= 2 * kSMs && tiles >= kWarps * 2 * c) || (units * 2 * c <= 2048 && tiles >= 48 * kWarps * 2 * c))) c *= 2;
    return c;
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
    int C = cluster_of(units, r.width * (p.ps / kKeys));
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
