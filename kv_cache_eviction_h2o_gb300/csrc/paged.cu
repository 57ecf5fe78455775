// paged.cu -- bookkeeping and writing of the paged cache: which pages and
// slots a step's new tokens take, and their key and value rows into them.
#include <algorithm>
#include <climits>

#include "common.cuh"
#include "paged.h"

namespace h2o {

namespace {

// ------------------------------------------------------------ block tables
//
// With b_i tokens before and t_i new ones, request i owns o_i = ceil(b_i / ps)
// pages and takes n_i = ceil((b_i + t_i) / ps) - o_i more from the free list,
// so with P_i = sum_{j<i} n_j and R_i = sum_{j<i} t_j
//   table[i][o_i + j] = free[P_i + j],   row R_i + x: pos = b_i + x,
//   slot = table[i][pos / ps] * ps + pos % ps.
// Every CTA makes both running sums over all requests for itself (8 bytes a
// request, read from L2) and then writes its share of the rows and pages, so
// one launch does it with no order between CTAs.  A slot is taken from the
// free list, not from the table entry another CTA may be writing.  Bound:
// launch latency for a decode step, the maps' 12 bytes a row for prompts.

enum TableError : int { kTableCount = 1, kTableRows = 2, kTablePages = 4, kTableWidth = 8 };

struct TableSums {
    long long rows, pages;
};

__device__ __forceinline__ TableSums sums_up(TableSums x, int d, int lane)
{
    const long long r = __shfl_up_sync(0xffffffffu, x.rows, d), p = __shfl_up_sync(0xffffffffu, x.pages, d);
    if (lane >= d) { x.rows += r; x.pages += p; }
    return x;
}

// the last i in [0, n) with start[i] <= x (start ascending, start[0] <= x)
__device__ __forceinline__ int owner_of(const int* start, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// x[i .. i + 3], zeros from n on
__device__ __forceinline__ int4 four_of(const int* x, int i, int n)
{
    if (i + 4 <= n && ((size_t)x & 15) == 0) return *reinterpret_cast<const int4*>(x + i);
    return make_int4(i < n ? x[i] : 0, i + 1 < n ? x[i + 1] : 0, i + 2 < n ? x[i + 2] : 0, i + 3 < n ? x[i + 3] : 0);
}

// A thread takes four requests at a time (i a multiple of four).
__global__ void __launch_bounds__(1024) page_tables_kernel(const TablesArgs a)
{
    extern __shared__ __align__(16) int sm[];
    const int n4 = (a.n + 4) & ~3;     // room for n + 1, in fours
    int* start = sm;                   // [n + 1] first row of each request
    int* first = sm + n4;              // [n + 1] first free-list entry of each
    int* before = sm + 2 * n4;         // [n]
    __shared__ TableSums warp_sum[32];
    __shared__ int warp_max[32], flags;
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int sh = __ffs(a.ps) - 1, up = a.ps - 1;
    const int per = ((a.n + nt - 1) / nt + 3) & ~3, i0 = min(a.n, tid * per), i1 = min(a.n, i0 + per);
    if (tid == 0) flags = 0;
    __syncthreads();

    TableSums mine{0, 0};
    int longest = 0, bad = 0;
    int4 b4 = make_int4(0, 0, 0, 0), t4 = b4;              // (the last four, which with up to 4096 requests are all)
    for (int i = i0; i < i1; i += 4) {
        b4 = four_of(a.before, i, a.n);
        t4 = four_of(a.fresh, i, a.n);
        *reinterpret_cast<int4*>(before + i) = b4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const long long b = (&b4.x)[j], t = (&t4.x)[j];
            if (b < 0 || t < 0) { bad |= kTableCount; continue; }
            const long long want = (b + t + up) >> sh;
            if (want > a.width) bad |= kTableWidth;
            mine.rows += t;
            mine.pages += want - ((b + up) >> sh);
            longest = max(longest, (int)min(b + t, (long long)INT_MAX));
        }
    }
    if (bad) atomicOr(&flags, bad);
    TableSums upto = mine;
    for (int d = 1; d < 32; d <<= 1) upto = sums_up(upto, d, lane);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 31) warp_sum[warp] = upto;
    if (lane == 0) warp_max[warp] = longest;
    __syncthreads();
    if (warp == 0) {
        const bool in = lane < (nt >> 5);
        TableSums w = in ? warp_sum[lane] : TableSums{0, 0};
        longest = __reduce_max_sync(0xffffffffu, in ? warp_max[lane] : 0);
        for (int d = 1; d < 32; d <<= 1) w = sums_up(w, d, lane);
        if (in) warp_sum[lane] = w;
        if (lane == 0) warp_max[0] = longest;
    }
    __syncthreads();
    const TableSums all = warp_sum[(nt >> 5) - 1];
    int err = flags;
    if (all.rows > a.cap) err |= kTableRows;
    if (all.pages > a.n_free) err |= kTablePages;
    const int rows = err ? 0 : (int)all.rows, pages = err ? 0 : (int)all.pages;

    // all or nothing: with an error no request gets rows or pages
    long long r = upto.rows - mine.rows + (warp ? warp_sum[warp - 1].rows : 0);
    long long p = upto.pages - mine.pages + (warp ? warp_sum[warp - 1].pages : 0);
    for (int i = i0; i < i1; i += 4) {
        if (per > 4) {
            b4 = four_of(a.before, i, a.n);
            t4 = four_of(a.fresh, i, a.n);
        }
        int4 s4 = make_int4(0, 0, 0, 0), f4 = s4;
        if (!err)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int b = (&b4.x)[j], t = (&t4.x)[j];
                (&s4.x)[j] = (int)r;
                (&f4.x)[j] = (int)p;
                r += t;
                p += ((b + t + up) >> sh) - ((b + up) >> sh);
            }
        *reinterpret_cast<int4*>(start + i) = s4;
        *reinterpret_cast<int4*>(first + i) = f4;
    }
    __syncthreads();                                       // (before start[n] goes behind the last four)
    if (tid == 0) {
        start[a.n] = rows;
        first[a.n] = pages;
        if (blockIdx.x == 0) {
            a.status[0] = rows;
            a.status[1] = pages;
            a.status[2] = err ? 0 : warp_max[0];
            a.status[3] = err;
        }
    }
    __syncthreads();

    const int g = blockIdx.x * nt + tid, stride = gridDim.x * nt;
    for (int i = g; i <= a.n; i += stride) {
        a.row_start[i] = start[i];
        if (i < a.n) a.after[i] = before[i] + (start[i + 1] - start[i]);
    }
    // (from the other end: the first CTAs have the loop above and the longer share of the one below)
    for (int x = stride - 1 - g; x < pages; x += stride) {
        const int i = owner_of(first, a.n, x);
        a.table[(size_t)i * a.width + ((before[i] + up) >> sh) + (x - first[i])] = a.free_pages[x];
    }
    // four rows a thread, written as 16 bytes where the maps lie on them
    const bool wide = (((size_t)a.row_seq | (size_t)a.row_pos | (size_t)a.slot) & 15) == 0;
    const int last = (INT_MAX - a.ps) >> sh;
    for (int x0 = g * 4; x0 < a.cap; x0 += stride * 4) {
        int4 seq = make_int4(-1, -1, -1, -1), pos = seq, slot = seq;
        if (x0 < rows) {
            int i = owner_of(start, a.n, x0);
            // the page of position `at` of request i; a table or free-list entry that is no page gives no slot
            auto slot_of = [&](int at) {
                const int owned = (before[i] + up) >> sh, pg = at >> sh;
                const int page = pg < owned ? a.table[(size_t)i * a.width + pg] : a.free_pages[first[i] + pg - owned];
                return page >= 0 && page <= last ? (page << sh) + (at & up) : -1;
            };
            const int at = before[i] + (x0 - start[i]);
            if (x0 + 4 <= start[i + 1] && (at & up) <= a.ps - 4) {
                // all in one page of one request, as most are
                const int s = slot_of(at);
                seq = make_int4(i, i, i, i);
                pos = make_int4(at, at + 1, at + 2, at + 3);
                if (s >= 0) slot = make_int4(s, s + 1, s + 2, s + 3);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int x = x0 + j;
                    if (x >= rows) break;
                    while (start[i + 1] <= x) ++i;
                    const int y = before[i] + (x - start[i]);
                    (&seq.x)[j] = i;
                    (&pos.x)[j] = y;
                    (&slot.x)[j] = slot_of(y);
                }
            }
        }
        if (wide && x0 + 4 <= a.cap) {
            *reinterpret_cast<int4*>(a.row_seq + x0) = seq;
            *reinterpret_cast<int4*>(a.row_pos + x0) = pos;
            *reinterpret_cast<int4*>(a.slot + x0) = slot;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (x0 + j >= a.cap) break;
                a.row_seq[x0 + j] = (&seq.x)[j];
                a.row_pos[x0 + j] = (&pos.x)[j];
                a.slot[x0 + j] = (&slot.x)[j];
            }
        }
    }
}

// ------------------------------------------------------------- page writes
//
// A row goes to page slot / ps, offset slot % ps, as it is; the row with a
// page's last offset also leaves the page's bounds, the smallest and largest
// value of each channel over its ps keys (NaN where one is NaN).  Bounds are
// made when a page fills, from all its keys, and not kept up to date row by
// row: a page that is not full is never ranked, and a page that was rolled
// back and filled again gets bounds of what it holds.  Keys of rows in this
// call are read from k (rows just before this one, which go to the page too),
// older ones from the page.  Bound: HBM.

template <typename T> struct Vec16;
template <> struct Vec16<float> {
    float x[4];
    __device__ __forceinline__ void load(const void* p)
    {
        const float4 w = *static_cast<const float4*>(p);
        x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
    }
    __device__ __forceinline__ void store(void* p) const { *static_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]); }
    __device__ __forceinline__ void low(const Vec16& o)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("min.NaN.f32 %0, %0, %1;" : "+f"(x[i]) : "f"(o.x[i]));
    }
    __device__ __forceinline__ void high(const Vec16& o)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(x[i]) : "f"(o.x[i]));
    }
};
template <> struct Vec16<__nv_bfloat16> {
    uint32_t x[4];
    __device__ __forceinline__ void load(const void* p)
    {
        const uint4 w = *static_cast<const uint4*>(p);
        x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
    }
    __device__ __forceinline__ void store(void* p) const { *static_cast<uint4*>(p) = make_uint4(x[0], x[1], x[2], x[3]); }
    __device__ __forceinline__ void low(const Vec16& o)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(x[i]) : "r"(o.x[i]));
    }
    __device__ __forceinline__ void high(const Vec16& o)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(x[i]) : "r"(o.x[i]));
    }
};

constexpr int kWriteThreads = 256;

// A CTA takes RPT * 256 / tx rows and tx 16-byte columns of them (all heads
// side by side): thread = column and every (256 / tx)-th row, all its loads
// before its stores.  Then, for each row among them that ends a page, the
// threads of a column share the page's keys, most of which L2 has just then.
// (32768 rows of 8 heads, 64-token pages: 49 us, of 40 at the copy bandwidth;
// 42 without bounds, 56 with CTAs apart for them.)
template <typename T, int D, int RPT>
__global__ void __launch_bounds__(kWriteThreads) page_write_kernel(const PagePool p, const T* __restrict__ k, const T* __restrict__ v,
                                                                   const long long k_stride, const long long v_stride,
                                                                   const int* __restrict__ slot, const int rows, const int tx)
{
    constexpr int E = 16 / sizeof(T), VPR = D / E;        // elements of a vector, vectors of a row's head
    __shared__ Vec16<T> part[2][kWriteThreads];
    __shared__ int near[kWriteThreads];                   // slots of this CTA's rows, behind those of the page size - 1 rows before
    const int sh = __ffs(p.ps) - 1, ty = kWriteThreads / tx, up = p.ps - 1;
    const int x = threadIdx.x & (tx - 1), y = threadIdx.x / tx, col = blockIdx.y * tx + x;
    const bool in = col < p.heads * VPR;
    const int h = col / VPR, e = (col & (VPR - 1)) * E;
    const int r0 = blockIdx.x * RPT * ty, nr = min(rows - r0, RPT * ty);
    T* K = static_cast<T*>(p.K);
    T* V = static_cast<T*>(p.V);
    const T* kc = k + (size_t)col * E;
    const T* vc = v + (size_t)col * E;
    {
        // (up + nr <= 127 + 128)
        const int r = r0 - up + (int)threadIdx.x;
        int s = -1;
        if (r >= 0 && (int)threadIdx.x < up + nr) s = slot[r];
        near[threadIdx.x] = s < (long long)p.pages * p.ps ? s : -1;
    }
    __syncthreads();
    auto place = [&](int s) {                             // of this column in slot s
        return (((size_t)(s >> sh) * p.heads + h) * p.ps + (s & up)) * D + e;
    };
    Vec16<T> kv[RPT], vv[RPT];
    int s[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = y + i * ty;
        s[i] = in && r < nr ? near[up + r] : -1;
        if (s[i] >= 0) {
            kv[i].load(kc + (r0 + r) * k_stride);
            vv[i].load(vc + (r0 + r) * v_stride);
        }
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i)
        if (s[i] >= 0) {
            kv[i].store(K + place(s[i]));
            vv[i].store(V + place(s[i]));
        }
    for (int r = 0; r < nr; ++r) {
        const int end = near[up + r];
        if (end < 0 || (end & up) != up) continue;        // (the same for the whole CTA)
        // The key at offset o is that of a row of this call, or one of before.  The row lies up - o before this one, or nearer
        // where the call leaves slots of the page out.
        bool gaps = false;
        for (int i = threadIdx.x & 31; i < up; i += 32) gaps |= (near[r + i] >> sh) == (end >> sh) && near[r + i] - i != end - up;
        gaps = __any_sync(0xffffffffu, gaps);
        Vec16<T> lo, hi;
        if (in) {
            const T* page = K + place(end) - (size_t)up * D;
            lo.load(kc + (r0 + r) * k_stride);
            hi = lo;
            auto take = [&](int o, int i) {
                Vec16<T> w;
                w.load(near[i] == end - up + o ? kc + (r0 - up + i) * k_stride : page + o * D);
                lo.low(w);
                hi.high(w);
            };
            if (gaps) {
                for (int o = y; o < up; o += ty) {
                    int i = r + o;
                    while (i < r + up && near[i] != end - up + o) ++i;
                    take(o, i);
                }
            } else {
#pragma unroll 8
                for (int o = y; o < up; o += ty) take(o, r + o);
            }
            part[0][threadIdx.x] = lo;
            part[1][threadIdx.x] = hi;
        }
        __syncthreads();
        if (in && y == 0) {
            for (int j = 1; j < ty; ++j) {
                lo.low(part[0][j * tx + x]);
                hi.high(part[1][j * tx + x]);
            }
            T* b = static_cast<T*>(p.bounds) + ((size_t)(end >> sh) * p.heads + h) * 2 * D + e;
            lo.store(b);
            hi.store(b + D);
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_page_tables(const TablesArgs& a, cudaStream_t st)
{
    const long long work = std::max<long long>(a.n, ((long long)a.cap + 3) / 4);
    const int threads = work <= 256 ? 256 : 1024;
    const int grid = (int)std::min<long long>(kSMs, std::max<long long>(1, (work + threads - 1) / threads));
    const size_t smem = 3 * sizeof(int) * (((size_t)a.n + 4) & ~(size_t)3);
    static SmemOnce once;                                  // (the kernel's own arrays count towards the 48 KB too)
    const cudaError_t e = once.allow(page_tables_kernel);
    if (e != cudaSuccess) return e;
    page_tables_kernel<<<grid, threads, smem, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_page_write(const PagePool& p, const void* k, const void* v, long long k_stride, long long v_stride,
                              const int* slot, int rows, cudaStream_t st)
{
    const int cols = p.heads * (p.D * (p.dtype ? 2 : 4) / 16);
    int tx = 8;
    while (tx < 64 && tx < cols) tx *= 2;
    const int ty = kWriteThreads / tx;
    // four rows a thread where that still makes two CTAs an SM
    const long long tiles = ((rows + 4LL * ty - 1) / (4 * ty)) * ((cols + tx - 1) / tx);
    auto go = [&](auto t, auto d, auto rpt) {
        using T = decltype(t);
        constexpr int R = decltype(rpt)::value;
        const dim3 grid((unsigned)((rows + (long long)R * ty - 1) / (R * ty)), (unsigned)((cols + tx - 1) / tx));
        page_write_kernel<T, decltype(d)::value, R><<<grid, kWriteThreads, 0, st>>>(p, static_cast<const T*>(k), static_cast<const T*>(v),
                                                                                    k_stride, v_stride, slot, rows, tx);
    };
    auto by_rows = [&](auto t, auto d) {
        if (tiles >= 2 * kSMs) go(t, d, std::integral_constant<int, 4>());
        else go(t, d, std::integral_constant<int, 1>());
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (p.dtype) p.D == 64 ? by_rows(__nv_bfloat16(), D64()) : by_rows(__nv_bfloat16(), D128());
    else p.D == 64 ? by_rows(float(), D64()) : by_rows(float(), D128());
    return cudaGetLastError();
}

}  // namespace h2o
