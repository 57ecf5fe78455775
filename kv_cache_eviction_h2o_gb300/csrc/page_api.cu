// page_api.cu -- the paged-cache calls of the C ABI (include/h2o.h): argument
// checks and launches.  They hold no state: the caller owns every buffer.
#include <climits>
#include <cmath>
#include <cstdlib>
#include <cstring>

#include "h2o.h"
#include "kernels.h"
#include "paged.h"

using namespace h2o;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// host-side fault injection for the failure-path tests, as for handles
bool inject_launch()
{
    const char* f = getenv("H2O_FAULT");
    return f && strcmp(f, "launch") == 0;
}

int launched(cudaError_t e, const char* where)
{
    return e == cudaSuccess ? H2O_OK : set_last_error(H2O_ERR_CUDA, "%s launch: %s", where, cudaGetErrorString(e));
}

int check_pool(const PagePool& p)
{
    if (!p.K || !p.V) return set_last_error(H2O_ERR_ARG, "K and V must be non-NULL");
    if (!aligned16(p.K) || !aligned16(p.V) || !aligned16(p.bounds))
        return set_last_error(H2O_ERR_ARG, "K, V and bounds must be 16-byte aligned");
    if (p.dtype == (H2O_BF16 | H2O_KV8) || p.dtype == H2O_KV8 || p.dtype == (H2O_BF16 | H2O_KV4) || p.dtype == H2O_KV4)
        return set_last_error(H2O_ERR_UNSUPPORTED, "H2O_KV8 / H2O_KV4 are not supported on paged caches");
    if (p.dtype != H2O_F32 && p.dtype != H2O_BF16) return set_last_error(H2O_ERR_ARG, "dtype must be H2O_F32 or H2O_BF16");
    if (p.D != 64 && p.D != 128) return set_last_error(H2O_ERR_ARG, "head_dim must be 64 or 128 (got %d)", p.D);
    if (p.ps != 16 && p.ps != 32 && p.ps != 64 && p.ps != 128)
        return set_last_error(H2O_ERR_ARG, "page_size must be 16, 32, 64 or 128 (got %d)", p.ps);
    if (p.pages < 1 || p.heads < 1 || p.heads > 65535)
        return set_last_error(H2O_ERR_ARG, "num_pages must be >= 1 and kv_heads in [1, 65535]");
    if ((long long)p.pages * p.heads > INT_MAX / p.ps)
        return set_last_error(H2O_ERR_ARG, "num_pages * kv_heads * page_size must be below 2^31");
    return H2O_OK;
}

// a row of `need` elements every `stride` elements, rows starting on 16 bytes
int check_stride(long long stride, long long need, int dtype, const char* what)
{
    const int per16 = dtype == H2O_BF16 ? 8 : 4;
    if (stride < need) return set_last_error(H2O_ERR_ARG, "%s rows are %lld elements apart, and hold %lld", what, stride, need);
    if (stride % per16) return set_last_error(H2O_ERR_ARG, "%s rows must start on 16-byte boundaries", what);
    return H2O_OK;
}

// Whether rows of q are written by other rows' results: q and out share memory and are neither the same rows nor different
// columns of the same rows (of a fused buffer).
bool rows_collide(const PageRows& r, long long need, int dtype)
{
    const long long size = dtype == H2O_BF16 ? 2 : 4, qs = r.q_stride * size, os = r.out_stride * size, n = need * size;
    const uintptr_t q = reinterpret_cast<uintptr_t>(r.q), o = reinterpret_cast<uintptr_t>(r.out);
    if (r.rows < 1 || q + (r.rows - 1) * qs + n <= o || o + (r.rows - 1) * os + n <= q) return false;
    if (r.rows == 1) return q != o;
    if (qs != os) return true;
    const long long by = (long long)(o > q ? o - q : q - o) % qs;
    return q != o && (by < n || by > qs - n);
}

int check_rows(const PagePool& p, const PageRows& r, double scale)
{
    if (r.rows < 0) return set_last_error(H2O_ERR_ARG, "rows must be >= 0 (got %d)", r.rows);
    if (r.G < 1 || r.G > kMaxPageGroups)
        return set_last_error(H2O_ERR_ARG, "groups must be in [1, %d] (got %d)", kMaxPageGroups, r.G);
    if (r.requests < 1) return set_last_error(H2O_ERR_ARG, "requests must be >= 1 (got %d)", r.requests);
    if (r.width < 1 || r.width > kMaxTableWidth)
        return set_last_error(H2O_ERR_ARG, "table_width must be in [1, %d] (got %d)", kMaxTableWidth, r.width);
    if (!(scale > 0.0) || !std::isfinite(scale)) return set_last_error(H2O_ERR_ARG, "scale must be finite and > 0");
    if (!(r.qscale > 0.f) || !std::isfinite(r.qscale)) return set_last_error(H2O_ERR_ARG, "scale is out of fp32's range");
    if ((long long)r.rows * p.heads > (1 << 24) / r.G)
        return set_last_error(H2O_ERR_ARG, "rows * kv_heads * groups must be at most 2^24");
    if (!r.table) return set_last_error(H2O_ERR_ARG, "table must be non-NULL");
    if (r.rows && (!r.q || !r.out || !r.seq || !r.pos))
        return set_last_error(H2O_ERR_ARG, "q, out, row_seq and row_pos must be non-NULL");
    if (!aligned16(r.q) || !aligned16(r.out)) return set_last_error(H2O_ERR_ARG, "q and out must be 16-byte aligned");
    if (!aligned4(r.seq) || !aligned4(r.pos) || !aligned4(r.table))
        return set_last_error(H2O_ERR_ARG, "row_seq, row_pos and table must be 4-byte aligned");
    int rc;
    const long long need = (long long)p.heads * r.G * p.D;
    if ((rc = check_stride(r.q_stride, need, p.dtype, "q")) || (rc = check_stride(r.out_stride, need, p.dtype, "out"))) return rc;
    if (rows_collide(r, need, p.dtype)) return set_last_error(H2O_ERR_ARG, "out overlaps other rows of q");
    return H2O_OK;
}

}  // namespace

extern "C" {

int h2o_page_tables(const int* len_before, const int* n_new, int requests, const int* free_pages, int n_free,
                    int page_size, int* table, int table_width, int* len_after, int* row_start, int* row_seq,
                    int* row_pos, int* slot, int rows_cap, int* status, void* cuda_stream)
{
    if (requests < 1 || requests > kMaxPageRequests)
        return set_last_error(H2O_ERR_ARG, "requests must be in [1, %d] (got %d)", kMaxPageRequests, requests);
    if (n_free < 0 || rows_cap < 0 || rows_cap > 1 << 30)
        return set_last_error(H2O_ERR_ARG, "n_free must be >= 0 and rows_cap in [0, 2^30]");
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
        return set_last_error(H2O_ERR_ARG, "page_size must be 16, 32, 64 or 128 (got %d)", page_size);
    if (table_width < 1 || table_width > kMaxTableWidth)
        return set_last_error(H2O_ERR_ARG, "table_width must be in [1, %d] (got %d)", kMaxTableWidth, table_width);
    if (!len_before || !n_new || !table || !len_after || !row_start || !status || (n_free && !free_pages) ||
        (rows_cap && (!row_seq || !row_pos || !slot)))
        return set_last_error(H2O_ERR_ARG, "the lengths, free_pages, table, the row maps and status must be non-NULL");
    const void* all[] = {len_before, n_new, free_pages, table, len_after, row_start, row_seq, row_pos, slot, status};
    for (const void* p : all)
        if (!aligned4(p)) return set_last_error(H2O_ERR_ARG, "h2o_page_tables arrays must be 4-byte aligned");
    // (CTAs read the inputs while others write: lengths updated in place would be taken for both)
    struct Range { const int* p; long long n; };
    const Range in[] = {{len_before, requests}, {n_new, requests}, {free_pages, n_free}};
    const Range out[] = {{table, (long long)requests * table_width}, {len_after, requests}, {row_start, requests + 1LL},
                         {row_seq, rows_cap}, {row_pos, rows_cap}, {slot, rows_cap}, {status, 4}};
    for (const Range& x : in)
        for (const Range& y : out)
            if (x.n && y.n && reinterpret_cast<uintptr_t>(x.p) < reinterpret_cast<uintptr_t>(y.p) + y.n * sizeof(int) &&
                reinterpret_cast<uintptr_t>(y.p) < reinterpret_cast<uintptr_t>(x.p) + x.n * sizeof(int))
                return set_last_error(H2O_ERR_ARG, "an output of h2o_page_tables overlaps an input");
    if (inject_launch()) return set_last_error(H2O_ERR_CUDA, "kernel launch failed (injected)");
    TablesArgs a = {};
    a.before = len_before; a.fresh = n_new; a.free_pages = free_pages; a.table = table; a.after = len_after;
    a.row_start = row_start; a.row_seq = row_seq; a.row_pos = row_pos; a.slot = slot; a.status = status;
    a.n = requests; a.n_free = n_free; a.ps = page_size; a.width = table_width; a.cap = rows_cap;
    return launched(launch_page_tables(a, reinterpret_cast<cudaStream_t>(cuda_stream)), "h2o_page_tables");
}

int h2o_page_write(const void* k, const void* v, long long k_stride, long long v_stride, const int* slot, int rows,
                   void* K, void* V, void* bounds, int num_pages, int kv_heads, int page_size, int head_dim, int dtype,
                   void* cuda_stream)
{
    PagePool p = {};
    p.K = K; p.V = V; p.bounds = bounds;
    p.pages = num_pages; p.heads = kv_heads; p.ps = page_size; p.D = head_dim; p.dtype = dtype;
    int rc = check_pool(p);
    if (rc) return rc;
    if (!bounds) return set_last_error(H2O_ERR_ARG, "bounds must be non-NULL");
    if (rows < 0) return set_last_error(H2O_ERR_ARG, "rows must be >= 0 (got %d)", rows);
    if (rows && (!k || !v || !slot)) return set_last_error(H2O_ERR_ARG, "k, v and slot must be non-NULL");
    if (!aligned16(k) || !aligned16(v)) return set_last_error(H2O_ERR_ARG, "k and v must be 16-byte aligned");
    if (!aligned4(slot)) return set_last_error(H2O_ERR_ARG, "slot must be 4-byte aligned");
    const long long need = (long long)kv_heads * head_dim;
    if ((rc = check_stride(k_stride, need, dtype, "k")) || (rc = check_stride(v_stride, need, dtype, "v"))) return rc;
    if (!rows) return H2O_OK;
    if (inject_launch()) return set_last_error(H2O_ERR_CUDA, "kernel launch failed (injected)");
    return launched(launch_page_write(p, k, v, k_stride, v_stride, slot, rows, reinterpret_cast<cudaStream_t>(cuda_stream)),
                    "h2o_page_write");
}

int h2o_page_attend(const void* q, long long q_stride, const int* row_seq, const int* row_pos, int rows, const void* K,
                    const void* V, const void* bounds, int num_pages, int kv_heads, int groups, int page_size,
                    int head_dim, int dtype, const int* table, int requests, int table_width, int budget, int recent,
                    double scale, void* out, long long out_stride, int* picked, void* cuda_stream)
{
    PagePool p = {};
    p.K = const_cast<void*>(K); p.V = const_cast<void*>(V); p.bounds = const_cast<void*>(bounds);
    p.pages = num_pages; p.heads = kv_heads; p.ps = page_size; p.D = head_dim; p.dtype = dtype;
    PageRows r = {};
    r.q = q; r.out = out; r.q_stride = q_stride; r.out_stride = out_stride; r.seq = row_seq; r.pos = row_pos;
    r.table = table; r.rows = rows; r.G = groups; r.requests = requests; r.width = table_width;
    r.qscale = (float)(scale * 1.4426950408889634);
    int rc;
    if ((rc = check_pool(p)) || (rc = check_rows(p, r, scale))) return rc;
    if (recent < 1 || recent > budget) return set_last_error(H2O_ERR_ARG, "recent must be in [1, budget] (got %d of %d)", recent, budget);
    if (budget < table_width) {
        if (budget > kMaxPickedPages)
            return set_last_error(H2O_ERR_ARG, "a budget below table_width must be at most %d pages (got %d)", kMaxPickedPages, budget);
        if (!bounds) return set_last_error(H2O_ERR_ARG, "bounds must be non-NULL when budget is below table_width");
    }
    if (!aligned4(picked)) return set_last_error(H2O_ERR_ARG, "picked must be 4-byte aligned");
    if (!rows) return H2O_OK;
    if (inject_launch()) return set_last_error(H2O_ERR_CUDA, "kernel launch failed (injected)");
    return launched(launch_page_attend(p, r, budget, recent, picked, PrefixPart{}, reinterpret_cast<cudaStream_t>(cuda_stream)),
                    "h2o_page_attend");
}

long long h2o_prefix_work_bytes(int rows, int kv_heads, int groups, int head_dim, int prefix_len, int dtype)
{
    if (rows < 0 || kv_heads < 1 || groups < 1 || groups > kMaxPageGroups || (head_dim != 64 && head_dim != 128) ||
        prefix_len < 0 || prefix_len > kMaxPrefix || (dtype != H2O_F32 && dtype != H2O_BF16) || (long long)rows * kv_heads > (1 << 24) / groups)
        return set_last_error(H2O_ERR_ARG, "h2o_prefix_work_bytes: sizes out of range");
    const long long qrows = (long long)rows * kv_heads * groups;
    // at least 16 bytes, so that the buffer is one
    return 16 + prefix_splits(rows, kv_heads, groups, head_dim, prefix_len, dtype) * qrows * (4LL * head_dim + 8);
}

int h2o_prefix_attend(const void* q, long long q_stride, const int* row_seq, const int* row_pos, int rows, const void* K,
                      const void* V, int num_pages, int kv_heads, int groups, int page_size, int head_dim, int dtype,
                      const int* prefix_table, int prefix_len, const int* table, int requests, int table_width,
                      double scale, void* out, long long out_stride, void* work, long long work_bytes, void* cuda_stream)
{
    PagePool p = {};
    p.K = const_cast<void*>(K); p.V = const_cast<void*>(V);
    p.pages = num_pages; p.heads = kv_heads; p.ps = page_size; p.D = head_dim; p.dtype = dtype;
    PageRows r = {};
    r.q = q; r.out = out; r.q_stride = q_stride; r.out_stride = out_stride; r.seq = row_seq; r.pos = row_pos;
    r.table = table; r.rows = rows; r.G = groups; r.requests = requests; r.width = table_width;
    r.qscale = (float)(scale * 1.4426950408889634);
    int rc;
    if ((rc = check_pool(p)) || (rc = check_rows(p, r, scale))) return rc;
    if (prefix_len < 0 || prefix_len > kMaxPrefix)
        return set_last_error(H2O_ERR_ARG, "prefix_len must be in [0, 2^30] (got %d)", prefix_len);
    if (prefix_len && (!prefix_table || !aligned4(prefix_table)))
        return set_last_error(H2O_ERR_ARG, "prefix_table must be non-NULL and 4-byte aligned");
    const long long need = h2o_prefix_work_bytes(rows, kv_heads, groups, head_dim, prefix_len, dtype);
    if (!work || !aligned16(work) || work_bytes < need)
        return set_last_error(H2O_ERR_ARG, "work must be 16-byte aligned and hold %lld bytes (got %lld)", need, work_bytes);
    if (!rows) return H2O_OK;
    if (inject_launch()) return set_last_error(H2O_ERR_CUDA, "kernel launch failed (injected)");
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
    PrefixPart part = {};
    part.splits = prefix_splits(rows, kv_heads, groups, head_dim, prefix_len, dtype);
    part.o = static_cast<float*>(work);
    part.ml = reinterpret_cast<float2*>(part.o + (size_t)part.splits * rows * kv_heads * groups * head_dim);
    cudaError_t e = cudaSuccess;
    if (part.splits) e = launch_prefix(p, r, prefix_table, prefix_len, part, st);
    if (e == cudaSuccess) e = launch_page_attend(p, r, 0, 0, nullptr, part, st);
    return launched(e, "h2o_prefix_attend");
}

}  // extern "C"
