// page_checks.h -- argument checks that the calls without a handle share.
#pragma once

#include <cmath>
#include <cstdlib>
#include <cstring>

#include "h2o.h"
#include "kernels.h"
#include "paged.h"

namespace h2o {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// host-side fault injection for the failure-path tests, as for handles
inline bool inject_launch()
{
    const char* f = getenv("H2O_FAULT");
    return f && strcmp(f, "launch") == 0;
}

inline int launched(cudaError_t e, const char* where)
{
    return e == cudaSuccess ? H2O_OK : set_last_error(H2O_ERR_CUDA, "%s launch: %s", where, cudaGetErrorString(e));
}

// a row of `need` elements every `stride` elements, rows starting on 16 bytes
inline int check_stride(long long stride, long long need, int dtype, const char* what)
{
    const int per16 = dtype == H2O_BF16 ? 8 : 4;
    if (stride < need) return set_last_error(H2O_ERR_ARG, "%s rows are %lld elements apart, and hold %lld", what, stride, need);
    if (stride % per16) return set_last_error(H2O_ERR_ARG, "%s rows must start on 16-byte boundaries", what);
    return H2O_OK;
}

// Whether rows of q are written by other rows' results: q and out share memory and are neither the same rows nor different
// columns of the same rows (of a fused buffer).
inline bool rows_collide(const PageRows& r, long long need, int dtype)
{
    const long long size = dtype == H2O_BF16 ? 2 : 4, qs = r.q_stride * size, os = r.out_stride * size, n = need * size;
    const uintptr_t q = reinterpret_cast<uintptr_t>(r.q), o = reinterpret_cast<uintptr_t>(r.out);
    if (r.rows < 1 || q + (r.rows - 1) * qs + n <= o || o + (r.rows - 1) * os + n <= q) return false;
    if (r.rows == 1) return q != o;
    if (qs != os) return true;
    const long long by = (long long)(o > q ? o - q : q - o) % qs;
    return q != o && (by < n || by > qs - n);
}

inline int check_rows(const PagePool& p, const PageRows& r, double scale)
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

}  // namespace h2o
