// prompt_api.cu -- rotary positions, prompt attention and quantised paged
// caches of the C ABI (include/h2o.h): argument checks and launches.  They
// hold no state: the caller owns every buffer.
#include <climits>

#include "h2o.h"
#include "kernels.h"
#include "page_checks.h"
#include "prompts.h"

using namespace h2o;

namespace {

// rows of `need` elements, `stride` apart
struct Rows {
    const void* p;
    long long stride, need;
};

// Whether an output's rows a share memory with b's and are neither the same rows nor other columns of the same rows.
bool collide(const Rows& a, long long na, const Rows& b, long long nb, int size)
{
    if (na < 1 || nb < 1 || !a.need || !b.need) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    const long long as = a.stride * size, bs = b.stride * size, an = a.need * size, bn = b.need * size;
    if (x + (na - 1) * as + an <= y || y + (nb - 1) * bs + bn <= x) return false;
    if (as != bs) return true;
    const long long by = x > y ? (as - (long long)(x - y) % as) % as : (long long)(y - x) % as;   // where b's columns begin in a's rows
    return by < an || by + bn > as;
}

bool same(const Rows& a, const Rows& b, int rows) { return a.p == b.p && (a.stride == b.stride || rows == 1); }

int check_head_dim(int d)
{
    return d == 64 || d == 128 ? H2O_OK : set_last_error(H2O_ERR_ARG, "head_dim must be 64 or 128 (got %d)", d);
}

int check_row_type(int dtype)
{
    return dtype == H2O_F32 || dtype == H2O_BF16 ? H2O_OK : set_last_error(H2O_ERR_ARG, "dtype must be H2O_F32 or H2O_BF16");
}

int make_pool(QuantPool& p, const void* K, const void* V, const float* ks, const float* vs, int pages, int heads, int ps, int D, int dtype)
{
    p.K = const_cast<void*>(K); p.V = const_cast<void*>(V); p.ks = const_cast<float*>(ks); p.vs = const_cast<float*>(vs);
    p.pages = pages; p.heads = heads; p.ps = ps; p.D = D;
    const int flag = dtype & (H2O_KV8 | H2O_KV4);
    p.dtype = dtype & ~(H2O_KV8 | H2O_KV4);
    if ((flag != H2O_KV8 && flag != H2O_KV4) || (p.dtype != H2O_F32 && p.dtype != H2O_BF16))
        return set_last_error(H2O_ERR_ARG, "dtype must be H2O_F32 or H2O_BF16, with H2O_KV8 or H2O_KV4");
    p.bits = flag == H2O_KV8 ? 8 : 4;
    if (!K || !V || !ks || !vs) return set_last_error(H2O_ERR_ARG, "K, V, kscale and vscale must be non-NULL");
    if (!aligned16(K) || !aligned16(V) || !aligned16(ks) || !aligned16(vs))
        return set_last_error(H2O_ERR_ARG, "K, V, kscale and vscale must be 16-byte aligned");
    int rc = check_head_dim(D);
    if (rc) return rc;
    if (ps != 16 && ps != 32 && ps != 64 && ps != 128)
        return set_last_error(H2O_ERR_ARG, "page_size must be 16, 32, 64 or 128 (got %d)", ps);
    if (pages < 1 || heads < 1 || heads > 65535)
        return set_last_error(H2O_ERR_ARG, "num_pages must be >= 1 and kv_heads in [1, 65535]");
    if ((long long)pages * heads > INT_MAX / ps)
        return set_last_error(H2O_ERR_ARG, "num_pages * kv_heads * page_size must be below 2^31");
    return H2O_OK;
}

// key and value rows beside a quantised pool
int check_kv_rows(const QuantPool& p, const void* k, long long k_stride, const void* v, long long v_stride, const int* slot, int rows)
{
    if (rows < 0) return set_last_error(H2O_ERR_ARG, "rows must be >= 0 (got %d)", rows);
    if ((long long)rows * p.heads > 1 << 28) return set_last_error(H2O_ERR_ARG, "rows * kv_heads must be at most 2^28");
    if (rows && (!k || !v || !slot)) return set_last_error(H2O_ERR_ARG, "k, v and slot must be non-NULL");
    if (!aligned16(k) || !aligned16(v)) return set_last_error(H2O_ERR_ARG, "k and v must be 16-byte aligned");
    if (!aligned4(slot)) return set_last_error(H2O_ERR_ARG, "slot must be 4-byte aligned");
    const long long need = (long long)p.heads * p.D;
    const int rc = check_stride(k_stride, need, p.dtype, "k");
    return rc ? rc : check_stride(v_stride, need, p.dtype, "v");
}

}  // namespace

extern "C" {

int h2o_rope_table(int rot_dim, double base, int kind, double factor, double original_len, double low, double high, long long* table)
{
    if (rot_dim < 2 || rot_dim > 128 || rot_dim % 2) return set_last_error(H2O_ERR_ARG, "rot_dim must be even and in [2, 128] (got %d)", rot_dim);
    if (!(base >= 1.0) || !std::isfinite(base)) return set_last_error(H2O_ERR_ARG, "base must be finite and >= 1");
    if (kind < H2O_ROPE_PLAIN || kind > H2O_ROPE_PARTS) return set_last_error(H2O_ERR_ARG, "kind must be one of H2O_ROPE_PLAIN to H2O_ROPE_PARTS");
    if (!table) return set_last_error(H2O_ERR_ARG, "table must be non-NULL");
    if (kind != H2O_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return set_last_error(H2O_ERR_ARG, "factor must be finite and >= 1");
    if (kind == H2O_ROPE_BASE && rot_dim < 4) return set_last_error(H2O_ERR_ARG, "H2O_ROPE_BASE needs a rot_dim of at least 4");
    if (kind == H2O_ROPE_PARTS && (!(original_len >= 1.0) || !std::isfinite(original_len) || !(low >= 0.0) || !(high > low) || !std::isfinite(high)))
        return set_last_error(H2O_ERR_ARG, "H2O_ROPE_PARTS needs original_len >= 1 and 0 <= low < high");
    const double two_pi = 6.283185307179586476925;
    if (kind == H2O_ROPE_BASE) base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
    if (!std::isfinite(base)) return set_last_error(H2O_ERR_ARG, "base * factor is out of range");
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (kind == H2O_ROPE_LINEAR) f /= factor;
        if (kind == H2O_ROPE_PARTS) {
            const double t = (original_len * f / two_pi - low) / (high - low), g = t < 0.0 ? 0.0 : t > 1.0 ? 1.0 : t;
            f *= (1.0 - g) / factor + g;
        }
        table[i] = std::llrint(std::ldexp(f / two_pi, 64));   // (f <= 1: below 2^62)
    }
    return H2O_OK;
}

int h2o_rope(const void* q, long long q_stride, void* q_out, long long q_out_stride, int heads, const void* k, long long k_stride, void* k_out,
             long long k_out_stride, int kv_heads, const int* row_pos, int rows, const long long* table, int rot_dim, int form, double amplitude,
             int head_dim, int dtype, void* cuda_stream)
{
    int rc;
    if ((rc = check_row_type(dtype)) || (rc = check_head_dim(head_dim))) return rc;
    if (rows < 0) return set_last_error(H2O_ERR_ARG, "rows must be >= 0 (got %d)", rows);
    if (heads < 1 || kv_heads < 0) return set_last_error(H2O_ERR_ARG, "heads must be >= 1 and kv_heads >= 0");
    if ((long long)rows * ((long long)heads + kv_heads) > 1 << 28 || (long long)heads + kv_heads > 1 << 20)
        return set_last_error(H2O_ERR_ARG, "rows * (heads + kv_heads) must be at most 2^28, and heads + kv_heads 2^20");
    if (rot_dim < 2 || rot_dim > head_dim || rot_dim % 2)
        return set_last_error(H2O_ERR_ARG, "rot_dim must be even and in [2, head_dim] (got %d)", rot_dim);
    if (form != H2O_ROPE_HALF && form != H2O_ROPE_PAIRS) return set_last_error(H2O_ERR_ARG, "form must be H2O_ROPE_HALF or H2O_ROPE_PAIRS");
    if (!std::isfinite(amplitude) || !std::isfinite((float)amplitude)) return set_last_error(H2O_ERR_ARG, "amplitude must be finite in fp32");
    if (!table || (reinterpret_cast<uintptr_t>(table) & 7u)) return set_last_error(H2O_ERR_ARG, "table must be non-NULL and 8-byte aligned");
    if (rows && (!q || !q_out || !row_pos)) return set_last_error(H2O_ERR_ARG, "q, q_out and row_pos must be non-NULL");
    if (rows && kv_heads && (!k || !k_out)) return set_last_error(H2O_ERR_ARG, "k and k_out must be non-NULL when there are kv_heads");
    if (!aligned4(row_pos)) return set_last_error(H2O_ERR_ARG, "row_pos must be 4-byte aligned");
    if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(k_out))
        return set_last_error(H2O_ERR_ARG, "q, k and their outputs must be 16-byte aligned");
    const Rows in[2] = {{q, q_stride, (long long)heads * head_dim}, {k, k_stride, (long long)kv_heads * head_dim}};
    const Rows out[2] = {{q_out, q_out_stride, in[0].need}, {k_out, k_out_stride, in[1].need}};
    const char* names[2][2] = {{"q", "q_out"}, {"k", "k_out"}};
    for (int i = 0; i < (kv_heads ? 2 : 1); ++i) {
        if ((rc = check_stride(in[i].stride, in[i].need, dtype, names[i][0])) || (rc = check_stride(out[i].stride, out[i].need, dtype, names[i][1])))
            return rc;
    }
    const int size = dtype == H2O_BF16 ? 2 : 4;
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            if (!(i == j && same(out[i], in[j], rows)) && collide(out[i], rows, in[j], rows, size))
                return set_last_error(H2O_ERR_ARG, "%s overlaps other rows of %s", names[i][1], names[j][0]);
    if (collide(out[0], rows, out[1], rows, size)) return set_last_error(H2O_ERR_ARG, "q_out overlaps k_out");
    if (!rows) return H2O_OK;
    if (inject_launch()) return set_last_error(H2O_ERR_CUDA, "kernel launch failed (injected)");
    RopeArgs a = {};
    for (int i = 0; i < 2; ++i) {
        a.in[i] = in[i].p; a.out[i] = const_cast<void*>(out[i].p);
        a.in_stride[i] = in[i].stride; a.out_stride[i] = out[i].stride;
    }
    a.heads[0] = heads; a.heads[1] = kv_heads;
    a.pos = row_pos; a.table = table; a.rows = rows; a.rot = rot_dim; a.amplitude = (float)amplitude;
    return launched(launch_rope(a, form, head_dim, dtype, reinterpret_cast<cudaStream_t>(cuda_stream)), "h2o_rope");
}

int h2o_prompt_attend(const void* q, long long q_stride, int rows, const void* k, long long k_stride, const void* v, long long v_stride, int k_rows,
                      int kv_heads, int groups, int head_dim, int dtype, const int* q_start, const int* k_start, int requests, double scale, void* out,
                      long long out_stride, void* cuda_stream)
{
    int rc;
    if ((rc = check_row_type(dtype)) || (rc = check_head_dim(head_dim))) return rc;
    if (rows < 0 || rows > kMaxPromptRows || k_rows < 0 || k_rows > kMaxPromptRows)
        return set_last_error(H2O_ERR_ARG, "rows and k_rows must be in [0, 2^24] (got %d and %d)", rows, k_rows);
    if (kv_heads < 1 || kv_heads > 65535) return set_last_error(H2O_ERR_ARG, "kv_heads must be in [1, 65535] (got %d)", kv_heads);
    if (groups < 1 || groups > kMaxPageGroups) return set_last_error(H2O_ERR_ARG, "groups must be in [1, %d] (got %d)", kMaxPageGroups, groups);
    if (requests < 1 || requests > kMaxPromptRequests)
        return set_last_error(H2O_ERR_ARG, "requests must be in [1, %d] (got %d)", kMaxPromptRequests, requests);
    if ((long long)rows * kv_heads > (1 << 28) / groups || (long long)k_rows * kv_heads > 1 << 28)
        return set_last_error(H2O_ERR_ARG, "rows * kv_heads * groups and k_rows * kv_heads must be at most 2^28");
    if ((long long)requests * kv_heads > 1 << 22) return set_last_error(H2O_ERR_ARG, "requests * kv_heads must be at most 2^22");
    PackedArgs a = {};
    a.qscale = (float)(scale * 1.4426950408889634);
    if (!(scale > 0.0) || !std::isfinite(scale)) return set_last_error(H2O_ERR_ARG, "scale must be finite and > 0");
    if (!(a.qscale > 0.f) || !std::isfinite(a.qscale)) return set_last_error(H2O_ERR_ARG, "scale is out of fp32's range");
    if (!q_start || !aligned4(q_start) || !aligned4(k_start)) return set_last_error(H2O_ERR_ARG, "q_start must be non-NULL, it and k_start 4-byte aligned");
    if ((rows && (!q || !out)) || (k_rows && (!k || !v))) return set_last_error(H2O_ERR_ARG, "q, k, v and out must be non-NULL");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return set_last_error(H2O_ERR_ARG, "q, k, v and out must be 16-byte aligned");
    const long long kn = (long long)kv_heads * head_dim, qn = kn * groups;
    if ((rc = check_stride(q_stride, qn, dtype, "q")) || (rc = check_stride(k_stride, kn, dtype, "k")) || (rc = check_stride(v_stride, kn, dtype, "v")) ||
        (rc = check_stride(out_stride, qn, dtype, "out")))
        return rc;
    const int size = dtype == H2O_BF16 ? 2 : 4;
    const Rows o = {out, out_stride, qn};
    if (collide(o, rows, {q, q_stride, qn}, rows, size) || collide(o, rows, {k, k_stride, kn}, k_rows, size) || collide(o, rows, {v, v_stride, kn}, k_rows, size))
        return set_last_error(H2O_ERR_ARG, "out overlaps q, k or v");
    if (!rows) return H2O_OK;
    if (inject_launch()) return set_last_error(H2O_ERR_CUDA, "kernel launch failed (injected)");
    a.q = q; a.k = k; a.v = v; a.out = out;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride; a.out_stride = out_stride;
    a.q_start = q_start; a.k_start = k_start ? k_start : q_start;
    a.rows = rows; a.k_rows = k_rows; a.heads = kv_heads; a.G = groups; a.requests = requests;
    return launched(launch_prompt_attend(a, head_dim, dtype, reinterpret_cast<cudaStream_t>(cuda_stream)), "h2o_prompt_attend");
}

int h2o_page_quant_write(const void* k, const void* v, long long k_stride, long long v_stride, const int* slot, int rows, void* K, void* V, float* kscale,
                         float* vscale, int num_pages, int kv_heads, int page_size, int head_dim, int dtype, void* cuda_stream)
{
    QuantPool p = {};
    int rc;
    if ((rc = make_pool(p, K, V, kscale, vscale, num_pages, kv_heads, page_size, head_dim, dtype)) ||
        (rc = check_kv_rows(p, k, k_stride, v, v_stride, slot, rows)))
        return rc;
    if (!rows) return H2O_OK;
    if (inject_launch()) return set_last_error(H2O_ERR_CUDA, "kernel launch failed (injected)");
    return launched(launch_page_quant_write(p, k, v, k_stride, v_stride, slot, rows, reinterpret_cast<cudaStream_t>(cuda_stream)), "h2o_page_quant_write");
}

int h2o_page_quant_read(const void* K, const void* V, const float* kscale, const float* vscale, int num_pages, int kv_heads, int page_size, int head_dim,
                        int dtype, const int* slot, int rows, void* k, long long k_stride, void* v, long long v_stride, void* cuda_stream)
{
    QuantPool p = {};
    int rc;
    if ((rc = make_pool(p, K, V, kscale, vscale, num_pages, kv_heads, page_size, head_dim, dtype)) ||
        (rc = check_kv_rows(p, k, k_stride, v, v_stride, slot, rows)))
        return rc;
    const long long need = (long long)kv_heads * head_dim;
    if (collide({k, k_stride, need}, rows, {v, v_stride, need}, rows, p.dtype == H2O_BF16 ? 2 : 4)) return set_last_error(H2O_ERR_ARG, "k overlaps v");
    if (!rows) return H2O_OK;
    if (inject_launch()) return set_last_error(H2O_ERR_CUDA, "kernel launch failed (injected)");
    return launched(launch_page_quant_read(p, slot, rows, k, k_stride, v, v_stride, reinterpret_cast<cudaStream_t>(cuda_stream)), "h2o_page_quant_read");
}

int h2o_page_quant_attend(const void* q, long long q_stride, const int* row_seq, const int* row_pos, int rows, const void* K, const void* V,
                          const float* kscale, const float* vscale, int num_pages, int kv_heads, int groups, int page_size, int head_dim, int dtype,
                          const int* table, int requests, int table_width, double scale, void* out, long long out_stride, void* cuda_stream)
{
    QuantPool p = {};
    PageRows r = {};
    r.q = q; r.out = out; r.q_stride = q_stride; r.out_stride = out_stride; r.seq = row_seq; r.pos = row_pos;
    r.table = table; r.rows = rows; r.G = groups; r.requests = requests; r.width = table_width;
    r.qscale = (float)(scale * 1.4426950408889634);
    int rc;
    if ((rc = make_pool(p, K, V, kscale, vscale, num_pages, kv_heads, page_size, head_dim, dtype))) return rc;
    PagePool shape = {};
    shape.heads = kv_heads; shape.D = head_dim; shape.dtype = p.dtype;
    if ((rc = check_rows(shape, r, scale))) return rc;
    if (!rows) return H2O_OK;
    if (inject_launch()) return set_last_error(H2O_ERR_CUDA, "kernel launch failed (injected)");
    return launched(launch_page_quant_attend(p, r, reinterpret_cast<cudaStream_t>(cuda_stream)), "h2o_page_quant_attend");
}

}  // extern "C"
