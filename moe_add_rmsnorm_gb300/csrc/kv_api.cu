// The C ABI of the paged, quantized key/value cache: argument checks (refusal by name, before any launch) and the calls.
#include <cuda_runtime.h>

#include "kernels.h"
#include "q8moe.h"

namespace q8 {
extern int model_fail(int code, const char* fmt, ...);
}

using namespace q8;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int64_t kMost = int64_t(1) << 30;  // rows, pages and positions: their sums stay within 32 bits

// Checks pages and batch and fills the kernels' view of them.
int check_view(const q8_kv_pages* pages, const q8_kv_batch* batch, int64_t rows, KvView* view) {
    model_fail(Q8_OK, "%s", "");
    if (!pages || !batch) return model_fail(Q8_EINVAL, "%s: null", pages ? "batch" : "pages");
    if (!pages->k || !pages->v || !pages->ks || !pages->vs) return model_fail(Q8_EINVAL, "pages: null words or scales");
    if (pages->words != Q8_KV_INT8 && pages->words != Q8_KV_E4M3)
        return model_fail(Q8_EINVAL, "pages: words %d", (int)pages->words);
    if (pages->pages < 1 || pages->kv_heads < 1)
        return model_fail(Q8_EINVAL, "pages: %lld pages of %lld heads", (long long)pages->pages, (long long)pages->kv_heads);
    if (pages->pages > kMost || pages->kv_heads > 1024)
        return model_fail(Q8_EUNSUPPORTED, "pages: %lld pages of %lld heads: at most 2^30 and 1024", (long long)pages->pages,
                          (long long)pages->kv_heads);
    if (pages->head_dim != 64 && pages->head_dim != 128)
        return model_fail(Q8_EUNSUPPORTED, "pages: head_dim %lld: 64 or 128", (long long)pages->head_dim);
    const int64_t ps = pages->page_size;
    if (ps < 16 || ps > 1024 || (ps & (ps - 1)))
        return model_fail(Q8_EUNSUPPORTED, "pages: page_size %lld: a power of two from 16 to 1024", (long long)ps);
    if (!aligned(pages->k, 32) || !aligned(pages->v, 32)) return model_fail(Q8_EINVAL, "pages: words not 32-byte aligned");
    if (!aligned(pages->ks, 16) || !aligned(pages->vs, 16)) return model_fail(Q8_EINVAL, "pages: scales not 16-byte aligned");
    // (a batch without sequences has no arrays: an empty tensor's address is null)
    if (batch->seqs != 0 && (!batch->row_start || !batch->kv_len || !batch->table))
        return model_fail(Q8_EINVAL, "batch: null row_start, kv_len or table");
    if (!aligned(batch->row_start, 4) || !aligned(batch->kv_len, 4) || !aligned(batch->table, 4) || !aligned(batch->error, 4))
        return model_fail(Q8_EINVAL, "batch: an array not 4-byte aligned");
    if (batch->seqs < 0 || rows < 0) return model_fail(Q8_EINVAL, "batch: seqs or rows negative");
    if (batch->seqs > 65536) return model_fail(Q8_EUNSUPPORTED, "batch: %lld sequences: at most 65536", (long long)batch->seqs);
    if (rows > (1 << 24)) return model_fail(Q8_EUNSUPPORTED, "rows %lld: at most 2^24", (long long)rows);
    if (batch->seqs != 0 && (batch->table_pages < 1 || batch->table_stride < batch->table_pages))
        return model_fail(Q8_EINVAL, "batch: %lld pages a table row, rows %lld apart", (long long)batch->table_pages,
                          (long long)batch->table_stride);
    if (batch->table_pages > kMost / ps || batch->table_stride > kMost)
        return model_fail(Q8_EUNSUPPORTED, "batch: a table row of more than 2^30 positions");
    int log2 = 4;
    while ((int64_t(1) << log2) < ps) ++log2;
    view->k = (int8_t*)pages->k;
    view->v = (int8_t*)pages->v;
    view->ks = pages->ks;
    view->vs = pages->vs;
    view->pages = (int)pages->pages;
    view->kv = (int)pages->kv_heads;
    view->page_log2 = log2;
    view->row_start = batch->row_start;
    view->kv_len = batch->kv_len;
    view->table = batch->table;
    view->table_stride = batch->table_stride;
    view->seqs = (int)batch->seqs;
    view->cap = (int)(batch->table_pages * ps);
    view->rows = (int)rows;
    view->error = batch->error;
    return Q8_OK;
}

// f32 rows of `width` values, `stride` apart (none: any address, that of an empty tensor among them).
int check_rows(const float* x, int64_t stride, int64_t width, int64_t rows, const char* name) {
    if (!x && rows != 0) return model_fail(Q8_EINVAL, "%s: null", name);
    if (!aligned(x, 16) || stride % 4) return model_fail(Q8_EINVAL, "%s: address or stride not 16-byte aligned", name);
    if (rows > 1 && stride < width)
        return model_fail(Q8_EINVAL, "%s: rows %lld apart, %lld values wide", name, (long long)stride, (long long)width);
    if (stride < 0 || stride > kMost) return model_fail(Q8_EINVAL, "%s: stride %lld", name, (long long)stride);
    return Q8_OK;
}

// Rows of one buffer written while those of another are read: q8_paged_attention's out and q, q8_kv_append's q_out and what
// it reads.  Columns of one buffer, the same
// distance apart, are rows that lie between one another's.
int check_apart(const float* x, int64_t x_stride, int64_t x_width, const char* x_name, const float* y, int64_t y_stride,
                int64_t y_width, const char* y_name, int64_t rows) {
    if (rows == 0) return Q8_OK;
    const int64_t xs = (rows - 1) * x_stride + x_width, ys = (rows - 1) * y_stride + y_width;
    const uintptr_t xa = (uintptr_t)x, ya = (uintptr_t)y;
    if (xa + 4 * (uint64_t)xs <= ya || ya + 4 * (uint64_t)ys <= xa) return Q8_OK;
    if (rows > 1 && x_stride == y_stride) {  // (both addresses are multiples of 16)
        const int64_t d = ((int64_t)(ya - xa) / 4 % x_stride + x_stride) % x_stride;
        if (d >= x_width && d + y_width <= x_stride) return Q8_OK;
    }
    return model_fail(Q8_EINVAL, "%s: overlaps %s", x_name, y_name);
}

// Whether two vectors of hd values lie over one another among rows x heads of them at r*rs + h*hs and the same ones `at` values
// on (at 0: any two different ones).  Exact: for each distance between heads only the two nearest between rows can do it.
bool vectors_meet(int64_t at, int64_t rows, int64_t rs, int64_t heads, int64_t hs, int64_t hd) {
    for (int64_t dh = 1 - heads; dh < heads; ++dh) {
        const int64_t d = at + dh * hs;  // to be undone by -dr * rs, to within hd - 1
        const int64_t near = rows > 1 ? d / rs : 0;
        for (int64_t dr = near - 1; dr <= near + 1; ++dr) {
            if (dr <= -rows || dr >= rows || (at == 0 && dh == 0 && dr == 0)) continue;
            const int64_t left = d - dr * rs;
            if (left > -hd && left < hd) return true;
        }
    }
    return false;
}

int done(cudaError_t e, const char* what) {
    return e == cudaSuccess ? Q8_OK : model_fail(Q8_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace

extern "C" {

int q8_rope_table(double theta, int64_t positions, int64_t head_dim, float* cos, float* sin, q8_stream stream) {
    model_fail(Q8_OK, "%s", "");
    if (!cos || !sin) return model_fail(Q8_EINVAL, "cos or sin: null");
    if (!aligned(cos, 4) || !aligned(sin, 4)) return model_fail(Q8_EINVAL, "cos or sin: not 4-byte aligned");
    if (!(theta > 0.0)) return model_fail(Q8_EINVAL, "theta: not positive");
    if (positions < 0 || head_dim < 2 || head_dim % 2)
        return model_fail(Q8_EINVAL, "positions %lld, head_dim %lld", (long long)positions, (long long)head_dim);
    if (positions > kMost || head_dim > 4096)
        return model_fail(Q8_EUNSUPPORTED, "positions %lld, head_dim %lld: at most 2^30 and 4096", (long long)positions,
                          (long long)head_dim);
    if (positions == 0) return Q8_OK;
    return done(launch_rope_table(cos, sin, (int)positions, (int)(head_dim / 2), theta, (cudaStream_t)stream),
                "q8_rope_table");
}

int q8_kv_append(const q8_kv_pages* pages, const q8_kv_batch* batch, int64_t rows, int64_t heads, const float* q,
                 int64_t q_stride, const float* k, int64_t k_stride, const float* v, int64_t v_stride,
                 const float* q_norm, const float* k_norm, float eps, const float* cos, const float* sin,
                 int64_t rope_positions, float* q_out, int64_t q_out_stride, q8_stream stream) {
    KvAppendCall c;
    if (int r = check_view(pages, batch, rows, &c.view)) return r;
    const int64_t hd = pages->head_dim, kv = pages->kv_heads;
    if (heads < 0 || heads > 1024 * 64) return model_fail(Q8_EINVAL, "heads %lld", (long long)heads);
    if (heads) {
        if (int r = check_rows(q, q_stride, heads * hd, rows, "q")) return r;
        if (int r = check_rows(q_out, q_out_stride, heads * hd, rows, "q_out")) return r;
    } else if (q) {
        return model_fail(Q8_EINVAL, "q: given without heads");
    }
    if (int r = check_rows(k, k_stride, kv * hd, rows, "k")) return r;
    if (int r = check_rows(v, v_stride, kv * hd, rows, "v")) return r;
    if (!(eps >= 0.f)) return model_fail(Q8_EINVAL, "eps: negative or NaN");
    if (!aligned(q_norm, 4) || !aligned(k_norm, 4)) return model_fail(Q8_EINVAL, "q_norm or k_norm: not 4-byte aligned");
    if ((cos == nullptr) != (sin == nullptr)) return model_fail(Q8_EINVAL, "cos and sin: one without the other");
    if (!aligned(cos, 16) || !aligned(sin, 16)) return model_fail(Q8_EINVAL, "cos or sin: not 16-byte aligned");
    if (cos && rope_positions < 1) return model_fail(Q8_EINVAL, "rope_positions %lld", (long long)rope_positions);
    if (rows == 0 || batch->seqs == 0) return Q8_OK;
    if (heads) {
        const int64_t qw = heads * hd, kw = kv * hd;
        if (q_out != q || (rows > 1 && q_out_stride != q_stride))
            if (int r = check_apart(q_out, q_out_stride, qw, "q_out", q, q_stride, qw, "q", rows)) return r;
        if (int r = check_apart(q_out, q_out_stride, qw, "q_out", k, k_stride, kw, "k", rows)) return r;
        if (int r = check_apart(q_out, q_out_stride, qw, "q_out", v, v_stride, kw, "v", rows)) return r;
    }
    c.hd = (int)hd;
    c.heads = (int)heads;
    c.words = (int)pages->words;
    c.q = q, c.k = k, c.v = v;
    c.q_stride = q_stride, c.k_stride = k_stride, c.v_stride = v_stride, c.q_out_stride = q_out_stride;
    c.q_norm = q_norm, c.k_norm = k_norm;
    c.eps = eps;
    c.cos_t = cos, c.sin_t = sin;
    c.rope_positions = rope_positions;
    c.q_out = q_out;
    return done(launch_kv_append(c, (cudaStream_t)stream), "q8_kv_append");
}

int q8_kv_read(const q8_kv_pages* pages, const q8_kv_batch* batch, int64_t rows, float* k_out, float* v_out,
               int64_t row_stride, int64_t head_stride, q8_stream stream) {
    KvReadCall c;
    if (int r = check_view(pages, batch, rows, &c.view)) return r;
    if (!k_out && !v_out && rows != 0) return model_fail(Q8_EINVAL, "k_out and v_out: both null");
    if (!aligned(k_out, 32) || !aligned(v_out, 32) || row_stride % 8 || head_stride % 8)
        return model_fail(Q8_EINVAL, "k_out, v_out: an address or stride not 32-byte aligned");
    const int64_t hd = pages->head_dim;
    if ((rows > 1 && row_stride < hd) || (pages->kv_heads > 1 && head_stride < hd) || row_stride < 0 || head_stride < 0)
        return model_fail(Q8_EINVAL, "k_out, v_out: rows %lld and heads %lld apart, %lld values each", (long long)row_stride,
                          (long long)head_stride, (long long)hd);
    if (row_stride > (int64_t(1) << 36) || head_stride > (int64_t(1) << 36))
        return model_fail(Q8_EUNSUPPORTED, "k_out, v_out: strides of more than 2^36");
    if (rows > 0) {
        // Rows within heads or heads within rows, as dense layouts are, is the quick answer.
        const int64_t kv = pages->kv_heads, span = (rows - 1) * row_stride + (kv - 1) * head_stride + hd;
        const bool nested = (rows == 1 || row_stride >= (kv - 1) * head_stride + hd) || (kv == 1 || head_stride >= (rows - 1) * row_stride + hd);
        if (!nested && vectors_meet(0, rows, row_stride, kv, head_stride, hd))
            return model_fail(Q8_EINVAL, "k_out, v_out: rows %lld and heads %lld apart overlap", (long long)row_stride,
                              (long long)head_stride);
        if (k_out && v_out && batch->seqs > 0) {
            const uintptr_t a = (uintptr_t)k_out, b = (uintptr_t)v_out;
            if (a < b + 4 * (uint64_t)span && b < a + 4 * (uint64_t)span &&
                (a == b || vectors_meet((int64_t)(b - a) / 4, rows, row_stride, kv, head_stride, hd)))
                return model_fail(Q8_EINVAL, "v_out: overlaps k_out");
        }
    }
    if (rows == 0 || batch->seqs == 0) return Q8_OK;
    c.hd = (int)hd;
    c.words = (int)pages->words;
    c.k_out = k_out, c.v_out = v_out;
    c.row_stride = row_stride, c.head_stride = head_stride;
    return done(launch_kv_read(c, (cudaStream_t)stream), "q8_kv_read");
}

static int attention(PagedAttnCall& c, const q8_kv_pages* pages, const q8_kv_batch* batch, int64_t rows, int64_t heads,
                     const float* q, int64_t q_stride, float scale, float* out, int64_t out_stride, float* lse, q8_ws* ws,
                     q8_stream stream) {
    if (int r = check_view(pages, batch, rows, &c.view)) return r;
    const int64_t kv = pages->kv_heads;
    if (heads < 1 || heads % kv) return model_fail(Q8_EINVAL, "heads %lld: not a multiple of the %lld key/value heads",
                                                   (long long)heads, (long long)kv);
    if (heads / kv > 64) return model_fail(Q8_EUNSUPPORTED, "heads %lld: more than 64 a key/value head", (long long)heads);
    if (int r = check_rows(q, q_stride, heads * pages->head_dim, rows, "q")) return r;
    if (int r = check_rows(out, out_stride, heads * pages->head_dim, rows, "out")) return r;
    if (q == out && rows != 0) return model_fail(Q8_EINVAL, "out: q itself");
    const int64_t width = heads * pages->head_dim;
    if (int r = check_apart(out, out_stride, width, "out", q, q_stride, width, "q", rows)) return r;
    if (!aligned(lse, 4)) return model_fail(Q8_EINVAL, "lse: not 4-byte aligned");
    if (!(scale > 0.f) || scale > 1e30f) return model_fail(Q8_EINVAL, "scale: not positive and finite");
    if (!ws) return model_fail(Q8_EINVAL, "ws: null");
    if (rows == 0 || batch->seqs == 0) return Q8_OK;
    c.hd = (int)pages->head_dim;
    c.heads = (int)heads;
    c.words = (int)pages->words;
    c.q = q;
    c.q_stride = q_stride, c.out_stride = out_stride;
    c.scale = scale;
    c.out = out;
    c.lse = lse;
    Carve cv = workspace_carve(ws);
    cudaError_t e = launch_paged_attention(c, cv, (cudaStream_t)stream);
    if (cv.overflow) return model_fail(Q8_ENOSPACE, "q8_paged_attention: workspace too small for the partial results");
    return done(e, "q8_paged_attention");
}

int q8_paged_attention(const q8_kv_pages* pages, const q8_kv_batch* batch, int64_t rows, int64_t heads, const float* q,
                       int64_t q_stride, float scale, float* out, int64_t out_stride, float* lse, q8_ws* ws,
                       q8_stream stream) {
    PagedAttnCall c;
    return attention(c, pages, batch, rows, heads, q, q_stride, scale, out, out_stride, lse, ws, stream);
}

int q8_paged_wait_selftest(const q8_kv_pages* pages, const q8_kv_batch* batch, int64_t rows, int64_t heads, const float* q,
                           int64_t q_stride, float scale, float* out, int64_t out_stride, q8_ws* ws, unsigned polls,
                           q8_stream stream) {
    model_fail(Q8_OK, "%s", "");
    if (polls < 1 || polls > (1u << 12)) return model_fail(Q8_EINVAL, "polls %u: 1 to 2^12", polls);
    PagedAttnCall c;
    c.polls = polls;
    c.missing = 16;
    return attention(c, pages, batch, rows, heads, q, q_stride, scale, out, out_stride, nullptr, ws, stream);
}

}  // extern "C"
