// The C ABI of the feed-forward block with 4-bit weights: argument checks (refusal by name, before any launch) and the calls.
#include <cuda_runtime.h>
#include <math.h>

#include "ffn4.h"
#include "q8moe.h"

namespace q8 {
extern int model_fail(int code, const char* fmt, ...);
}

using namespace q8;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// A call's byte ranges, to refuse outputs that lie over inputs or over one another.
struct Range {
    uintptr_t at = 0;
    int64_t bytes = 0;
    Range() {}
    Range(const void* p, int64_t n) : at((uintptr_t)p), bytes(p ? n : 0) {}
    bool meets(const Range& o) const {
        return bytes > 0 && o.bytes > 0 && at < o.at + (uintptr_t)o.bytes && o.at < at + (uintptr_t)bytes;
    }
};

int check_q4(const q4_mat* W, const char* name) {
    if (!W) return model_fail(Q8_EINVAL, "%s: null matrix", name);
    if (!W->q || !W->s) return model_fail(Q8_EINVAL, "%s: null words or scales", name);
    if (W->rows < 1 || W->cols < 1)
        return model_fail(Q8_EINVAL, "%s: %lld x %lld", name, (long long)W->rows, (long long)W->cols);
    if (W->group != 32 && W->group != 64 && W->group != 128)
        return model_fail(Q8_EUNSUPPORTED, "%s: group %lld: 32, 64 or 128", name, (long long)W->group);
    if (W->cols % W->group)
        return model_fail(Q8_EUNSUPPORTED, "%s: %lld columns, not whole groups of %lld", name, (long long)W->cols,
                          (long long)W->group);
    if (W->cols > 32768 || W->rows > (int64_t(1) << 30))
        return model_fail(Q8_EUNSUPPORTED, "%s: %lld x %lld: at most 2^30 rows of 32768", name, (long long)W->rows,
                          (long long)W->cols);
    if (W->scale_type != Q4_SCALE_F16 && W->scale_type != Q4_SCALE_BF16)
        return model_fail(Q8_EINVAL, "%s: scale type %d", name, (int)W->scale_type);
    if (!aligned(W->q, 16)) return model_fail(Q8_EINVAL, "%s: words not 16-byte aligned", name);
    if (!aligned(W->s, 2)) return model_fail(Q8_EINVAL, "%s: scales not 2-byte aligned", name);
    return Q8_OK;
}

Q4View view_of(const q4_mat* W) {
    Q4View v;
    v.q = W->q;
    v.s = (const uint16_t*)W->s;
    v.z = W->z;
    v.rows = W->rows;
    v.cols = (int)W->cols;
    v.group_log2 = W->group == 32 ? 5 : W->group == 64 ? 6 : 7;
    v.bf16 = W->scale_type == Q4_SCALE_BF16;
    return v;
}

// The activation of a product: f32 rows or quantized ones, `cols` values each.
int check_q4_act(const float* x, int64_t stride, const q8_act* xq, int64_t rows, int64_t cols, const char* name, Q4Act* out) {
    if (rows * cols > (int64_t(1) << 33))
        return model_fail(Q8_EUNSUPPORTED, "%s: %lld rows of %lld values: at most 2^33", name, (long long)rows, (long long)cols);
    if (!x && !xq) return model_fail(Q8_EINVAL, "%s: null, as is its quantized form", name);
    if (x && xq) return model_fail(Q8_EINVAL, "%s: given as values and as words", name);
    if (x) {
        if (!aligned(x, 16) || stride % 4) return model_fail(Q8_EINVAL, "%s: address or stride not of 16 bytes", name);
        if (stride < cols && rows > 1)
            return model_fail(Q8_EINVAL, "%s: rows %lld apart, of %lld values", name, (long long)stride, (long long)cols);
        out->x = x;
        out->stride = stride;
        return Q8_OK;
    }
    if (!xq->q || !xq->s) return model_fail(Q8_EINVAL, "%s: null words or scales", name);
    if (!aligned(xq->q, 32) || (xq->lo && !aligned(xq->lo, 32)))
        return model_fail(Q8_EINVAL, "%s: words not 32-byte aligned", name);
    if (!aligned(xq->s, 4)) return model_fail(Q8_EINVAL, "%s: scales not 4-byte aligned", name);
    out->q = xq->q;
    out->lo = xq->lo;
    out->s = xq->s;
    out->stride = cols;
    return Q8_OK;
}

// Whether two sets of `rows` rows, equally far apart, are columns beside one another.
bool beside(const float* a, int64_t a_cols, const float* b, int64_t b_cols, int64_t stride, int64_t rows) {
    if (rows < 2 || stride < 1 || ((uintptr_t)a - (uintptr_t)b) % 4) return false;
    int64_t at = (int64_t)((intptr_t)b - (intptr_t)a) / 4 % stride;  // where b's columns start in a's rows
    if (at < 0) at += stride;
    return at >= a_cols && at + b_cols <= stride;
}

// Whether `out` meets the activation (its `rows` rows of cols values) or the matrix.
bool meets_act(const Range& out, const Q4Act& a, int64_t rows, int64_t cols) {
    if (a.x) return out.meets(Range(a.x, 4 * ((rows - 1) * a.stride + cols)));
    return out.meets(Range(a.q, rows * cols)) || out.meets(Range(a.lo, rows * cols)) || out.meets(Range(a.s, rows * cols / 8));
}
bool meets_mat(const Range& out, const q4_mat* W) {
    const int64_t groups = W->rows * (W->cols / W->group);
    return out.meets(Range(W->q, W->rows * W->cols / 2)) || out.meets(Range(W->s, 2 * groups)) || out.meets(Range(W->z, groups));
}

int check_plan4(const q8_moe_plan* plan) {
    if (!plan->counts || !plan->offsets || !plan->lists || !plan->active) return model_fail(Q8_EINVAL, "plan: null array");
    if (!aligned(plan->counts, 4) || !aligned(plan->offsets, 4) || !aligned(plan->lists, 4) || !aligned(plan->active, 4))
        return model_fail(Q8_EINVAL, "plan: not 4-byte aligned");
    return Q8_OK;
}

// Whether `out` meets the arrays of a plan that several rows are multiplied by.
bool meets_plan(const Range& out, const q8_moe_plan* plan, int64_t experts, int64_t rows, int k) {
    return rows > 1 && (out.meets(Range(plan->offsets, 4 * (experts + 1))) || out.meets(Range(plan->active, 4 * (experts + 1))) ||
                        out.meets(Range(plan->lists, 4 * rows * k)));
}

PlanPtrs plan_ptrs(const q8_moe_plan* plan) {
    PlanPtrs p;
    p.counts = plan->counts;
    p.offsets = plan->offsets;
    p.lists = plan->lists;
    p.active = plan->active;
    return p;
}

// What moe_gate_up_q4 and moe_down_combine_q4 check alike.
int check_experts(int64_t rows, int k, const int32_t* ids, const q8_moe_plan* plan, q8_ws* ws) {
    if (rows < 0) return model_fail(Q8_EINVAL, "rows negative");
    if (k < 1 || k > 32) return model_fail(Q8_EUNSUPPORTED, "k %d: 1 to 32 experts a row", k);
    if (rows * k > (int64_t(1) << 24) || rows > (int64_t(1) << 24))
        return model_fail(Q8_EUNSUPPORTED, "rows*k %lld: at most 2^24 choices", (long long)(rows * k));
    if (rows == 0) return Q8_OK;
    if (!ids || !ws) return model_fail(Q8_EINVAL, "ids or ws: null");
    if (!aligned(ids, 4)) return model_fail(Q8_EINVAL, "ids: not 4-byte aligned");
    if (rows > 1 && !plan) return model_fail(Q8_EINVAL, "plan: null (%lld rows are grouped by expert)", (long long)rows);
    if (plan) return check_plan4(plan);
    return Q8_OK;
}

int finish(cudaError_t e, const Carve& cv, const char* who) {
    if (cv.overflow) return model_fail(Q8_ENOSPACE, "%s: workspace too small", who);
    return e == cudaSuccess ? Q8_OK : model_fail(Q8_ECUDA, "%s: %s", who, cudaGetErrorString(e));
}

}  // namespace

extern "C" {

int postnorm_add_rmsnorm_q8(const float* a, const float* b, const float* w_post, const float* w_pre, const float* gate,
                            int64_t gate_row_stride, int64_t gate_stride, float scale, int64_t rows, int64_t d, float eps,
                            float* sum_out, float* y_out, const q8_act* yq, q8_stream stream) {
    model_fail(Q8_OK, "%s", "");
    if (rows < 0 || d < 1) return model_fail(Q8_EINVAL, "rows %lld, d %lld", (long long)rows, (long long)d);
    if (d > 16384) return model_fail(Q8_EUNSUPPORTED, "d %lld: a row kernel holds at most 16384 values", (long long)d);
    if (rows > 0x7fffffff) return model_fail(Q8_EUNSUPPORTED, "rows: too many");
    if (!(eps >= 0.f)) return model_fail(Q8_EINVAL, "eps: negative or NaN");
    if (gate_row_stride < 0 || gate_stride < 0) return model_fail(Q8_EINVAL, "gate: negative stride");
    if (yq && d % 32)
        return model_fail(Q8_EUNSUPPORTED, "d %lld: the int8 epilogue needs whole 32-value blocks", (long long)d);
    if (!sum_out && !y_out && !yq) return model_fail(Q8_EINVAL, "no output requested");
    if (rows == 0) return Q8_OK;
    if (!a || !b) return model_fail(Q8_EINVAL, "%s: null", a ? "b" : "a");
    if (!w_pre && (y_out || yq)) return model_fail(Q8_EINVAL, "w_pre: null");
    const void* words[] = {a, b, w_post, w_pre, gate, sum_out, y_out};
    const char* names[] = {"a", "b", "w_post", "w_pre", "gate", "sum_out", "y_out"};
    for (int i = 0; i < 7; ++i)
        if (!aligned(words[i], 4)) return model_fail(Q8_EINVAL, "%s: not 4-byte aligned", names[i]);
    if (yq) {
        if (!yq->q || !yq->s) return model_fail(Q8_EINVAL, "yq: null words or scales");
        if (!aligned(yq->q, 32) || (yq->lo && !aligned(yq->lo, 32)))
            return model_fail(Q8_EINVAL, "yq: words not 32-byte aligned");
        if (!aligned(yq->s, 4)) return model_fail(Q8_EINVAL, "yq: scales not 4-byte aligned");
    }
    const int64_t n = rows * d;
    const Range in[] = {{a, 4 * n}, {b, 4 * n}, {w_post, 4 * d}, {w_pre, 4 * d},
                        {gate, 4 * ((rows - 1) * gate_row_stride + (d - 1) * gate_stride + 1)}};
    const Range out[] = {{sum_out, 4 * n}, {y_out, 4 * n}, {yq ? yq->q : nullptr, n}, {yq ? yq->lo : nullptr, n},
                         {yq ? yq->s : nullptr, n / 8}};
    const char* outs[] = {"sum_out", "y_out", "yq", "yq's low words", "yq's scales"};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < 5; ++j)
            if (out[i].meets(in[j]) && !(i < 2 && j < 2 && out[i].at == in[j].at))
                return model_fail(Q8_EINVAL, "%s: overlaps %s", outs[i], names[j]);
        for (int j = 0; j < i; ++j)
            if (out[i].meets(out[j])) return model_fail(Q8_EINVAL, "%s: overlaps %s", outs[i], outs[j]);
    }
    PostnormCall c;
    c.a = a;
    c.b = b;
    c.w_post = w_post;
    c.w_pre = w_pre;
    c.gate = gate;
    c.gate_row = gate_row_stride;
    c.gate_col = gate_stride;
    c.scale = scale;
    c.eps = eps;
    c.rows = rows;
    c.d = d;
    c.sum = sum_out;
    c.y = y_out;
    c.yq = yq ? yq->q : nullptr;
    c.yl = yq ? yq->lo : nullptr;
    c.ys = yq ? yq->s : nullptr;
    return finish(launch_postnorm(c, (cudaStream_t)stream), Carve(), "postnorm_add_rmsnorm_q8");
}

int moe_route_scored(const float* logits, int64_t stride, int64_t rows, int64_t experts, const q8_route_rule* rule, int k,
                     int32_t* ids, float* gates, const q8_moe_plan* plan, q8_ws* ws, q8_stream stream) {
    model_fail(Q8_OK, "%s", "");
    if (rows < 0 || experts < 1) return model_fail(Q8_EINVAL, "rows %lld, experts %lld", (long long)rows, (long long)experts);
    if (experts > 1024) return model_fail(Q8_EUNSUPPORTED, "%lld experts: at most 1024", (long long)experts);
    if (!rule) return model_fail(Q8_EINVAL, "rule: null");
    if (rule->score != Q8_SCORE_SOFTMAX && rule->score != Q8_SCORE_SIGMOID)
        return model_fail(Q8_EINVAL, "rule: score %d", (int)rule->score);
    if (rule->groups < 1 || rule->groups > 32) return model_fail(Q8_EUNSUPPORTED, "rule: %d groups: 1 to 32", rule->groups);
    if (experts % rule->groups)
        return model_fail(Q8_EINVAL, "rule: %lld experts in %d groups", (long long)experts, rule->groups);
    if (rule->keep_groups < 1 || rule->keep_groups > rule->groups)
        return model_fail(Q8_EINVAL, "rule: keep_groups %d of %d", rule->keep_groups, rule->groups);
    if (rule->group_top != 1 && rule->group_top != 2) return model_fail(Q8_EINVAL, "rule: group_top %d: 1 or 2", rule->group_top);
    if (rule->renorm != 0 && rule->renorm != 1) return model_fail(Q8_EINVAL, "rule: renorm %d: 0 or 1", rule->renorm);
    if (!isfinite(rule->scale)) return model_fail(Q8_EINVAL, "rule: scale not finite");
    if (k < 1 || k > 32) return model_fail(Q8_EUNSUPPORTED, "k %d: the router keeps 1 to 32 experts", k);
    if (k > experts / rule->groups * rule->keep_groups)
        return model_fail(Q8_EINVAL, "k %d above the %lld experts of the kept groups", k,
                          (long long)(experts / rule->groups * rule->keep_groups));
    if (rows > (int64_t(1) << 24) || rows * k > (int64_t(1) << 24))
        return model_fail(Q8_EUNSUPPORTED, "rows*k %lld: at most 2^24 choices", (long long)(rows * k));
    if (rows == 0) return Q8_OK;
    if (!logits || !ids || !gates) return model_fail(Q8_EINVAL, "logits, ids or gates: null");
    if (!aligned(logits, 4) || !aligned(ids, 4) || !aligned(gates, 4) || !aligned(rule->bias, 4))
        return model_fail(Q8_EINVAL, "logits, bias, ids or gates: not 4-byte aligned");
    if (rows > 1 && stride < experts)
        return model_fail(Q8_EINVAL, "logits: rows %lld apart, of %lld values", (long long)stride, (long long)experts);
    const Range in(logits, 4 * ((rows - 1) * stride + experts)), biases(rule->bias, 4 * experts);
    const Range out[] = {{ids, 4 * rows * k}, {gates, 4 * rows * k}};
    if (out[0].meets(out[1]) || out[0].meets(in) || out[1].meets(in) || out[0].meets(biases) || out[1].meets(biases))
        return model_fail(Q8_EINVAL, "ids or gates: overlaps the logits, the bias or the other");
    if (plan) {
        if (int r = check_plan4(plan)) return r;
        if (!ws) return model_fail(Q8_EINVAL, "ws: null (the choices are grouped)");
        const Range made[] = {{plan->counts, 4 * experts}, {plan->offsets, 4 * (experts + 1)}, {plan->lists, 4 * rows * k},
                              {plan->active, 4 * (experts + 1)}};
        for (int i = 0; i < 4; ++i) {
            bool bad = made[i].meets(in) || made[i].meets(biases) || made[i].meets(out[0]) || made[i].meets(out[1]);
            for (int j = 0; j < i; ++j) bad = bad || made[i].meets(made[j]);
            if (bad) return model_fail(Q8_EINVAL, "plan: overlaps the logits, the bias, ids, gates or itself");
        }
    }
    RouteScoredCall c;
    c.logits = logits;
    c.stride = stride;
    c.rows = rows;
    c.E = (int)experts;
    c.K = k;
    c.rule = *rule;
    c.ids = ids;
    c.gates = gates;
    if (plan) c.plan = plan_ptrs(plan);
    Carve cv;
    if (plan) cv = workspace_carve(ws);
    const cudaError_t e = launch_route_scored(c, cv, (cudaStream_t)stream);
    return finish(e, cv, "moe_route_scored");
}

int q4_gemv(const q4_mat* W, const float* x, int64_t x_stride, const q8_act* xq, int64_t rows, float* y, int64_t y_stride,
            q8_ws* ws, q8_stream stream) {
    model_fail(Q8_OK, "%s", "");
    if (int r = check_q4(W, "W")) return r;
    if (rows < 0) return model_fail(Q8_EINVAL, "rows negative");
    if (rows > 65536) return model_fail(Q8_EUNSUPPORTED, "rows %lld: at most 65536", (long long)rows);
    if (rows == 0) return Q8_OK;
    Q4Call c;
    if (int r = check_q4_act(x, x_stride, xq, rows, W->cols, "x", &c.act)) return r;
    if (!y || !aligned(y, 4)) return model_fail(Q8_EINVAL, "y: null or not 4-byte aligned");
    if (rows > 1 && y_stride < W->rows)
        return model_fail(Q8_EINVAL, "y: rows %lld apart, of %lld values", (long long)y_stride, (long long)W->rows);
    if (rows > 1 && !ws) return model_fail(Q8_EINVAL, "ws: null (several rows)");
    const Range out(y, 4 * ((rows - 1) * y_stride + W->rows));
    if (meets_mat(out, W) ||
        (meets_act(out, c.act, rows, W->cols) &&
         !(x && x_stride == y_stride && beside(x, W->cols, y, W->rows, y_stride, rows))))
        return model_fail(Q8_EINVAL, "y: overlaps an input");
    c.kind = Q4_DENSE;
    c.w0 = view_of(W);
    c.out_rows = W->rows;
    c.R = rows;
    c.y = y;
    c.y_stride = y_stride;
    Carve cv;
    if (ws) cv = workspace_carve(ws);
    const cudaError_t e = launch_q4(c, cv, (cudaStream_t)stream);
    return finish(e, cv, "q4_gemv");
}

int moe_gate_up_q4(const q4_mat* gate, const q4_mat* up, int64_t dff, const float* x, const q8_act* xq, int64_t rows, int k,
                   const int32_t* ids, const q8_moe_plan* plan, float* h, q8_ws* ws, q8_stream stream) {
    model_fail(Q8_OK, "%s", "");
    if (int r = check_q4(gate, "gate")) return r;
    if (int r = check_q4(up, "up")) return r;
    if (gate->rows != up->rows || gate->cols != up->cols || gate->group != up->group || gate->scale_type != up->scale_type ||
        !gate->z != !up->z)
        return model_fail(Q8_EINVAL, "gate and up differ in shape, group, scale type or zero points");
    if (dff < 1 || gate->rows % dff)
        return model_fail(Q8_EINVAL, "dff %lld does not divide the %lld stacked rows", (long long)dff, (long long)gate->rows);
    if (int r = check_experts(rows, k, ids, plan, ws)) return r;
    if (rows == 0) return Q8_OK;
    Q4Call c;
    if (int r = check_q4_act(x, gate->cols, xq, rows, gate->cols, "x", &c.act)) return r;
    if (!h || !aligned(h, 4)) return model_fail(Q8_EINVAL, "h: null or not 4-byte aligned");
    const Range out(h, 4 * rows * k * dff);
    if (meets_act(out, c.act, rows, gate->cols) || meets_mat(out, gate) || meets_mat(out, up) ||
        out.meets(Range(ids, 4 * rows * k)) || meets_plan(out, plan, gate->rows / dff, rows, k))
        return model_fail(Q8_EINVAL, "h: overlaps an input");
    c.kind = Q4_GATE_UP;
    c.w0 = view_of(gate);
    c.w1 = view_of(up);
    c.E = gate->rows / dff;
    c.out_rows = dff;
    c.R = rows;
    c.K = k;
    c.ids = ids;
    if (plan && rows > 1) c.plan = plan_ptrs(plan);
    c.y = h;
    c.y_stride = dff;
    Carve cv = workspace_carve(ws);
    const cudaError_t e = launch_q4(c, cv, (cudaStream_t)stream);
    return finish(e, cv, "moe_gate_up_q4");
}

int moe_down_combine_q4(const q4_mat* down, int64_t d, const float* h, const q8_act* hq, int64_t rows, int k,
                        const int32_t* ids, const float* gates, const q8_moe_plan* plan, const float* residual, float* y,
                        q8_ws* ws, q8_stream stream) {
    model_fail(Q8_OK, "%s", "");
    if (int r = check_q4(down, "down")) return r;
    if (d < 1 || down->rows % d)
        return model_fail(Q8_EINVAL, "d %lld does not divide the %lld stacked rows", (long long)d, (long long)down->rows);
    if (int r = check_experts(rows, k, ids, plan, ws)) return r;
    if (rows == 0) return Q8_OK;
    Q4Call c;
    if (int r = check_q4_act(h, down->cols, hq, rows * k, down->cols, "h", &c.act)) return r;
    if (!gates || !aligned(gates, 4)) return model_fail(Q8_EINVAL, "gates: null or not 4-byte aligned");
    if (!y || !aligned(y, 4) || !aligned(residual, 4)) return model_fail(Q8_EINVAL, "y: null, or y or residual not 4-byte aligned");
    const Range out(y, 4 * rows * d);
    if (meets_act(out, c.act, rows * k, down->cols) || meets_mat(out, down) || out.meets(Range(ids, 4 * rows * k)) ||
        out.meets(Range(gates, 4 * rows * k)) || (residual != y && out.meets(Range(residual, 4 * rows * d))) ||
        meets_plan(out, plan, down->rows / d, rows, k))
        return model_fail(Q8_EINVAL, "y: overlaps an input");
    c.kind = Q4_DOWN;
    c.w0 = view_of(down);
    c.E = down->rows / d;
    c.out_rows = d;
    c.R = rows;
    c.K = k;
    c.ids = ids;
    c.gates = gates;
    if (plan && rows > 1) c.plan = plan_ptrs(plan);
    c.residual = residual;
    c.y = y;
    c.y_stride = d;
    Carve cv = workspace_carve(ws);
    const cudaError_t e = launch_q4(c, cv, (cudaStream_t)stream);
    return finish(e, cv, "moe_down_combine_q4");
}

}  // extern "C"
