// Products of 4-bit weights with several activation rows: the launches (q4_rows.cuh has the kernels).
#include "q4_rows.cuh"

namespace q8 {
namespace {

// y[r] = residual[r] + sum_j gates[r][j] out[r][j], in the order of the choices.
__global__ void __launch_bounds__(256) q4_combine_kernel(const RowsParams p) {
    griddep_wait();
    const int64_t n = (int64_t)p.R * p.out_rows, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
        const int64_t r = i / p.out_rows, o = i - r * p.out_rows;
        float sum = 0.f;
        for (int j = 0; j < p.K; ++j) {
            const int64_t c = r * p.K + j;
            const int e = p.ids[c];
            if (e >= 0 && e < p.E) sum = fmaf(p.gates[c], p.out[c * p.out_rows + o], sum);
        }
        p.y[i] = p.residual ? p.residual[i] + sum : sum;
    }
}

}  // namespace

bool q4_row_fits(const Q4Call& c);
cudaError_t launch_q4_row(const Q4Call& c, cudaStream_t st);

cudaError_t launch_q4(const Q4Call& c, Carve& ws, cudaStream_t st) {
    if (c.R == 1 && q4_row_fits(c)) return launch_q4_row(c, st);
    const int form = c.act.x ? FORM_F32 : c.act.lo ? FORM_TWO : FORM_ONE;
    RowsParams p = {};
    p.w0 = c.w0;
    p.w1 = c.w1;
    p.act = c.act;
    p.kind = c.kind;
    p.E = c.E;
    p.out_rows = c.out_rows;
    p.R = (int)c.R;
    p.K = c.K;
    p.act_rows = c.kind == Q4_DOWN ? c.R * c.K : c.R;
    p.plan = c.plan;
    p.ids = c.ids;
    p.gates = c.gates;
    p.residual = c.residual;
    p.y = c.y;
    p.y_stride = c.y_stride;
    p.chunks = (c.w0.cols + 127) / 128;
    p.row_tiles = (int)((c.out_rows + (c.kind == Q4_GATE_UP ? 15 : 31)) / (c.kind == Q4_GATE_UP ? 16 : 32));
    p.parts = ws.take<uint4>((size_t)p.act_rows * p.chunks * 16 * (form == FORM_ONE ? 1 : 2));
    p.scales = ws.take<float>((size_t)p.act_rows * (form == FORM_F32 ? 1 : p.chunks * 4 * form));
    if (c.kind == Q4_DOWN) p.out = ws.take<float>((size_t)c.R * c.K * c.out_rows);
    if (ws.overflow) return cudaSuccess;
    const int64_t groups = c.kind == Q4_DENSE ? 1 : c.R == 1 ? c.K : min(c.E, c.R * c.K);
    const cudaError_t e = form == FORM_F32   ? launch_rows_f32(p, groups, st)
                          : form == FORM_ONE ? launch_rows_one(p, groups, st)
                                             : launch_rows_two(p, groups, st);
    if (e != cudaSuccess || c.kind != Q4_DOWN) return e;
    const int64_t n = c.R * c.out_rows;
    return launch(q4_combine_kernel, dim3((unsigned)min((n + 255) / 256, (int64_t)device_info().sms * 16)), dim3(256), 0, st, 1, p);
}

}  // namespace q8
