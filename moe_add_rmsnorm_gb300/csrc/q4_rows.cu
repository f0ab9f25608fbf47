// Products of 4-bit weights with several activation rows: the launches (q4_rows.cuh has the kernels).
#include "q4_rows.cuh"

namespace q8 {

cudaError_t launch_q4_warps(const Q4Call& c, int64_t groups, int form, float* out, Carve& ws, cudaStream_t st) {
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
    p.y = c.y;
    p.y_stride = c.y_stride;
    p.chunks = (c.w0.cols + 127) / 128;
    p.row_tiles = (int)((c.out_rows + (c.kind == Q4_GATE_UP ? 15 : 31)) / (c.kind == Q4_GATE_UP ? 16 : 32));
    p.parts = ws.take<uint4>((size_t)p.act_rows * p.chunks * 16 * (form == FORM_ONE ? 1 : 2));
    p.scales = ws.take<float>((size_t)p.act_rows * (form == FORM_F32 ? 1 : p.chunks * 4 * form));
    p.out = out;
    if (ws.overflow) return cudaSuccess;
    return form == FORM_F32   ? launch_rows_f32(p, groups, st)
           : form == FORM_ONE ? launch_rows_one(p, groups, st)
                              : launch_rows_two(p, groups, st);
}

}  // namespace q8
