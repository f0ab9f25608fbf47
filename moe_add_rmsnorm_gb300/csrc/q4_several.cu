// Products of 4-bit weights with several activation rows: which kernel takes them (q4_rows.cuh, q4_mma.cuh), and the sum over
// the choices.
#include "q4_mma.cuh"

namespace q8 {
namespace {

struct CombineParams {
    int64_t E, d;
    int R, K;
    const int32_t* ids;
    const float *gates, *residual, *out;
    float* y;
    const int* failed;  // of products whose waits can give up, the workspace's word; else NULL
};

// y[r] = residual[r] + sum_j gates[r][j] out[r][j], in the order of the choices.  Nothing where the products' waits gave up, in
// this call or in an earlier one: `out` then holds an earlier call's sums.
__global__ void __launch_bounds__(256) q4_combine_kernel(const CombineParams p) {
    griddep_wait();
    const int failed = p.failed ? __ldcg(p.failed) : 0;  // (looked at only with the sums: its load is one among theirs)
    const int64_t o = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (o >= p.d) return;
    for (int64_t r = blockIdx.y; r < p.R; r += gridDim.y) {
        float sum = 0.f;
#pragma unroll 8
        for (int j = 0; j < p.K; ++j) {  // (independent loads: eight of them on their way together)
            const int64_t c = r * p.K + j;
            const int e = p.ids[c];
            const float g = p.gates[c], v = p.out[c * p.d + o];
            if (e >= 0 && e < p.E) sum = fmaf(g, v, sum);
        }
        sum = p.residual ? p.residual[r * p.d + o] + sum : sum;
        if (failed == 0) p.y[r * p.d + o] = sum;
    }
}

// The CUDA driver API's tensor-map encoder, found once through the runtime's entry-point lookup, so that the library does not
// link against libcuda.
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
Encode encoder() {
    static const Encode fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return (Encode) nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    return fn;
}

}  // namespace

bool q4_map(CUtensorMap* map, const Q4View& w, int box_rows) {
    const Encode encode = encoder();
    if (!encode) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)w.cols / 2, (cuuint64_t)w.rows}, stride[1] = {(cuuint64_t)w.cols / 2};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows}, step[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(w.q), dims, stride, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool q4_row_fits(const Q4Call& c);
cudaError_t launch_q4_row(const Q4Call& c, cudaStream_t st);
cudaError_t launch_q4_warps(const Q4Call& c, int64_t groups, int form, float* out, Carve& ws, cudaStream_t st);

namespace {

cudaError_t launch_q4_tensor(const Q4Call& c, int64_t groups, int form, float* out, Carve& ws, cudaStream_t st) {
    MmaParams p = {};
    p.w0 = c.w0;
    p.w1 = c.w1;
    p.act = c.act;
    p.kind = c.kind;
    p.E = c.E;
    p.out_rows = c.out_rows;
    p.R = (int)c.R;
    p.K = c.K;
    p.plan = c.plan;
    p.ids = c.ids;
    p.y = c.y;
    p.y_stride = c.y_stride;
    p.out = out;
    p.failed = ws.failed;
    p.chunks = (c.w0.cols + 127) / 128;
    const int tile_rows = c.kind == Q4_GATE_UP ? 64 : 128;
    p.row_tiles = (int)((c.out_rows + tile_rows - 1) / tile_rows);
    p.slots = c.kind == Q4_DENSE ? (c.R + 7) & ~int64_t(7) : (c.R * c.K + 8 * groups + 15) & ~int64_t(7);
    p.parts = ws.take<char>((size_t)p.slots / 8 * p.chunks * (form == FORM_ONE ? 2048 : 4096));
    p.scales = ws.take<float>(form == FORM_F32 ? (size_t)p.slots : (size_t)p.slots / 8 * p.chunks * 32);
    if (ws.overflow) return cudaSuccess;
    return form == FORM_F32   ? launch_mma_f32(p, groups, ws, st)
           : form == FORM_ONE ? launch_mma_one(p, groups, ws, st)
                              : launch_mma_two(p, groups, ws, st);
}

// A call whose rows fit the workspace.
cudaError_t launch_q4_rows(const Q4Call& c, int form, Carve& ws, cudaStream_t st) {
    if (c.R == 1 && q4_row_fits(c)) return launch_q4_row(c, st);
    const int64_t groups = c.kind == Q4_DENSE ? 1 : c.R == 1 ? c.K : min(c.E, c.R * c.K);
    float* out = c.kind == Q4_DOWN ? ws.take<float>((size_t)c.R * c.K * c.out_rows) : nullptr;
    if (ws.overflow) return cudaSuccess;
    // Up to 16 columns (an activation's parts) a group on average, the warp-wide products are as fast or faster: they start
    // sooner and unpack with all their warps.  From there on the tensor cores' rows share what was unpacked.  Measured, warps and
    // tensor cores, us: 8192 x 4096, group 128, f32: 8 rows 12 and 16, 16 rows 19 and 16, 64 rows 40 and 23; 6 of 64 experts of
    // 2048 x 1408, group 32, f32: 24 rows (2.3 an expert) 109 and 154, 60 (5.6) 151 and 176, 100 (9.4) 200 and 184, 256 (24) 412 and
    // 254.
    const int64_t columns = c.R * c.K * (form == FORM_ONE ? 1 : 2);
    const bool warps = columns <= 16 * groups;
    const cudaError_t e = warps ? launch_q4_warps(c, groups, form, out, ws, st) : launch_q4_tensor(c, groups, form, out, ws, st);
    if (e != cudaSuccess || ws.overflow || c.kind != Q4_DOWN) return e;
    const CombineParams p = {c.E, c.out_rows, (int)c.R, c.K, c.ids, c.gates, c.residual, out, c.y, warps ? nullptr : ws.failed};
    const dim3 grid((unsigned)((c.out_rows + 127) / 128), (unsigned)min(c.R, (int64_t)65535));
    return launch(q4_combine_kernel, grid, dim3(128), 0, st, 1, p);
}

}  // namespace

cudaError_t launch_q4(const Q4Call& call, Carve& ws, cudaStream_t st) {
    const int form = call.act.x ? FORM_F32 : call.act.lo ? FORM_TWO : FORM_ONE;
    if (call.kind != Q4_DENSE || call.R == 1) return launch_q4_rows(call, form, ws, st);
    // A projection of more rows than the workspace holds operands of takes them so many at a time.
    const size_t row = (size_t)((call.w0.cols + 127) / 128) * (form == FORM_ONE ? 256 + 16 : 512 + 16) + 8;
    const size_t joins = size_t(6) << 20;  // the sums of weights that are cut (a tile of 64 rows by 128 an SM), and edges
    const size_t room = ws.size > ws.used + joins ? (ws.size - ws.used - joins) / row : 0;
    if (room < 64 || (size_t)call.R <= room) return launch_q4_rows(call, form, ws, st);
    Q4Call c = call;
    for (int64_t left = call.R; left > 0; left -= c.R) {
        c.R = min(left, (int64_t)(room & ~size_t(63)));
        Carve own = ws;  // (the blocks' launches follow one another)
        const cudaError_t e = launch_q4_rows(c, form, own, st);
        ws.overflow = own.overflow;
        if (e != cudaSuccess || ws.overflow) return e;
        c.y += c.R * c.y_stride;
        if (form == FORM_F32) {
            c.act.x += c.R * c.act.stride;
        } else {
            c.act.q += c.R * c.w0.cols;
            if (form == FORM_TWO) c.act.lo += c.R * c.w0.cols;
            c.act.s += c.R * (c.w0.cols / 32);
        }
    }
    return cudaSuccess;
}

}  // namespace q8
