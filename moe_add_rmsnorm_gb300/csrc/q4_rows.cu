// Products with 4-bit weights.
#include <cuda_fp16.h>

#include "common.cuh"
#include "ffn4.h"

namespace q8 {
namespace {

__device__ __forceinline__ float q4_scale_of(const Q4View& w, int64_t i) {
    const uint16_t u = w.s[i];
    return w.bf16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
}

// A warp's dot of weight row o with activation row r.
__device__ float row_dot(const Q4View& w, int64_t o, const Q4Act& act, int64_t r) {
    const int lane = threadIdx.x & 31;
    float sum = 0.f;
    for (int t = lane; t < w.cols; t += 32) {
        const int64_t g = o * (w.cols >> w.group_log2) + (t >> w.group_log2);
        const int word = (w.q[o * (w.cols / 2) + t / 2] >> (t & 1 ? 4 : 0)) & 15;
        const float wv = (float)(word - (w.z ? w.z[g] : 8)) * q4_scale_of(w, g);
        float x;
        if (act.x) {
            x = act.x[r * act.stride + t];
        } else {
            x = act.q[r * w.cols + t];
            if (act.lo) x += act.lo[r * w.cols + t] * 0.0078125f;
            x *= act.s[(r * w.cols + t) >> 5];
        }
        sum = fmaf(wv, x, sum);
    }
    return group_sum<32>(sum);
}

__global__ void __launch_bounds__(256) q4_kernel(const Q4Call c) {
    const int64_t rows = c.R * (c.kind == Q4_GATE_UP ? c.K : 1);
    const int64_t n = rows * c.out_rows, step = (int64_t)gridDim.x * 8;
    for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += step) {
        const int64_t r = i / c.out_rows, o = i % c.out_rows;
        if (c.kind == Q4_DENSE) {
            const float v = row_dot(c.w0, o, c.act, r);
            if ((threadIdx.x & 31) == 0) c.y[r * c.y_stride + o] = v;
        } else if (c.kind == Q4_GATE_UP) {
            const int64_t e = c.ids[r];
            if (e < 0 || e >= c.E) continue;
            const float g = row_dot(c.w0, e * c.out_rows + o, c.act, r / c.K);
            const float u = row_dot(c.w1, e * c.out_rows + o, c.act, r / c.K);
            if ((threadIdx.x & 31) == 0) c.y[r * c.y_stride + o] = silu_f32(g) * u;
        } else {
            float v = c.residual ? c.residual[r * c.out_rows + o] : 0.f, sum = 0.f;
            for (int j = 0; j < c.K; ++j) {
                const int64_t e = c.ids[r * c.K + j];
                if (e < 0 || e >= c.E) continue;
                sum = fmaf(c.gates[r * c.K + j], row_dot(c.w0, e * c.out_rows + o, c.act, r * c.K + j), sum);
            }
            if ((threadIdx.x & 31) == 0) c.y[r * c.y_stride + o] = v + sum;
        }
    }
}

}  // namespace

cudaError_t launch_q4_row(const Q4Call& c, cudaStream_t st);

cudaError_t launch_q4(const Q4Call& c, Carve&, cudaStream_t st) {
    if (c.R == 1) return launch_q4_row(c, st);
    return launch(q4_kernel, dim3((unsigned)device_info().sms * 8), dim3(256), 0, st, 0, c);
}

}  // namespace q8
