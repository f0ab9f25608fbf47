// Launch interface between the C ABI of the 4-bit feed-forward block (ffn4_api.cu) and its kernels.  Host code only.
#pragma once
#include <atomic>

#include "kernels.h"

namespace q8 {

// Allows `kernel` `bytes` of dynamic shared memory, once a device (the call takes longer than the checks of a whole call).
template <typename Kern>
cudaError_t allow_smem(Kern kernel, size_t bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// ---- the norms around a block (postnorm.cu) ---------------------------------------------------------------------
struct PostnormCall {
    const float *a = nullptr, *b = nullptr, *w_post = nullptr, *w_pre = nullptr, *gate = nullptr;
    int64_t gate_row = 0, gate_col = 0;  // strides of gate
    float scale = 1.f, eps = 0.f;
    int64_t rows = 0, d = 0;
    float *sum = nullptr, *y = nullptr;
    int8_t *yq = nullptr, *yl = nullptr;
    float* ys = nullptr;
};
cudaError_t launch_postnorm(const PostnormCall& c, cudaStream_t st);

// ---- the scored router (route_scored.cu) ----------------------------------------------------------------------------
struct RouteScoredCall {
    const float* logits = nullptr;
    int64_t stride = 0, rows = 0;
    int E = 0, K = 0;
    q8_route_rule rule = {};
    int32_t* ids = nullptr;
    float* gates = nullptr;
    PlanPtrs plan;  // filled when plan.counts != nullptr
};
cudaError_t launch_route_scored(const RouteScoredCall& c, Carve& ws, cudaStream_t st);

// ---- products with 4-bit weights (q4_row.cu, q4_rows.cu) -------------------------------------------------------------
struct Q4View {
    const uint8_t* q = nullptr;
    const uint16_t* s = nullptr;
    const uint8_t* z = nullptr;
    int cols = 0, group_log2 = 0, bf16 = 0;
    int64_t rows = 0;
};

// Rows of activations: f32, or words (and low words) with a scale for every 32.
struct Q4Act {
    const float* x = nullptr;
    int64_t stride = 0;
    const int8_t *q = nullptr, *lo = nullptr;
    const float* s = nullptr;
};

enum { Q4_DENSE = 0, Q4_GATE_UP = 1, Q4_DOWN = 2 };

struct Q4Call {
    int kind = Q4_DENSE;
    Q4View w0, w1;                // gate-up: gate and up
    int64_t E = 1, out_rows = 0;  // out_rows a group (dense: the matrix's; dff; d)
    Q4Act act;
    int64_t R = 1;
    int K = 1;
    const int32_t* ids = nullptr;
    const float* gates = nullptr;
    PlanPtrs plan;                // several rows
    const float* residual = nullptr;
    float* y = nullptr;           // dense: y; gate-up: h; down: y
    int64_t y_stride = 0;
};
cudaError_t launch_q4(const Q4Call& c, Carve& ws, cudaStream_t st);

}  // namespace q8
