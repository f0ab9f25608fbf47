// Products of 4-bit weights with several rows of f32 activations on the tensor cores (q4_mma.cuh).
#include "q4_mma.cuh"

namespace q8 {

cudaError_t launch_mma_f32(const MmaParams& p, int64_t groups, Carve& ws, cudaStream_t st) {
    return launch_mma<FORM_F32>(p, groups, ws, st);
}

}  // namespace q8
