// Products of 4-bit weights with several rows of activations of one int8 word a value on the tensor cores (q4_mma.cuh).
#include "q4_mma.cuh"

namespace q8 {

cudaError_t launch_mma_one(const MmaParams& p, int64_t groups, Carve& ws, cudaStream_t st) {
    return launch_mma<FORM_ONE>(p, groups, ws, st);
}

}  // namespace q8
