// Products of 4-bit weights with several rows of f32 activations (q4_rows.cuh).
#include "q4_rows.cuh"

namespace q8 {

cudaError_t launch_rows_f32(const RowsParams& p, int64_t groups, cudaStream_t st) { return launch_rows<FORM_F32>(p, groups, st); }

}  // namespace q8
