// Products of 4-bit weights with several rows of activations of one int8 word a value (q4_rows.cuh).
#include "q4_rows.cuh"

namespace q8 {

cudaError_t launch_rows_one(const RowsParams& p, int64_t groups, cudaStream_t st) { return launch_rows<FORM_ONE>(p, groups, st); }

}  // namespace q8
