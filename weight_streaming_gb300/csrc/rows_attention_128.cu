// Heads of 128 columns (see rows_attention.cu).
#include "rows_attention.cuh"

namespace vp {
template cudaError_t launch_rows<128, 1>(const RowsArgs&, int, const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
template cudaError_t launch_rows<128, 2>(const RowsArgs&, int, const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
}  // namespace vp
