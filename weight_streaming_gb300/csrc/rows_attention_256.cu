// Heads of 256 columns (see rows_attention.cu).
#include "rows_attention.cuh"

namespace vp {
template cudaError_t launch_rows<256, 2>(const RowsArgs&, int, const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
template cudaError_t launch_rows<256, 1>(const RowsArgs&, int, const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
}  // namespace vp
