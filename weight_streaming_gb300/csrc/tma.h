// Host side of tiled TMA copies: the driver's tensor-map encoder, looked up once (no link to libcuda).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include "verify.h"

namespace vp {

vp_status tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* fn);  // errors.cu

}  // namespace vp
