// See errors.h.
#include "errors.h"

#include <atomic>

#include "tma.h"

namespace vp {

namespace {
thread_local int g_last_cuda_error = 0;
}

vp_status cuda_fail(cudaError_t e) {
  g_last_cuda_error = (int)e;
  return VP_ERR_CUDA;
}

int last_cuda_error() { return g_last_cuda_error; }

vp_status tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* fn) {
  static std::atomic<void*> cached{nullptr};
  void* p = cached.load();
  if (!p) {
    cudaDriverEntryPointQueryResult res;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &res);
    if (e != cudaSuccess) return cuda_fail(e);
    if (res != cudaDriverEntryPointSuccess || !p) return VP_ERR_UNSUPPORTED;
    cached.store(p);
  }
  *fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  return VP_OK;
}

}  // namespace vp
