// Linear layer of a block-quantised FP8 checkpoint on block-quantised activations
// (vp_linear_fp8_block).
//
// Mathematics: y[m][n] = sum_b xs[m][b] ws[n / 128][b] (sum_{k in b} xq[m][k] w[n][k]).  The products are
// exact in fp32 (e4m3 has 4 significant bits); the scales differ from block to block, so each inner
// sum of 128 products leaves the accumulator, is scaled and added to an fp32 register.
// First form: CUDA cores, a 64 x 64 output tile per CTA, 4 x 4 outputs per thread.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "errors.h"
#include "fp8_block.h"
#include "internal.h"
#include "ptx.cuh"
#include "verify.h"

namespace vp {

namespace {

__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float (&v)[4]) {
  uint32_t lo, hi;
  e4m3x4_to_f16x2x2(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

__global__ void __launch_bounds__(256) linear_simple(const uint8_t* __restrict__ w, const float* __restrict__ ws,
                                                     const uint8_t* __restrict__ xq, const float* __restrict__ xs,
                                                     void* __restrict__ y, int f32, int M, int N, int K) {
  __shared__ float sx[32][65], sw[32][65];  // [k][row]
  const int n0 = blockIdx.x * 64, m0 = blockIdx.y * 64, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int KB = qblocks(K);
  float acc[4][4] = {};
  for (int kb = 0; kb < KB; ++kb) {
    float part[4][4] = {};
    for (int k0 = 0; k0 < kQBlock; k0 += 32) {
      for (int i = tid; i < 512; i += 256) {  // 64 rows x 8 words of each operand
        const int r = i >> 3, c = i & 7, k = kb * kQBlock + k0 + 4 * c;
        float v[4];
        uint32_t word = 0;
        if (m0 + r < M && k < K) word = *reinterpret_cast<const uint32_t*>(xq + (size_t)(m0 + r) * K + k);
        e4m3x4_to_f32(word, v);
        for (int e = 0; e < 4; ++e) sx[4 * c + e][r] = v[e];
        const int n = n0 + r;
        word = 0;
        if (n < N)
          word = *reinterpret_cast<const uint32_t*>(w + ((size_t)(n >> 7) * KB + kb) * kQTileBytes +
                                                    qtile_offset(n & 127, (k0 >> 4) + (c >> 2)) + 4 * (c & 3));
        e4m3x4_to_f32(word, v);
        for (int e = 0; e < 4; ++e) sw[4 * c + e][r] = v[e];
      }
      __syncthreads();
      for (int k = 0; k < 32; ++k)
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j) part[i][j] = fmaf(sx[k][ty + 16 * i], sw[k][tx + 16 * j], part[i][j]);
      __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m < M && n < N) acc[i][j] = fmaf(part[i][j], xs[(size_t)m * KB + kb] * ws[(size_t)(n >> 7) * KB + kb], acc[i][j]);
      }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= M || n >= N) continue;
      if (f32)
        static_cast<float*>(y)[(size_t)m * N + n] = acc[i][j];
      else
        static_cast<__nv_bfloat16*>(y)[(size_t)m * N + n] = __float2bfloat16_rn(acc[i][j]);
    }
}

bool al(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int kMaxMq = 1 << 20;

}  // namespace

}  // namespace vp

using namespace vp;

extern "C" {

size_t vp_linear_fp8_block_workspace_bytes(int M, int N, int K) {
  if (M < 1 || M > kMaxMq || !q_shape_ok(N, K)) return 0;
  return 256;
}

vp_status vp_linear_fp8_block(const void* w_packed, const float* w_scales, const void* xq, const float* x_scales,
                              void* y, int y_type, int M, int N, int K, void* ws, size_t ws_bytes, void* stream) {
  if (!w_packed || !w_scales || !xq || !x_scales || !y || !ws || (y_type != VP_BF16 && y_type != VP_F32))
    return VP_ERR_INVALID_ARG;
  const size_t need = vp_linear_fp8_block_workspace_bytes(M, N, K);
  if (need == 0) return VP_ERR_SHAPE;
  if (!al(w_packed, 16) || !al(w_scales, 4) || !al(xq, 16) || !al(x_scales, 4) || !al(y, 16) || !al(ws, 256))
    return VP_ERR_ALIGNMENT;
  if (ws_bytes < need) return VP_ERR_WORKSPACE;
  int sms = 0;
  const vp_status st = device_sm_count(&sms);
  if (st != VP_OK) return st;
  linear_simple<<<dim3((unsigned)((N + 63) / 64), (unsigned)((M + 63) / 64)), 256, 0, (cudaStream_t)stream>>>(
      static_cast<const uint8_t*>(w_packed), w_scales, static_cast<const uint8_t*>(xq), x_scales, y, y_type == VP_F32,
      M, N, K);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VP_OK : cuda_fail(e);
}

}  // extern "C"
