// Producers of block-scaled e4m3 operands: the weight packer (vp_pack_fp8_block), the quantiser
// (vp_quant_fp8), and the residual addition + RMSNorm with a quantised output (vp_add_rmsnorm_fp8).
//
// Mathematics: a group of 128 values shares s = max(max|x| / 448, 2^-126), so that |x / s| <= 448 up to
// one rounding, and q = e4m3(x * (1 / s)): the reciprocal is one fp32 rounding away from the quotient,
// which moves a value across a border of e4m3 (steps of 2^-3 relative) for about 1 in 2^19 values.
// e4m3's half step is 2^-4 of the value: the 8 bits the tensor core multiplies.  The maximum is taken
// on the magnitude's bits as integers, where NaN is above infinity: both reach the scale.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "errors.h"
#include "fp8_block.h"
#include "verify.h"

namespace vp {

namespace {

__device__ __forceinline__ void unpack_bf16x2(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xFFFF0000u);
}
// Eight consecutive values of a row of x (16-byte aligned).
template <bool kF32>
__device__ __forceinline__ void load8(const void* x, size_t at, float (&v)[8]) {
  if (kF32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(x) + at));
    const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(x) + at + 4));
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at));
    unpack_bf16x2(a.x, v[0], v[1]);
    unpack_bf16x2(a.y, v[2], v[3]);
    unpack_bf16x2(a.z, v[4], v[5]);
    unpack_bf16x2(a.w, v[6], v[7]);
  }
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
// The half warp's 16 x 8 values are one group: its scale (returned to every lane) and this lane's codes.
__device__ __forceinline__ float quant_group(const float (&v)[8], uint2& codes) {
  const uint32_t half = 0xFFFFu << (threadIdx.x & 16);  // the other half warp may be past the row's end
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(half, m, o));
  float s = __uint_as_float(m) / kE4m3Max;
  if (s < 1.17549435e-38f) s = 1.17549435e-38f;  // 2^-126: its reciprocal is finite (NaN stays)
  const float r = 1.0f / s;
  codes.x = e4m3x4(v[0] * r, v[1] * r, v[2] * r, v[3] * r);
  codes.y = e4m3x4(v[4] * r, v[5] * r, v[6] * r, v[7] * r);
  return s;
}

// One half warp per (row, group).  Bounded by the bytes: 2 or 4 read and about 1 written per value.
template <bool kF32>
__global__ void __launch_bounds__(256) quant_kernel(const void* __restrict__ x, long long ld, int M, int K,
                                                    uint8_t* __restrict__ q, float* __restrict__ scales) {
  const int KB = qblocks(K), lane = threadIdx.x & 15;
  const long long n = (long long)M * KB, step = (long long)gridDim.x * 16;
  for (long long u = (long long)blockIdx.x * 16 + (threadIdx.x >> 4); u < n; u += step) {
    const int m = (int)(u / KB), b = (int)(u - (long long)m * KB), k = b * kQBlock + lane * 8;
    const bool ok = k < K;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (ok) load8<kF32>(x, (size_t)m * ld + k, v);
    uint2 c;
    const float s = quant_group(v, c);
    if (ok) *reinterpret_cast<uint2*>(q + (size_t)m * K + k) = c;
    if (lane == 0) scales[u] = s;
  }
}

// One CTA per row, kC chunks of 8 values per thread in registers (one pass over the data).
template <bool kF32, int kC>
__global__ void __launch_bounds__(1024) norm_kernel(const void* x, long long ld, const uint16_t* residual,
                                                    const float* __restrict__ weight, float eps, int K, uint16_t* h,
                                                    uint8_t* __restrict__ q, float* __restrict__ scales) {
  __shared__ float red[32];
  __shared__ double redd[32];
  const int m = blockIdx.x, tid = threadIdx.x, T = blockDim.x, KB = qblocks(K);
  float v[kC][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const int k = (tid + i * T) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
    if (k >= K) continue;
    load8<kF32>(x, (size_t)m * ld + k, v[i]);
    if (residual) {
      float r[8];
      load8<false>(residual, (size_t)m * K + k, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] += r[e];
    }
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[i][2 * e], v[i][2 * e + 1]);  // the residual stream is bf16
      w[e] = *reinterpret_cast<const uint32_t*>(&p);
      unpack_bf16x2(w[e], v[i][2 * e], v[i][2 * e + 1]);
    }
    if (h) *reinterpret_cast<uint4*>(h + (size_t)m * K + k) = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
  if ((tid & 31) == 0) red[tid >> 5] = ss;
  __syncthreads();
  ss = 0.0f;
  for (int w = 0; w < (T + 31) / 32; ++w) ss += red[w];
  float inv = 1.0f / sqrtf(ss / (float)K + eps);
  double invd = 0.0;
  const bool wide = !(ss >= 1e-30f && ss <= 3.0e38f);  // squares outside fp32 (or a zero or NaN row): fp64
  if (wide) {
    double sd = 0.0;
#pragma unroll
    for (int i = 0; i < kC; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) sd += (double)v[i][e] * (double)v[i][e];
    for (int o = 16; o; o >>= 1) sd += __shfl_xor_sync(0xFFFFFFFFu, sd, o);
    if ((tid & 31) == 0) redd[tid >> 5] = sd;
    __syncthreads();
    sd = 0.0;
    for (int w = 0; w < (T + 31) / 32; ++w) sd += redd[w];
    invd = 1.0 / sqrt(sd / (double)K + (double)eps);
  }
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const int k = (tid + i * T) * 8;
    if ((k & ~127) >= K) continue;  // uniform over the half warp
    float y[8], wt[8] = {1, 1, 1, 1, 1, 1, 1, 1};
    if (weight && k < K) {
#pragma unroll
      for (int e = 0; e < 8; ++e) wt[e] = __ldg(weight + k + e);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      y[e] = wide ? (float)((double)v[i][e] * invd * (double)wt[e]) : v[i][e] * inv * wt[e];
    uint2 c;
    const float s = quant_group(y, c);
    if (k < K) *reinterpret_cast<uint2*>(q + (size_t)m * K + k) = c;
    if ((tid & 15) == 0) scales[(size_t)m * KB + k / kQBlock] = s;
  }
}

__global__ void pack_block_kernel(const uint8_t* __restrict__ w, int N, int K, uint8_t* __restrict__ out) {
  const int KB = qblocks(K);
  const long long n = (long long)qblocks(N) * KB * (kQTileBytes / 16);
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    const long long tile = i >> 10;
    const int r = (int)(i >> 3) & 127, c = (int)i & 7;
    const int nb = (int)(tile / KB), kb = (int)(tile - (long long)nb * KB);
    const int row = nb * kQBlock + r, k = kb * kQBlock + c * 16;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < N && k < K) v = *reinterpret_cast<const uint4*>(w + (size_t)row * K + k);
    *reinterpret_cast<uint4*>(out + tile * kQTileBytes + qtile_offset(r, c)) = v;
  }
}

bool al(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

vp_status check_rows(const void* x, int x_type, int64_t ld_x, int M, int K, int max_k, const void* q,
                     const float* scales) {
  if (!x || !q || !scales || (x_type != VP_BF16 && x_type != VP_F32)) return VP_ERR_INVALID_ARG;
  if (M < 1 || M > (1 << 24) || K < 16 || K % 16 || K > max_k || ld_x < K || ld_x > (1LL << 40)) return VP_ERR_SHAPE;
  if (!al(x, 16) || ld_x % (x_type == VP_F32 ? 4 : 8) || !al(q, 16) || !al(scales, 4)) return VP_ERR_ALIGNMENT;
  return VP_OK;
}

}  // namespace

}  // namespace vp

using namespace vp;

extern "C" {

size_t vp_packed_bytes_fp8_block(int N, int K) {
  if (!q_shape_ok(N, K)) return 0;
  return (size_t)qblocks(N) * (size_t)qblocks(K) * kQTileBytes;
}

vp_status vp_pack_fp8_block(const void* w, int N, int K, void* packed, size_t packed_bytes, void* stream) {
  if (!w || !packed) return VP_ERR_INVALID_ARG;
  const size_t need = vp_packed_bytes_fp8_block(N, K);
  if (need == 0) return VP_ERR_SHAPE;
  if (packed_bytes < need) return VP_ERR_INVALID_ARG;
  if (!al(w, 16) || !al(packed, 16)) return VP_ERR_ALIGNMENT;
  int sms = 0;
  const vp_status st = device_sm_count(&sms);
  if (st != VP_OK) return st;
  const long long n = (long long)(need / 16);
  pack_block_kernel<<<(unsigned)std::min<long long>((n + 255) / 256, 16LL * sms), 256, 0, (cudaStream_t)stream>>>(
      static_cast<const uint8_t*>(w), N, K, static_cast<uint8_t*>(packed));
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VP_OK : cuda_fail(e);
}

vp_status vp_quant_fp8(const void* x, int x_type, int64_t ld_x, int M, int K, void* q, float* scales, void* stream) {
  vp_status st = check_rows(x, x_type, ld_x, M, K, 65536, q, scales);
  if (st != VP_OK) return st;
  int sms = 0;
  if ((st = device_sm_count(&sms)) != VP_OK) return st;
  const long long n = (long long)M * qblocks(K);
  const unsigned grid = (unsigned)std::min<long long>((n + 15) / 16, 64LL * sms);
  auto* kern = x_type == VP_F32 ? quant_kernel<true> : quant_kernel<false>;
  kern<<<grid, 256, 0, (cudaStream_t)stream>>>(x, ld_x, M, K, static_cast<uint8_t*>(q), scales);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VP_OK : cuda_fail(e);
}

vp_status vp_add_rmsnorm_fp8(const void* x, int x_type, int64_t ld_x, const void* residual, const float* weight,
                             float eps, int M, int K, void* h, void* q, float* scales, void* stream) {
  vp_status st = check_rows(x, x_type, ld_x, M, K, 16384, q, scales);
  if (st != VP_OK) return st;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return VP_ERR_INVALID_ARG;
  if (h && h == x && (x_type != VP_BF16 || ld_x != K)) return VP_ERR_INVALID_ARG;
  if ((residual && !al(residual, 16)) || (weight && !al(weight, 4)) || (h && !al(h, 16))) return VP_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = device_sm_count(&sms)) != VP_OK) return st;
  const int chunks = K / 8;
  const int threads = std::min(1024, (chunks + 31) / 32 * 32);
  const bool two = chunks > threads;
  auto* kern = x_type == VP_F32 ? (two ? norm_kernel<true, 2> : norm_kernel<true, 1>)
                                : (two ? norm_kernel<false, 2> : norm_kernel<false, 1>);
  kern<<<(unsigned)M, threads, 0, (cudaStream_t)stream>>>(x, ld_x, static_cast<const uint16_t*>(residual), weight, eps,
                                                          K, static_cast<uint16_t*>(h), static_cast<uint8_t*>(q),
                                                          scales);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VP_OK : cuda_fail(e);
}

}  // extern "C"
