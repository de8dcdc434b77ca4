// Producers of block-scaled e4m3 operands: the weight packer (vp_pack_fp8_block), the quantiser
// (vp_quant_fp8), and the residual addition + RMSNorm with a quantised output (vp_add_rmsnorm_fp8).
//
// Mathematics: a group of 128 values shares s = max(max|x| / 448, 2^-126), so that |x / s| <= 448 up to
// one rounding, and q = e4m3(x * 448 / max|x|), or e4m3(x 2^126) where s is 2^-126.  Of bf16 values, and after a
// norm, the codes are those of the exact quotient (e4m3's half step, 2^-4 of the value, is the only rounding; at
// s = 2^-126 the norm's own rounding comes before); of fp32 values three fp32 roundings come before, which move
// about 1 value in 2^18 across a border between two codes.  Infinities and NaN reach the scale of their group,
// and nothing else.
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
__device__ __forceinline__ void unpack8(uint4 a, float (&v)[8]) {
  unpack_bf16x2(a.x, v[0], v[1]);
  unpack_bf16x2(a.y, v[2], v[3]);
  unpack_bf16x2(a.z, v[4], v[5]);
  unpack_bf16x2(a.w, v[6], v[7]);
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min_abs(float a, float b, float c) {  // of magnitudes (a has no sign); NaN loses
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {  // of the magnitudes, NaN if either is; signs mean nothing
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
constexpr float kScaleFloor = 1.17549435e-38f;  // 2^-126: its reciprocal is finite
// Of a group whose values are f times those at hand, with the maximum m at hand:
// s = max(m f / 448, 2^-126), and the factor r = 448 / m of the values at hand (f 2^126 at the floor).  The
// quotient is the dividend times the constant's reciprocal with its remainder added back (exact in an fma, so
// the result is the rounded quotient); r is the hardware's approximation with one Newton step towards
// 448 / m: about 12 instructions in place of two divisions' 40, in a kernel that issues as much as it loads.
__device__ __forceinline__ void scale_of(float m, float f, float& s, float& r) {
  constexpr float kInv = 1.0f / kE4m3Max, kTiny = kScaleFloor;
  const float mf = m * f, q = mf * kInv;
  s = fmaf(fmaf(-q, kE4m3Max, mf), kInv, q);
  float r0;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(fmaxf(m * kInv, kTiny)));
  r = fmaf(fmaf(-r0, m, kE4m3Max) * kInv, r0, r0);
  if (!(s > kTiny)) {  // NaN is put right below
    s = kTiny;
    r = fminf(f * 8.50705917e37f, 3e38f);  // 2^126; finite, for zeros under a large f
  }
  if (!(mf <= 3.402823466e38f)) s = mf, r = mf == mf ? 0.0f : mf;  // an infinity: finite values over it are 0; NaN
}
// This lane's eight codes of values times r.
__device__ __forceinline__ uint2 codes_of(const float (&v)[8], float r) {
  return make_uint2(e4m3x4(v[0] * r, v[1] * r, v[2] * r, v[3] * r), e4m3x4(v[4] * r, v[5] * r, v[6] * r, v[7] * r));
}
// The largest magnitude of the half warp's 16 x 8 values (one group).
__device__ __forceinline__ float group_max(const float (&v)[8]) {
  const uint32_t half = 0xFFFFu << (threadIdx.x & 16);  // the other half warp may be past the row's end
  float m = max_nan(fabsf(v[0]), fabsf(v[1]));
#pragma unroll
  for (int e = 2; e < 8; e += 2) m = max_nan(m, fabsf(v[e]), fabsf(v[e + 1]));
#pragma unroll
  for (int o = 8; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(half, m, o));
  return m;
}
// The group's scale (returned to every lane) and this lane's codes.
__device__ __forceinline__ float quant_group(const float (&v)[8], uint2& codes) {
  float s, r;
  scale_of(group_max(v), 1.0f, s, r);
  codes = codes_of(v, r);
  return s;
}
// The same of eight bf16 values (times f; m: the largest before that) as loaded: the maximum is taken two at a time.
// Where f is not 1, m lies well inside fp32's range and the scale above the floor, or the result is not used.
__device__ __forceinline__ float quant_group(uint4 w, float f, uint2& codes, float& m) {
  const uint32_t half = 0xFFFFu << (threadIdx.x & 16);
  uint32_t m2 = max_bf16x2(max_bf16x2(w.x, w.y), max_bf16x2(w.z, w.w));
#pragma unroll
  for (int o = 8; o; o >>= 1) m2 = max_bf16x2(m2, __shfl_xor_sync(half, m2, o));
  float s, r, v[8];
  m = max_nan(fabsf(__uint_as_float(m2 << 16)), fabsf(__uint_as_float(m2 & 0xFFFF0000u)));
  scale_of(m, f, s, r);
  unpack8(w, v);
  // Values of 8 bits hit e4m3's ties: x 448 / m is k 2^j with an odd k below 32, or 2^-13 and more away from it.
  // So r a little larger (its error and the product's are below 2^-22) and the product cut to 16 bits give the
  // tie itself, and leave every other value on its side: the codes are those of the exact quotient.
  const uint32_t keep = s > kScaleFloor ? 0xFFFFFF00u : ~0u;  // at the floor r is f over a power of two
  r = s > kScaleFloor ? r * (1.0f + 4.76837158e-7f) : r;      // 2^-21
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(__float_as_uint(v[e] * r) & keep);
  codes = codes_of(v, 1.0f);
  return s;
}

// A half warp takes kU (row, group) pairs in a row, all loads first.  kFlat: whole groups in a dense matrix, so
// the pairs are consecutive in memory and need no row arithmetic.  2051 rows of 17408 in bf16 (108 MB): 21 us
// from memory (5.2 TB/s, of 6.8 that a copy reaches), 19 us when L2 holds a part (23 and 21 with the maximum taken
// over the magnitudes' bits as integers).  The integer pipe bounds it: product, cut and conversion of every value
// are what is left.  One pair each: 29 us before the last steps.  fp32 input (179 MB): 27 us, 6.7 TB/s.
// 4 rows of 6144: 4.2 us, a launch.
template <bool kF32, int kU, bool kFlat>
__global__ void __launch_bounds__(256) quant_kernel(const void* __restrict__ x, long long ld, int M, int K,
                                                    uint8_t* __restrict__ q, float* __restrict__ scales) {
  const int KB = qblocks(K), lane = threadIdx.x & 15;
  const long long n = (long long)M * KB, u0 = ((long long)blockIdx.x * 16 + (threadIdx.x >> 4)) * kU;
  if (u0 >= n) return;
  int m = 0, b = 0;
  if (!kFlat) {
    m = n >> 32 ? (int)(u0 / KB) : (int)((uint32_t)u0 / (uint32_t)KB);
    b = (int)(u0 - (long long)m * KB);
  }
  uint4 w[kU][kF32 ? 2 : 1];
  size_t at[kU];  // of the codes; ~0: nothing there
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    const int k = b * kQBlock + lane * 8;
    bool ok;
    size_t src;
    if (kFlat) {
      ok = u0 + i < n;
      src = (size_t)u0 * kQBlock + lane * 8 + i * kQBlock;
      at[i] = src;
    } else {
      ok = m < M && k < K;
      src = (size_t)m * ld + k;
      at[i] = ok ? (size_t)m * K + k : ~(size_t)0;
      if (++b == KB) b = 0, ++m;
    }
    w[i][0] = w[i][kF32 ? 1 : 0] = make_uint4(0, 0, 0, 0);
    if (!ok) continue;
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) + src * (kF32 ? 4 : 2));
    w[i][0] = __ldg(p);
    if (kF32) w[i][kF32 ? 1 : 0] = __ldg(p + 1);
  }
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    if (u0 + i >= n) break;
    uint2 c;
    float s;
    if constexpr (kF32) {
      const uint4 a = w[i][0], d = w[i][1];
      const float v[8] = {__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w),
                          __uint_as_float(d.x), __uint_as_float(d.y), __uint_as_float(d.z), __uint_as_float(d.w)};
      s = quant_group(v, c);
    } else {
      float m;
      s = quant_group(w[i][0], 1.0f, c, m);
    }
    if (kFlat || at[i] != ~(size_t)0) *reinterpret_cast<uint2*>(q + at[i]) = c;
    if (lane == 0) scales[u0 + i] = s;
  }
}

// The border between two e4m3 codes that lies nearest above or below t >= 0 (to some steps of fp32): the middle
// of the normal codes' interval is where the lower 20 bits read 0x80000.  The codes below 2^-6 lie 2^-9 apart, as
// those from there to 2^-5 do, so adding 2^-6 makes them look alike.
__device__ __forceinline__ float border_of(float t) {
  const bool sub = t < 0.015625f;
  const float s = sub ? fminf(t + 0.015625f, 0.031249998f) : t;  // below 2^-5
  const float b = __uint_as_float((__float_as_uint(s) & 0xFFF00000u) | 0x80000u);
  return sub ? b - 0.015625f : b;
}
// The codes of a group of values h w (eight per lane, weights at w; 0 past the row), for the groups that fp32 does
// not decide.  y = hi + lo and the maximum m + ml are exact pairs, and 448 y is compared with (m + ml) times the
// border at hand (both over 512, so that nothing overflows).  The values have 35 and 37 bits: where they differ
// they do so by 2^-37 of themselves and more, and what the sum below rounds is under 2^-46 of them where they
// agree; so the sign is the exact one, a tie is one, and e4m3's rounding the only one.
__device__ __forceinline__ uint2 codes_pair(uint4 a, const float* w, bool valid) {
  const uint32_t half = 0xFFFFu << (threadIdx.x & 16);
  float hi[8], lo[8], ml = 0.0f;
  unpack8(a, hi);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = hi[e], g = valid ? __ldg(w + e) : 0.0f;
    hi[e] = __fmul_rn(x, g);
    lo[e] = fmaf(x, g, -hi[e]);
  }
  float m = group_max(hi);
  const float r = m > 0.0f ? kE4m3Max / m : 0.0f;  // the other half warp's group may be the open one, and this one zero
  ml = -m;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (fabsf(hi[e]) == m) ml = fmaxf(ml, copysignf(1.0f, hi[e]) * lo[e]);
#pragma unroll
  for (int o = 8; o; o >>= 1) ml = fmaxf(ml, __shfl_xor_sync(half, ml, o));
  m *= 0.001953125f, ml *= 0.001953125f;  // 1 / 512
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // 448 / 512; products that the compiler does not fuse with what follows
    const float h = fabsf(hi[e]), b = border_of(h * r), x = __fmul_rn(h, 0.875f), y = __fmul_rn(b, m);
    const float rest = (x - y) + ((fmaf(h, 0.875f, -x) - fmaf(b, m, -y)) +
                                  fmaf(hi[e] < 0.0f ? -lo[e] : lo[e], 0.875f, -__fmul_rn(b, ml)));
    const int up = fabsf(rest) <= y * 2.27373675e-13f ? 0 : rest > 0.0f ? 1 : -1;  // 2^-42
    hi[e] = copysignf(__int_as_float(__float_as_int(b) + up), hi[e]);
  }
  return codes_of(hi, 1.0f);
}

// h: the sum, rounded to fp32, then to the residual stream's bf16.
__device__ __forceinline__ uint4 residual_sum(float (&v)[8], uint4 r) {
  float t[8];
  unpack8(r, t);
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * e] + t[2 * e], v[2 * e + 1] + t[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A chunk of the residual stream again, from memory: h where it was written, else the inputs (which then still
// stand).  What follows is rare, and kept apart so that the ordinary path holds no registers for it.
template <bool kF32>
__device__ __forceinline__ uint4 reload(const void* x, long long at_x, const uint16_t* residual, const uint16_t* h, size_t at) {
  if (h) return *reinterpret_cast<const uint4*>(h + at);
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) + at_x * (kF32 ? 4 : 2));
  const uint4 b = p[0];
  float v[8];
  if (kF32) {
    const uint4 c = p[1];
    const uint32_t u[8] = {b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(u[e]);
  } else {
    unpack8(b, v);
  }
  constexpr uint32_t kNone = 0x80008000u;  // -0: adding it leaves a zero's sign, too
  return residual_sum(v, residual ? *reinterpret_cast<const uint4*>(residual + at) : make_uint4(kNone, kNone, kNone, kNone));
}
// The group of this lane's chunk `a` in fp64; w: the chunk's weights, or NULL.  h w has 32 bits, so it, 448 h w and
// its maximum are exact; the product with 448 / m is off by less than 2^-51, ties lie in 5 bits and every other
// quotient 2^-37 away from them, so rounding it to 41 bits gives each its side.  It is then cut to fp32 with a last
// bit for what was cut, and e4m3's rounding decides.  (At the scale's floor the values carry the row's factor and
// its rounding.)  Few fp64 operations, the rest on the bits: 4099 rows of 5120 that all come here take 0.67 ms.
__device__ __noinline__ void group64(uint4 a, const float* w, double inv, bool valid, uint8_t* q, float* scale) {
  const uint32_t half = 0xFFFFu << (threadIdx.x & 16);
  float v[8], s;
  uint2 c;
  unpack8(a, v);
  const bool some = ((a.x | a.y | a.z | a.w) & 0x7FFF7FFFu) != 0;
  if (__any_sync(half, some) || !(fabs(inv) <= 1e300)) {
    auto product = [&](int e) -> double {  // of v[0], the lane's value e; rotating, so that the loops stay loops
      return (double)v[0] * (double)(valid && w ? __ldg(w + e) : 1.0f);
    };
    auto rotate = [&](float x) {
#pragma unroll
      for (int i = 0; i < 7; ++i) v[i] = v[i + 1];
      v[7] = x;
    };
    unsigned long long top = 0;  // the largest magnitude's bits: NaN above infinity above the finite ones
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
      top = max(top, (unsigned long long)__double_as_longlong(product(e)) & ~(1ull << 63));
      rotate(v[0]);
    }
#pragma unroll 1
    for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(half, top, o));
    const double m = __longlong_as_double((long long)top), ym = m * inv, sd = ym / (double)kE4m3Max;
    const bool least = !(sd > (double)kScaleFloor), none = !(ym <= 1.7e308);  // infinite, or no value
    s = none ? (float)ym : least ? kScaleFloor : (float)sd;
    const double r = none ? 1.0 / ym : least ? inv * 8.507059173023462e37 : (double)kE4m3Max / m;  // 2^126
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
      const double t = product(e) * r;
      const long long bits = (__double_as_longlong(t) + 0x800) & ~0xFFFll;
      const float f = __double2float_rz(__longlong_as_double(bits));
      // finite values over an infinity are 0, the others NaN
      rotate(none ? (float)t : (bits & 0x1FFFFFFF) ? __int_as_float(__float_as_int(f) | 1) : f);
    }
    c = codes_of(v, 1.0f);
  } else {  // zeros (a padding row's): theirs, or a NaN weight's
    if (valid && w)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= __ldg(w + e);
    s = quant_group(v, c);
  }
  if (valid) *reinterpret_cast<uint2*>(q) = c;
  if ((threadIdx.x & 15) == 0) *scale = s;
}
// The chunk at column k of row m again: its codes from pairs of floats; all of it in fp64 where the products
// or the scale leave fp32's range (`far`).
template <bool kF32>
__device__ __noinline__ void redo_chunk(const void* x, long long ld, const uint16_t* residual, const float* weight, int m,
                                        int k, int K, const uint16_t* h, float inv, bool far, uint8_t* q, float* scale) {
  const bool valid = k < K;
  const size_t at = (size_t)m * K + k;
  const uint4 a = valid ? reload<kF32>(x, m * ld + k, residual, h, at) : make_uint4(0, 0, 0, 0);
  if (far) {
    group64(a, weight ? weight + k : nullptr, inv, valid, q + at, scale);
  } else if (weight) {  // without weights: the other half warp's group is the one
    const uint2 c = codes_pair(a, weight + k, valid);
    if (valid) *reinterpret_cast<uint2*>(q + at) = c;
  }
}
// A row whose squares leave fp32's range (or a zero or NaN row): all of it in fp64.
template <bool kF32>
__device__ __noinline__ void redo_row(const void* x, long long ld, const uint16_t* residual, const float* weight, int m,
                                      int K, const uint16_t* h, float eps, uint8_t* q, float* scales, double* red) {
  double sum = 0.0;
#pragma unroll 1
  for (int k = threadIdx.x * 8; k < K; k += blockDim.x * 8) {
    float v[8];
    const uint4 a = reload<kF32>(x, m * ld + k, residual, h, (size_t)m * K + k);
    if (((a.x | a.y | a.z | a.w) & 0x7FFF7FFFu) == 0) continue;
    unpack8(a, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += (double)v[e] * (double)v[e];
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = 0.0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) sum += red[w];
  const double inv = 1.0 / sqrt(sum / (double)K + (double)eps);
#pragma unroll 1
  for (int k = threadIdx.x * 8; (k & ~127) < K; k += blockDim.x * 8) {
    const bool valid = k < K;
    const size_t at = (size_t)m * K + k;
    group64(valid ? reload<kF32>(x, m * ld + k, residual, h, at) : make_uint4(0, 0, 0, 0), weight ? weight + k : nullptr,
            inv, valid, q + at, scales + (size_t)m * qblocks(K) + k / kQBlock);
  }
}

// One CTA per row, kC chunks of 8 values per thread, held in registers as the bf16 pairs that the residual
// stream is rounded to: one pass over the data, every load issued before the first use.  Many rows: four
// chunks per thread, so that an SM holds several rows' CTAs and 100 KB and more of loads in flight while
// others reduce; few rows: one chunk per thread, the shortest path through a row.  4099 rows of 5120 in bf16
// with a residual (148 MB) from memory, by the weights: random 24-bit ones 31.6 us (32.8 between other work), 4.7 TB/s of the 6.8 that a copy
// reaches (fp32 input 35.3, 5.4 TB/s); none 26.8; bf16 ones (as checkpoints hold them), whose products with bf16
// values meet e4m3's ties, 35 to 38; all one 51.  Looking at the borders below 2^-6 costs 0.7 us of these.  With
// the rare paths inline, over chunks held in registers, 33 us; two chunks per thread 33 us; a resident grid that
// copies a row ahead into shared memory 37 us (fewer warps to hide a row's reductions).  8 rows: 4.6 us, 1.4 more if
// one of them has an open group; 4.2 us is a launch.
template <bool kF32, int kC>
__global__ void __launch_bounds__(1024) norm_kernel(const void* x, long long ld, const uint16_t* residual,
                                                    const float* __restrict__ weight, int vec, float eps, float ss_max, int K,
                                                    uint16_t* h, uint8_t* __restrict__ q, float* __restrict__ scales) {
  __shared__ float red[32];
  __shared__ double redd[32];
  const int m = blockIdx.x, tid = threadIdx.x, step = blockDim.x * 8, KB = qblocks(K), warps = blockDim.x >> 5;
  const int k0 = tid * 8;  // the thread's first chunk; the others follow at `step`
  const uint8_t* px = static_cast<const uint8_t*>(x) + ((size_t)m * ld + k0) * (kF32 ? 4 : 2);
  const size_t row = (size_t)m * K + k0;
  uint4 a[kC], b[kF32 ? kC : 1], r[kC];
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    a[i] = r[i] = make_uint4(0, 0, 0, 0);
    if (kF32) b[i] = make_uint4(0, 0, 0, 0);
    if (k0 + i * step >= K) continue;
    const uint4* p = reinterpret_cast<const uint4*>(px + i * step * (kF32 ? 4 : 2));
    a[i] = p[0];
    if (kF32) b[i] = p[1];
    if (residual) r[i] = *reinterpret_cast<const uint4*>(residual + row + i * step);
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const int k = k0 + i * step;
    float v[8];
    if (kF32) {
      const uint32_t w[8] = {a[i].x, a[i].y, a[i].z, a[i].w, b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
    } else {
      unpack8(a[i], v);
    }
    if (residual) {
      float t[8];
      unpack8(r[i], t);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += t[e];
    }
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);  // the residual stream is bf16
      w[e] = *reinterpret_cast<const uint32_t*>(&p);
    }
    a[i] = make_uint4(w[0], w[1], w[2], w[3]);
    if (h && k < K) *reinterpret_cast<uint4*>(h + row + i * step) = a[i];
    unpack8(a[i], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
  if ((tid & 31) == 0) red[tid >> 5] = ss;
  __syncthreads();
  ss = 0.0f;
  for (int w = 0; w < warps; ++w) ss += red[w];
  const float* pw = weight + k0;
  if (ss >= 1e-30f && ss <= ss_max) {
    const float inv = 1.0f / sqrtf(ss / (float)K + eps);
    // The values at hand are h w: the row's factor cancels from the codes and enters the scales only.
    unsigned open = 0, far = 0;  // chunks of the thread that fp32 leaves open, or that leave its range
    auto outside = [&](float most, float s) {  // NaN too; a group of zeros is done
      return most != 0.0f && !(most >= 1e-25f && most <= 1e30f && s > 2.0f * kScaleFloor);
    };
    if (!weight) {
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        const int k = k0 + i * step;
        if ((k & ~127) >= K) break;  // uniform over the half warp
        uint2 c;
        float most;
        const float s = quant_group(a[i], inv, c, most);
        if (outside(most, s)) far |= 1u << i;
        if (k < K) *reinterpret_cast<uint2*>(q + row + i * step) = c;
        if ((tid & 15) == 0) scales[(size_t)m * KB + k / kQBlock] = s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        const int k = k0 + i * step;
        if ((k & ~127) >= K) break;
        float v[8];
        unpack8(a[i], v);
        if (k < K) {
          if (vec) {
            const float4 c = __ldg(reinterpret_cast<const float4*>(pw + i * step)), d = __ldg(reinterpret_cast<const float4*>(pw + i * step) + 1);
            v[0] *= c.x, v[1] *= c.y, v[2] *= c.z, v[3] *= c.w, v[4] *= d.x, v[5] *= d.y, v[6] *= d.z, v[7] *= d.w;
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= __ldg(pw + i * step + e);
          }
        }
        float s, r;
        const float most = group_max(v);
        scale_of(most, inv, s, r);
        // Products within 5 steps of fp32 of a border of e4m3's (see border_of): three fp32 roundings leave those
        // open.  The borders below 2^-6 are looked at only where a value lies there (normal values: 2 % of the warps).
        unsigned near = ~0u;
        float least = 1.0f;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          v[e] *= r, v[e + 1] *= r;
          near = __vimin3_u32(near, (__float_as_uint(v[e]) << 12) - (0x7FFFBu << 12), (__float_as_uint(v[e + 1]) << 12) - (0x7FFFBu << 12));
          least = min_abs(least, v[e], v[e + 1]);
        }
        if (least < 0.015625f) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float t = fabsf(v[e]);
            if (t < 0.015625f) near = min(near, (__float_as_uint(t + 0.015625f) << 12) - (0x7FFFBu << 12));
          }
        }
        const uint2 c = codes_of(v, 1.0f);
        if (near <= 10u << 12) open |= 1u << i;
        if (most == 0.0f || outside(most, s)) far |= 1u << i;  // zero, or lost
        if (k < K) *reinterpret_cast<uint2*>(q + row + i * step) = c;
        if ((tid & 15) == 0) scales[(size_t)m * KB + k / kQBlock] = s;
      }
    }
    open = __reduce_or_sync(0xFFFFFFFFu, open | far);
#pragma unroll 1
    for (int i = 0; open >> i; ++i) {  // 1 group in 760 with random 24-bit weights, 1 in 16 to 26 with bf16 ones
      const int k = k0 + i * step;
      if (!(open >> i & 1) || (k & ~127) >= K) continue;
      redo_chunk<kF32>(x, ld, residual, weight, m, k, K, h, inv, far >> i & 1, q, scales + (size_t)m * KB + k / kQBlock);
    }
    return;
  }
  redo_row<kF32>(x, ld, residual, weight, m, K, h, eps, q, scales, redd);
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
  const bool wide = x_type == VP_F32, many = n >= 512LL * sms;  // enough pairs to fill the SMs four at a time
  const long long per = many ? 64 : 16, blocks = (n + per - 1) / per;
  const bool flat = ld_x == K && K % kQBlock == 0;
  auto* kern = !many ? (wide ? quant_kernel<true, 1, false> : quant_kernel<false, 1, false>)
               : flat ? (wide ? quant_kernel<true, 4, true> : quant_kernel<false, 4, true>)
                      : (wide ? quant_kernel<true, 4, false> : quant_kernel<false, 4, false>);
  kern<<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(x, ld_x, M, K, static_cast<uint8_t*>(q), scales);
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
  const int per = M >= 2 * sms ? 4 : chunks > 1024 ? 2 : 1;
  const int threads = (chunks + 32 * per - 1) / (32 * per) * 32;
  const bool wide = x_type == VP_F32;
  const float ss_max = eps <= 1e37f ? 3.0e38f : 0.0f;  // up to here the sum of squares, and the mean plus eps, are finite
  auto* kern = per == 4 ? (wide ? norm_kernel<true, 4> : norm_kernel<false, 4>)
                        : per == 2 ? (wide ? norm_kernel<true, 2> : norm_kernel<false, 2>)
                                   : (wide ? norm_kernel<true, 1> : norm_kernel<false, 1>);
  kern<<<(unsigned)M, threads, 0, (cudaStream_t)stream>>>(x, ld_x, static_cast<const uint16_t*>(residual), weight,
                                                          al(weight, 16), eps, ss_max, K, static_cast<uint16_t*>(h),
                                                          static_cast<uint8_t*>(q), scales);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VP_OK : cuda_fail(e);
}

}  // extern "C"
