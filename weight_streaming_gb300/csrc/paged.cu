// New rows into a paged KV cache with the attention layer's Q/K norm and rotary embedding on the way
// (vp_paged_append), and into an 8-bit one (vp_paged_append_fp8).
//
// Mathematics: per head, y = x / sqrt(mean x^2 + eps) * w (optional), then the pairs of the first rot_dim
// elements turn by the angle pos * f_j.  Only the angle modulo one turn matters, and pos is an integer:
// the host gives f_j / 2 pi modulo 1 as a 64-bit binary fraction F_j, and pos * F_j wraps around 2^64
// by itself to the fraction of a turn -- exact but for F_j's own rounding (2^-54 of a turn per
// position: 3e-8 of a turn at 2^29 positions), with one integer product and no fp64.
//
// D / 8 lanes hold one head, each both elements of its four pairs; the sum of squares comes by shuffles.  A
// block serves one row and a group of heads; its sines and cosines are formed once.  The bytes bound it for
// prompts (each read and written once), the latency of one load, the reduction and one store for single
// tokens.  6001 rows of 48 x 128 heads (147 MB): 26 us, 5.6 TB/s of the 6.8 that a copy reaches (29 us when
// the norm's code stands in the same kernel: its instructions outgrow their cache), 37 us with Q/K norms; of 32 x
// 256 heads with Q/K norms (197 MB) 65 us; 48 rows of 32 x 256 heads: 6.2 us.
//
// Into 8 bits 6001 rows of 32 + 16 x 128 heads (135 MB) take 60 us, 2.3 TB/s: instructions, at 88 registers a quarter of the warp
// slots (one to three heads per group of lanes: 75, 67, 62 us), and the heads that are formed again in fp64 for an open code.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "errors.h"
#include "paged.h"
#include "ptx.cuh"
#include "verify.h"

namespace vp {

namespace {

constexpr int kThreadsP = 128;
constexpr int kMaxPairs = 128;

struct AppendArgs {
  const uint16_t *q, *k, *v;
  long long ld_q, ld_k, ld_v;
  const float *q_norm, *k_norm;
  float eps;
  int rot, interleaved;
  const int32_t *row_start, *ctx, *pages;
  int S, M, Hq, Hkv, n_pages, log_page, max_pages;
  void *k_cache, *v_cache;
  uint8_t *k_scales, *v_scales;  // 8-bit cache
  uint16_t* q_out;
  int32_t* kv_len;
  int* status;
  unsigned long long turn[kMaxPairs];  // f_j / 2 pi mod 1, in units of 2^-64
};

__device__ __forceinline__ void unpack8(uint4 a, float (&v)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(w[e] << 16);
    v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The sequence whose rows hold row r (the last s with row_start[s] <= r), or -1 for a padding row.
__device__ __forceinline__ int find_seq(const int32_t* start, int S, int r) {
  if (r < start[0] || r >= start[S]) return -1;
  int lo = 0, hi = S;  // start[lo] <= r; the answer lies in [lo, hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= r) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __noinline__ double square64(float v) { return (double)v * (double)v; }
__device__ __noinline__ float scale64(float v, double s, float w) { return (float)((double)v * s * (double)w); }

// One head over its root mean square, times the weights at w0 (first four values) and w1; kL lanes hold 8 values each.
template <int kL>
__device__ __forceinline__ void norm_head(float (&x)[8], const float* w0, const float* w1, float eps, uint32_t mask) {
  float ss = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
  for (int o = kL / 2; o; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
  if (ss >= 1e-30f && ss <= 3.0e38f && eps <= 1e37f) {  // the mean plus eps is finite
    const float inv = 1.0f / sqrtf(ss / (float)(8 * kL) + eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * __ldg(e < 4 ? w0 + e : w1 + e - 4);
  } else {  // squares outside fp32's range (or a zero or NaN head): fp64, in calls so that no other head pays for it
    double sd = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) sd += square64(x[e]);
#pragma unroll
    for (int o = kL / 2; o; o >>= 1) sd += __shfl_xor_sync(mask, sd, o);
    const double id = 1.0 / sqrt(sd / (double)(8 * kL) + (double)eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = scale64(x[e], id, __ldg(e < 4 ? w0 + e : w1 + e - 4));
  }
}
__device__ __forceinline__ void turn(float& x0, float& x1, float c, float s) {
  const float a = x0, b = x1;
  x0 = fmaf(a, c, -(b * s));
  x1 = fmaf(a, s, b * c);
}

// ------------------------------------------------------------------ the 8-bit cache
// A head's codes are e4m3(x / 2^e), e the smallest exponent (from kMinExp on) with max |x| <= 448 2^e: the power of two
// costs at most one of e4m3's 17 binades and no digit, and code * 2^e is a bf16 value, so that reading the cache back
// rounds nothing.
constexpr int kMinExp = -118;    // codes times 2^-118 are bf16 values down to e4m3's smallest, 2^-9
// What fp32 may be off by, of a pair's length: the angle as a fraction of a half turn pi u / 2, sine and cosine 2 u each, products
// and sum 2 u (u = 2^-24): below 8 u; the norm 20 u more.
constexpr float kOpenTurn = 0x1p-21f, kOpenNorm = 0x1p-19f;

// e of a maximum by its bits: max = f 2^E, 1/2 <= f < 1, against 448 = 7/8 2^9.
__device__ __forceinline__ int scale_exp(uint32_t bits) {
  return max((int)(bits >> 23) - 126 - 9 + ((bits & 0x7FFFFF) > 0x600000), kMinExp);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The head again in fp64, for heads whose scale or a code fp32 leaves open (next to 448 2^e, or half way between two codes):
// the exact value's codes and exponent.  rows: raw bf16; w0, w1: weights or NULL; turn0: the row's first turn for this
// lane's pairs (NULL: not turned); split: pairs (j, j + 4) of the lane's eight, else neighbours.
template <int kL>
__device__ __noinline__ int quant64(uint4 raw, const float* w0, const float* w1, float eps, const unsigned long long* turns,
                                    unsigned long long pos, bool split, uint32_t mask, uint2& codes) {
  double x[8];
  const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) x[2 * k] = __uint_as_float(in[k] << 16), x[2 * k + 1] = __uint_as_float(in[k] & 0xFFFF0000u);
  if (w0) {
    double ss = 0.0;
#pragma unroll
    for (int k = 0; k < 8; ++k) ss += x[k] * x[k];
#pragma unroll
    for (int o = kL / 2; o; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
    const double inv = 1.0 / sqrt(ss / (8 * kL) + (double)eps);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = x[k] * inv * (double)__ldg(k < 4 ? w0 + k : w1 + k - 4);
  }
  if (turns) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      double s, c;
      sincospi((double)(long long)(pos * turns[j]) * 0x1p-63, &s, &c);
      double &p = x[split ? j : 2 * j], &q = x[split ? j + 4 : 2 * j + 1];
      const double u = p, v = q;
      p = u * c - v * s;
      q = u * s + v * c;
    }
  }
  double top = 0.0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = fmax(top, fabs(x[k]));
#pragma unroll
  for (int o = kL / 2; o; o >>= 1) top = fmax(top, __shfl_xor_sync(mask, top, o));
  const long long b = __double_as_longlong(top);
  const int e = max((int)(b >> 52) - 1022 - 9 + ((b & 0xFFFFFFFFFFFFFLL) > 0xC000000000000LL), kMinExp);
  const double inv = __longlong_as_double((long long)(1023 - e) << 52);
  float y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {  // rounded once, to a multiple of the step at its size
    const double v = x[k] * inv;
    const int n = max((int)(__double_as_longlong(fabs(v)) >> 52) - 1023, -6) - 3;
    y[k] = (float)(rint(v * __longlong_as_double((long long)(1023 - n) << 52)) * __longlong_as_double((long long)(1023 + n) << 52));
  }
  codes.x = e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16;
  codes.y = e4m3x2(y[4], y[5]) | e4m3x2(y[6], y[7]) << 16;
  return e;
}

// Eight codes of a lane and, by the head's first lane, the exponent (128: NaN).
__device__ __forceinline__ void store8(const AppendArgs& a, void* cache, uint8_t* scales, int h, int page, long long pos, int off0,
                                       int off1, int lane, int D, uint2 codes, int ex) {
  const size_t at = (((size_t)page * a.Hkv + h) << a.log_page) + (pos & ((1 << a.log_page) - 1));
  uint8_t* dst = static_cast<uint8_t*>(cache) + at * D;
  *reinterpret_cast<uint32_t*>(dst + off0) = codes.x;
  *reinterpret_cast<uint32_t*>(dst + off1) = codes.y;
  if (lane == 0) scales[at] = (uint8_t)(ex + 127);
}

// kB: heads per group of lanes.  Every load of the block's heads is issued first: they depend on nothing
// that the row's position has to be looked up for.
template <int D, int kB, bool kNorm, bool kFp8>
__global__ void __launch_bounds__(kThreadsP) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kL = D / 8;                    // lanes per head
  constexpr int kGroups = kThreadsP / kL;      // heads at a time
  __shared__ __align__(16) float s_cos[kMaxPairs], s_sin[kMaxPairs];
  const int r = blockIdx.x, tid = threadIdx.x;
  const int lane = tid & (kL - 1), nq = a.q ? a.Hq : 0, heads = nq + 2 * a.Hkv;
  const int h0 = blockIdx.y * kB * kGroups + tid / kL;
  // A lane's eight values: two runs of four.  Half-split pairs: elements 4 l .. and half + 4 l .. for the lanes of
  // the rotated part, so that both elements of a pair are the lane's own; else eight in a row.
  const int half = a.rot >> 1, rl = half >> 2;  // rl: lanes of the rotated part (both pairings)
  const bool turns = lane < rl, split = turns && !a.interleaved;
  const int off0 = split ? 4 * lane : 8 * lane, off1 = split ? half + 4 * lane : 8 * lane + 4;
  // the row's arrays, each as if its heads had the numbers that they have here (q, then k, then v)
  const uint16_t* q_row = a.q + (size_t)r * a.ld_q;
  const uint16_t* k_row = a.k + (ptrdiff_t)r * a.ld_k - nq * D;
  const uint16_t* v_row = a.v + (ptrdiff_t)r * a.ld_v - (nq + a.Hkv) * D;
  uint4 raw[kB];
#pragma unroll
  for (int i = 0; i < kB; ++i) {
    const int hh = h0 + i * kGroups;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (hh >= heads) continue;
    const uint16_t* src = (hh < nq ? q_row : hh < nq + a.Hkv ? k_row : v_row) + hh * D;
    const uint2 u = *reinterpret_cast<const uint2*>(src + off0), v = *reinterpret_cast<const uint2*>(src + off1);
    raw[i] = make_uint4(u.x, u.y, v.x, v.y);
  }
  // the lengths after this call, by the first blocks
  if (a.kv_len && blockIdx.y == 0) {
    for (long long s = (long long)r * kThreadsP + tid; s < a.S; s += (long long)gridDim.x * kThreadsP) {
      const long long n = a.row_start ? (long long)a.row_start[s + 1] - a.row_start[s] : 1;
      a.kv_len[s] = (int32_t)min((long long)a.ctx[s] + n, 0x7FFFFFFFLL);
    }
  }
  if (a.row_start && r == 0 && blockIdx.y == 0 && tid == 0 && a.status && (a.row_start[0] < 0 || a.row_start[a.S] > a.M))
    report_unless(a.status, VP_ERR_SHAPE, VP_ERR_TIMEOUT);  // rows that this call does not have
  int s = r;
  if (a.row_start) {
    if (a.S <= 2 * kThreadsP) {  // the number of sequences that start at or before the row: two loads for all
      s = -1 + __syncthreads_count(tid < a.S && a.row_start[tid] <= r);
      if (a.S > kThreadsP) s += __syncthreads_count(tid + kThreadsP < a.S && a.row_start[tid + kThreadsP] <= r);
      if (s >= 0 && r >= a.row_start[a.S]) s = -1;
    } else {
      s = find_seq(a.row_start, a.S, r);
    }
  }
  if (s < 0) return;
  const long long pos = (long long)a.ctx[s] + (a.row_start ? r - a.row_start[s] : 0);
  int page = -1;
  if (pos >= 0 && (pos >> a.log_page) < a.max_pages) page = a.pages[(size_t)s * a.max_pages + (pos >> a.log_page)];
  for (int j = tid; j < half; j += kThreadsP) {
    const unsigned long long f = (unsigned long long)pos * a.turn[j];
    // the nearest signed fraction of a turn, in half turns
    sincospif((float)(int32_t)(f >> 32) * 4.656612873077393e-10f, &s_sin[j], &s_cos[j]);
  }
  const bool ok = page >= 0 && page < a.n_pages;
  if (!ok && tid == 0 && blockIdx.y == 0 && a.status) report_unless(a.status, VP_ERR_SHAPE, VP_ERR_TIMEOUT);
  __syncthreads();
  float4 cs = make_float4(1.0f, 1.0f, 1.0f, 1.0f), sn = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (turns) {  // of pairs 4 lane .. 4 lane + 3, the same for every head
    cs = *reinterpret_cast<const float4*>(s_cos + 4 * lane);
    sn = *reinterpret_cast<const float4*>(s_sin + 4 * lane);
  }
  if (!ok) {  // nothing to append; the row's queries are zero
    for (int hh = h0, i = 0; i < kB && hh < nq; ++i, hh += kGroups)
      *reinterpret_cast<uint4*>(a.q_out + ((size_t)r * a.Hq + hh) * D + 8 * lane) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int head_step = D << a.log_page;  // from one head's slot to the next one's in a page
  const ptrdiff_t slot = (((ptrdiff_t)page * a.Hkv << a.log_page) + (pos & ((1 << a.log_page) - 1))) * D;
  uint16_t* q_dst = a.q_out + (size_t)r * a.Hq * D;
  uint16_t* k_dst = static_cast<uint16_t*>(a.k_cache) + (slot - (ptrdiff_t)nq * head_step);
  uint16_t* v_dst = static_cast<uint16_t*>(a.v_cache) + (slot - (ptrdiff_t)(nq + a.Hkv) * head_step);
  const uint32_t mask = kL == 32 ? 0xFFFFFFFFu : ((1u << (kL & 31)) - 1) << ((tid & 31) & ~(kL - 1));
#pragma unroll
  for (int i = 0; i < kB; ++i) {
    const int hh = h0 + i * kGroups;
    if (hh >= heads) break;
    const bool isq = hh < nq, isk = !isq && hh < nq + a.Hkv;
    uint16_t* dst = isq ? q_dst + hh * D : (isk ? k_dst : v_dst) + (ptrdiff_t)hh * head_step;
    uint4 out = raw[i];
    const float* w = !kNorm ? nullptr : isq ? a.q_norm : isk ? a.k_norm : nullptr;
    // (8-bit keys: all lanes of a head together, as they share its maximum)
    if ((isq || isk) && (w || turns || (kFp8 && isk && a.rot))) {
      float x[8];
      unpack8(raw[i], x);
      if (kNorm && w) norm_head<kL>(x, w + off0, w + off1, a.eps, mask);
      if (split) {
        turn(x[0], x[4], cs.x, sn.x);
        turn(x[1], x[5], cs.y, sn.y);
        turn(x[2], x[6], cs.z, sn.z);
        turn(x[3], x[7], cs.w, sn.w);
      } else if (turns) {
        turn(x[0], x[1], cs.x, sn.x);
        turn(x[2], x[3], cs.y, sn.y);
        turn(x[4], x[5], cs.z, sn.z);
        turn(x[6], x[7], cs.w, sn.w);
      }
      if (kFp8 && isk) {
        // codes and exponent, and whether what fp32 may be off by could change one of them
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
        top = __reduce_max_sync(mask, top);
        int ex = scale_exp(top);
        const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
        const float off = kNorm ? kOpenNorm : turns ? kOpenTurn : 0.0f;
        bool open = false;
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int p = split ? e : 2 * e, q = split ? e + 4 : 2 * e + 1;  // a pair
          const float d = (fabsf(x[p]) + fabsf(x[q])) * off;
          lo[e] = e4m3x2((x[p] - d) * inv, (x[q] - d) * inv);
          hi[e] = e4m3x2((x[p] + d) * inv, (x[q] + d) * inv);
          open = open || lo[e] != hi[e];
        }
        // 64 fp32 steps are 2^-18 to 2^-17 of the maximum, more than it may be off by (a pair's length is at most sqrt 2 of it)
        open = open || scale_exp(top - min(top, 64u)) != scale_exp(top + 64u);
        uint2 codes;
        if (split) {
          codes.x = __byte_perm(__byte_perm(lo[0], lo[1], 0x0040), __byte_perm(lo[2], lo[3], 0x0040), 0x5410);
          codes.y = __byte_perm(__byte_perm(lo[0], lo[1], 0x0051), __byte_perm(lo[2], lo[3], 0x0051), 0x5410);
        } else {
          codes.x = lo[0] | lo[1] << 16, codes.y = lo[2] | lo[3] << 16;
        }
        if (top >= 0x7F800000u) {  // a value that is none: the head is none
          codes = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu), ex = 128;
        } else if (__any_sync(mask, open)) {
          ex = quant64<kL>(raw[i], w ? w + off0 : nullptr, w ? w + off1 : nullptr, a.eps, turns ? a.turn + 4 * lane : nullptr,
                           (unsigned long long)pos, split, mask, codes);
        }
        store8(a, a.k_cache, a.k_scales, hh - nq, page, pos, off0, off1, lane, D, codes, ex);
        continue;
      }
      out = pack8(x);
    }
    if (kFp8 && !isq) {  // values, or keys as they came: exact in fp32
      float x[8];
      unpack8(raw[i], x);
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
      top = __reduce_max_sync(mask, top);
      int ex = scale_exp(top);
      const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
      uint2 codes = make_uint2(e4m3x2(x[0] * inv, x[1] * inv) | e4m3x2(x[2] * inv, x[3] * inv) << 16,
                               e4m3x2(x[4] * inv, x[5] * inv) | e4m3x2(x[6] * inv, x[7] * inv) << 16);
      if (top >= 0x7F800000u) codes = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu), ex = 128;
      store8(a, isk ? a.k_cache : a.v_cache, isk ? a.k_scales : a.v_scales, isk ? hh - nq : hh - nq - a.Hkv, page, pos, off0,
             off1, lane, D, codes, ex);
      continue;
    }
    *reinterpret_cast<uint2*>(dst + off0) = make_uint2(out.x, out.y);
    *reinterpret_cast<uint2*>(dst + off1) = make_uint2(out.z, out.w);
  }
}

bool al(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace

vp_status check_cache(const vp_paged_cache* c) {
  if (!c || !c->k || !c->v || !c->pages) return VP_ERR_INVALID_ARG;
  const int P = c->page_size;
  if ((c->D != 64 && c->D != 128 && c->D != 256) || (P != 16 && P != 32 && P != 64 && P != 128) || c->Hkv < 1 ||
      c->Hkv > 1024 || c->n_pages < 1 || c->max_pages < 1 || (long long)c->n_pages * c->Hkv * P >= (1LL << 31) ||
      (long long)c->max_pages * P >= (1LL << 31))
    return VP_ERR_SHAPE;
  if (!al(c->k, 16) || !al(c->v, 16) || !al(c->pages, 4)) return VP_ERR_ALIGNMENT;
  return VP_OK;
}

}  // namespace vp

using namespace vp;

namespace {

// Both appends; the cache is checked.
template <bool kFp8>
vp_status append(const vp_paged_cache& c, uint8_t* k_scales, uint8_t* v_scales, const void* q, int64_t ld_q, const void* k,
                 int64_t ld_k, const void* v, int64_t ld_v, const float* q_norm, const float* k_norm, float eps,
                 const vp_rope* rope, const int32_t* row_start, const int32_t* ctx, int S, int M, int Hq, void* q_out,
                 int32_t* kv_len, int* status, void* stream) {
  vp_status st;
  if (!k || !v || !ctx || (q && !q_out) || kv_len == ctx) return VP_ERR_INVALID_ARG;
  if ((q_norm || k_norm) && !(eps > 0.0f && std::isfinite(eps))) return VP_ERR_INVALID_ARG;
  if (M < 1 || M > (1 << 24) || S < 1 || S > 65536 || (!row_start && M != S)) return VP_ERR_SHAPE;
  const long long kd = (long long)c.Hkv * c.D, qd = (long long)Hq * c.D;
  if (ld_k < kd || ld_v < kd || ld_k > (1LL << 40) || ld_v > (1LL << 40)) return VP_ERR_SHAPE;
  if (q && (Hq < 1 || Hq > 4096 || ld_q < qd || ld_q > (1LL << 40))) return VP_ERR_SHAPE;
  if (q && q_out == q && ld_q != qd) return VP_ERR_INVALID_ARG;
  if (!al(k, 16) || !al(v, 16) || ld_k % 8 || ld_v % 8 || (q && (!al(q, 16) || ld_q % 8 || !al(q_out, 16))) ||
      (q_norm && !al(q_norm, 4)) || (k_norm && !al(k_norm, 4)) || (row_start && !al(row_start, 4)) || !al(ctx, 4) ||
      (kv_len && !al(kv_len, 4)) || (status && !al(status, 4)))
    return VP_ERR_ALIGNMENT;
  AppendArgs a;
  a.rot = a.interleaved = 0;
  if (rope && rope->rot_dim) {
    if (!rope->inv_freq) return VP_ERR_INVALID_ARG;
    if (rope->rot_dim < 0 || rope->rot_dim % 16 || rope->rot_dim > c.D) return VP_ERR_SHAPE;
    a.rot = rope->rot_dim;
    a.interleaved = rope->interleaved != 0;
    for (int j = 0; j < a.rot / 2; ++j) {
      const double f = rope->inv_freq[j] / 6.283185307179586476925;
      if (!std::isfinite(f)) return VP_ERR_INVALID_ARG;
      const double t = f - std::floor(f);  // [0, 1]: 1 wraps to 0
      // the top 32 bits and the rest, each exact: 2^64 itself does not fit the integer
      const double top = std::floor(t * 4294967296.0), low = (t * 4294967296.0 - top) * 4294967296.0;
      a.turn[j] = ((unsigned long long)top << 32) + (unsigned long long)low;
    }
  }
  int sms = 0;
  if ((st = device_sm_count(&sms)) != VP_OK) return st;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.ld_q = ld_q, a.ld_k = ld_k, a.ld_v = ld_v;
  a.q_norm = q_norm, a.k_norm = k_norm, a.eps = eps;
  a.row_start = row_start, a.ctx = ctx, a.pages = c.pages;
  a.S = S, a.M = M, a.Hq = Hq, a.Hkv = c.Hkv, a.n_pages = c.n_pages, a.max_pages = c.max_pages;
  a.log_page = 4;
  while ((1 << a.log_page) < c.page_size) ++a.log_page;
  a.k_cache = c.k, a.v_cache = c.v;
  a.k_scales = k_scales, a.v_scales = v_scales;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.kv_len = kv_len, a.status = status;
  const int heads = (q ? Hq : 0) + 2 * c.Hkv, at_once = kThreadsP / (c.D / 8);
  // Few rows: one head per group of lanes (more blocks, the shortest path through each).  Many: a row's heads
  // over the fewest blocks of at most six per group, evenly (every block looks the row's position up; 6001
  // rows of 48 heads, with the norm's code: 45, 32, 30 us at 2 x 256, 3 x 128 and 6 x 128 heads x threads).
  const int turns = (heads + at_once - 1) / at_once;
  const bool many = (long long)M * turns >= 16LL * sms;
  const int blocks = many ? (turns + 5) / 6 : turns, per = (turns + blocks - 1) / blocks;
  using Kernel = void (*)(const AppendArgs);
  auto pick = [&](auto norm) -> Kernel {
    constexpr bool N = decltype(norm)::value;
    static const Kernel kernels[3][6] = {
        {append_kernel<64, 1, N, kFp8>, append_kernel<64, 2, N, kFp8>, append_kernel<64, 3, N, kFp8>, append_kernel<64, 4, N, kFp8>, append_kernel<64, 5, N, kFp8>, append_kernel<64, 6, N, kFp8>},
        {append_kernel<128, 1, N, kFp8>, append_kernel<128, 2, N, kFp8>, append_kernel<128, 3, N, kFp8>, append_kernel<128, 4, N, kFp8>, append_kernel<128, 5, N, kFp8>, append_kernel<128, 6, N, kFp8>},
        {append_kernel<256, 1, N, kFp8>, append_kernel<256, 2, N, kFp8>, append_kernel<256, 3, N, kFp8>, append_kernel<256, 4, N, kFp8>, append_kernel<256, 5, N, kFp8>, append_kernel<256, 6, N, kFp8>}};
    return kernels[c.D == 64 ? 0 : c.D == 128 ? 1 : 2][per - 1];
  };
  const Kernel kern = (q && q_norm) || k_norm ? pick(std::true_type()) : pick(std::false_type());
  kern<<<dim3((unsigned)M, (unsigned)blocks), kThreadsP, 0, (cudaStream_t)stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VP_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

vp_status vp_paged_append(const vp_paged_cache* cache, const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                          int64_t ld_v, const float* q_norm, const float* k_norm, float eps, const vp_rope* rope,
                          const int32_t* row_start, const int32_t* ctx, int S, int M, int Hq, void* q_out, int32_t* kv_len,
                          int* status, void* stream) {
  const vp_status st = check_cache(cache);
  if (st != VP_OK) return st;
  return append<false>(*cache, nullptr, nullptr, q, ld_q, k, ld_k, v, ld_v, q_norm, k_norm, eps, rope, row_start, ctx, S, M, Hq,
                       q_out, kv_len, status, stream);
}

vp_status vp_paged_append_fp8(const vp_paged_cache_fp8* cache, const void* q, int64_t ld_q, const void* k, int64_t ld_k,
                              const void* v, int64_t ld_v, const float* q_norm, const float* k_norm, float eps,
                              const vp_rope* rope, const int32_t* row_start, const int32_t* ctx, int S, int M, int Hq,
                              void* q_out, int32_t* kv_len, int* status, void* stream) {
  const vp_status st = check_cache_fp8(cache);
  if (st != VP_OK) return st;
  const vp_paged_cache c = {cache->k, cache->v, cache->pages, cache->n_pages, cache->page_size, cache->max_pages, cache->Hkv,
                            cache->D};
  return append<true>(c, cache->k_scales, cache->v_scales, q, ld_q, k, ld_k, v, ld_v, q_norm, k_norm, eps, rope, row_start, ctx,
                      S, M, Hq, q_out, kv_len, status, stream);
}

}  // extern "C"
