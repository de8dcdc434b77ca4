// Attention of one new token per sequence over a paged KV cache (vp_paged_attention).
//
// Mathematics: t_i = scale q . k_i; one pass keeps m = max t, l = sum e^(t - m), o = sum e^(t - m) v, and
// two partial results join as m = max(m1, m2), l = l1 e^(m1 - m) + l2 e^(m2 - m) (o alike).
// First form: one CTA per (q head, sequence); its warps take every fourth position.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "errors.h"
#include "internal.h"
#include "paged.h"
#include "verify.h"

namespace vp {

namespace {

struct PagedArgs {
  const uint16_t *q, *k, *v, *gate;
  uint16_t* out;
  float* lse;
  const int32_t *kv_len, *pages;
  int S, Hq, Hkv, n_pages, log_page, max_pages;
  float scale;
  int* status;
};

template <int D>
__global__ void __launch_bounds__(128) attend_simple(const PagedArgs a) {
  constexpr int kE = D / 32;
  __shared__ float so[4][D], sm[4], sl[4];
  const int h = blockIdx.x, s = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = h / (a.Hq / a.Hkv);
  int n = a.kv_len[s];
  if (n < 0 || n > (a.max_pages << a.log_page)) {
    if (threadIdx.x == 0) atomicExch(a.status, (int)VP_ERR_SHAPE);
    n = 0;
  }
  auto bf = [](uint16_t x) { return __uint_as_float((uint32_t)x << 16); };
  const size_t row = ((size_t)s * a.Hq + h) * D;
  float q[kE], o[kE], m = -INFINITY, l = 0.0f;
  for (int e = 0; e < kE; ++e) q[e] = bf(a.q[row + lane + 32 * e]), o[e] = 0.0f;
  for (int p = warp; p < n; p += 4) {
    const int page = a.pages[(size_t)s * a.max_pages + (p >> a.log_page)];
    if (page < 0 || page >= a.n_pages) {
      if (lane == 0) atomicExch(a.status, (int)VP_ERR_SHAPE);
      continue;
    }
    const size_t at = ((((size_t)page * a.Hkv + g) << a.log_page) + (p & ((1 << a.log_page) - 1))) * D;
    float t = 0.0f;
    for (int e = 0; e < kE; ++e) t = fmaf(q[e], bf(a.k[at + lane + 32 * e]), t);
    for (int x = 16; x; x >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, x);
    t *= a.scale;
    const float mn = fmaxf(m, t);
    const float c = m == -INFINITY ? 0.0f : expf(m - mn), w = t == -INFINITY ? 0.0f : expf(t - mn);
    m = mn;
    l = l * c + w;
    for (int e = 0; e < kE; ++e) o[e] = o[e] * c + w * bf(a.v[at + lane + 32 * e]);
  }
  for (int e = 0; e < kE; ++e) so[warp][lane + 32 * e] = o[e];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  __syncthreads();
  float M = -INFINITY, L = 0.0f;
  for (int w = 0; w < 4; ++w) M = fmaxf(M, sm[w]);
  float c[4];
  for (int w = 0; w < 4; ++w) L += sl[w] * (c[w] = sm[w] == -INFINITY ? 0.0f : expf(sm[w] - M));
  for (int d = threadIdx.x; d < D; d += 128) {
    float y = 0.0f;
    for (int w = 0; w < 4; ++w) y += so[w][d] * c[w];
    y = L == 0.0f ? 0.0f : y / L;
    if (a.gate) y /= 1.0f + expf(-bf(a.gate[row + d]));
    a.out[row + d] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
  }
  if (threadIdx.x == 0 && a.lse) a.lse[(size_t)s * a.Hq + h] = L == 0.0f ? -INFINITY : M + logf(L);
}

bool al(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool attend_shape_ok(int S, int Hq, int Hkv, int D) {
  return S >= 1 && S <= 8192 && Hkv >= 1 && Hkv <= 1024 && (long long)S * Hkv <= 65536 && Hq >= Hkv && Hq % Hkv == 0 &&
         Hq / Hkv <= 16 && (D == 64 || D == 128 || D == 256);
}

}  // namespace

}  // namespace vp

using namespace vp;

extern "C" {

size_t vp_paged_attention_workspace_bytes(int S, int Hq, int Hkv, int D) {
  if (!attend_shape_ok(S, Hq, Hkv, D)) return 0;
  return 256;
}

vp_status vp_paged_attention(const vp_paged_cache* cache, const void* q, const int32_t* kv_len, int S, int Hq,
                             float scale, const void* gate, void* out, float* lse, void* ws, size_t ws_bytes,
                             void* stream) {
  vp_status st = check_cache(cache);
  if (st != VP_OK) return st;
  if (!q || !kv_len || !out || !ws || !std::isfinite(scale)) return VP_ERR_INVALID_ARG;
  const vp_paged_cache& c = *cache;
  if (!attend_shape_ok(S, Hq, c.Hkv, c.D)) return VP_ERR_SHAPE;
  if (!al(q, 16) || !al(kv_len, 4) || (gate && !al(gate, 16)) || !al(out, 16) || (lse && !al(lse, 4)) || !al(ws, 256))
    return VP_ERR_ALIGNMENT;
  if (ws_bytes < vp_paged_attention_workspace_bytes(S, Hq, c.Hkv, c.D)) return VP_ERR_WORKSPACE;
  int sms = 0;
  if ((st = device_sm_count(&sms)) != VP_OK) return st;
  PagedArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(c.k);
  a.v = static_cast<const uint16_t*>(c.v);
  a.gate = static_cast<const uint16_t*>(gate);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.kv_len = kv_len, a.pages = c.pages;
  a.S = S, a.Hq = Hq, a.Hkv = c.Hkv, a.n_pages = c.n_pages, a.max_pages = c.max_pages;
  a.log_page = 4;
  while ((1 << a.log_page) < c.page_size) ++a.log_page;
  a.scale = scale;
  a.status = static_cast<int*>(ws);
  const dim3 grid((unsigned)Hq, (unsigned)S);
  cudaStream_t s = (cudaStream_t)stream;
  if (c.D == 64)
    attend_simple<64><<<grid, 128, 0, s>>>(a);
  else if (c.D == 128)
    attend_simple<128><<<grid, 128, 0, s>>>(a);
  else
    attend_simple<256><<<grid, 128, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VP_OK : cuda_fail(e);
}

}  // extern "C"
