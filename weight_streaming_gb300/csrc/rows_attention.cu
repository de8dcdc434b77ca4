// Attention of several new rows per sequence: whole prompts (vp_prompt_attention), chunks over a paged cache
// (vp_paged_attention_rows) and over an 8-bit one (vp_paged_attention_rows_fp8).  The kernel stands in rows_attention.cuh.
//
// Mathematics: as for single tokens (paged_attention.cu): one pass over the keys keeps a reference m, l = sum 2^(t - m) and o =
// sum 2^(t - m) v of t = scale log2(e) q . k; two parts join as m = max(m1, m2), l = l1 2^(m1 - m) + l2 2^(m2 - m), o alike.  m is
// the running maximum of some earlier block: it follows only where the maximum has grown by 2^8, so o is seldom scaled.
// l sums the weights in fp32; the tensor cores take them in bf16, one rounding of at most 2^-8 each (the values are bf16, and both
// operands of a product have one type).  Outputs are 1.1 to 1.4 times as far from the definition as with weights in 32 bits.  A second
// bf16 part, as single tokens have it in paged_attention.cu, would mean these products twice, half as much tensor work again where
// that is the bound.
//
// Design: 4 D flops a key, row and query head on the tensor cores (bf16, fp32 sums in tensor memory).
//  * Rows: the G query heads of a key-value head are rows of their own (row = token * G + head), so that the keys are read
//    once for all of them and a few tokens fill a tile.  An item is 128 or 256 rows of one sequence and key-value head.
//  * Two tiles of 128 rows share the keys.  With 64 or 128 columns both lie in one CTA (scores and outputs fill the tensor
//    memory; one tile's softmax runs beside the other's products).  With 256 columns a CTA pair (cta_group::2) takes a
//    tile each, holds half of every key and value block, and has two score buffers.  A single CTA would take 64 bytes of L2 a
//    cycle there and stay at half the rate (12,289 rows of 24 / 4 x 256 heads: 2.0 ms, in pairs 1.8 at first, 1.29 now).
//  * One tile (sequences with few rows): queries in tensor memory, two score buffers; with at most 32 rows every softmax warp
//    takes all rows and a quarter of the keys (61 single tokens over an 8-bit cache: 299 us without, 198 with, at that time).
//  * Warps: a scheduler, two that start copies (TMA, 128-byte swizzle; a block's pages), one that issues products, four or
//    eight that prepare operands, a softmax warp per 32 rows of a tile.  Weights go back into tensor memory over the scores, 64
//    keys at a time, and the products start with the first 64.
//  * Values that a row of the item does not see have a weight of zero, which times infinity or NaN is not zero: in blocks that
//    some row does not see whole (its own diagonal, the sequence's end) the preparing warps look at the values first, make
//    those zeros and note their columns and first keys; the rows that see them get NaN at the end.
//  * 8-bit cache: the preparing warps expand codes to bf16 operand tiles.  A code's bits three places lower are its value times
//    2^-120 as bf16; one product with 2^(120 + scale - 127) gives the exact value.
//  * Work: the items of all sequences and heads form one line of keys plus a fixed cost each, cut into equal parts, one per CTA or
//    pair (the lengths are read on the device: each CTA sums the line up and finds its part).  At most two items of a CTA are
//    cut; their parts lie in the workspace and a second launch joins them.  No counters: nothing to reset.
//
// What bounds it (2,048 rows behind 30,000 positions): 24 / 4 x 256 heads 938 us, 1.67 PFLOP/s, 86 % of the measured bf16 rate: the
// tensor cores.  32 / 8 x 128 heads 880 us, 1.18 PFLOP/s: a tile's chain of softmax (two warps of a scheduler share its instruction
// slots and caches) and products, an estimated 2,900 cycles a block against 2,048 of products.  64 columns: 754 us, 0.69 PFLOP/s, the
// exponentials and the same chain.  Few rows: the cache's bytes in bf16 (64 x 8,001 positions of 8 x 128 heads 327 us, 6.4
// TB/s); in 8 bits the expansion and the softmax of 128 keys take longer than their bytes (291 us, 3.6 TB/s).
// Loops are kept short on purpose: a scheduler's warps share its instruction cache.  With the softmax unrolled over 128 keys and
// copies of the waits' slow halves 61 single tokens over an 8-bit cache took 566 us in place of 290 (now 192).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "errors.h"
#include "internal.h"
#include "paged.h"
#include "rows_attention.cuh"
#include "serve_ws.h"
#include "tma.h"

namespace vp {

namespace {

constexpr int kJoinThreads = 256, kJoinRows = 16;  // CTAs of an item's rows

// Joins the items that were cut: the CTA (c, y) those whose first part is CTA c's last piece, the y-th share of its rows.
// The parts' weights first; then each output value is summed by one thread, or, where there are fewer values than threads, by
// several that take every n-th part, in a fixed order both times.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ RowsArgs a, int part_rows) {
  __shared__ float s_w[kJoinRows][kRowsGrid], s_m[kJoinRows], s_l[kJoinRows];
  __shared__ float4 s_sum[kJoinThreads];
  __shared__ int s_cnt;
  const int c = blockIdx.x, tid = threadIdx.x, grid = gridDim.x;
  const int4 d = a.desc[2 * c + 1];
  if (d.z < 0 || *(volatile int*)a.status == VP_ERR_TIMEOUT) return;
  const int rows = d.w & (kPartEnds - 1), per = (rows + gridDim.y - 1) / gridDim.y, r0 = blockIdx.y * per;
  const int nr = min(per, rows - r0);
  if (nr <= 0) return;
  if (tid == 0) s_cnt = grid - 1 - c;
  __syncthreads();
  for (int k = tid; c + 1 + k < grid; k += kJoinThreads) {  // parts behind the first
    const int4 e = a.desc[2 * (c + 1 + k)];
    if (e.z != d.z || e.x != d.x || e.y != d.y)
      atomicMin(&s_cnt, k);
    else if (e.w & kPartEnds)
      atomicMin(&s_cnt, k + 1);
  }
  __syncthreads();
  const int cnt = s_cnt + 1;
  auto part = [&](int x) { return (size_t)(c + x) * 2 + (x == 0); };
  for (int i = tid; i < nr * cnt; i += kJoinThreads) s_w[i / cnt][i % cnt] = __ldcg(a.part_ml + (part(i % cnt) * 256 + r0 + i / cnt) * 2);
  __syncthreads();
  if (tid < nr) {
    float m = -INFINITY, l = 0.0f;
#pragma unroll 8
    for (int x = 0; x < cnt; ++x) m = fmaxf(m, s_w[tid][x]);
#pragma unroll 8
    for (int x = 0; x < cnt; ++x) {
      const float mx = s_w[tid][x], f = mx == -INFINITY ? 0.0f : ra_ex2(mx - m);
      s_w[tid][x] = f;
      l += f * __ldcg(a.part_ml + (part(x) * 256 + r0 + tid) * 2 + 1);  // NaN stays NaN
    }
    s_m[tid] = m, s_l[tid] = l;
  }
  __syncthreads();
  const int n = nr * (D / 4), groups = n < kJoinThreads ? kJoinThreads / n : 1;
  for (int i0 = 0; i0 < n; i0 += kJoinThreads) {
    const int g = groups > 1 ? tid / n : 0, i = groups > 1 ? tid - g * n : i0 + tid;
    const bool work = i < n && g < groups;
    const int r = work ? i % nr : 0, d4 = work ? i / nr : 0;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (work) {
#pragma unroll 8
      for (int x = g; x < cnt; x += groups) {
        const float f = s_w[r][x];
        const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o) + (part(x) * (D / 4) + d4) * part_rows + r0 + r);
        y.x = fmaf(f, v.x, y.x), y.y = fmaf(f, v.y, y.y), y.z = fmaf(f, v.z, y.z), y.w = fmaf(f, v.w, y.w);
      }
    }
    if (groups > 1) {
      s_sum[tid] = y;
      __syncthreads();
      if (g != 0 || !work) continue;
      for (int k = 1; k < groups; ++k) {
        const float4 v = s_sum[k * n + i];
        y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
      }
    }
    if (!work) continue;
    const float l = s_l[r], inv = l == 0.0f ? 0.0f : 1.0f / l;
    const size_t orow = (size_t)(d.z + (r0 + r) / a.G) * a.Hq + d.y * a.G + (r0 + r) % a.G;
    y.x *= inv, y.y *= inv, y.z *= inv, y.w *= inv;
    if (a.gate) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(a.gate + orow * D + 4 * d4));
      ra_gate2(y.x, y.y, w.x);
      ra_gate2(y.z, y.w, w.y);
    }
    *reinterpret_cast<uint2*>(a.out + orow * D + 4 * d4) = make_uint2(ra_bf16x2(y.x, y.y), ra_bf16x2(y.z, y.w));
    if (d4 == 0 && a.lse) a.lse[orow] = ra_lse(s_m[r], l);
  }
}

bool al(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int kMaxGroup = 64;  // query heads per key-value head

bool rows_shape_ok(int S, int M, int Hq, int Hkv, int D) {
  return S >= 1 && S <= 65536 && M >= 1 && M <= (1 << 24) && Hkv >= 1 && Hkv <= 1024 && Hq >= Hkv && Hq % Hkv == 0 &&
         Hq / Hkv <= kMaxGroup && (D == 64 || D == 128 || D == 256) && (long long)M * Hkv <= (1LL << 30);
}

struct RowsWs {
  size_t desc, part_ml, part_o, total;
};
RowsWs rows_ws(int D) {
  RowsWs w;
  w.desc = kServeData;
  w.part_ml = w.desc + sizeof(int4) * kRowsGrid * 2;
  w.part_o = w.part_ml + sizeof(float) * kRowsGrid * 2 * 256 * 2;
  w.total = w.part_o + sizeof(float) * kRowsGrid * 2 * (size_t)(D == 256 ? 128 : 256) * D;  // a pair: 256 rows
  return w;
}

// Two tiles of 128 rows share every key and value that is read; where a sequence has fewer rows (on average: the lengths are
// on the device) one tile does, with a second score buffer.  16 sequences of 4,000 positions, one / two tiles in us: of 128 columns
// (32 / 8 heads) with 4, 32, 128, 160, 256 rows per key head 62 / 72, 70 / 79, 76 / 83, 113 / 98, 115 / 104, in 8 bits 61 / 85, 68 / 91, 82 / 97,
// 123 / 108, 130 / 115; of 64 the same way, 65 / 72 at 128 and 91 / 78 at 160; of 256 (24 / 4 heads) 64 / 72 at 6, 75 / 81 at 96, 96 / 86 at 144,
// 107 / 93 at 240.  Against the rule: 256 columns in 8 bits, where one tile stays ahead (107 / 122 at 240, 266 / 323 at 768), and batches
// whose sequences differ (39 single tokens and 2,001 rows, by the average two tiles: 223 / 271 of 128 columns, 208 / 230 of 256).
int rows_tiles(int S, int M, int Hq, int Hkv) { return (long long)M * (Hq / Hkv) <= 128LL * S ? 1 : 2; }

// Rows and columns of the key (0) and value (1) tiles.
int tile_rows(int D, int tiles, int kv) { return kv ? rows_block(D, tiles) : rows_key_rows(D, tiles); }
int tile_cols(int D, int tiles, int kv) { return kv ? rows_value_cols(D, tiles) : D; }

// What the three calls share: the arguments that they have in common, checked, and the launches.
struct Common {
  const void* q;
  long long ld_q;
  int S, M, Hq, Hkv, D;
  float scale;
  const void* gate;
  void* out;
  float* lse;
  void* ws;
  size_t ws_bytes;
};
vp_status check_common(const Common& x) {
  if (!x.q || !x.out || !x.ws || !std::isfinite(x.scale * 1.4426950408889634f)) return VP_ERR_INVALID_ARG;
  if (!rows_shape_ok(x.S, x.M, x.Hq, x.Hkv, x.D) || x.ld_q < (long long)x.Hq * x.D || x.ld_q > (1LL << 38)) return VP_ERR_SHAPE;
  if (!al(x.q, 16) || x.ld_q % 8 || (x.gate && !al(x.gate, 16)) || !al(x.out, 16) || (x.lse && !al(x.lse, 4)) || !al(x.ws, 256))
    return VP_ERR_ALIGNMENT;
  if (x.ws_bytes < rows_ws(x.D).total) return VP_ERR_WORKSPACE;
  return VP_OK;
}
vp_status run_rows(const Common& x, RowsArgs a, int source, const CUtensorMap& kmap, const CUtensorMap& vmap, int sms,
                   cudaStream_t s) {
  const RowsWs w = rows_ws(x.D);
  uint8_t* b = static_cast<uint8_t*>(x.ws);
  a.q = static_cast<const uint16_t*>(x.q);
  a.gate = static_cast<const uint16_t*>(x.gate);
  a.out = static_cast<uint16_t*>(x.out);
  a.lse = x.lse;
  a.ld_q = x.ld_q;
  a.S = x.S, a.M = x.M, a.Hq = x.Hq, a.Hkv = x.Hkv, a.G = x.Hq / x.Hkv;
  a.scale2 = x.scale == 0.0f ? 1.0f : std::fabs(x.scale) * 1.4426950408889634f;
  a.q_and = x.scale == 0.0f ? 0u : 0xFFFFFFFFu;
  a.q_flip = x.scale < 0.0f ? 0x80008000u : 0u;
  a.desc = reinterpret_cast<int4*>(b + w.desc);
  a.part_ml = reinterpret_cast<float*>(b + w.part_ml);
  a.part_o = reinterpret_cast<float*>(b + w.part_o);
  a.status = reinterpret_cast<int*>(b);
  const int tiles = rows_tiles(x.S, x.M, x.Hq, x.Hkv);
  a.tok_tile = 128 * tiles / a.G;
  a.g_inv = (65536 + a.G - 1) / a.G;
  // Starting and ending an item, in keys: 64 to 2,560 tried over 16 calls of each width (prompts of 2,000 to 16,384 rows, one to 40 a
  // call, chunks, drafts, single tokens), without and with gates, which are read at an item's end.  40 prompts of 16,000 rows:
  // pairs 512, 640, 768: 309, 299, 310 us, with gates 640, 1,024, 1,280: 441, 397, 409; 64 columns (two tiles) 128, 256, 448: 228, 195,
  // 221, with gates 268, 213, 225; 128 columns 256, 448, 640: 313, 276, 301, with gates 373, 307, 316.  60 single tokens in 8 bits of
  // 128 columns 256, 448, 640: 193, 178, 174.  The other calls come within 4 % of their best at these values.
  const bool pair = x.D == 256 && tiles == 2;
  a.item_cost = pair ? (x.gate ? 1024 : 640) : x.D == 64 && tiles == 2 ? 256 : 448;
  const int grid = std::min(sms, kRowsGrid);
  // Polls after which a wait for an item gives up: kMbarPolls and one per 32 keys of a CTA's part of the line, were every sequence as long as it
  // can be.  A role that has nothing to do in an item (a tile without rows, queries loaded ahead, the issuing warp of a pair's second
  // CTA) waits for as long as the others work on it, up to the CTA's whole time.  A poll takes 4 us (measured, whatever the
  // hint), 32 keys 0.6 us at most: kMbarPolls alone, 0.26 s, ran out where 192 rows saw 2^31 positions (0.35 s an item).
  const long long longest = source == kDense ? x.M : (long long)a.max_pages << a.log_page;
  const long long line = ((long long)x.S + x.M / a.tok_tile) * (longest + a.item_cost) * x.Hkv;
  a.polls = kMbarPolls + (uint32_t)std::min((line / (pair ? grid / 2 : grid) + 2 * kMinKeys) / 32, 1LL << 31);
  cudaError_t e;
  if (x.D == 256)
    e = tiles == 2 ? launch_rows<256, 2>(a, source, kmap, vmap, grid, s) : launch_rows<256, 1>(a, source, kmap, vmap, grid, s);
  else if (x.D == 128)
    e = tiles == 2 ? launch_rows<128, 2>(a, source, kmap, vmap, grid, s) : launch_rows<128, 1>(a, source, kmap, vmap, grid, s);
  else
    e = tiles == 2 ? launch_rows<64, 2>(a, source, kmap, vmap, grid, s) : launch_rows<64, 1>(a, source, kmap, vmap, grid, s);
  if (e != cudaSuccess) return cuda_fail(e);
  const dim3 jg((unsigned)(pair ? grid / 2 : grid), kJoinRows);
  if (x.D == 256)
    join_kernel<256><<<jg, kJoinThreads, 0, s>>>(a, 128 * tiles);
  else if (x.D == 128)
    join_kernel<128><<<jg, kJoinThreads, 0, s>>>(a, 128 * tiles);
  else
    join_kernel<64><<<jg, kJoinThreads, 0, s>>>(a, 128 * tiles);
  e = cudaGetLastError();
  return e == cudaSuccess ? VP_OK : cuda_fail(e);
}

int log_page(int P) {
  int l = 4;
  while ((1 << l) < P) ++l;
  return l;
}

}  // namespace

vp_status check_cache_fp8(const vp_paged_cache_fp8* c) {
  if (!c || !c->k_scales || !c->v_scales) return VP_ERR_INVALID_ARG;
  const vp_paged_cache plain = {c->k, c->v, c->pages, c->n_pages, c->page_size, c->max_pages, c->Hkv, c->D};
  const vp_status st = check_cache(&plain);
  if (st != VP_OK) return st;
  return al(c->k_scales, 16) && al(c->v_scales, 16) ? VP_OK : VP_ERR_ALIGNMENT;
}

}  // namespace vp

using namespace vp;

extern "C" {

size_t vp_prompt_attention_workspace_bytes(int S, int M, int Hq, int Hkv, int D) {
  return rows_shape_ok(S, M, Hq, Hkv, D) ? rows_ws(D).total : 0;
}

vp_status vp_prompt_attention(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                              const int32_t* row_start, int S, int M, int Hq, int Hkv, int D, float scale, const void* gate,
                              void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  if (!k || !v || !row_start) return VP_ERR_INVALID_ARG;
  const Common x = {q, ld_q, S, M, Hq, Hkv, D, scale, gate, out, lse, ws, ws_bytes};
  vp_status st = check_common(x);
  if (st != VP_OK) return st;
  const long long kd = (long long)Hkv * D;
  if (ld_k < kd || ld_v < kd || ld_k > (1LL << 38) || ld_v > (1LL << 38)) return VP_ERR_SHAPE;
  if (!al(k, 16) || !al(v, 16) || ld_k % 8 || ld_v % 8 || !al(row_start, 4)) return VP_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = device_sm_count(&sms)) != VP_OK) return st;
  PFN_cuTensorMapEncodeTiled_v12000 encode;
  if ((st = tensor_map_encoder(&encode)) != VP_OK) return st;
  // rows of [Hkv D / 64][64]: a box is a block's rows of one head, its 64-column groups one behind the other
  CUtensorMap maps[2];
  const int tiles = rows_tiles(S, M, Hq, Hkv);
  for (int i = 0; i < 2; ++i) {
    const cuuint64_t dims[3] = {64, (cuuint64_t)M, (cuuint64_t)(kd / 64)};
    const cuuint64_t strides[2] = {(cuuint64_t)(i ? ld_v : ld_k) * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)tile_rows(D, tiles, i), (cuuint32_t)tile_cols(D, tiles, i) / 64}, step[3] = {1, 1, 1};
    if (encode(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(i ? v : k), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return VP_ERR_UNSUPPORTED;
  }
  RowsArgs a = {};
  a.row_start = row_start;
  return run_rows(x, a, kDense, maps[0], maps[1], sms, (cudaStream_t)stream);
}

size_t vp_paged_attention_rows_workspace_bytes(int S, int M, int Hq, int Hkv, int D) {
  return rows_shape_ok(S, M, Hq, Hkv, D) ? rows_ws(D).total : 0;
}

vp_status vp_paged_attention_rows(const vp_paged_cache* cache, const void* q, const int32_t* row_start, const int32_t* kv_len,
                                  int S, int M, int Hq, float scale, const void* gate, void* out, float* lse, void* ws,
                                  size_t ws_bytes, void* stream) {
  vp_status st = check_cache(cache);
  if (st != VP_OK) return st;
  if (!kv_len) return VP_ERR_INVALID_ARG;
  const vp_paged_cache& c = *cache;
  const Common x = {q, (long long)Hq * c.D, S, M, Hq, c.Hkv, c.D, scale, gate, out, lse, ws, ws_bytes};
  if ((st = check_common(x)) != VP_OK) return st;
  if (!row_start && M != S) return VP_ERR_SHAPE;
  if ((row_start && !al(row_start, 4)) || !al(kv_len, 4)) return VP_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = device_sm_count(&sms)) != VP_OK) return st;
  PFN_cuTensorMapEncodeTiled_v12000 encode;
  if ((st = tensor_map_encoder(&encode)) != VP_OK) return st;
  // as [D / 64][rows of all pages and heads][64]: a box is a block's rows, or a page's where pages are shorter (one
  // 64-column group of it then: the next one lies a block's rows further on in shared memory)
  const int tiles = rows_tiles(S, M, Hq, c.Hkv);
  CUtensorMap maps[2];
  for (int i = 0; i < 2; ++i) {
    const int all = tile_rows(c.D, tiles, i), rows = std::min(c.page_size, all);
    const cuuint64_t dims[3] = {64, (cuuint64_t)c.n_pages * c.Hkv * c.page_size, (cuuint64_t)c.D / 64};
    const cuuint64_t strides[2] = {(cuuint64_t)c.D * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)rows, rows == all ? (cuuint32_t)tile_cols(c.D, tiles, i) / 64 : 1u}, step[3] = {1, 1, 1};
    if (encode(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, i ? c.v : c.k, dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return VP_ERR_UNSUPPORTED;
  }
  RowsArgs a = {};
  a.row_start = row_start, a.kv_len = kv_len, a.pages = c.pages;
  a.n_pages = c.n_pages, a.log_page = log_page(c.page_size), a.max_pages = c.max_pages;
  return run_rows(x, a, kPaged, maps[0], maps[1], sms, (cudaStream_t)stream);
}

vp_status vp_paged_attention_rows_fp8(const vp_paged_cache_fp8* cache, const void* q, const int32_t* row_start,
                                      const int32_t* kv_len, int S, int M, int Hq, float scale, const void* gate, void* out,
                                      float* lse, void* ws, size_t ws_bytes, void* stream) {
  vp_status st = check_cache_fp8(cache);
  if (st != VP_OK) return st;
  if (!kv_len) return VP_ERR_INVALID_ARG;
  const vp_paged_cache_fp8& c = *cache;
  const Common x = {q, (long long)Hq * c.D, S, M, Hq, c.Hkv, c.D, scale, gate, out, lse, ws, ws_bytes};
  if ((st = check_common(x)) != VP_OK) return st;
  if (!row_start && M != S) return VP_ERR_SHAPE;
  if ((row_start && !al(row_start, 4)) || !al(kv_len, 4)) return VP_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = device_sm_count(&sms)) != VP_OK) return st;
  PFN_cuTensorMapEncodeTiled_v12000 encode;
  if ((st = tensor_map_encoder(&encode)) != VP_OK) return st;
  const int tiles = rows_tiles(S, M, Hq, c.Hkv);
  CUtensorMap maps[2];  // rows of D codes; a box is a tile's rows, or a page's
  for (int i = 0; i < 2; ++i) {
    const cuuint64_t dims[2] = {(cuuint64_t)c.D, (cuuint64_t)c.n_pages * c.Hkv * c.page_size}, strides[1] = {(cuuint64_t)c.D};
    const cuuint32_t box[2] = {(cuuint32_t)tile_cols(c.D, tiles, i), (cuuint32_t)std::min(c.page_size, tile_rows(c.D, tiles, i))}, step[2] = {1, 1};
    if (encode(&maps[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, i ? c.v : c.k, dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return VP_ERR_UNSUPPORTED;
  }
  RowsArgs a = {};
  a.row_start = row_start, a.kv_len = kv_len, a.pages = c.pages;
  a.k_scales = c.k_scales, a.v_scales = c.v_scales;
  a.n_pages = c.n_pages, a.log_page = log_page(c.page_size), a.max_pages = c.max_pages;
  return run_rows(x, a, kPagedFp8, maps[0], maps[1], sms, (cudaStream_t)stream);
}

}  // extern "C"
