// Attention of one new token per sequence over a paged KV cache (vp_paged_attention).
//
// Mathematics: t_i = scale q . k_i; one pass keeps m = max t, l = sum e^(t - m), o = sum e^(t - m) v, and
// two partial results join as m = max(m1, m2), l = l1 e^(m1 - m) + l2 e^(m2 - m) (o alike).
//
// What bounds it: every cached key and value is read once for the G = Hq / Hkv query heads that share it
// (G flops per byte at most), so the bytes do; everything else hides behind the copies.
//  * The cached positions of all (sequence, key-value head)s form one line of pieces of 8 KB of keys and
//    8 KB of values (16, 32 or 64 positions at D = 256, 128, 64).  One CTA per SM; the lengths are read on
//    the device, where each CTA sums them up and finds its first piece.  The line is cut into equal runs;
//    where there are few (sequence, head)s each is cut by itself into even parts; short ones are not cut.
//  * A producer warp walks the run, looks the pages up and issues the TMA loads (box = the piece's rows
//    of one page, 128-byte swizzle) into a ring of 16 KB stages; five warps (four above 8 heads) take the pieces in
//    turn, each with its own running maximum, sum and output in registers: no synchronisation between
//    them until the (sequence, head) ends, where they are joined through shared memory.
//  * The tensor core's 16 rows hold up to 16 query heads.  P is split in two bf16 parts, hi + lo (about
//    2^-17 relative): with G <= 8 heads the parts are the tile's upper and lower 8 rows of one MMA, and
//    their sums are added at the end; above, two MMAs.
//  * A (sequence, head) that crosses CTAs goes through fp32 partials in the workspace (two per CTA at
//    most: its first and its last one), announced after the CTA's last copy (a GPU-scope fence waits
//    for the copies in flight); the last contributor joins them in order.
// Measured, from memory: 131,071 positions of 4 x 256 heads (537 MB) in 91 us, 5.9 TB/s with start and join (7.1
// TB/s while it streams; a copy reaches 6.8 of reads and writes); 61 sequences of 300 to 9,000 positions, 8 x 128
// heads (1.18 GB) in 182 us, 6.5 TB/s; 4 sequences of up to 700 positions in 14.3 us: launch, lengths, first
// copies, join.
// Waits are bounded: a warp whose wait ran out reports VP_ERR_TIMEOUT, takes no further stage and goes on to the
// end, so the CTA ends; the warps that issue copies see them land first, whatever ran out, and no join copies start
// once something has.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "errors.h"
#include "internal.h"
#include "paged.h"
#include "ptx.cuh"
#include "serve_ws.h"
#include "tma.h"
#include "verify.h"

namespace vp {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPaGrid = 152;                  // CTAs at most: one per SM
constexpr int kPieceBytes = 8192;             // of keys, and of values
constexpr int kMinPieces = 5;                 // pieces per CTA at least: one per warp (8: 4 sequences of 700 12.9 us, 5: 12.3)
constexpr int kJoinCost = 18;                 // joining parts of a (sequence, head) costs as much as these many pieces

struct PagedArgs {
  const uint16_t *q, *gate;
  uint16_t* out;
  float* lse;
  const int32_t *kv_len, *pages;
  int S, Hq, Hkv, G, n_pages, log_page, max_pages, log_box;
  float scale2;        // scale * log2(e)
  unsigned* counters;  // [S][Hkv]
  float* part_o;       // [grid][2][16][D]
  float* part_ml;      // [grid][2][16][2]: maximum (log2 units), sum
  int* status;
};

__device__ __forceinline__ void ldsm_x4(uint32_t a, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t a, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two fp32 values as bf16 pairs: hi = bf16(x) (a in the low half), lo = bf16(x - hi).
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  const __nv_bfloat162 l = __floats2bfloat162_rn(a - __low2float(h), b - __high2float(h));
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar,
                                            uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, "
      "%4}], [%5], %6;" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(pol)
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("{ .reg .b64 st; mbarrier.arrive.shared::cta.b64 st, [%0]; }" ::"r"(smem_addr(bar)) : "memory");
}
template <int kThreads>
__device__ __forceinline__ void named_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}
__device__ __forceinline__ float bfv(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

// The usable length of sequence s (0 when it is out of range).
__device__ __forceinline__ int seq_len(const PagedArgs& a, int s) {
  const int n = __ldg(a.kv_len + s);
  return n < 0 || n > ((long long)a.max_pages << a.log_page) ? 0 : n;
}

// Four output values of row r of a (sequence, head group) from the joined sums; M in log2 units.
template <int D>
__device__ __forceinline__ void finish(const PagedArgs& a, size_t qrow, int r, int d, float4 y, float M, float L, uint2 gate) {
  const size_t at = qrow + (size_t)r * D + d;
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  float v[4] = {y.x * inv, y.y * inv, y.z * inv, y.w * inv};
  if (a.gate) {
    const float g[4] = {bfv(gate.x & 0xFFFF), bfv(gate.x >> 16), bfv(gate.y & 0xFFFF), bfv(gate.y >> 16)};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // 2 ulp, but 0 where the sum is above 2^126.  Far below that 1 + e^-g is e^-g, and half the gate twice keeps
      // what a large value leaves of it.
      const float half = expf(0.5f * g[e]);
      v[e] = g[e] < -60.0f ? v[e] * half * half : __fdividef(v[e], 1.0f + expf(-g[e]));
    }
  }
  const __nv_bfloat162 p0 = __floats2bfloat162_rn(v[0], v[1]), p1 = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(a.out + at) = make_uint2(*reinterpret_cast<const uint32_t*>(&p0), *reinterpret_cast<const uint32_t*>(&p1));
  if (a.lse && d == 0) a.lse[qrow / D + r] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// a / b in 32 bits where that holds a (a 64-bit division is a call of some hundred instructions).
__device__ __forceinline__ long long div64(long long a, int b) {
  return a >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

template <int D, bool kWide>
struct PaCfg {
  static constexpr int kRows = kPieceBytes / (2 * D);      // positions per piece
  // Consumer warps, two stages each: a warp takes every kWarps-th piece, so it alone waits on its stages'
  // barriers and sees each of their phases (copies of other warps' stages may land in any order).
  static constexpr int kWarps = kWide ? 4 : 5;
  static constexpr int kStages = 2 * kWarps;
  static constexpr int kThreads = (kWarps + 1) * 32, kConsumers = kWarps * 32;
  static constexpr int kM = kWide ? 16 : 8;                // query rows kept
  static constexpr int kLd = D + 8;                        // padded row of the join buffer
  static constexpr int kJoin = kWarps * kM * kLd * 4 > 16 * kPaGrid * 4 ? kWarps * kM * kLd * 4 : 16 * kPaGrid * 4;
  static constexpr int kSmem = 1024 + kStages * 2 * kPieceBytes + kJoin;
  static_assert(kSmem <= 225 * 1024, "shared memory of one CTA");
};

// A run of pieces of one (sequence, head): [p0, p1) of its np; u = the line's index of its piece 0.
struct Segment {
  int s, h, p0, p1, np, len;
  long long u;
};
struct Walk {
  long long u, u1;       // next piece and end of the run
  int s, h, p, np, len;  // the piece's sequence, head and number; the sequence's pieces and length
  bool whole;            // (sequence, head)s are not cut: those that start in the run, to their ends
  template <int kRows>
  __device__ bool next(const PagedArgs& a, Segment& g) {
    if (u >= u1) return false;
    while (p >= np) {  // the next head, or the next sequence that has positions
      p = 0;
      if (np > 0 && ++h < a.Hkv) continue;
      h = 0;
      do {
        if (++s >= a.S) return false;
        len = seq_len(a, s);
        np = (len + kRows - 1) / kRows;
      } while (np == 0);
    }
    g.s = s;
    g.h = h;
    g.p0 = p;
    g.p1 = whole ? np : (int)min((long long)np, p + u1 - u);
    g.np = np;
    g.len = len;
    g.u = u - p;
    u += g.p1 - p;
    p = g.p1;
    return true;
  }
};

template <int D, bool kWide>
__global__ void __launch_bounds__(PaCfg<D, kWide>::kThreads, 1)
    paged_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap) {
  using C = PaCfg<D, kWide>;
  constexpr int kR = C::kRows, kM = C::kM, kLd = C::kLd;
  constexpr int kPaWarps = C::kWarps, kPaThreads = C::kThreads, kPaConsumers = C::kConsumers;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t full[C::kStages], empty[C::kStages], s_join;
  __shared__ int s_bad[C::kStages];          // boxes of the stage whose page is out of range (bit per box)
  __shared__ long long s_scan[kPaThreads / 32];
  __shared__ int s_most[kPaThreads / 32];
  __shared__ int s_first[6], s_abort, s_last[2];
  __shared__ float s_ml[kPaWarps][kM][2], s_row[16];
  const uint32_t ring = (smem_addr(dyn) + 1023u) & ~1023u;
  float* join = reinterpret_cast<float*>(dyn + (ring - smem_addr(dyn)) + C::kStages * 2 * kPieceBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
#ifdef VP_WAIT_TEST
  // Wait-test hook (workspace word kWsTestSkip), for the first CTA: 1 leaves out the arrival that frees its first
  // stage, 2 the copies of its first piece; 3, for every CTA that joins parts: a copy of theirs; 4: its first
  // consumer warp's first wait runs out at once.
  const int hook = ((const volatile int*)a.status)[kWsTestSkip / sizeof(int)];
#else
  constexpr int hook = 0;
#endif
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&s_join, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (tid < 6) s_first[tid] = 0;
  // Sequences without positions: zeros, and the status of those out of range.
  for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
    if (seq_len(a, s) > 0) continue;
    if (tid == 0 && __ldg(a.kv_len + s) != 0) report_unless(a.status, VP_ERR_SHAPE, VP_ERR_TIMEOUT);
    uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)s * a.Hq * D);
    for (int i = tid; i < a.Hq * D / 8; i += kPaThreads) o[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int i = tid; i < a.Hq; i += kPaThreads) a.lse[(size_t)s * a.Hq + i] = -INFINITY;
  }
  // The line: pieces before each thread's share of the sequences, and in all.
  const int per = (a.S + kPaThreads - 1) / kPaThreads, sa = min(a.S, tid * per), sb = min(a.S, sa + per);
  long long mine = 0;
  int most = 0;  // pieces of the longest sequence
  for (int s = sa; s < sb; ++s) {
    const int np = (seq_len(a, s) + kR - 1) / kR;
    mine += np;
    most = max(most, np);
  }
  long long pre = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xFFFFFFFFu, pre, o);
    if (lane >= o) pre += v;
  }
  most = (int)__reduce_max_sync(0xFFFFFFFFu, (unsigned)most);
  if (lane == 31) s_scan[warp] = pre, s_most[warp] = most;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kPaThreads / 32; ++w) {
    if (w < warp) pre += s_scan[w];
    total += s_scan[w];
    most = max(most, s_most[w]);
  }
  pre -= mine;  // exclusive
  const long long U = total * a.Hkv;
  // Short sequences are not cut: a CTA takes those that start in its run.  The longest one then adds to the run
  // (or is the run, where there are fewer (sequence, head)s than CTAs), and nothing has to be joined.  64
  // sequences of 100 to 300 positions, 8 x 128 heads: 25 us cut, 20 us whole.
  const long long run = max((U + gridDim.x - 1) / gridDim.x, (long long)kMinPieces);
  const bool whole = most + (a.S * a.Hkv > (int)gridDim.x ? run : 0) <= run + kJoinCost;
  const int c = blockIdx.x;
  // Few (sequence, head)s: each is cut by itself into equal parts of at most `part` pieces, one per CTA.  A run of
  // the line would end one and start another, two results to join in turn; the parts are longer than the
  // runs, but not by more than that costs.  One sequence of 2,000 positions: 21 us in runs, 13 us in parts.
  const int heads = a.S * a.Hkv;
  const long long part = heads < (int)gridDim.x ? max((U + gridDim.x - heads - 1) / (gridDim.x - heads), (long long)kMinPieces) : 0;
  const bool even = !whole && heads < (int)gridDim.x && part - run <= kJoinCost;
  int ctas;
  Walk walk;
  if (even) {
    const int L = (int)part;
    int parts = 0;  // of the thread's sequence (fewer sequences than threads here)
    if (tid < a.S) parts = ((seq_len(a, tid) + kR - 1) / kR + L - 1) / L;
    int before = parts;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
      if (lane >= o) before += v;
    }
    __syncthreads();  // s_most is read
    if (lane == 31) s_most[warp] = before;
    __syncthreads();
    ctas = 0;
#pragma unroll
    for (int w = 0; w < kPaThreads / 32; ++w) {
      if (w < warp) before += s_most[w];
      ctas += s_most[w];
    }
    ctas *= a.Hkv;
    if (c >= ctas) return;
    const int at = (before - parts) * a.Hkv;
    if (c >= at && c < before * a.Hkv) {
      const int np = (seq_len(a, tid) + kR - 1) / kR, h = (c - at) / parts, x = c - at - h * parts;
      s_first[0] = tid;
      s_first[1] = h;
      s_first[2] = (int)((long long)x * np / parts);
      s_first[3] = (int)((long long)(x + 1) * np / parts);
      s_first[4] = c - x;
      s_first[5] = c - x + parts - 1;
    }
    __syncthreads();
    walk.u = 0;
    walk.u1 = s_first[3] - s_first[2];
  } else {
    ctas = whole ? (int)min((long long)gridDim.x, U) : (int)min((long long)gridDim.x, (U + kMinPieces - 1) / kMinPieces);
    if (c >= ctas) return;
    const long long u0 = div64(c * U, ctas), u1 = div64((c + 1) * U, ctas);
    if (u0 >= pre * a.Hkv && u0 < (pre + mine) * a.Hkv) {
      long long at = pre * a.Hkv;
      for (int s = sa; s < sb; ++s) {
        const int np = (seq_len(a, s) + kR - 1) / kR;
        if (u0 < at + (long long)np * a.Hkv) {
          s_first[0] = s;
          const int h = (int)div64(u0 - at, np);
          s_first[1] = h;
          s_first[2] = (int)(u0 - at - (long long)h * np);
          break;
        }
        at += (long long)np * a.Hkv;
      }
    }
    __syncthreads();
    walk.u = u0;
    walk.u1 = u1;
  }
  walk.s = s_first[0];
  walk.h = s_first[1];
  walk.p = s_first[2];
  walk.len = seq_len(a, walk.s);
  walk.np = (walk.len + kR - 1) / kR;
  walk.whole = whole;
  if (whole && walk.p > 0) {  // this one starts in an earlier run
    walk.u += walk.np - walk.p;
    walk.p = walk.np;
  }
  Segment g;

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {  // a converged warp
    for (uint32_t i = hook == 4 && c == 0 && warp == 0 && bar == full ? kMbarPolls : 0; i < kMbarPolls; ++i) {
      if (__all_sync(0xFFFFFFFFu, mbar_try_wait_hint(bar, parity, 20000u))) return true;
      if (__any_sync(0xFFFFFFFFu, *(volatile int*)&s_abort)) return false;
    }
    *(volatile int*)&s_abort = 1;
    atomicExch(a.status, (int)VP_ERR_TIMEOUT);
    return false;
  };

  if (warp == kPaWarps) {
    // ------------------------------------------------------------ producer
    // 32 pieces at a time: each lane looks up the pages of one, then they are issued in turn.
    const uint64_t pol = l2_evict_first_policy();
    const int boxes = kR >> a.log_box, box_bytes = 2 * D << a.log_box, slots = (1 << a.log_page) - 1;
    constexpr int kMaxBoxes = kR / 16;
    int n = 0, st = 0;
    uint32_t par = 1;  // the first round of empty stages passes
    bool ok = true;
    while (ok && walk.template next<kR>(a, g)) {
      const int32_t* table = a.pages + (size_t)g.s * a.max_pages;
      for (int base = g.p0; ok && base < g.p1; base += 32) {
        int rows[kMaxBoxes], bad = 0, good = 0;
        const int p = base + lane;
#pragma unroll
        for (int j = 0; j < kMaxBoxes; ++j) {
          const int pos = p * kR + (j << a.log_box);
          rows[j] = -1;
          if (j >= boxes || p >= g.p1 || pos >= g.len) continue;
          const int pg = __ldg(table + (pos >> a.log_page));
          if (pg >= 0 && pg < a.n_pages) {
            rows[j] = ((pg * a.Hkv + g.h) << a.log_page) + (pos & slots);
            ++good;
          } else {
            bad |= 1 << j;
          }
        }
        if (bad) report_unless(a.status, VP_ERR_SHAPE, VP_ERR_TIMEOUT);
        const int cnt = min(32, g.p1 - base);
        for (int i = 0; i < cnt; ++i, ++n) {
          int row[kMaxBoxes];
#pragma unroll
          for (int j = 0; j < kMaxBoxes; ++j) row[j] = __shfl_sync(0xFFFFFFFFu, rows[j], i);
          const int bd = __shfl_sync(0xFFFFFFFFu, bad, i), gd = __shfl_sync(0xFFFFFFFFu, good, i);
          if (!(ok = wait(&empty[st], par))) break;
          if (elect_one()) {
            s_bad[st] = bd;
            const uint32_t bar = smem_addr(&full[st]), dst = ring + st * 2 * kPieceBytes;
            mbar_arrive_expect_tx(&full[st], gd * 2 * box_bytes);
#pragma unroll
            for (int j = 0; j < kMaxBoxes; ++j) {
              if (row[j] < 0 || (hook == 2 && blockIdx.x == 0 && n == 0)) continue;
              tma_load_3d(dst + j * box_bytes, &kmap, 0, row[j], 0, bar, pol);
              tma_load_3d(dst + kPieceBytes + j * box_bytes, &vmap, 0, row[j], 0, bar, pol);
            }
          }
          __syncwarp();
          if (++st == C::kStages) st = 0, par ^= 1;
        }
      }
    }
    // Every copy lands before this warp leaves, and with it the shared memory: a consumer whose wait ran out may
    // have left without them, after this warp's last wait.
    for (int i = 0; i < min(n, C::kStages); ++i) mbar_wait_bounded(&full[i], ((n - 1 - i) / C::kStages) & 1);
    return;
  }

  // -------------------------------------------------------------- consumers
  const int gq = lane >> 2, cq = lane & 3;
  int n = 0;                       // the run's pieces before the segment
  int st = warp;                   // the warp's next stage (warp or warp + kWarps), and its phase
  uint32_t par = 0;
  // A wait of this warp ran out: it takes and frees no more stages.  Its phases would be out of step (a parity two
  // uses ahead of an unfinished phase reads as complete), and a stage freed so would be armed a second time.
  bool dead = false;
  int pend_s[2] = {-1, -1}, pend_h[2] = {0, 0};
  int pend_first[2] = {0, 0}, pend_last[2] = {0, 0};
  const int sub = 128 << a.log_box;  // bytes between a box's 64-column groups
  while (walk.template next<kR>(a, g)) {
    const size_t qrow = ((size_t)g.s * a.Hq + (size_t)g.h * a.G) * D;
    // Q fragments: rows gq (and gq + 8) of the group's heads; rows past G are zero
    uint32_t qf[D / 16][kWide ? 4 : 2];
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
      for (int e = 0; e < (kWide ? 4 : 2); ++e) {
        const int r = kWide ? gq + 8 * (e & 1) : gq, d = 16 * ks + 2 * cq + 8 * (kWide ? e >> 1 : e);
        qf[ks][e] = r < a.G ? __ldg(reinterpret_cast<const uint32_t*>(a.q + qrow + (size_t)r * D + d)) : 0u;
      }
    }
    if (a.gate)  // used at the segment's end: on its way meanwhile (16 positions of one sequence: 7.3 -> 6.8 us)
      for (int i = tid; i < a.G * D / 64; i += kPaConsumers)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(a.gate + qrow + 64 * i));
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    constexpr int kH = kWide ? 2 : 1;  // row groups with maxima of their own
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    // the segment's first piece of this warp: the run's pieces go round the warps
    const int skip = (warp - n % kPaWarps + kPaWarps) % kPaWarps;
    n += g.p1 - g.p0;
    for (int p = g.p0 + skip; p < g.p1; p += kPaWarps) {
      if (dead || !wait(&full[st], par)) {
        dead = true;
        break;
      }
      const int at = st;
      st += kPaWarps;
      if (st >= C::kStages) st = warp, par ^= 1;
      const uint32_t kb = ring + at * 2 * kPieceBytes, vb = kb + kPieceBytes;
      const int valid = g.len - p * kR, bad = *(volatile int*)&s_bad[at];
      const bool masked = valid < kR || bad;
      auto seen = [&](int key) { return key < valid && !((bad >> (key >> a.log_box)) & 1); };
      if (masked) {
        // values of positions that take no part: zeros (0 * NaN would not vanish)
        for (int i = lane; i < kR * (D / 8); i += 32) {
          const int r = i / (D / 8), ch = i % (D / 8);
          if (!seen(r))
            sts128(vb + (r >> a.log_box) * (2 * D << a.log_box) + (ch >> 3) * sub + (r & ((1 << a.log_box) - 1)) * 128 + ((ch & 7) << 4),
                   make_uint4(0, 0, 0, 0));
        }
        __syncwarp();
      }
      // S = Q K^T: 16 positions (two n-tiles) at a time
      float s[kR / 8][4];
#pragma unroll
      for (int i = 0; i < kR / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll
      for (int t = 0; t < kR / 16; ++t) {
        const int r = 16 * t + ((lane >> 4) << 3) + (lane & 7);
        const uint32_t row = kb + (r >> a.log_box) * (2 * D << a.log_box) + (r & ((1 << a.log_box) - 1)) * 128;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const int ch = 2 * ks + ((lane >> 3) & 1);
          uint32_t b0, b1, b2, b3;
          ldsm_x4(row + (ch >> 3) * sub + (((ch & 7) ^ (lane & 7)) << 4), b0, b1, b2, b3);
          if constexpr (kWide) {
            mma_bf16(s[2 * t], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b0, b1);
            mma_bf16(s[2 * t + 1], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b2, b3);
          } else {
            mma_bf16(s[2 * t], qf[ks][0], 0u, qf[ks][1], 0u, b0, b1);
            mma_bf16(s[2 * t + 1], qf[ks][0], 0u, qf[ks][1], 0u, b2, b3);
          }
        }
      }
      // online softmax (log2 units)
      float mx[2] = {m[0], m[1]};
#pragma unroll
      for (int i = 0; i < kR / 8; ++i)
#pragma unroll
        for (int e = 0; e < 2 * kH; ++e) {
          float v = s[i][e] * a.scale2;
          if (masked && !seen(8 * i + 2 * cq + (e & 1))) v = -INFINITY;
          s[i][e] = v;
          mx[e >> 1] = fmaxf(mx[e >> 1], v);
        }
      bool grow = false;
      float alpha[2] = {1.0f, 1.0f};
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 2));
        if (mx[h] > m[h]) {
          alpha[h] = exp2f(m[h] - mx[h]);
          grow = true;
        }
        m[h] = mx[h];
        l[h] *= alpha[h];
      }
      if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= alpha[0];
          o[i][1] *= alpha[0];
          o[i][2] *= alpha[kWide ? 1 : 0];
          o[i][3] *= alpha[kWide ? 1 : 0];
        }
      }
      const float m0 = m[0] == -INFINITY ? 0.0f : m[0], m1 = m[1] == -INFINITY ? 0.0f : m[1];
      uint32_t hi[kR / 8][kH], lo[kR / 8][kH];
#pragma unroll
      for (int i = 0; i < kR / 8; ++i)
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          const float mm = h ? m1 : m0, x = exp2f(s[i][2 * h] - mm), y = exp2f(s[i][2 * h + 1] - mm);
          l[h] += x + y;
          split_bf16(x, y, hi[i][h], lo[i][h]);
        }
      // O += P V
#pragma unroll
      for (int t = 0; t < kR / 16; ++t) {
        const int r = 16 * t + (lane & 15);
        const uint32_t row = vb + (r >> a.log_box) * (2 * D << a.log_box) + (r & ((1 << a.log_box) - 1)) * 128;
#pragma unroll
        for (int np = 0; np < D / 16; ++np) {
          const int ch = 2 * np + (lane >> 4);
          uint32_t b0, b1, b2, b3;
          ldsm_x4_t(row + (ch >> 3) * sub + (((ch & 7) ^ (lane & 7)) << 4), b0, b1, b2, b3);
          if constexpr (kWide) {
            mma_bf16(o[2 * np], hi[2 * t][0], hi[2 * t][1], hi[2 * t + 1][0], hi[2 * t + 1][1], b0, b1);
            mma_bf16(o[2 * np], lo[2 * t][0], lo[2 * t][1], lo[2 * t + 1][0], lo[2 * t + 1][1], b0, b1);
            mma_bf16(o[2 * np + 1], hi[2 * t][0], hi[2 * t][1], hi[2 * t + 1][0], hi[2 * t + 1][1], b2, b3);
            mma_bf16(o[2 * np + 1], lo[2 * t][0], lo[2 * t][1], lo[2 * t + 1][0], lo[2 * t + 1][1], b2, b3);
          } else {  // rows 0..7: hi, rows 8..15: lo
            mma_bf16(o[2 * np], hi[2 * t][0], lo[2 * t][0], hi[2 * t + 1][0], lo[2 * t + 1][0], b0, b1);
            mma_bf16(o[2 * np + 1], hi[2 * t][0], lo[2 * t][0], hi[2 * t + 1][0], lo[2 * t + 1][0], b2, b3);
          }
        }
      }
      if (masked) fence_proxy_async_smem();  // the zeros, before the stage's next copy
      __syncwarp();
      if (lane == 0 && !(hook == 1 && c == 0 && at == 0 && par == 0)) mbar_arrive(&empty[at]);
    }
    // ---- the warps' results of this (sequence, head)
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
      l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
      if (cq == 0) {
        s_ml[warp][gq + 8 * h][0] = m[h];
        s_ml[warp][gq + 8 * h][1] = l[h];
      }
    }
    float* jw = join + (size_t)warp * kM * kLd;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const int d = 8 * i + 2 * cq;
      if constexpr (kWide) {
        *reinterpret_cast<float2*>(jw + gq * kLd + d) = make_float2(o[i][0], o[i][1]);
        *reinterpret_cast<float2*>(jw + (gq + 8) * kLd + d) = make_float2(o[i][2], o[i][3]);
      } else {
        *reinterpret_cast<float2*>(jw + gq * kLd + d) = make_float2(o[i][0] + o[i][2], o[i][1] + o[i][3]);
      }
    }
    named_sync<kPaConsumers>();
    const bool complete = g.p0 == 0 && g.p1 == g.np;
    const int slot = g.p0 == 0 ? 1 : 0;
    for (int i = tid; i < a.G * (D / 4); i += kPaConsumers) {
      const int r = i / (D / 4), d = 4 * (i % (D / 4));
      float M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int w = 0; w < kPaWarps; ++w) M = fmaxf(M, s_ml[w][r][0]);
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kPaWarps; ++w) {
        const float mw = s_ml[w][r][0], f = mw == -INFINITY ? 0.0f : exp2f(mw - M);
        const float4 v = *reinterpret_cast<const float4*>(join + ((size_t)w * kM + r) * kLd + d);
        L += f * s_ml[w][r][1];
        y.x += f * v.x;
        y.y += f * v.y;
        y.z += f * v.z;
        y.w += f * v.w;
      }
      if (complete) {
        uint2 gate = make_uint2(0, 0);
        if (a.gate) gate = __ldg(reinterpret_cast<const uint2*>(a.gate + qrow + (size_t)r * D + d));
        finish<D>(a, qrow, r, d, y, M, L, gate);
      } else {
        const size_t ps = (size_t)c * 2 + slot;
        __stcg(reinterpret_cast<float4*>(a.part_o + (ps * 16 + r) * D + d), y);
        if (d == 0) __stcg(reinterpret_cast<float2*>(a.part_ml + (ps * 16 + r) * 2), make_float2(M, L));
      }
    }
    if (!complete) {
      pend_s[slot] = g.s;
      pend_h[slot] = g.h;
      // the CTAs that own the (sequence, head)'s first and last piece
      if (even) {
        pend_first[slot] = s_first[4];
        pend_last[slot] = s_first[5];
      } else {
        const long long a0 = (g.u + 1) * ctas - 1, a1 = (g.u + g.np) * ctas - 1;
        pend_first[slot] = U >> 31 ? (int)(a0 / U) : (int)div64(a0, (int)U);
        pend_last[slot] = U >> 31 ? (int)(a1 / U) : (int)div64(a1, (int)U);
      }
      // in range whatever is written to kv_len meanwhile
      pend_first[slot] = max(0, min(pend_first[slot], ctas - 1));
      pend_last[slot] = max(pend_first[slot], min(pend_last[slot], ctas - 1));
    }
    named_sync<kPaConsumers>();  // the join buffer is free
  }
  // -------------------------------------------------------------- results shared with other CTAs
  if (pend_s[0] < 0 && pend_s[1] < 0) return;
  __threadfence();
  named_sync<kPaConsumers>();
  if (tid < 2 && pend_s[tid] >= 0) {
    unsigned* cnt = a.counters + (size_t)pend_s[tid] * a.Hkv + pend_h[tid];
    const unsigned old = atom_add_acq_rel_gpu(cnt, 1);
    s_last[tid] = old == (unsigned)(pend_last[tid] - pend_first[tid]);
    if (s_last[tid]) *cnt = 0;  // every contributor has arrived
  }
  named_sync<kPaConsumers>();
  // The last contributor's copies land in the ring, which is free: every part's maxima and sums (one copy, at
  // the ring's end) and the parts' outputs, as many at a time as fit, a copy per lane of the first warp.
  constexpr int kItems = (kM * (D / 4) + kPaConsumers - 1) / kPaConsumers;  // float4 sums per thread
  constexpr int kMlBytes = 256 * kPaGrid, kRing = C::kStages * 2 * kPieceBytes - kMlBytes;
  const uint8_t* ring_p = dyn + (ring - smem_addr(dyn));
  const float* ml = reinterpret_cast<const float*>(ring_p + kRing);      // [2 part - 1][16][2]
  float(*s_w)[kPaGrid] = reinterpret_cast<float(*)[kPaGrid]>(join);      // [row][part]: the parts' weights
  const int part_bytes = a.G * D * 4, room = kRing / part_bytes;
  uint32_t jpar = 0;
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    if (pend_s[e] < 0 || !*(volatile int*)&s_last[e]) continue;
    const int first = pend_first[e], cnt = pend_last[e] - first + 1;
    const size_t qrow = ((size_t)pend_s[e] * a.Hq + (size_t)pend_h[e] * a.G) * D;
    // part x lies in its CTA's end slot when it is the first, else in the start slot
    // The first warp: parts x0 .. x0 + n - 1, and every part's maxima.  False, and nothing copied, once a wait of
    // the CTA has run out: its ring may not be free, nor the barrier's last phase complete.
    auto fetch = [&](int x0, int n, bool with_ml) -> bool {
      if (__any_sync(0xFFFFFFFFu, *(volatile int*)&s_abort)) return false;
      const uint32_t bar = smem_addr(&s_join), ml_bytes = (2 * cnt - 1) * 128;
      asm volatile("fence.proxy.async;" ::: "memory");  // the other CTAs' stores, before these copies read them
      if (lane == 0) {
        mbar_arrive_expect_tx(&s_join, n * part_bytes + (with_ml ? ml_bytes : 0));
        if (with_ml && hook != 3) bulk_load(ring + kRing, a.part_ml + ((size_t)first * 2 + 1) * 32, ml_bytes, bar);
      }
      __syncwarp();
      for (int x = x0 + lane; x < x0 + n; x += 32)
        bulk_load(ring + (x - x0) * part_bytes, a.part_o + ((size_t)(first + x) * 2 + (x == 0)) * (16 * D), part_bytes, bar);
      return true;
    };
    // The warp that copied does not leave before its copies have landed, even if the wait is called off.
    auto landed = [&](bool copied) {
      if (!wait(&s_join, jpar) && copied) mbar_wait_bounded(&s_join, jpar);
      jpar ^= 1;
    };
    bool copied = warp == 0 && fetch(0, min(room, cnt), true);
    // the gate, while the parts are on their way
    uint2 gate[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int i = tid + k * kPaConsumers;
      gate[k] = make_uint2(0, 0);
      if (a.gate && i < a.G * (D / 4))
        gate[k] = __ldg(reinterpret_cast<const uint2*>(a.gate + qrow + (size_t)(i / (D / 4)) * D + 4 * (i % (D / 4))));
    }
    landed(copied);
    // part 0's maxima and sums lie first, part x's at index 2 x - 1 (the slots in between are other tiles')
    for (int i = tid; i < a.G * cnt; i += kPaConsumers) {
      const int r = i / cnt, x = i - r * cnt;
      float M = -INFINITY;
#pragma unroll 8
      for (int z = 0; z < cnt; ++z) M = fmaxf(M, ml[max(2 * z - 1, 0) * 32 + 2 * r]);
      const float m = ml[max(2 * x - 1, 0) * 32 + 2 * r];
      s_w[r][x] = m == -INFINITY ? 0.0f : exp2f(m - M);
      if (x == 0) s_row[r] = M;
    }
    named_sync<kPaConsumers>();
    float4 y[kItems];
    float L[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) y[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f), L[k] = 0.0f;
    for (int x0 = 0; x0 < cnt; x0 += room) {
      const int n = min(room, cnt - x0);
      if (x0) {
        named_sync<kPaConsumers>();  // the ring is read
        copied = warp == 0 && fetch(x0, n, false);
        landed(copied);
      }
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const int i = tid + k * kPaConsumers;
        if (i >= a.G * (D / 4)) break;
        const int r = i / (D / 4);
        const float* w = s_w[r] + x0;
        const uint8_t* src = ring_p + 16 * i;
#pragma unroll 8
        for (int x = 0; x < n; ++x) {  // in order
          const float f = w[x];
          L[k] += f * ml[max(2 * (x0 + x) - 1, 0) * 32 + 2 * r + 1];
          const float4 v = *reinterpret_cast<const float4*>(src + x * part_bytes);
          y[k].x += f * v.x;
          y[k].y += f * v.y;
          y[k].z += f * v.z;
          y[k].w += f * v.w;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int i = tid + k * kPaConsumers;
      if (i >= a.G * (D / 4)) break;
      const int r = i / (D / 4);
      finish<D>(a, qrow, r, 4 * (i % (D / 4)), y[k], s_row[r], L[k], gate[k]);
    }
    named_sync<kPaConsumers>();
  }
}

bool al(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool attend_shape_ok(int S, int Hq, int Hkv, int D) {
  return S >= 1 && S <= 8192 && Hkv >= 1 && Hkv <= 1024 && (size_t)S * Hkv <= kServeMaxCounters && Hq >= Hkv && Hq % Hkv == 0 &&
         Hq / Hkv <= 16 && (D == 64 || D == 128 || D == 256);
}

struct PagedWs {
  size_t part_o, part_ml, total;
};
PagedWs paged_ws(int D) {  // the counters, one per (sequence, head), lie at kServeCounters
  PagedWs w;
  w.part_o = kServeData;
  w.part_ml = w.part_o + sizeof(float) * kPaGrid * 2 * 16 * (size_t)D;
  w.total = w.part_ml + sizeof(float) * kPaGrid * 2 * 16 * 2;
  return w;
}

template <int D, bool kWide>
cudaError_t launch_paged(const PagedArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, int grid, cudaStream_t s) {
  constexpr int kSmem = PaCfg<D, kWide>::kSmem;
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !done[dev].load()) {
    e = cudaFuncSetAttribute(paged_kernel<D, kWide>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev].store(true);
  }
  paged_kernel<D, kWide><<<grid, (PaCfg<D, kWide>::kThreads), kSmem, s>>>(a, kmap, vmap);
  return cudaGetLastError();
}

}  // namespace

}  // namespace vp

using namespace vp;

extern "C" {

size_t vp_paged_attention_workspace_bytes(int S, int Hq, int Hkv, int D) {
  if (!attend_shape_ok(S, Hq, Hkv, D)) return 0;
  return paged_ws(D).total;
}

vp_status vp_paged_attention(const vp_paged_cache* cache, const void* q, const int32_t* kv_len, int S, int Hq,
                             float scale, const void* gate, void* out, float* lse, void* ws, size_t ws_bytes,
                             void* stream) {
  vp_status st = check_cache(cache);
  if (st != VP_OK) return st;
  if (!q || !kv_len || !out || !ws || !std::isfinite(scale * kLog2e)) return VP_ERR_INVALID_ARG;
  const vp_paged_cache& c = *cache;
  if (!attend_shape_ok(S, Hq, c.Hkv, c.D)) return VP_ERR_SHAPE;
  if (!al(q, 16) || !al(kv_len, 4) || (gate && !al(gate, 16)) || !al(out, 16) || (lse && !al(lse, 4)) || !al(ws, 256))
    return VP_ERR_ALIGNMENT;
  if (ws_bytes < vp_paged_attention_workspace_bytes(S, Hq, c.Hkv, c.D)) return VP_ERR_WORKSPACE;
  int sms = 0;
  if ((st = device_sm_count(&sms)) != VP_OK) return st;
  PFN_cuTensorMapEncodeTiled_v12000 encode;
  if ((st = tensor_map_encoder(&encode)) != VP_OK) return st;
  const PagedWs w = paged_ws(c.D);
  uint8_t* b = static_cast<uint8_t*>(ws);
  PagedArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.gate = static_cast<const uint16_t*>(gate);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.kv_len = kv_len, a.pages = c.pages;
  a.S = S, a.Hq = Hq, a.Hkv = c.Hkv, a.G = Hq / c.Hkv, a.n_pages = c.n_pages, a.max_pages = c.max_pages;
  a.log_page = 4;
  while ((1 << a.log_page) < c.page_size) ++a.log_page;
  const int rows = kPieceBytes / (2 * c.D);
  a.log_box = 4;
  while ((1 << a.log_box) < std::min(rows, c.page_size)) ++a.log_box;
  a.scale2 = scale * kLog2e;
  a.counters = reinterpret_cast<unsigned*>(b + kServeCounters);
  a.part_o = reinterpret_cast<float*>(b + w.part_o);
  a.part_ml = reinterpret_cast<float*>(b + w.part_ml);
  a.status = reinterpret_cast<int*>(b);
  // keys and values as [D / 64][rows of all pages and heads][64]: a box is the piece's rows, all columns
  CUtensorMap maps[2];
  for (int i = 0; i < 2; ++i) {
    const cuuint64_t dims[3] = {64, (cuuint64_t)c.n_pages * c.Hkv * c.page_size, (cuuint64_t)c.D / 64};
    const cuuint64_t strides[2] = {(cuuint64_t)c.D * 2, 128};
    const cuuint32_t box[3] = {64, 1u << a.log_box, (cuuint32_t)c.D / 64}, step[3] = {1, 1, 1};
    if (encode(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, i ? c.v : c.k, dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return VP_ERR_UNSUPPORTED;
  }
  const int grid = std::min(sms, kPaGrid);
  cudaStream_t s = (cudaStream_t)stream;
  const bool wide = a.G > 8;
  cudaError_t e;
  if (c.D == 64)
    e = wide ? launch_paged<64, true>(a, maps[0], maps[1], grid, s) : launch_paged<64, false>(a, maps[0], maps[1], grid, s);
  else if (c.D == 128)
    e = wide ? launch_paged<128, true>(a, maps[0], maps[1], grid, s) : launch_paged<128, false>(a, maps[0], maps[1], grid, s);
  else
    e = wide ? launch_paged<256, true>(a, maps[0], maps[1], grid, s) : launch_paged<256, false>(a, maps[0], maps[1], grid, s);
  return e == cudaSuccess ? VP_OK : cuda_fail(e);
}

}  // extern "C"
