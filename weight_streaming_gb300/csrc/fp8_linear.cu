// Linear layer of a block-quantised FP8 checkpoint on block-quantised activations
// (vp_linear_fp8_block).
//
// Mathematics: y[m][n] = sum_b xs[m][b] ws[n / 128][b] (sum_{k in b} xq[m][k] w[n][k]).  The products are
// exact in fp32 (e4m3 has 4 significant bits); the scales differ from block to block, so each inner
// sum of 128 products leaves the tensor core's accumulator, is scaled and added to an fp32 register.
//
// Design: one persistent CTA per SM; a producer warp, an MMA warp and eight epilogue warps.  Above 128
// tokens two CTAs form a pair (cta_group::2) on a tile of 256 tokens x 256 weight rows: each loads its
// 128 tokens and half of the weights, 32 KB a K block in place of 48 KB.
//  * Operands: one stage of the shared-memory ring is one 128-wide K block: the tokens by a tiled TMA
//    load (128-byte swizzle; rows past M and columns past K read zero), the weights by one bulk copy
//    of 16 KB per 128 rows (packed in the swizzled order).
//  * tcgen05.mma kind::f8f6f4, 128 lanes x kBC columns, four K = 32 steps per block, into one of
//    512 / kBC tensor-memory buffers (each block starts from zero); the epilogue warps read the buffer
//    (tcgen05.ld), scale and accumulate in registers while the next block's MMAs run.
//  * Tokens on the lanes for M > 64 (the factor xs ws is one scalar per thread and block), weights on
//    the lanes for M <= 64 (16, 32 or 64 token columns; the factors come by shuffles): a small batch
//    then pads to 16 columns instead of 128 lanes, and the weight stream is what it waits for.
//  * Work: whole rounds of output tiles first; each remaining tile is cut along K into as many parts as
//    there are CTAs for it (at most 16).  Where few narrow tiles are all of the work, a tile's parts are
//    a cluster and join through shared memory; else they go through fp32 partials in the workspace,
//    which the last CTA to arrive (a counter, nobody waits) adds.  In K order both times, so results
//    do not depend on the arrival order.
//
// What bounds it, N x K: 8 tokens, 5120 x 17408 (89.5 MB of weights) take 20.8 us, 4.3 TB/s: the stream at about
// 6.5 TB/s and 7 us of launch, first copies, last block and join.  200 tokens, 16384 x 5120: 26 us, 64 pairs
// with a tile each.  100 tokens, 5120 x 17408: 28.7 us; 34816 x 5120, more tiles than CTAs: 29.6 us for 8 tokens
// (6.0 TB/s), 38.8 for 100.  4096 tokens, 17408 x 5120: 283 to 291 us at the power limit, 2.5 PFLOP/s, 258 us in the
// first calls (cuBLAS' bf16 1.9 PFLOP/s): 62 % of the tensor cycles.  A K block of a pair's tile is 512 cycles of
// MMAs and about 330 of reading and scaling its sums, and takes 760; two tensor-memory buffers (all there is at 128 x
// 256 sums) would allow 512, so about 680 cycles of a buffer's turn are commits, arrivals and waits.
//
// Waits are bounded: on a timeout the CTA reports VP_ERR_TIMEOUT, waits (again with a limit) for its copies and
// MMAs and frees its tensor memory.  Timed out or not, the copying warp leaves last: see its end.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "errors.h"
#include "fp8_block.h"
#include "internal.h"
#include "ptx.cuh"
#include "serve_ws.h"
#include "tma.h"
#include "verify.h"

namespace vp {

namespace {

constexpr int kLinThreads = 384;  // warp 0 copies, warp 1 MMAs, warps 2 and 3 idle, warps 4..11 epilogue
constexpr int kLinGrid = 152;     // CTAs at most: one per SM
constexpr int kEpiThreads = 256;
constexpr int kSmemRing = 216 * 1024;
constexpr int kMaxStages = 12;
constexpr int kMaxCluster = 8;    // CTAs of a cluster that joins parts
constexpr int kMaxSplit = 16;     // parts along K: each costs the last one a read of its sums

struct LinArgs {
  const uint8_t* w;
  const float *ws, *xs;
  void* y;
  int f32, M, N, KB;
  int vec_x, vec_w;           // the scales' rows can be read 16 bytes at a time
  int tile_m, tile_n;         // output tiles along the tokens, along the weight rows
  int dp_rounds, cut_tiles;   // whole tiles per CTA (pair); the tiles after them, each cut into
  int split;                  // this many parts along K, one per CTA (pair), at multiples of
  int unit, units;            // this many K blocks; ceil(KB / unit)
  int cluster;                // > 1: the parts of a tile are the CTAs of a cluster and join in shared memory
  unsigned* counters;         // [cut_tiles][2 CTAs of a pair][8 epilogue warps]
  float* partials;            // [grid][kBC][128]
  int* status;
};

template <int kBC, bool kPair>
struct LinCfg {
  // K blocks per stage, barrier and tensor-memory buffer: waits, commits and loop cost the MMA warp about 650
  // cycles a block when they are taken for each, more than a block of a narrow tile takes to arrive.
  static constexpr int kG = kBC == 16 ? 4 : kBC <= 64 ? 2 : 1;
  static constexpr int kBlock = 16384 + (kPair ? kBC / 2 : kBC) * 128;  // a pair's CTAs hold half of the columns each
  static constexpr int kStage = kG * kBlock;
  static constexpr int kStages = kPair ? 5 : kSmemRing / kStage < kMaxStages ? kSmemRing / kStage : kMaxStages;
  static constexpr int kOut = kPair ? 8 * 8192 : 0;  // output staging: 8 KB per epilogue warp
  static constexpr int kBufs = 512 / (kBC * kG) < 8 ? 512 / (kBC * kG) : 8;
  static constexpr int kCols = kBC * kG * kBufs;  // tensor-memory columns (512)
  static constexpr int kSmem = kStages * kStage + kOut + 1024;
};

struct Item {
  int tile, kb0, kb1;
};
// The pieces of work of CTA (pair) c in turn: its whole tiles, then one part of a tile that is cut along K.
struct Sched {
  int c, G, i;
  // pair: the CTAs 2 c and 2 c + 1 work on the same tiles
  __device__ explicit Sched(int pair) : c(blockIdx.x >> pair), G(gridDim.x >> pair), i(0) {}
  __device__ bool next(const LinArgs& a, Item& it) {
    if (i < a.dp_rounds) {
      it.tile = i++ * G + c;
      it.kb0 = 0;
      it.kb1 = a.KB;
      return true;
    }
    if (i > a.dp_rounds || c >= a.cut_tiles * a.split) return false;
    ++i;
    const int t = c / a.split, part = c - t * a.split;
    it.tile = a.dp_rounds * G + t;
    it.kb0 = part * a.units / a.split * a.unit;
    it.kb1 = min(a.KB, (part + 1) * a.units / a.split * a.unit);
    return true;
  }
};

// Tile order: groups of 8 token tiles, weight tiles across, so that the CTAs of one round share rows
// of both operands in L2.
__device__ __forceinline__ void tile_at(const LinArgs& a, int t, int& mt, int& nt) {
  constexpr int kGroup = 8;
  const int per = kGroup * a.tile_n, g = t / per, r = t - g * per, gm = min(kGroup, a.tile_m - g * kGroup);
  nt = r / gm;
  mt = g * kGroup + r - nt * gm;
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// K-major operand with the 128-byte swizzle: 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
template <bool kPair>
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  if constexpr (kPair)
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
  else
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// Arrives on `bar` (in both CTAs of a pair, at the same offset; or in those of `mask`) when every MMA issued so
// far by this thread has completed.
template <bool kPair>
__device__ __forceinline__ void mma_commit(uint64_t* bar, uint16_t mask = 3) {
  if constexpr (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(mask)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
template <bool kPair>
__device__ __forceinline__ void lin_tmem_alloc(uint32_t* dst, uint32_t cols) {
  if constexpr (kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst, cols);
  }
}
template <bool kPair>
__device__ __forceinline__ void lin_tmem_dealloc(uint32_t t, uint32_t cols) {
  if constexpr (kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(cols) : "memory");
  else
    tmem_dealloc(t, cols);
}
// Pair forms: loads into this CTA's shared memory that complete on a barrier of the pair's first CTA, the
// address of that CTA's copy of a variable, an arrival there, and the pair's barrier.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, "
      "%4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
               "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ uint32_t leader_addr(uint32_t a) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}
// The rest of a bounded wait of a converged warp.
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, int* abort, int* status) {
  for (uint32_t i = 0; i < kMbarPolls; ++i) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity), "r"(20000u)
                 : "memory");
    if (__all_sync(0xFFFFFFFFu, ok != 0)) return true;
    if (__any_sync(0xFFFFFFFFu, *(volatile int*)abort)) return false;
  }
  *(volatile int*)abort = 1;
  atomicExch(status, (int)VP_ERR_TIMEOUT);
  return false;
}
// acc += x * f, in its place among the volatile loads.
__device__ __forceinline__ void fma_here(float& acc, uint32_t x, float f) {
  asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(acc) : "f"(__uint_as_float(x)), "f"(f));
}
// p[k .. k + 3] as far as it lies before n (k a multiple of 4; vec: p + k is 16-byte aligned and n too).
__device__ __forceinline__ float4 load4(const float* p, int k, int n, int vec) {
  if (vec) return __ldg(reinterpret_cast<const float4*>(p + k));
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  v.x = __ldg(p + k);
  if (k + 1 < n) v.y = __ldg(p + k + 1);
  if (k + 2 < n) v.z = __ldg(p + k + 2);
  if (k + 3 < n) v.w = __ldg(p + k + 3);
  return v;
}
__device__ __forceinline__ float pick4(const float4& v, int k) {
  const float lo = k & 1 ? v.y : v.x, hi = k & 1 ? v.w : v.z;
  return k & 2 ? hi : lo;
}
// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
// A float of the cluster's CTA `rank`, at this CTA's shared address.
__device__ __forceinline__ float ld_cluster(uint32_t addr, int rank) {
  uint32_t r;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("{ .reg .b64 st; mbarrier.arrive.shared::cta.b64 st, [%0]; }" ::"r"(bar) : "memory");
}
// kN consecutive 32-bit columns of the warp's lane: the load, and the wait for it, which takes the
// registers as operands so that no use of them can move in front of it.
template <int kN>
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t* r) {
  if constexpr (kN == 32) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t)
        : "memory");
  } else if constexpr (kN == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t));
  } else {
    static_assert(kN == 8, "");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t)
                 : "memory");
  }
}
template <int kN>
__device__ __forceinline__ void tmem_wait(uint32_t* r) {
  if constexpr (kN == 32) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
  } else if constexpr (kN == 16) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
  } else {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
  }
}
// kBC: columns of a tile (token columns when kSwap, else weight rows: 128, or a pair's 256).  kPair: two CTAs (a
// cluster) work on one tile of 256 tokens x 256 weight rows, 128 tokens' sums in each one's tensor memory; the first
// CTA's MMA warp issues for both.
template <int kBC, bool kSwap, bool kPair>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_kernel(const __grid_constant__ LinArgs a, const __grid_constant__ CUtensorMap xmap,
                  const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap ymap) {
  using C = LinCfg<kBC, kPair>;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], tfull[8], tempty[8], drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const uint32_t ring = (smem_addr(dyn) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kPair ? (int)cluster_rank() : 0;
#ifdef VP_WAIT_TEST
  // Wait-test hook (workspace word kWsTestSkip): the first CTA (5: the second) leaves out, of its first block,
  // 1 the commit to the epilogue, 2 the commit that frees the stage, 3 an arrival that frees the tensor-memory
  // buffer, 4 and 5 the copies; 6: its first epilogue warp's first wait runs out at once.
  const int hook = ((const volatile int*)a.status)[kWsTestSkip / sizeof(int)];
  const bool hooked = blockIdx.x == (hook == 5 ? 1 : 0);
#else
  constexpr int hook = 0;
  constexpr bool hooked = false;
#endif
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], (kPair ? 2 : 1) * kEpiThreads / 32);
    }
    mbar_init(&drain, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) lin_tmem_alloc<kPair>(&s_tmem, C::kCols);
  tmem_fence_before();
  if constexpr (kPair) {
    __syncthreads();
    cluster_sync();  // the other CTA's barriers exist
  } else {           // the copying warp made the barriers and needs nothing else: it starts at once
    __syncwarp();
    if (warp == 0)
      asm volatile("bar.arrive 2, %0;" ::"n"(kLinThreads) : "memory");
    else
      asm volatile("bar.sync 2, %0;" ::"n"(kLinThreads) : "memory");
  }
  tmem_fence_after();
  const uint32_t tmem = *(volatile uint32_t*)&s_tmem;

  // A bounded wait of a converged warp; false when it ran out here or elsewhere in the CTA.
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    if (hooked && hook == 6 && warp == 4) {
      *(volatile int*)&s_abort = 1;
      atomicExch(a.status, (int)VP_ERR_TIMEOUT);
      return false;
    }
    if (__all_sync(0xFFFFFFFFu, mbar_try(bar, parity))) return true;
    return wait_slow(bar, parity, &s_abort, a.status);
  };

  // Registers: launched at 168 a thread; the four warps that only issue keep 40, the epilogue's eight get
  // 232 (4 x 40 + 8 x 232 = 12 x 168).
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    Sched sched(kPair);
    Item it;
    // Whole warps run the two issuing loops, one elected lane issues: the operands stay warp-uniform.
    if (warp == 0) {
      int n = 0, s = 0;
      uint32_t par = 1;  // of the empty barriers: the first round passes
      bool ok = true;
      while (ok && sched.next(a, it)) {
        int mt, nt;
        tile_at(a, it.tile, mt, nt);
        // the weight tile of this output tile (a pair's CTAs take one each; past the last row block the last one
        // again, whose products are not stored)
        const int nb = kPair ? min(2 * nt + rank, qblocks(a.N) - 1) : nt;
        const int rows = kSwap ? kBC : 128, m0 = kPair ? mt * 256 + rank * 128 : mt * rows;
        for (int kb0 = it.kb0; kb0 < it.kb1; kb0 += C::kG, ++n) {
          if (!(ok = wait(smem_addr(&empty[s]), par))) break;
          if (elect_one()) {
            const int cnt = min(C::kG, it.kb1 - kb0);
            if constexpr (kPair) {
              if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::kStage);  // both CTAs' copies
            } else {
              mbar_arrive_expect_tx(&full[s], cnt * (rows * 128 + kQTileBytes));
            }
#pragma unroll
            for (int g = 0; g < C::kG; ++g) {
              if (g >= cnt || (hooked && (hook == 4 || hook == 5) && n == 0)) break;
              const int kb = kb0 + g;
              const uint32_t st = ring + s * C::kStage + g * C::kBlock;
              // lanes' operand first (16 KB), columns' operand behind it
              const uint32_t dst_w = kSwap ? st : st + 16384, dst_x = kSwap ? st + 16384 : st;
              if constexpr (kPair) {
                const uint32_t bar = leader_addr(smem_addr(&full[s]));
                tma_load_2d_pair(dst_x, &xmap, kb * kQBlock, m0, bar);
                tma_load_3d_pair(dst_w, &wmap, 0, 0, nb * a.KB + kb, bar);
              } else {
                const uint32_t bar = smem_addr(&full[s]);
                tma_load_2d(dst_x, &xmap, kb * kQBlock, m0, bar);
                bulk_load(dst_w, a.w + ((size_t)nb * a.KB + kb) * kQTileBytes, kQTileBytes, bar);
              }
            }
          }
          __syncwarp();
          if (++s == C::kStages) s = 0, par ^= 1;
        }
      }
      // Nothing may be on its way to this CTA's shared memory, or from here to the pair's other CTA, when the CTA
      // ends: each stage's last commit says that its copies have landed and been read, and it is itself the last
      // arrival from the pair's first CTA.  Where the MMAs have stopped the wait takes its whole limit, a
      // second, in which whatever was on its way arrives (the other CTA waits for this one at the end).
      for (int i = 0; i < min(n, C::kStages); ++i)
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&empty[i], ((n - 1 - i) / C::kStages) & 1))) {
          *(volatile int*)&s_abort = 1;
          atomicExch(a.status, (int)VP_ERR_TIMEOUT);
          break;
        }
    }
    if (warp == 1 && rank == 0) {
      int s = 0, b = 0;
      uint32_t par = 0, tpar = 1;
      bool ok = true, first = true;  // first: only the wait-test build asks
      // e4m3 x e4m3 -> fp32, 128 rows (a pair's two CTAs: 256)
      constexpr uint32_t idesc = 1u << 4 | (uint32_t)(kBC >> 3) << 17 | (kPair ? 16u : 8u) << 24;
      while (ok && sched.next(a, it)) {
        for (int kb0 = it.kb0; kb0 < it.kb1; kb0 += C::kG) {
          const int cnt = min(C::kG, it.kb1 - kb0);
          const uint64_t da = smem_desc(ring) + (uint64_t)(s * (C::kStage >> 4)), db = da + (16384 >> 4);
          if (!(ok = wait(smem_addr(&full[s]), par))) break;
          if (!(ok = wait(smem_addr(&tempty[b]), tpar))) break;
          tmem_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int g = 0; g < C::kG; ++g) {
              if (g >= cnt) break;
#pragma unroll
              for (int k = 0; k < 4; ++k)  // 32 bytes along K inside the swizzle atom
                mma_f8<kPair>(tmem + (b * C::kG + g) * kBC, da + g * (C::kBlock >> 4) + 2 * k,
                              db + g * (C::kBlock >> 4) + 2 * k, idesc, k > 0);
            }
            if (!(hooked && hook == 1 && first)) mma_commit<kPair>(&tfull[b]);
            if (!(hooked && hook == 2 && first)) mma_commit<kPair>(&empty[s]);
          }
          first = false;
          __syncwarp();
          if (++s == C::kStages) s = 0, par ^= 1;
          if (++b == C::kBufs) b = 0, tpar ^= 1;
        }
      }
      if (!ok) {
        if (elect_one()) mma_commit<kPair>(&drain, 1);  // here alone
        __syncwarp();
        mbar_wait_bounded(&drain, 0);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    Sched sched(kPair);
    Item it;
    constexpr int kW = kBC / 2;                   // columns per warp
    constexpr int kCh = kW < 32 ? kW : 32;        // columns per tensor-memory load
    const int quad = warp & 3, half = (warp - 4) >> 2, row = quad * 32 + lane, c0 = half * kW;
    const uint32_t tm = tmem + ((uint32_t)(quad * 32) << 16) + c0;
    const uint32_t tfull0 = smem_addr(tfull), tempty0 = kPair ? leader_addr(smem_addr(tempty)) : smem_addr(tempty);
    int b = 0;
    uint32_t par = 0;
    bool ok = true;
    // Factors of four blocks at a time: each of a warp's 32 rows is a cache line of its own, so a load per
    // block would keep the load unit busy for 256 cycles of the block's 512.  The next tile's first
    // factors are loaded before this tile's output is stored.
    const float *px, *pw;
    float4 fx, fw;          // tokens on the lanes: the current four blocks'
    float4 ax[4], aw[4];    // weights on the lanes: the next sixteen blocks'
    int mt, nt, next_mt = 0, next_nt = 0;
    Item next;
    auto fetch = [&]() -> bool {
      if (!sched.next(a, next)) return false;
      tile_at(a, next.tile, next_mt, next_nt);
      // the factor of this thread's row (tokens on the lanes) or of column c0 + lane (weights there); what is
      // past the last row or column is computed with another's factor and not stored
      const int m = kSwap ? next_mt * kBC + c0 + lane : kPair ? next_mt * 256 + rank * 128 + row : next_mt * 128 + row;
      const int nb = kPair ? 2 * next_nt + half : next_nt;
      px = a.xs + (size_t)min(m, a.M - 1) * a.KB;
      pw = a.ws + (size_t)min(nb, qblocks(a.N) - 1) * a.KB;
      if constexpr (kSwap) {
#pragma unroll
        for (int d = 0; d < 4; ++d)
          if (next.kb0 + 4 * d < next.kb1) {
            ax[d] = load4(px, next.kb0 + 4 * d, a.KB, a.vec_x);
            aw[d] = load4(pw, next.kb0 + 4 * d, a.KB, a.vec_w);
          }
      } else {
        fx = load4(px, next.kb0 & ~3, a.KB, a.vec_x);
        fw = load4(pw, next.kb0 & ~3, a.KB, a.vec_w);
      }
      return true;
    };
    // Writes the warp's part of tile (mt, nt).
    auto store = [&](const float (&acc)[kW], int mt, int nt) {
      const int m = kPair ? mt * 256 + rank * 128 + row : mt * 128 + row;  // tokens on the lanes
      if (kSwap) {
        const int nn = nt * 128 + row;
        if (nn < a.N) {
#pragma unroll
          for (int j = 0; j < kW; ++j) {
            const int mm = mt * kBC + c0 + j;
            if (mm >= a.M) continue;
            const size_t at = (size_t)mm * a.N + nn;
            if (a.f32)
              static_cast<float*>(a.y)[at] = acc[j];
            else
              static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(acc[j]);
          }
        }
      } else if (kPair) {
        // through shared memory (128-byte swizzled rows) to asynchronous tile stores, which cut off at M and N
        const uint32_t stage = ring + C::kStages * C::kStage + (warp - 4) * 8192;
        const int y0 = mt * 256 + rank * 128 + quad * 32;
        const uint32_t swz = (uint32_t)(lane & 7);
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the staging's last stores have read it
        __syncwarp();
        if (a.f32) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {  // boxes of 32 columns
            const uint32_t box = stage + (q & 1) * 4096, r = box + lane * 128;
            if (q == 2) {
              asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
              __syncwarp();
            }
#pragma unroll
            for (int c = 0; c < 8; ++c)
              sts128(r + ((c ^ swz) << 4), make_uint4(__float_as_uint(acc[32 * q + 4 * c]), __float_as_uint(acc[32 * q + 4 * c + 1]),
                                                      __float_as_uint(acc[32 * q + 4 * c + 2]), __float_as_uint(acc[32 * q + 4 * c + 3])));
            fence_proxy_async_smem();
            __syncwarp();
            const int x = nt * 256 + half * 128 + q * 32;
            if (elect_one()) {
              if (y0 < a.M && x < a.N) tma_store_2d(&ymap, x, y0, box);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            __syncwarp();
          }
        } else {
#pragma unroll
          for (int q = 0; q < 2; ++q) {  // boxes of 64 columns
            const uint32_t box = stage + q * 4096, r = box + lane * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(acc[64 * q + 8 * c + 2 * e], acc[64 * q + 8 * c + 2 * e + 1]);
                w[e] = *reinterpret_cast<const uint32_t*>(&p);
              }
              sts128(r + ((c ^ swz) << 4), make_uint4(w[0], w[1], w[2], w[3]));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (elect_one()) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int x = nt * 256 + half * 128 + q * 64;
              if (y0 < a.M && x < a.N) tma_store_2d(&ymap, x, y0, stage + q * 4096);
            }
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
          __syncwarp();
        }
      } else if (m < a.M) {
        const int n0 = nt * kBC + c0;
#pragma unroll
        for (int j = 0; j < kW; j += 8) {
          if (n0 + j >= a.N) continue;
          const size_t at = (size_t)m * a.N + n0 + j;
          if (a.f32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.y) + at);
            o[0] = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
            o[1] = make_float4(acc[j + 4], acc[j + 5], acc[j + 6], acc[j + 7]);
          } else {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 p = __floats2bfloat162_rn(acc[j + 2 * e], acc[j + 2 * e + 1]);
              w[e] = *reinterpret_cast<const uint32_t*>(&p);
            }
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + at) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    };
    bool more = fetch();
    while (more) {
      it = next;
      mt = next_mt;
      nt = next_nt;
      float acc[kW];
#pragma unroll
      for (int j = 0; j < kW; ++j) acc[j] = 0.0f;
      if constexpr (kSwap) {
        // A few columns per block.  The factors come 16 blocks ahead (four blocks per load, four loads in
        // registers): behind the weight stream a miss takes microseconds.
        for (int kb4 = it.kb0; ok && kb4 < it.kb1; kb4 += 16) {
#pragma unroll
          for (int d = 0; d < 4; ++d) {
#pragma unroll
            for (int h = 0; h < 4; h += C::kG) {  // one buffer of kG blocks
              const int kb = kb4 + 4 * d + h;
              if (!ok || kb >= it.kb1) break;
              if (!(ok = wait(tfull0 + 8 * b, par))) break;
              tmem_fence_after();
              const uint32_t tb = tm + b * C::kG * kBC;
              uint32_t r[C::kG][kW];
#pragma unroll
              for (int g = 0; g < C::kG; ++g)
                if (kb + g < it.kb1) tmem_ld<kW>(tb + g * kBC, r[g]);
#pragma unroll
              for (int g = 0; g < C::kG; ++g) tmem_wait<kW>(r[g]);
              tmem_fence_before();
              __syncwarp();
              if (elect_one() && !(hooked && hook == 3 && warp == 4 && b == 0 && par == 0)) mbar_arrive(tempty0 + 8 * b);
#pragma unroll
              for (int g = 0; g < C::kG; ++g) {
                if (kb + g >= it.kb1) break;
                const float f = pick4(ax[d], h + g) * pick4(aw[d], h + g);
#pragma unroll
                for (int j = 0; j < kW; ++j)
                  acc[j] = fmaf(__uint_as_float(r[g][j]), __shfl_sync(0xFFFFFFFFu, f, j), acc[j]);
              }
              if (++b == C::kBufs) b = 0, par ^= 1;
            }
            if (kb4 + 4 * d + 16 < it.kb1) {
              ax[d] = load4(px, kb4 + 4 * d + 16, a.KB, a.vec_x);
              aw[d] = load4(pw, kb4 + 4 * d + 16, a.KB, a.vec_w);
            }
          }
        }
      }
      for (int kb = it.kb0; !kSwap && kb < it.kb1; ++kb) {
        if (!(ok = wait(tfull0 + 8 * b, par))) break;
        tmem_fence_after();
        const uint32_t tb = tm + b * kBC;
        // chunk by chunk; the next chunk's load is in flight while this one is accumulated
        constexpr int kNCh = kW / kCh;
        uint32_t r[2][kCh];
        tmem_ld<kCh>(tb, r[0]);
        const float f = pick4(fx, kb) * pick4(fw, kb);
        if ((kb & 3) == 3 && kb + 1 < it.kb1) {
          fx = load4(px, kb + 1, a.KB, a.vec_x);
          fw = load4(pw, kb + 1, a.KB, a.vec_w);
        }
#pragma unroll
        for (int i = 0; i < kNCh; ++i) {
          tmem_wait<kCh>(r[i & 1]);
          if (i + 1 < kNCh) {
            tmem_ld<kCh>(tb + (i + 1) * kCh, r[(i + 1) & 1]);
          } else {  // the buffer is read: the next MMAs may have it
            tmem_fence_before();
            __syncwarp();
            if (elect_one() && !(hooked && hook == 3 && warp == 4 && b == 0 && par == 0)) {
              if (kPair)
                mbar_arrive_cluster(tempty0 + 8 * b);
              else
                mbar_arrive(tempty0 + 8 * b);
            }
          }
#pragma unroll
          for (int j = 0; j < kCh; ++j) {
            const int col = i * kCh + j;
            fma_here(acc[col], r[i & 1][j], f);
          }
        }
        if (++b == C::kBufs) b = 0, par ^= 1;
      }
      if (!ok) break;
      more = fetch();
      if (kSwap && a.cluster > 1) {  // a part: left in the ring, which is free, for the cluster (below)
#pragma unroll
        for (int j = 0; j < kW; ++j)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(ring + ((c0 + j) * 128 + row) * 4), "f"(acc[j]) : "memory");
        continue;
      }
      if (it.kb1 - it.kb0 < a.KB) {
        // A part of the tile's K blocks: left in the workspace, and the last contributor adds them up.  Each
        // warp joins its own part of the tile (8 counters per tile and CTA): no CTA-wide wait.
        const size_t slot = (size_t)kBC * 128;
        float* mine = a.partials + blockIdx.x * slot + c0 * 128 + row;
#pragma unroll
        for (int j = 0; j < kW; ++j) __stcg(mine + j * 128, acc[j]);
        __threadfence();
        __syncwarp();
        const int t = sched.c / a.split;
        unsigned old = 0, *counter = a.counters + (t * 2 + rank) * 8 + warp - 4;
        if (lane == 0) old = atom_add_acq_rel_gpu(counter, 1);
        if (__shfl_sync(0xFFFFFFFFu, old, 0) != (unsigned)(a.split - 1)) continue;
        if (lane == 0) *counter = 0;  // every contributor has arrived
        __threadfence();
#pragma unroll
        for (int j = 0; j < kW; ++j) acc[j] = 0.0f;
        for (int e = 0; e < a.split; ++e) {  // in K order
          const int c = t * a.split + e;
          const float* p = a.partials + (kPair ? 2 * c + rank : c) * slot + c0 * 128 + row;
#pragma unroll
          for (int j = 0; j < kW; ++j) acc[j] += __ldcg(p + j * 128);
        }
      }
      store(acc, mt, nt);
    }
  }
  if (kPair) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the thread's output stores are done
  __syncwarp();
  if constexpr (kSwap && kBC <= 32) {
    if (a.cluster > 1) {
      cluster_sync();  // every part lies in its CTA's shared memory
      if (warp >= 4) {  // each CTA adds every cluster-th token's sums, in K order
        Sched sched(0);
        Item it;
        int mt, nt;
        sched.next(a, it);
        tile_at(a, it.tile, mt, nt);
        const int c0 = ((warp - 4) >> 2) * (kBC / 2), row = (warp & 3) * 32 + lane, nn = nt * 128 + row;
        for (int j = (int)cluster_rank(); j < kBC / 2; j += a.cluster) {
          const int mm = mt * kBC + c0 + j;
          if (mm >= a.M) break;
          const uint32_t at = ring + ((c0 + j) * 128 + row) * 4;
          float y = 0.0f;
#pragma unroll
          for (int e = 0; e < kMaxCluster; ++e) {
            if (e >= a.cluster) break;
            y += ld_cluster(at, e);
          }
          if (nn >= a.N) continue;
          if (a.f32)
            static_cast<float*>(a.y)[(size_t)mm * a.N + nn] = y;
          else
            static_cast<__nv_bfloat16*>(a.y)[(size_t)mm * a.N + nn] = __float2bfloat16_rn(y);
        }
      }
      __syncwarp();
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (kPair || (kSwap && a.cluster > 1)) cluster_sync();  // nobody reads or signals this CTA's shared memory any more
  tmem_fence_after();
  if (warp == 1) lin_tmem_dealloc<kPair>(tmem, C::kCols);
}

bool al(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int kMaxMq = 1 << 20;

// The tile form of a shape.
struct LinPlan {
  int bc;
  bool swap, pair;
  int tile_m, tile_n, tiles;
  size_t total;  // workspace bytes
};

LinPlan lin_plan(int M, int N) {
  LinPlan p;
  p.swap = M <= 64;
  p.pair = M > 128;
  p.bc = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
  p.tile_m = p.swap ? 1 : p.pair ? (M + 255) / 256 : 1;
  p.tile_n = p.swap ? qblocks(N) : (N + p.bc - 1) / p.bc;
  p.tiles = p.tile_m * p.tile_n;
  static_assert(kLinGrid * 2 * (kEpiThreads / 32) <= kServeMaxCounters, "counters");
  p.total = kServeData + sizeof(float) * kLinGrid * (size_t)p.bc * 128;
  return p;
}

// Parts along K of a tile that has `most` CTAs (pairs): the fewest microseconds of KB / s blocks (0.25 each for
// the narrow tiles, 0.4 for 128 and 256 columns) and, for s > 1, of the fence and the last part's read of all s
// parts (2, and a tile's 4 * 128 * bc bytes at about 70 GB/s for each).  1024 x 5120 x 5120, 4 tiles left of 80:
// 50 us in 16 parts, 37 us in 3.
int lin_split(int bc, int KB, int most) {
  const double block = bc >= 128 ? 0.4 : 0.25, read = bc * 512.0 / 70e3;
  int best = 1;
  double least = KB * block;
  for (int s = 2; s <= most; ++s) {
    const double t = (KB + s - 1) / s * block + 2.0 + read * s;
    if (t < least) least = t, best = s;
  }
  return best;
}

// Narrow tiles that are all cut join in clusters where every cluster is resident at once (clusters of 7 leave
// SMs of most GPCs idle, for one).  5120 x 17408, 3 parts: 8 tokens 19.6 us through the workspace, 18.3 in
// clusters; 32 tokens 21.0 and 20.7; 64 tokens 22.8 and 23.7 (32 KB a part), so those keep the workspace.
template <int kBC, bool kSwap, bool kPair>
cudaError_t launch_linear(LinArgs& a, const CUtensorMap& xmap, const CUtensorMap& wmap, const CUtensorMap& ymap,
                          int grid, cudaStream_t s) {
  constexpr int kSmem = LinCfg<kBC, kPair>::kSmem;
  auto* kern = linear_kernel<kBC, kSwap, kPair>;
  static std::atomic<bool> done[64];
  static std::atomic<int> resident[64][kMaxCluster + 1];  // clusters of a size, plus one; 0: not asked yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < 64;
  if (!known || !done[dev].load()) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (known) done[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = kPair ? 2 : 1;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  a.cluster = 1;
  if (kSwap && kBC <= 32 && known && a.dp_rounds == 0 && a.split > 1 && a.split <= kMaxCluster) {
    int n = resident[dev][a.split].load();
    if (n == 0) {
      at.val.clusterDim.x = (unsigned)a.split;
      if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;
      }
      resident[dev][a.split].store(++n);
      at.val.clusterDim.x = 1;
    }
    if (a.cut_tiles <= n - 1) {
      a.cluster = a.split;
      at.val.clusterDim.x = (unsigned)a.split;
    }
  }
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const LinArgs>(a), xmap, wmap, ymap);
}

}  // namespace

}  // namespace vp

using namespace vp;

extern "C" {

size_t vp_linear_fp8_block_workspace_bytes(int M, int N, int K) {
  if (M < 1 || M > kMaxMq || !q_shape_ok(N, K)) return 0;
  return lin_plan(M, N).total;
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
  vp_status st = device_sm_count(&sms);
  if (st != VP_OK) return st;
  PFN_cuTensorMapEncodeTiled_v12000 encode;
  if ((st = tensor_map_encoder(&encode)) != VP_OK) return st;
  const LinPlan p = lin_plan(M, N);
  CUtensorMap xmap, wmap, ymap;
  {
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)M}, strides[1] = {(cuuint64_t)K};
    const cuuint32_t box[2] = {kQBlock, (cuuint32_t)(p.swap ? p.bc : 128)}, step[2] = {1, 1};
    if (encode(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(xq), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return VP_ERR_UNSUPPORTED;
  }
  if (p.pair) {  // one packed tile per box (already in the swizzled order)
    const cuuint64_t dims[3] = {kQBlock, kQBlock, (cuuint64_t)qblocks(N) * qblocks(K)};
    const cuuint64_t strides[2] = {kQBlock, kQTileBytes};
    const cuuint32_t box[3] = {kQBlock, kQBlock, 1}, step[3] = {1, 1, 1};
    if (encode(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(w_packed), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return VP_ERR_UNSUPPORTED;
    const bool f32 = y_type == VP_F32;  // boxes of 128 bytes x 32 rows
    const cuuint64_t ydims[2] = {(cuuint64_t)N, (cuuint64_t)M}, ystrides[1] = {(cuuint64_t)N * (f32 ? 4 : 2)};
    const cuuint32_t ybox[2] = {f32 ? 32u : 64u, 32u}, ystep[2] = {1, 1};
    if (encode(&ymap, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, y, ydims, ystrides, ybox,
               ystep, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return VP_ERR_UNSUPPORTED;
  } else {
    wmap = ymap = xmap;
  }
  uint8_t* b = static_cast<uint8_t*>(ws);
  LinArgs a;
  a.w = static_cast<const uint8_t*>(w_packed);
  a.ws = w_scales;
  a.xs = x_scales;
  a.y = y;
  a.f32 = y_type == VP_F32;
  a.M = M, a.N = N, a.KB = qblocks(K);
  a.vec_x = a.KB % 4 == 0 && al(x_scales, 16);
  a.vec_w = a.KB % 4 == 0 && al(w_scales, 16);
  a.tile_m = p.tile_m, a.tile_n = p.tile_n;
  int grid = std::min(sms, kLinGrid) / (p.pair ? 2 : 1);  // CTAs, or pairs
  a.dp_rounds = p.tiles / grid;
  a.cut_tiles = p.tiles - a.dp_rounds * grid;
  a.unit = p.swap ? 4 : 1;
  a.units = (a.KB + a.unit - 1) / a.unit;
  a.split = a.cut_tiles ? lin_split(p.bc, a.KB, std::min({grid / a.cut_tiles, a.units, kMaxSplit})) : 1;
  if (a.dp_rounds == 0) grid = a.cut_tiles * a.split;
  if (p.pair) grid *= 2;
  a.counters = reinterpret_cast<unsigned*>(b + kServeCounters);
  a.partials = reinterpret_cast<float*>(b + kServeData);
  a.status = reinterpret_cast<int*>(b);
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  switch (p.bc) {
    case 16: e = launch_linear<16, true, false>(a, xmap, wmap, ymap, grid, s); break;
    case 32: e = launch_linear<32, true, false>(a, xmap, wmap, ymap, grid, s); break;
    case 64: e = launch_linear<64, true, false>(a, xmap, wmap, ymap, grid, s); break;
    case 128: e = launch_linear<128, false, false>(a, xmap, wmap, ymap, grid, s); break;
    default: e = launch_linear<256, false, true>(a, xmap, wmap, ymap, grid, s); break;
  }
  return e == cudaSuccess ? VP_OK : cuda_fail(e);
}

}  // extern "C"
