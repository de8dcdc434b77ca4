// The kernel of rows_attention.cu.
#pragma once
#include <cuda_bf16.h>

#include <atomic>

#include "internal.h"
#include "ptx.cuh"
#include "rows_attention.h"
#include "verify.h"

namespace vp {

namespace {

// ------------------------------------------------------------------ instructions
__device__ __forceinline__ bool ra_elect() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}
// A value that is the same in the whole warp, as one that the compiler knows to be (the products' operands are uniform
// registers).
__device__ __forceinline__ int ra_uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }
__device__ __forceinline__ void ra_arrive(uint32_t bar) {
  asm volatile("{ .reg .b64 st; mbarrier.arrive.shared::cta.b64 st, [%0]; }" ::"r"(bar) : "memory");
}
// An arrival at the barrier's copy in the pair's first CTA, after this thread's work.
__device__ __forceinline__ void ra_arrive_first(uint32_t bar, uint32_t rank = 0) {
  asm volatile(
      "{ .reg .b32 a; mapa.shared::cluster.u32 a, %0, %1;\n mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a]; }" ::"r"(bar),
      "r"(rank)
      : "memory");
}
// One poll of at most `ns`.  kPair: the arrivals may come from the pair's other CTA.
template <bool kPair>
__device__ __forceinline__ bool ra_try(uint32_t bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  if constexpr (kPair)
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(ns)
        : "memory");
  else
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity), "r"(ns)
                 : "memory");
  return ok != 0;
}
constexpr uint32_t kRaShort = 64;
// A bounded wait of a converged warp; false when it ran out here or elsewhere in the CTA.  polls: kMbarPolls where the others
// are at work on the same block, RowsArgs::polls where they may be at work on a whole item.
template <bool kPair>
__device__ __forceinline__ bool ra_wait(uint32_t bar, uint32_t parity, uint32_t polls, int* abort, int* status) {
  uint32_t left = polls + kRaShort;  // short polls first, then of 4 us (the hint's 20 are cut)
  while (!__all_sync(0xFFFFFFFFu, ra_try<kPair>(bar, parity, left > polls ? 0 : 20000))) {
    --left;
    if (left > polls) continue;
    if (__any_sync(0xFFFFFFFFu, *(volatile int*)abort)) return false;
    if (left == 0) {
      *(volatile int*)abort = 1;
      atomicExch(status, (int)VP_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
// The same without ordering this thread's memory accesses (what it announces lies in tensor memory, or is another's).
__device__ __forceinline__ void ra_arrive_first_relaxed(uint32_t bar) {
  asm volatile(
      "{ .reg .b32 a; mapa.shared::cluster.u32 a, %0, 0;\n mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [a]; }" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ uint32_t ra_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void ra_pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word of the shared memory of the pair's CTA `rank`, at this CTA's address.
__device__ __forceinline__ int ra_ld_pair(const void* p, uint32_t rank) {
  int v;
  asm volatile("{ .reg .b32 a; mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.s32 %0, [a]; }"
               : "=r"(v)
               : "r"(smem_addr(p)), "r"(rank)
               : "memory");
  return v;
}
__device__ __forceinline__ void ra_tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void ra_tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// Into this CTA's shared memory, completing on a barrier of the pair's first CTA.
__device__ __forceinline__ void ra_tma_3d_first(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "{ .reg .b32 a; mapa.shared::cluster.u32 a, %5, 0;\n"
      " cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], "
      "[a]; }" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// kRelease: with what this thread has written for those who wait behind the products.
template <bool kRelease>
__device__ __forceinline__ void ra_expect_first(uint32_t bar, uint32_t bytes) {
  if constexpr (kRelease)
    asm volatile(
        "{ .reg .b32 a; mapa.shared::cluster.u32 a, %0, 0;\n"
        " mbarrier.arrive.expect_tx.release.cluster.shared::cluster.b64 _, [a], %1; }" ::"r"(bar),
        "r"(bytes)
        : "memory");
  else
    asm volatile(
        "{ .reg .b32 a; mapa.shared::cluster.u32 a, %0, 0;\n"
        " mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [a], %1; }" ::"r"(bar),
        "r"(bytes)
        : "memory");
}
// 16 bytes by this lane, and its arrival once all of them have landed.
__device__ __forceinline__ void ra_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ra_copy16_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// Shared-memory operands with the 128-byte swizzle.  K-major (queries, keys): rows 128 bytes apart, groups of 8 rows
// 1024.  MN-major (values: 64 columns of 16 bits are the 128 bytes, keys the rows): 64-column groups `group` bytes apart.
__device__ __forceinline__ uint64_t ra_desc_k(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
__device__ __forceinline__ uint64_t ra_desc_mn(uint32_t addr, uint32_t group) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(group >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// D(tensor memory) (+)= A B: A in shared memory, or in tensor memory.  kPair: 256 rows, 128 in each CTA, which also holds half
// of B; issued by the first CTA.
template <bool kPair>
__device__ __forceinline__ void ra_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  if constexpr (kPair)
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
  else
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
template <bool kPair>
__device__ __forceinline__ void ra_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  if constexpr (kPair)
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
  else
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// Arrives on `bar` (in both CTAs of a pair) when every product issued so far by this thread has ended.
template <bool kPair>
__device__ __forceinline__ void ra_commit(uint64_t* bar) {
  if constexpr (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
// 32 columns of the warp's lanes: load, the wait that ties the loaded registers to it, and store.
__device__ __forceinline__ void ra_ld32(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void ra_wait32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void ra_st32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
      "r"(t)
      : "memory");
}
__device__ __forceinline__ void ra_st16(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(t)
      : "memory");
}
__device__ __forceinline__ void ra_ld16(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ float ra_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float ra_max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint64_t ra_pair(float lo, float hi) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ void ra_unpair(uint64_t p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ uint64_t ra_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t ra_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t ra_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t ra_bmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Two e4m3 codes (bytes 0, 1 with 0x9180, bytes 2, 3 with 0xB3A2: each and its sign, eight times) as bf16 bits of their values
// times 2^-120: the sign, then exponent and digits three places below.  (0x7F is not told apart: 480.)
template <uint32_t kSel>
__device__ __forceinline__ uint32_t ra_code2(uint32_t w) {
  uint32_t x;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(x) : "r"(w), "n"(kSel));
  return (x << 4) & 0x87F087F0u;
}
__device__ __forceinline__ void ra_prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ uint4 ra_ldg128(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// Whether one of a pair's bf16 values is infinite or NaN: the exponent's ones carry into the sign.
__device__ __forceinline__ uint32_t ra_special(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// v *= sigmoid(g) for two bf16 gates.  By half the exponential twice: e^g itself leaves fp32's range long before the product
// does (NaN stays NaN).
__device__ __forceinline__ void ra_gate2(float& v0, float& v1, uint32_t w) {
  constexpr float kHalfLog2e = 0.7213475204444817f;
  const float g0 = __uint_as_float(w << 16), g1 = __uint_as_float(w & 0xFFFF0000u);
  const float h0 = ra_ex2(-kHalfLog2e * fabsf(g0)), h1 = ra_ex2(-kHalfLog2e * fabsf(g1));
  const float n0 = g0 < 0.0f ? h0 : 1.0f, n1 = g1 < 0.0f ? h1 : 1.0f;
  v0 = __fdividef(v0 * n0 * n0, fmaf(h0, h0, 1.0f));
  v1 = __fdividef(v1 * n1 * n1, fmaf(h1, h1, 1.0f));
}
// What is subtracted from the scores for a reference: nothing where there is none yet; NaN, which every weight of the row then is,
// where a score is infinite or beyond fp32's range (finite scores less infinity would be weights of zero).
__device__ __forceinline__ float ra_less(float m) {
  return m == -INFINITY ? 0.0f : m == INFINITY ? __int_as_float(0x7FFFFFFF) : m;
}
// log sum exp from the reference in log2 units and the sum of 2^(t - m).
__device__ __forceinline__ float ra_lse(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Codes to bf16: a tile of kRowsT rows of kCols codes, then a scale byte per row, to an operand tile, by 128 threads.  Eight
// lanes take 64 codes of each of two rows, of neighbouring column groups where there are several: reads and writes then meet
// every bank once.  Scales from 2^8 on (the factor leaves bf16's range; 255 is NaN) are left to ra_expand_rare, for which this
// says whether there are any among the first `left` rows (behind them lies what nobody sees: a scale there may be anything, and costs
// nothing).  (A code 0x7F under another scale, which the append does not write, comes out as 480.)
template <int kCols, int kRowsT>
struct RaUnit {  // unit u (of kRowsT * kCols / 16) of thread tid: 16 codes
  int row, ch, i;
  __device__ RaUnit(int tid, int u) {
    constexpr int kChunks = kCols / 64;
    const int qd = (tid >> 3) + 16 * u, rsel = tid >> 2 & 1;
    row = 2 * (qd / kChunks) + rsel;
    ch = kChunks > 1 ? (qd % kChunks) ^ rsel : 0;
    i = tid & 3;
  }
  __device__ uint32_t in(uint32_t src) const { return src + row * kCols + ch * 64 + i * 16; }
  __device__ uint32_t scale(uint32_t src) const { return src + kRowsT * kCols + row; }
  __device__ uint32_t out(uint32_t dst, int k) const {  // of the k-th eight values
    return dst + ch * (kRowsT * 128) + row * 128 + (((2 * i + k) ^ (row & 7)) << 4);
  }
};
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
template <int kCols, int kRowsT>
__device__ __forceinline__ bool ra_expand(uint32_t src, uint32_t dst, int tid, int left) {
  constexpr int kUnits = kRowsT * kCols / 16 / 128, kAtOnce = 4;
  bool rare = false;
#pragma unroll 1
  for (int u0 = 0; u0 < kUnits; u0 += kAtOnce) {
    uint4 w[kAtOnce];
    uint32_t e[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const RaUnit<kCols, kRowsT> u(tid, u0 + k);
      w[k] = lds128(u.in(src));
      e[k] = lds8(u.scale(src));
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const RaUnit<kCols, kRowsT> u(tid, u0 + k);
      const uint32_t in[4] = {w[k].x, w[k].y, w[k].z, w[k].w}, f = (e[k] + 120) * 0x00800080u;  // 2^(120 + scale - 127)
      uint32_t o[8];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        o[2 * x] = ra_bmul2(ra_code2<0x9180>(in[x]), f);
        o[2 * x + 1] = ra_bmul2(ra_code2<0xB3A2>(in[x]), f);
      }
      rare = rare || (e[k] > 134 && u.row < left);
      sts128(u.out(dst, 0), make_uint4(o[0], o[1], o[2], o[3]));
      sts128(u.out(dst, 1), make_uint4(o[4], o[5], o[6], o[7]));
    }
  }
  return rare;
}
template <int kCols, int kRowsT>
__device__ __forceinline__ void ra_expand_rare(uint32_t src, uint32_t dst, int tid) {
#pragma unroll 1
  for (int k = 0; k < kRowsT * kCols / 128; ++k) {
    const RaUnit<kCols, kRowsT> u(tid, k >> 4);
    const uint32_t code = lds8(u.in(src) + (k & 15)), e = lds8(u.scale(src));
    const uint32_t bits = (code & 0x80) << 8 | (code & 0x7F) << 4, one = e == 0 ? 0x40u : e << 7;
    uint32_t v = ra_bmul2(ra_bmul2(bits, 0x7B80u), one) & 0xFFFFu;
    if (e == 255) v = 0x7FFFu;
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(u.out(dst, k >> 3 & 1) + (k & 7) * 2), "h"((uint16_t)v) : "memory");
  }
}
// A value tile with keys that some row does not see, or without keys in part (rows from `left` on, `bad` groups of 16 rows):
// what lies in those becomes zeros (weights of zero times what lies there), and, where the block is an edge block, so do
// infinite and NaN values, whose key is noted by column.
template <int kCols, int kRowsT>
__device__ __forceinline__ void ra_look(uint32_t tile, int tid, int left, uint32_t bad, bool edge, int key0, int* poison, int* special) {
#pragma unroll 1
  for (int u = tid; u < kRowsT * kCols / 8; u += 128) {
    const int ch = u / (kRowsT * 8), row = (u >> 3) % kRowsT, d = ch * 64 + (((u & 7) ^ (row & 7)) << 3);
    const uint32_t at = tile + u * 16;
    if (row >= left || (bad >> (row >> 4) & 1)) {
      sts128(at, make_uint4(0, 0, 0, 0));
      continue;
    }
    if (!edge) continue;
    const uint4 w = lds128(at);
    if (!(ra_special(w.x) | ra_special(w.y) | ra_special(w.z) | ra_special(w.w))) continue;
    *(volatile int*)special = 1;
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
      uint16_t v;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at + 2 * k));
      if ((v & 0x7F80) != 0x7F80) continue;
      atomicMin(poison + d + k, key0 + row);
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + 2 * k), "h"((uint16_t)0) : "memory");
    }
  }
}

// ------------------------------------------------------------------ work
// A sequence: n new rows from row0 on, which see the L cached positions up to their own.  A blank one has L = 0 and outputs of zero:
// an empty slot (no row_start, no positions), or a bad one, whose lengths do not fit.
struct RaSeq {
  int row0, n, L;
  bool blank, bad;
};
template <int kSrc>
__device__ __forceinline__ RaSeq ra_seq(const RowsArgs& a, int s) {
  RaSeq q;
  int r0 = s, r1 = s + 1;
  if (a.row_start) r0 = __ldg(a.row_start + s), r1 = __ldg(a.row_start + s + 1);
  q.bad = r0 < 0 || r1 > a.M || r1 < r0;
  r0 = max(r0, 0), r1 = min(r1, a.M);
  q.row0 = r0;
  q.n = r1 > r0 ? r1 - r0 : 0;
  q.L = q.n;
  bool empty = false;
  if (kSrc != kDense) {
    q.L = __ldg(a.kv_len + s);
    empty = !a.row_start && q.L == 0;
    q.bad = !empty && (q.bad || q.L < q.n || q.L > (long long)a.max_pages << a.log_page);
  }
  q.blank = q.bad || empty;
  if (q.blank) q.L = 0;
  return q;
}
// The work is one line: for every sequence, key-value head and item (tok_tile tokens) in turn, the item's keys and
// item_cost.  Its blocks lie at multiples of kBlock keys from the item's start; a CTA (a pair) owns the blocks that begin in
// its part of the line.
constexpr int kMinKeys = 256;   // of the line per CTA at least

// The line up to item t of one head.
__device__ __forceinline__ long long ra_upto(const RowsArgs& a, const RaSeq& q, int t) {
  if (q.blank) return (long long)t * a.item_cost;
  return (long long)t * ((long long)(q.L - q.n) + a.item_cost) + (long long)a.tok_tile * ((long long)t * (t + 1) / 2);
}
// Blocks of B keys; keys may be any int from 0 on.
template <int B>
__device__ __forceinline__ int ra_blocks(int keys) { return (int)(((uint32_t)keys + (B - 1)) / B); }
__device__ __forceinline__ int ra_items(const RowsArgs& a, const RaSeq& q) { return (q.n + a.tok_tile - 1) / a.tok_tile; }
__device__ __forceinline__ long long ra_line(const RowsArgs& a, const RaSeq& q) {
  if (q.n == 0) return 0;
  return ra_upto(a, q, ra_items(a, q) - 1) + q.L + a.item_cost;
}

// One piece of work, in shared memory: blocks b0 .. b1 - 1 of an item.
struct RaItem {
  int s, h;            // s < 0: the end
  int row;             // global row of the first token
  int kv_row;          // global row of the sequence's first key (dense)
  int toks;
  int lim0;            // keys that the first token sees; each further token one more
  int keys;            // that the last one sees (0: a blank sequence)
  int b0, b1;
  int cnt[2];          // blocks of each tile of 128 rows in this piece
  int edge;            // first block that some token does not see whole
  int slot;            // -1: the whole item; 0, 1: the CTA's first, last part
};

// kTiles: tiles of 128 rows per item.  Two lie in one CTA, or, with 256 columns, in the two CTAs of a pair, each of which
// holds half of every key and value block.
template <int D, int kTiles, int kSrc>
struct RaCfg {
  static constexpr bool kFp8 = kSrc == kPagedFp8, kPair = D == 256 && kTiles == 2;
  static constexpr int kSub = kPair ? 1 : kTiles;                    // tiles in a CTA
  // warps that prepare operands (with codes, four expand keys and four values), softmax warps
  static constexpr int kPrep = kFp8 ? 8 : 4, kSoft = 4 * kSub, kThreads = 32 * (4 + kPrep + kSoft);
  static constexpr int kBlock = rows_block(D, kTiles);
  static constexpr int kRows = 128 * kTiles;
  // operand tiles in a CTA: key rows and columns; a pair's CTA holds half of the keys, and half of the values' columns
  static constexpr int kKRows = kPair ? kBlock / 2 : kBlock, kVCols = kPair ? D / 2 : D;
  static constexpr int kTile = kKRows * D * 2;                       // bytes, of either
  static_assert(kTile == kBlock * kVCols * 2, "");
  static constexpr int kRaw = kTile / 2 + 128;                       // the same in codes, and the scales' bytes
  // One tile with at most 32 rows: every softmax warp takes all of them and a quarter of each block's keys (else three of the
  // four would have nothing to do, and the fourth would take longer than codes take to arrive); the quarters are joined here.
  static constexpr int kJoin = kTiles == 1 ? 4 * 4096 : 0;
  static constexpr bool kQSmem = kTiles == 2;                        // else the queries lie in tensor memory
  static constexpr int kQ = kQSmem ? kSub * 128 * D * 2 : 0;
  // stages of keys and of values, rings of their own (with codes: of bf16 tiles, and of codes)
  static constexpr int kKSt = kFp8 ? (D == 64 ? 3 : 2) : D == 64 ? 4 : kTiles == 2 ? 2 : 3, kVSt = !kFp8 && D > 64 && kTiles == 2 ? 3 : kKSt;
  static constexpr int kStages = kKSt + kVSt;
  static constexpr int kRawSt = !kFp8 ? 0 : D == 64 ? 4 : kTiles == 2 ? 1 : 2, kRawStages = 2 * kRawSt;
  static constexpr int kRing = kPair ? 2 : 3;                        // items
  static constexpr int kParts = kBlock / 64;                         // of a block's weights: the products take the first ones early
  // tensor memory: scores (two tiles, or two buffers of one), outputs, queries
  static constexpr int kColS = kBlock;                               // from one score buffer to the next
  static constexpr int kColO = 2 * kColS;
  static constexpr int kColQ = kColO + D;
  // registers: what issues keeps few, what prepares operands some, the softmax warps take the rest of the launch's
  static constexpr int kLaunch = 65536 / kThreads / 8 * 8;
  static constexpr int kRegIssue = kThreads == 640 ? 48 : kSub == 2 || kFp8 ? 64 : 104,
                       kRegPrep = kThreads == 640 ? 56 : kSub == 2 ? 64 : kFp8 ? 96 : 168,
                       kRegSoft = kThreads == 640 ? 160 : kSub == 2 ? 192 : 232;
  static_assert(4 * kRegIssue + kPrep * kRegPrep + kSoft * kRegSoft <= kThreads / 32 * kLaunch, "");
  static_assert(kColO + kSub * D <= 512 && (kQSmem || kColQ + D / 2 <= 512), "");
};
template <int D, int kTiles, int kSrc>
struct RaShared {
  using C = RaCfg<D, kTiles, kSrc>;
  uint64_t full[C::kStages], ready[C::kStages], empty[C::kStages];
  uint64_t rfull[C::kRawStages + 1], rempty[C::kRawStages + 1];
  uint64_t sfull[2], pfull[2][2], ofull[2], opart[2], qfull[2], qfree[2], meet[2];
  uint64_t ifull[C::kRing], iempty[C::kRing], drain;
  unsigned long long scan[C::kThreads / 32];
  unsigned long long x0, x1, base;
  RaItem item[C::kRing];
  int special[C::kRing];    // whether poison has an entry
  int poison[C::kRing][D];  // per column: the first key of the item's edge blocks whose value is infinite or NaN
  uint32_t bad[16];         // per block: the groups of 16 keys whose page does not exist
  float quarter[kTiles == 1 ? 4 : 1][kTiles == 1 ? 32 : 1][2];  // maxima and sums of the quarters
  int s0;
  uint32_t tmem;
  int abort;
};
template <int D, int kTiles, int kSrc>
constexpr int ra_smem() {
  using C = RaCfg<D, kTiles, kSrc>;
  return C::kQ + C::kStages * C::kTile + C::kJoin + C::kRawStages * C::kRaw + (int)sizeof(RaShared<D, kTiles, kSrc>);
}

template <int D, int kTiles, int kSrc>
__global__ void __launch_bounds__(RaCfg<D, kTiles, kSrc>::kThreads, 1)
    rows_kernel(const __grid_constant__ RowsArgs a, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
  using C = RaCfg<D, kTiles, kSrc>;
  constexpr bool kPair = C::kPair;
  constexpr int BN = C::kBlock, kSub = C::kSub;
  constexpr int kChunks = D / 64, kVChunks = C::kVCols / 64;                    // 128-byte column groups of keys, of values
  constexpr uint32_t kKGroup = C::kKRows * 128, kVGroup = BN * 128;             // bytes from one to the next
  extern __shared__ __align__(1024) uint8_t dyn[];
  uint8_t* const q_p = dyn;
  uint8_t* const ring_p = q_p + C::kQ;
  uint8_t* const join_p = ring_p + C::kStages * C::kTile;
  uint8_t* const raw_p = join_p + C::kJoin;
  auto& sh = *reinterpret_cast<RaShared<D, kTiles, kSrc>*>(raw_p + C::kRawStages * C::kRaw);
  const uint32_t q_s = smem_addr(q_p), ring = smem_addr(ring_p), raw = smem_addr(raw_p);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kPair ? (int)ra_rank() : 0;
  const int c = kPair ? blockIdx.x >> 1 : blockIdx.x, workers = kPair ? gridDim.x >> 1 : gridDim.x;  // CTAs or pairs
#ifdef VP_WAIT_TEST
  // Wait-test hook (workspace word kWsTestSkip): the first CTA (a pair's second one with 6, 7 in place of 2, 4) leaves out
  // 1 its first scores' commit, 2 a softmax warp's first arrival, 3 its first copies, 4 the first arrival of the warps
  // that prepare operands, 5 its first item.
  const int word = ((const volatile int*)a.status)[kWsTestSkip / sizeof(int)];
  const int hook = blockIdx.x == 0 && word < 6 ? word : blockIdx.x == 1 && word == 6 ? 2 : blockIdx.x == 1 && word == 7 ? 4 : 0;
#else
  constexpr int hook = 0;
#endif

  // -------------------------------------------------------------- the CTA's (pair's) part of the line
  if (threadIdx.x == 0) {
    if (rank == 0) a.desc[2 * c] = a.desc[2 * c + 1] = make_int4(0, 0, -1, 0);
    sh.abort = 0;
  }
  {
    const int per = (a.S + C::kThreads - 1) / C::kThreads, s0 = min((int)threadIdx.x * per, a.S), s1 = min(s0 + per, a.S);
    unsigned long long mine = 0;
    bool falls = false;
    for (int s = s0; s < s1; ++s) {
      const RaSeq q = ra_seq<kSrc>(a, s);
      falls = falls || (a.row_start && __ldg(a.row_start + s + 1) < __ldg(a.row_start + s));
      if (q.bad && blockIdx.x == 0) report_unless(a.status, VP_ERR_SHAPE, VP_ERR_TIMEOUT);
      mine += (unsigned long long)ra_line(a, q) * a.Hkv;
    }
    unsigned long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) sh.scan[warp] = upto;
    // Sequences that overlap could have any number of rows: no work is begun.
    if (__syncthreads_or(falls)) return;
    unsigned long long total = 0, before = 0;
#pragma unroll 1
    for (int w = 0; w < C::kThreads / 32; ++w) {
      if (w == warp) before = total;
      total += sh.scan[w];
    }
    const unsigned long long most = total / kMinKeys;
    const int parts = most < 1 ? 1 : most < workers ? (int)most : workers;
    if (total == 0 || c >= parts) return;
    const unsigned long long each = total / parts, more = total % parts;
    const unsigned long long x0 = each * c + more * c / parts, x1 = each * (c + 1) + more * (c + 1) / parts;
    before += upto - mine;
    if (x0 >= before && x0 < before + mine) {  // the sequence that holds the part's start
      unsigned long long at = before;
      int s = s0;
      for (; s + 1 < s1; ++s) {
        const unsigned long long u = (unsigned long long)ra_line(a, ra_seq<kSrc>(a, s)) * a.Hkv;
        if (at + u > x0) break;
        at += u;
      }
      sh.s0 = s, sh.base = at, sh.x0 = x0, sh.x1 = x1;
    }
  }
  constexpr int kBoth = kPair ? 2 : 1;  // CTAs that arrive at the first one's barriers
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.ready[i], (C::kFp8 ? 4 : 5) * kBoth);  // four preparing warps and the copying one, or that one in their place
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < C::kRawStages; ++i) {
      mbar_init(&sh.rfull[i], 33);  // the copies of codes, and every lane's of scales
      mbar_init(&sh.rempty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.sfull[i], 1);
      for (int k = 0; k < 2; ++k) mbar_init(&sh.pfull[i][k], 4 * kBoth);
      mbar_init(&sh.ofull[i], 1);
      mbar_init(&sh.opart[i], 1);
      mbar_init(&sh.qfull[i], 4 * kBoth);
      mbar_init(&sh.qfree[i], 4);
      mbar_init(&sh.meet[i], 4);
    }
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(&sh.ifull[i], 1);
      mbar_init(&sh.iempty[i], 3 + C::kPrep + C::kSoft * kBoth);  // copying (two), issuing, preparing and softmax warps (a pair's: of both)
    }
    mbar_init(&sh.drain, 1);
    fence_mbar_init();
  }
  __syncwarp();  // the sequence's finder comes back: the allocation is a whole warp's
  if (warp == 1) {
    if constexpr (kPair) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem)) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(&sh.tmem, 512);
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (kPair) ra_pair_sync();  // the other CTA's barriers exist
  tmem_fence_after();
  const uint32_t tmem = ra_uniform(*(volatile uint32_t*)&sh.tmem);

  // Bounded waits of a converged warp; false when one ran out here or elsewhere in the CTA.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return ra_wait<kPair>(smem_addr(bar), parity, kMbarPolls, &sh.abort, a.status);
  };
  auto wait_item = [&](uint64_t* bar, uint32_t parity) -> bool {
    return ra_wait<kPair>(smem_addr(bar), parity, a.polls, &sh.abort, a.status);
  };
  // One lane's arrival for its warp, here, or where the products are issued.
  auto arrive = [&](uint64_t* bar) { ra_arrive(smem_addr(bar)); };
  auto arrive_first = [&](uint64_t* bar) {
    if constexpr (kPair)
      ra_arrive_first(smem_addr(bar));
    else
      ra_arrive(smem_addr(bar));
  };
  auto arrive_first_relaxed = [&](uint64_t* bar) {
    if constexpr (kPair)
      ra_arrive_first_relaxed(smem_addr(bar));
    else
      ra_arrive(smem_addr(bar));
  };
  // Four warps meet (a bounded wait, unlike a hardware barrier: another warp may have given up).
  auto meet = [&](int i, uint32_t& parity) -> bool {
    __syncwarp();
    if (lane == 0) arrive(&sh.meet[i]);
    const bool there = wait(&sh.meet[i], parity);
    parity ^= 1;
    return there;
  };
  // The it-th item, for every role but the scheduler; null when a wait ran out.
  auto get = [&](int it) -> const RaItem* {
    if (!wait_item(&sh.ifull[it % C::kRing], (it / C::kRing) & 1)) return nullptr;
    return &sh.item[it % C::kRing];
  };
  auto release = [&](int it) {
    __syncwarp();
    if (lane == 0) arrive(&sh.iempty[it % C::kRing]);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegIssue));
    if (warp == 3) {
      // ---------------------------------------------------------- scheduler: the pieces in turn (a pair's CTAs: the same ones)
      const long long x0 = (long long)sh.x0, x1 = (long long)sh.x1;
      long long at = (long long)sh.base;       // the line at the current sequence's (head's, item's) start
      int s = sh.s0, h = 0, t = 0, cached = -1, it = 0;
      int c_row = 0, c_n = 0, c_L = 0, c_blank = 0;  // lane l: sequence cached + l
      bool ok = true, jump = true;
      while (ok && s < a.S && at < x1) {
        if ((s & ~31) != cached) {
          cached = s & ~31;
          c_n = 0;
          if (cached + lane < a.S) {
            const RaSeq q = ra_seq<kSrc>(a, cached + lane);
            c_row = q.row0, c_n = q.n, c_L = q.L, c_blank = q.blank;
          }
        }
        RaSeq q;
        q.n = __shfl_sync(0xFFFFFFFFu, c_n, s & 31);
        if (q.n == 0) {  // the next sequence that has rows
          const uint32_t have = __ballot_sync(0xFFFFFFFFu, c_n > 0) >> (s & 31);
          s = have ? s + __ffs(have) - 1 : cached + 32;
          continue;
        }
        q.row0 = __shfl_sync(0xFFFFFFFFu, c_row, s & 31);
        q.L = __shfl_sync(0xFFFFFFFFu, c_L, s & 31);
        q.blank = __shfl_sync(0xFFFFFFFFu, c_blank, s & 31);
        const int items = ra_items(a, q);
        if (jump) {  // to the item that holds x0
          jump = false;
          const long long line = ra_line(a, q);
          if (x0 > at) {
            h = (int)min((x0 - at) / line, (long long)a.Hkv - 1);
            at += h * line;
            int lo = 0, hi = items;  // upto(lo) <= x0 - at; the answer lies in [lo, hi)
            while (hi - lo > 1) {
              const int mid = (lo + hi) >> 1;
              if (ra_upto(a, q, mid) <= x0 - at) lo = mid; else hi = mid;
            }
            t = lo;
            at += ra_upto(a, q, t);
          }
        }
        const int tok0 = t * a.tok_tile, toks = min(a.tok_tile, q.n - tok0);
        const int keys = q.blank ? 0 : q.L - q.n + tok0 + toks, nb = ra_blocks<BN>(keys);
        // blocks whose place on the line lies in [x0, x1); a blank sequence's item by its start
        const long long f = x0 - at, e = x1 - at;
        const int b0 = f <= 0 ? 0 : (int)min((f + BN - 1) / BN, (long long)nb), b1 = (int)min((e + BN - 1) / BN, (long long)nb);
        const bool mine = nb ? b0 < b1 : f <= 0;
        if (mine) {
          const int slot = it % C::kRing;
          if (it >= C::kRing && !(ok = wait_item(&sh.iempty[slot], (it / C::kRing - 1) & 1))) break;
          for (int d = lane; d < D; d += 32) sh.poison[slot][d] = 0x7FFFFFFF;
          if (lane == 0) {
            sh.special[slot] = 0;
            RaItem& i = sh.item[slot];
            i.s = s, i.h = h;
            i.row = q.row0 + tok0;
            i.kv_row = q.row0;
            i.toks = toks;
            i.lim0 = q.blank ? 0 : q.L - q.n + tok0 + 1;
            i.keys = keys;
            i.b0 = b0, i.b1 = b1;
            // Of two tiles in a CTA the first sees no further than its last token, and the second is there only if there
            // are more than 128 rows.
            const int rows = toks * a.G, k0 = q.blank ? 0 : i.lim0 + min(toks - 1, 127 / a.G);
            i.cnt[0] = kSub == 1 ? b1 - b0 : max(min(b1, ra_blocks<BN>(k0)) - b0, 0);
            i.cnt[1] = kSub == 2 && rows > 128 ? b1 - b0 : 0;
            i.edge = i.lim0 / BN;
            const bool starts = b0 == 0, ends = b1 == nb;
            i.slot = starts && ends ? -1 : starts ? 1 : 0;
            if (i.slot >= 0 && rank == 0) a.desc[2 * c + i.slot] = make_int4(s, h, q.row0 + tok0, rows | (ends ? kPartEnds : 0));
          }
          __syncwarp();
          if (lane == 0 && !(hook == 5 && it == 0)) arrive(&sh.ifull[slot]);
          ++it;
        }
        at += (long long)keys + a.item_cost;
        if (++t == items) {
          t = 0;
          if (++h == a.Hkv) h = 0, ++s;
        }
      }
      const int slot = it % C::kRing;
      if (ok && (it < C::kRing || wait_item(&sh.iempty[slot], (it / C::kRing - 1) & 1))) {
        if (lane == 0) {
          sh.item[slot].s = -1;
          arrive(&sh.ifull[slot]);
        }
      }
      __syncwarp();
    } else if (warp == 0 || warp == 2) {
      // ---------------------------------------------------------- copies: a warp for keys, one for values (starting a copy takes
      // about 130 cycles, and a block of pages of 16 has up to 32 of them)
      const int kv = warp >> 1;
      const int base = !kv ? 0 : C::kFp8 ? C::kRawSt : C::kKSt, stages = C::kFp8 ? C::kRawSt : kv ? C::kVSt : C::kKSt;
      uint64_t* const empty = C::kFp8 ? sh.rempty : sh.empty;
      const int P = 1 << a.log_page;
      int cur = 0, nxt = 0, cur_s = -1, cur_w = -1, nxt_w = -1;  // lane l: page table entry cur_w + l
      int st = base, g = 0;
      uint32_t par = 1;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const RaItem* pi = get(it);
        if (!pi || pi->s < 0) break;
        const int i_s = pi->s, i_h = pi->h, i_kv = pi->kv_row, i_keys = pi->keys, i_b0 = pi->b0, i_b1 = pi->b1, i_edge = pi->edge;
        for (int b = i_b0; ok && b < i_b1; ++b, ++g) {
          const int key0 = b * BN, last = (i_keys - 1) >> a.log_page;
          uint32_t wrong = 0;  // the block's pages that do not exist
          if (kSrc != kDense) {
            const int p0 = key0 >> a.log_page, w = p0 & ~31;
            if (i_s != cur_s || w != cur_w) {
              const int32_t* tab = a.pages + (size_t)i_s * a.max_pages;
              cur = i_s == cur_s && w == nxt_w ? nxt : w + lane < a.max_pages ? __ldg(tab + w + lane) : 0;
              cur_s = i_s, cur_w = w, nxt_w = w + 32;
              nxt = nxt_w + lane < a.max_pages ? __ldg(tab + nxt_w + lane) : 0;
            }
            const int box = min(P, BN), have = min(BN / box, last - p0 + 1);
            const int page = __shfl_sync(0xFFFFFFFFu, cur, (p0 - w + lane) & 31);
            wrong = __ballot_sync(0xFFFFFFFFu, lane < have && (page < 0 || page >= a.n_pages));
            uint32_t bad = 0;
            if (wrong) {
              const int per = box / 16;  // groups of 16 keys of a page
              for (int k = 0; k < have; ++k)
                if (wrong >> k & 1) bad |= ((1u << per) - 1) << (k * per);
              if (lane == 0) report_unless(a.status, VP_ERR_SHAPE, VP_ERR_TIMEOUT);
            }
            if (lane == 0) sh.bad[g & 15] = bad;  // (by both warps, the same; its announcement below releases it)
          }
          {
            if (!(ok = wait(&empty[st], par))) break;
            const bool skip = hook == 3 && g + kv == 0;
            // Values that some row does not see whole go by the preparing warps; what else is copied as it is announces itself
            // where the products are issued.
            const bool look = kv && b >= i_edge;
            auto announce = [&](uint32_t bytes) {
              if (look) {
                if (lane == 0) mbar_arrive_expect_tx(&sh.full[st], bytes);
                if (lane == 1) arrive_first_relaxed(&sh.ready[st]);
              } else if (lane == 0) {
                if constexpr (kPair)
                  ra_expect_first<kSrc != kDense>(smem_addr(&sh.ready[st]), bytes);  // pages: lane 0 has noted the missing ones
                else
                  mbar_arrive_expect_tx(&sh.ready[st], bytes);
              } else if (lane < 5) {
                arrive_first_relaxed(&sh.ready[st]);
              }
              __syncwarp();
            };
            auto copy3d = [&](uint32_t dst, int y, int z) {
              const CUtensorMap* map = kv ? &vmap : &kmap;
              if (!kPair || look)
                ra_tma_3d(dst, map, 0, y, z, smem_addr(look ? &sh.full[st] : &sh.ready[st]));
              else
                ra_tma_3d_first(dst, map, 0, y, z, smem_addr(&sh.ready[st]));
            };
            // this CTA's rows and columns of the block
            const int rows = kv ? BN : C::kKRows, key = key0 + (kPair && !kv ? rank * C::kKRows : 0);
            const int chunks = kv ? kVChunks : kChunks, chunk0 = kPair && kv ? rank * kVChunks : 0;
            if constexpr (kSrc == kDense) {
              announce(C::kTile);
              if (lane == 0 && !skip) copy3d(ring + st * C::kTile, i_kv + key, i_h * kChunks + chunk0);
            } else {
              const int box = min(P, rows), p0 = key >> a.log_page, in_page = key & (P - 1);
              const int have = max(min(rows / box, last - p0 + 1), 0);  // pages with keys
              // lane -> page, and column group where a page's rows are not the whole tile's
              const bool apart = !C::kFp8 && box < rows;
              const int of = apart ? lane / chunks : lane;
              const int page = __shfl_sync(0xFFFFFFFFu, cur, (p0 - cur_w + of) & 31);
              const bool real = page >= 0 && page < a.n_pages;
              const int y = ((page * a.Hkv + i_h) << a.log_page) + in_page;
              if constexpr (kSrc == kPaged) {
                const uint32_t dst = ring + st * C::kTile;
                const int none = a.n_pages * a.Hkv << a.log_page;  // behind the cache: zeros
                announce(have * box * chunks * 128);
                if (!skip && (apart ? lane < have * chunks : lane < have)) {
                  const int ch = apart ? lane % chunks : 0;
                  copy3d(dst + (ch * rows + of * box) * 128, real ? y : none, chunk0 + ch);
                }
              } else {
                const uint32_t dst = raw + st * C::kRaw, bar = smem_addr(&sh.rfull[st]);
                const bool copy = lane < have && real;
                const int copies = __popc(__ballot_sync(0xFFFFFFFFu, copy));
                if (lane == 0) mbar_arrive_expect_tx(&sh.rfull[st], copies * box * chunks * 64);
                __syncwarp();
                if (!skip && copy) ra_tma_2d(dst + lane * box * chunks * 64, kv ? &vmap : &kmap, chunk0 * 64, y, bar);
                // the scales, 16 a lane: lane l those of the tile's rows 16 l ..
                const int sp = lane / (box / 16), spage = __shfl_sync(0xFFFFFFFFu, cur, (p0 - cur_w + sp) & 31);
                if (sp < have && spage >= 0 && spage < a.n_pages)
                  ra_copy16(dst + rows * chunks * 64 + lane * 16,
                            (kv ? a.v_scales : a.k_scales) + ((size_t)(spage * a.Hkv + i_h) << a.log_page) + in_page + lane % (box / 16) * 16);
                ra_copy16_arrive(bar);
              }
            }
            __syncwarp();
            if (++st == base + stages) st = base, par ^= 1;
          }
        }
        if (ok) release(it);
      }
      // Nothing may be on its way to this CTA's shared memory when it ends.  Copies of codes: they have landed, whatever ran
      // out.  Others: a stage's last commit says that its copies have been read, and is itself the last arrival; where the
      // products have stopped this takes the wait's whole limit, in which whatever was on its way arrives.
      for (int i = 0; i < min(g, stages); ++i) {
        const int e = g - 1 - (g - 1 - i) % stages;  // the last copy into the ring's stage i
        uint64_t* const bar = (C::kFp8 ? sh.rfull : sh.empty) + base + i;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, (e / stages) & 1))) {
          *(volatile int*)&sh.abort = 1;
          atomicExch(a.status, (int)VP_ERR_TIMEOUT);
          break;
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- matrix products
      constexpr uint32_t kIdesc = 1u << 4 | 1u << 7 | 1u << 10 | (kPair ? 16u : 8u) << 24;  // bf16 x bf16 -> fp32, rows
      constexpr uint32_t kIdS = kIdesc | (uint32_t)(BN >> 3) << 17, kIdO = kIdesc | 1u << 16 | (uint32_t)(D >> 3) << 17;
      int ks = 0, vs = C::kKSt, g = 0;         // stages; blocks so far (one tile: of the score buffers)
      uint32_t kpar = 0, vpar = 0, qpar = 0, ppar = 0;  // of the stages, queries, weights (a bit per tile or buffer)
      bool ok = true, first = true;
      // Four products at a time in a loop (the warps of a scheduler share its instruction cache).
      auto scores = [&](int i, int stage) {  // tile i, or buffer i of the one tile
        uint64_t db = ra_desc_k(ring + stage * C::kTile), da = ra_desc_k(q_s + (kSub == 2 ? i * 128 * D * 2 : 0));
        uint32_t d = tmem + i * C::kColS, qa = tmem + C::kColQ;
#pragma unroll 1
        for (int ch = 0; ch < kChunks; ++ch) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (C::kQSmem)
              ra_mma_ss<kPair>(d, da + 2 * k, db + 2 * k, kIdS, ch + k > 0);
            else
              ra_mma_ts<kPair>(d, qa + 8 * k, db + 2 * k, kIdS, ch + k > 0);
          }
          db += kKGroup >> 4, da += 16384 >> 4, qa += 32;
        }
      };
      // weights of score buffer i, from block part on, into output o
      auto outputs = [&](int i, int o, int stage, int part, bool accumulate) {
        const uint64_t db = ra_desc_mn(ring + stage * C::kTile, kVGroup) + (uint64_t)(part * 4 * (2048 >> 4));
        const uint32_t p = tmem + i * C::kColS + part * 32, d = tmem + C::kColO + o * D;
#pragma unroll
        for (int k = 0; k < 4; ++k) ra_mma_ts<kPair>(d, p + 8 * k, db + (uint64_t)(k * (2048 >> 4)), kIdO, accumulate || k > 0);
      };
      auto q_ready = [&](int i) -> bool {
        const bool there = wait(&sh.qfull[i], qpar >> i & 1);
        qpar ^= 1u << i;
        return there;
      };
      // Outputs of block j from buffer i as its weights come, a part at a time.
      auto weigh = [&](int i, int o, int stage, bool accumulate) -> bool {
#pragma unroll 1
        for (int part = 0; part < C::kParts; ++part) {
          if (!wait(&sh.pfull[i][part], ppar >> i & 1)) return false;
          tmem_fence_after();
          if (ra_elect()) {
            outputs(i, o, stage, part, accumulate || part > 0);
            if (part + 1 < C::kParts) ra_commit<kPair>(&sh.opart[i]);
          }
          __syncwarp();
        }
        ppar ^= 1u << i;
        return true;
      };
      auto next_k = [&]() {
        if (++ks == C::kKSt) ks = 0, kpar ^= 1;
      };
      auto next_v = [&]() {
        if (++vs == C::kStages) vs = C::kKSt, vpar ^= 1;
      };
      for (int it = 0; ok; ++it) {
        const RaItem* pi = get(it);
        if (!pi || ra_uniform(pi->s) < 0) break;
        if (kPair && rank) {  // the first CTA issues
          release(it);
          continue;
        }
        const int nblk = ra_uniform(pi->b1 - pi->b0), cnt0 = ra_uniform(pi->cnt[0]), cnt1 = ra_uniform(pi->cnt[1]);
        if (cnt0 > 0) ok = q_ready(0);
        if (kSub == 2 && ok && cnt1 > 0) ok = q_ready(1);
        // Scores of block j + 1 and outputs of block j.  With two tiles one's softmax runs beside the other's products, with one
        // its next scores lie in a second buffer.
        for (int j = -1; ok && j < nblk; ++j) {
          if constexpr (kSub == 1) {
            if (j + 1 < nblk) {
              if (!(ok = wait(&sh.ready[ks], kpar))) break;
              tmem_fence_after();
              if (ra_elect()) {
                scores((g + j + 1) & 1, ks);
                if (!(hook == 1 && first)) ra_commit<kPair>(&sh.sfull[(g + j + 1) & 1]);
                ra_commit<kPair>(&sh.empty[ks]);
              }
              first = false;
              __syncwarp();
              next_k();
            }
            if (j >= 0) {
              const int buf = (g + j) & 1;
              if (!(ok = wait(&sh.ready[vs], vpar) && weigh(buf, 0, vs, j > 0))) break;
              if (ra_elect()) {
                ra_commit<kPair>(&sh.ofull[buf]);
                ra_commit<kPair>(&sh.empty[vs]);
              }
              __syncwarp();
              next_v();
            }
          } else {
            bool have_v = false, have_k = false;
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
              const int cnt = i ? cnt1 : cnt0;
              if (ok && j >= 0 && j < cnt) {
                if (!have_v) ok = have_v = wait(&sh.ready[vs], vpar);
                ok = ok && weigh(i, i, vs, j > 0);
                if (ok && ra_elect()) ra_commit<kPair>(&sh.ofull[i]);
                __syncwarp();
              }
              if (ok && j + 1 < cnt) {
                if (!have_k) ok = have_k = wait(&sh.ready[ks], kpar);
                tmem_fence_after();
                if (ok && ra_elect()) {
                  scores(i, ks);
                  if (!(hook == 1 && first)) ra_commit<kPair>(&sh.sfull[i]);
                }
                first = false;
                __syncwarp();
              }
            }
            if (!ok) break;
            // every block is some tile's: the second's where there are more than 128 rows, else the first's
            if (ra_elect()) {
              if (j >= 0) ra_commit<kPair>(&sh.empty[vs]);
              if (j + 1 < nblk) ra_commit<kPair>(&sh.empty[ks]);
            }
            __syncwarp();
            if (j >= 0) next_v();
            if (j + 1 < nblk) next_k();
          }
        }
        if (!ok) break;
        g += nblk;
        release(it);
      }
      // every product has ended before the tensor memory goes
      if (!kPair || rank == 0) {
        if (ra_elect()) ra_commit<kPair>(&sh.drain);
        __syncwarp();
        mbar_wait_bounded(&sh.drain, 0);
      }
    }
  } else if (warp < 4 + C::kPrep) {
    // ------------------------------------------------------------ queries, values that need a look, 8-bit tiles
    if constexpr (C::kRegPrep < C::kLaunch)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegPrep));
    const int group = warp >> 3, tid = threadIdx.x - 128 - 128 * group, quad = warp & 3;  // group 1: values of codes
    // rings: with codes this group's, else the values'
    const int base = C::kFp8 && !group ? 0 : C::kKSt, stages = C::kFp8 && !group ? C::kKSt : C::kVSt, rbase = group * C::kRawSt;
    int st = base, g = 0, rst = rbase, done = 0;
    int nq0 = 0, nq1 = 0;  // query tiles so far
    uint32_t mpar = 0, fpar = 0, wpar = 1, rpar = 0;  // of the meetings, the full barriers (a bit each: their phases are the looks'), the stages, the codes
    bool ok = true;
    // This warp's 32 rows of the CTA's tile w; rows that are not there read as zeros, warps without rows load nothing.
    auto load_q = [&](const RaItem& i, int w, int before) -> bool {
      auto free = [&]() -> bool { return before == 0 || wait_item(&sh.qfree[w], (before - 1) & 1); };
      bool waited = false;
      const int row0 = kTiles == 1 && i.toks * a.G <= 32 ? 0 : (kPair ? rank : w) * 128 + quad * 32;  // of the item
      if (row0 * a.g_inv >> 16 < i.toks) {
        if constexpr (C::kQSmem) {  // into shared memory, a row's lanes together
          constexpr int kLanes = D / 8, kAt = 32 / kLanes, kAtOnce = kSub == 2 ? 8 : 16;
          const int piece = lane % kLanes;
          const uint32_t dst = q_s + w * 128 * D * 2 + (piece >> 3) * 16384;
          const uint16_t* src = a.q + (size_t)i.row * a.ld_q + (size_t)i.h * a.G * D + piece * 8;
#pragma unroll 1
          for (int k0 = 0; k0 < kLanes; k0 += kAtOnce) {
            uint4 v[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
              const int r = row0 + (k0 + k) * kAt + lane / kLanes, t = r * a.g_inv >> 16;
              v[k] = make_uint4(0, 0, 0, 0);
              if (t < i.toks) v[k] = ra_ldg128(src + t * a.ld_q + (r - t * a.G) * D);
            }
            if (!waited && !free()) return false;  // the first ones are on their way meanwhile
            waited = true;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
              const int row = quad * 32 + (k0 + k) * kAt + lane / kLanes;
              sts128(dst + row * 128 + (((piece & 7) ^ (row & 7)) << 4),
                     make_uint4((v[k].x & a.q_and) ^ a.q_flip, (v[k].y & a.q_and) ^ a.q_flip, (v[k].z & a.q_and) ^ a.q_flip,
                                (v[k].w & a.q_and) ^ a.q_flip));
            }
          }
          fence_proxy_async_smem();
        } else {  // into tensor memory, a row per lane
          const int r = row0 + lane, t = r * a.g_inv >> 16;
          const bool there = t < i.toks;
          const uint16_t* src = a.q + (size_t)(i.row + (there ? t : 0)) * a.ld_q + (size_t)(i.h * a.G + r - t * a.G) * D;
#pragma unroll 2
          for (int ch = 0; ch < kChunks; ++ch) {
            uint32_t x[32];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              uint4 u = make_uint4(0, 0, 0, 0);
              if (there) u = ra_ldg128(src + ch * 64 + k * 8);
              x[4 * k] = (u.x & a.q_and) ^ a.q_flip, x[4 * k + 1] = (u.y & a.q_and) ^ a.q_flip;
              x[4 * k + 2] = (u.z & a.q_and) ^ a.q_flip, x[4 * k + 3] = (u.w & a.q_and) ^ a.q_flip;
            }
            __syncwarp();
            if (!waited && !free()) return false;
            if (!waited) tmem_fence_after();
            waited = true;
            ra_st32(tmem + ((uint32_t)(quad * 32) << 16) + C::kColQ + ch * 32, x);
          }
          tmem_wait_st();
          tmem_fence_before();
        }
      }
      __syncwarp();
      if (!waited && !free()) return false;  // (every phase is waited for)
      if (lane == 0) arrive_first(&sh.qfull[w]);
      return true;
    };
    for (int it = 0; ok; ++it) {
      const RaItem* pi = get(it);
      if (!pi || pi->s < 0) break;
      const int b0 = pi->b0, b1 = pi->b1, edge = pi->edge, keys = pi->keys;
      int* const poison = sh.poison[it % C::kRing] + (kPair ? rank * C::kVCols : 0);
      int* const special = &sh.special[it % C::kRing];
      // the queries and gates on their way to L2, ahead of those who read them
      for (int u = tid; u < min(pi->toks * a.G - (kPair ? rank * 128 : 0), kSub * 128) * kChunks && group == 0; u += 128) {
        const int row = u / kChunks + (kPair ? rank * 128 : 0), t = row * a.g_inv >> 16, hd = pi->h * a.G + row - t * a.G;
        if (it > 0) ra_prefetch(a.q + (size_t)(pi->row + t) * a.ld_q + (size_t)hd * D + u % kChunks * 64);
        if (a.gate) ra_prefetch(a.gate + ((size_t)(pi->row + t) * a.Hq + hd) * D + u % kChunks * 64);
      }
      // the queries, once the last item's scores are done with theirs
      if (group == 0) {
        if (pi->cnt[0] > 0) ok = load_q(*pi, 0, nq0++);
        if (kSub == 2 && ok && pi->cnt[1] > 0) ok = load_q(*pi, 1, nq1++);
        if (!ok) break;
      }
      for (int b = b0; ok && b < b1; ++b, ++g) {
        if constexpr (C::kFp8) {  // every tile: this group's keys, or values
          const uint32_t tile = ring + st * C::kTile, src = raw + rst * C::kRaw;
          if (!(ok = wait(&sh.rfull[rst], rpar) && wait(&sh.empty[st], wpar))) break;
          if (C::kKRows == BN || group) {
            if (ra_expand<C::kVCols, BN>(src, tile, tid, keys - b * BN)) ra_expand_rare<C::kVCols, BN>(src, tile, tid);
          } else {
            if (ra_expand<D, C::kKRows>(src, tile, tid, keys - b * BN - rank * C::kKRows)) ra_expand_rare<D, C::kKRows>(src, tile, tid);
          }
          const uint32_t bad = *(volatile uint32_t*)&sh.bad[g & 15];
          if (group && (b >= edge || bad)) {
            if (!(ok = meet(1, mpar))) break;  // other threads' values are looked at
            ra_look<C::kVCols, BN>(tile, tid, keys - b * BN, bad, b >= edge, b * BN, poison, special);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (!(hook == 4 && done == 0 && warp == 4)) arrive_first(&sh.ready[st]);
            arrive(&sh.rempty[rst]);
          }
          ++done;
          if (++rst == rbase + C::kRawSt) rst = rbase, rpar ^= 1;
          if (++st == base + stages) st = base, wpar ^= 1;
        } else {  // values of edge blocks
          if (b >= edge) {
            if (!(ok = wait_item(&sh.full[st], fpar >> st & 1))) break;
            fpar ^= 1u << st;
            ra_look<C::kVCols, BN>(ring + st * C::kTile, tid, keys - b * BN, 0, true, b * BN, poison, special);  // (no pages: zeros)
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && !(hook == 4 && done == 0 && warp == 4)) arrive_first(&sh.ready[st]);
            ++done;
          }
          if (++st == base + stages) st = base;
        }
      }
      if (ok) release(it);
    }
    if (C::kFp8)  // no commit is on its way when the CTA ends: a stage's last one frees it
      for (int i = 0; i < min(done, stages); ++i) {
        const int e = done - 1 - (done - 1 - i) % stages;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&sh.empty[base + i], (e / stages) & 1))) break;
      }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegSoft));
    // ------------------------------------------------------------ softmax: rows of the CTA's tile w, a thread per row
    const int w = (warp - 4 - C::kPrep) >> 2, quad = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const uint64_t scale_2 = ra_pair(a.scale2, a.scale2);
    int g = 0, npv = 0;  // blocks (one tile: of the score buffers) and outputs so far
    uint32_t mpar = 0;   // of the meetings
    bool ok = true;
    // The outputs of block n (one tile), or of this tile's block v, are there.
    auto outputs_of = [&](int n, int v) -> bool {
      return kSub == 1 ? wait(&sh.ofull[n & 1], n >> 1 & 1) : wait(&sh.ofull[w], v & 1);
    };
    for (int it = 0; ok; ++it) {
      const RaItem* pi = get(it);
      if (!pi || pi->s < 0) break;
      const int b0 = pi->b0, cnt = pi->cnt[w], nblk = pi->b1 - b0, toks = pi->toks;
      const bool few = kTiles == 1 && toks * a.G <= 32;  // every warp has the rows, for a quarter of the keys
      const int row0 = few ? 0 : (kPair ? rank : w) * 128 + quad * 32, r = row0 + lane;  // of the item
      const int tok = r * a.g_inv >> 16, first_tok = row0 * a.g_inv >> 16;
      const int lim = tok < toks ? min(pi->lim0 + tok, pi->keys) : pi->keys;  // keys that this row sees
      const int lim_min = __reduce_min_sync(0xFFFFFFFFu, lim);
      const bool idle = first_tok >= toks;  // no row of the warp is there
      float m = -INFINITY, mc = 0.0f;       // reference of the exponents (log2 units), and what is subtracted
      uint64_t l2[2] = {0, 0};              // sums of the weights
      // (a second tile may have had no rows in the items before)
      if (kSub == 2 && cnt > 0 && !(ok = wait_item(&sh.sfull[w], npv & 1))) break;
      for (int j = 0; ok && j < cnt; ++j) {
        const int n = g + j, buf = kSub == 2 ? w : n & 1;
        // Every phase of the outputs' barriers is waited for in turn: a wait tells a phase from the one before it only.  The
        // last outputs on the barriers end before these scores do: no time passes for them.
        if (j >= 3 - kSub && !(ok = outputs_of(n - 2, npv - 1))) break;
        if (kSub == 1 && C::kParts > 1 && n >= 2 && !(ok = wait(&sh.opart[buf], (n >> 1) - 1 & 1))) break;
        if (!(ok = wait(&sh.sfull[buf], kSub == 2 ? npv & 1 : n >> 1 & 1))) break;
        if (j == cnt - 1) {  // the queries have been read
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) arrive(&sh.qfree[w]);
          __syncwarp();
        }
        if (idle) {  // whatever the products make of the scores is not read
          tmem_fence_before();
          __syncwarp();
          if (lane < C::kParts) arrive_first_relaxed(&sh.pfull[buf][lane]);
        } else if (kTiles == 1 && few) {
          constexpr int kQ = BN / 4;
          tmem_fence_after();
          const uint32_t ts = lanes + buf * C::kColS;
          const uint32_t groups = kSrc == kDense ? 0 : *(volatile uint32_t*)&sh.bad[n & 15] >> (quad * (kQ / 16));
          const int sees = lim - (b0 + j) * BN - quad * kQ;
          uint32_t x[kQ];
#pragma unroll
          for (int k = 0; k < kQ; k += 16) ra_ld16(ts + quad * kQ + k, x + k);
          if (sees < kQ || groups) {
#pragma unroll
            for (int k = 0; k < kQ; ++k)
              if (k >= sees || (groups >> (k >> 4) & 1)) x[k] = 0xFF800000u;
          }
          __syncwarp();
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < kQ; k += 2) mx[k / 2 % 2] = ra_max3(mx[k / 2 % 2], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
          const float top = fmaxf(mx[0], mx[1]) * a.scale2;
          const bool grow = top > m + 8.0f || (m == -INFINITY && top > m);
          if (__any_sync(0xFFFFFFFFu, grow)) {  // as below
            const float to = grow ? top : m, f = grow ? ra_ex2(m - to) : 1.0f;
            m = to;
            mc = ra_less(m);
            __syncwarp();
            if (j > 0) {
              const uint64_t ff = ra_pair(f, f), zero = 0;
              l2[0] = ra_fma2(l2[0], ff, zero), l2[1] = ra_fma2(l2[1], ff, zero);
              if (!(ok = outputs_of(n - 1, 0))) break;
              tmem_fence_after();
#pragma unroll 1
              for (int d = 0; d < D; d += 16) {
                uint32_t y[16];
                ra_ld16(lanes + C::kColO + d, y);
#pragma unroll
                for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
                ra_st16(lanes + C::kColO + d, y);
              }
            }
          }
          const uint64_t mc2 = ra_pair(-mc, -mc);
          uint32_t p[16], none[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) p[e] = none[e] = 0;
#pragma unroll
          for (int e = 0; e < kQ / 2; ++e) {
            float lo, hi;
            ra_unpair(ra_fma2(ra_pair(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), scale_2, mc2), lo, hi);
            lo = ra_ex2(lo), hi = ra_ex2(hi);
            l2[e & 1] = ra_add2(l2[e & 1], ra_pair(lo, hi));
            p[e] = ra_bf16x2(lo, hi);
          }
          if (kQ == 16 && (quad & 1)) {  // the second half of 16 columns
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e + 8] = p[e], p[e] = 0;
          }
#pragma unroll
          for (int k = 0; k < BN / 32; ++k) {  // weights of zero for the other warps' keys
            if (k == quad * kQ / 32)
              ra_st16(ts + k * 16, p);
            else
              ra_st16(ts + k * 16, none);
          }
          tmem_wait_st();
          tmem_fence_before();
          __syncwarp();
          if (lane < C::kParts && !(hook == 2 && it == 0 && j == 0 && warp == 4 + C::kPrep)) arrive_first_relaxed(&sh.pfull[buf][lane]);
        } else {
          tmem_fence_after();
          const uint32_t ts = lanes + buf * C::kColS;
          const uint32_t bad = kSrc == kDense ? 0 : *(volatile uint32_t*)&sh.bad[n & 15];
          uint32_t x[64];
          ra_ld32(ts, x);
          ra_ld32(ts + 32, x + 32);
          // 64 keys at a time, whose weights the products can start with
#pragma unroll 1
          for (int part = 0; part < C::kParts; ++part) {
            const int key0 = (b0 + j) * BN + part * 64;
            ra_wait32(x);
            ra_wait32(x + 32);
            const uint32_t groups = bad >> (part * 4);
            if (lim_min - key0 < 64 || (groups & 15)) {  // keys that a row does not see
              const int sees = lim - key0;
#pragma unroll
              for (int k = 0; k < 64; ++k)
                if (k >= sees || (groups >> (k >> 4) & 1)) x[k] = 0xFF800000u;
            }
            float mx[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx[e] = ra_max3(__uint_as_float(x[3 * e]), __uint_as_float(x[3 * e + 1]), __uint_as_float(x[3 * e + 2]));
#pragma unroll
            for (int k = 12; k < 64; k += 2)
              mx[k / 2 % 4] = ra_max3(mx[k / 2 % 4], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
            const float top = fmaxf(ra_max3(mx[0], mx[1], mx[2]), mx[3]) * a.scale2;
            // The reference follows the maximum only where that has grown by 2^8: a weight may reach 2^8, which costs bf16
            // nothing, and the outputs are seldom scaled again.
            const bool grow = top > m + 8.0f || (m == -INFINITY && top > m);
            if (__any_sync(0xFFFFFFFFu, grow)) {
              const float to = grow ? top : m, f = grow ? ra_ex2(m - to) : 1.0f;
              m = to;
              mc = ra_less(m);
              __syncwarp();
              if (j + part > 0) {
                const uint64_t ff = ra_pair(f, f), zero = 0;
                l2[0] = ra_fma2(l2[0], ff, zero), l2[1] = ra_fma2(l2[1], ff, zero);
                // the last block's outputs, and those of this block's first weights
                if (kSub == 1 && j > 0 && !(ok = outputs_of(n - 1, 0))) break;
                if (part > 0 && !(ok = wait(&sh.opart[buf], kSub == 2 ? npv & 1 : n >> 1 & 1))) break;
                tmem_fence_after();
                const uint32_t to_ = lanes + C::kColO + w * D;
#pragma unroll 1
                for (int d = 0; d < D; d += 16) {
                  uint32_t y[16];
                  ra_ld16(to_ + d, y);
#pragma unroll
                  for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
                  ra_st16(to_ + d, y);
                }
              }
            }
            const uint64_t mc2 = ra_pair(-mc, -mc);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t p[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float lo, hi;
                ra_unpair(ra_fma2(ra_pair(__uint_as_float(x[32 * h + 2 * e]), __uint_as_float(x[32 * h + 2 * e + 1])), scale_2, mc2),
                          lo, hi);
                lo = ra_ex2(lo), hi = ra_ex2(hi);
                l2[e & 1] = ra_add2(l2[e & 1], ra_pair(lo, hi));
                p[e] = ra_bf16x2(lo, hi);
              }
              ra_st16(ts + part * 32 + h * 16, p);  // over the scores, behind what is still read
            }
            if (part + 1 < C::kParts) {
              ra_ld32(ts + (part + 1) * 64, x);
              ra_ld32(ts + (part + 1) * 64 + 32, x + 32);
            }
            tmem_wait_st();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0 && !(hook == 2 && it == 0 && j == 0 && warp == 4 + C::kPrep)) arrive_first_relaxed(&sh.pfull[buf][part]);
            __syncwarp();
          }
          if (!ok) break;
        }
        if (kSub == 2 && !(ok = wait(&sh.opart[w], npv & 1))) break;
        ++npv;
      }
      if (!ok) break;
      g += nblk;
      // ---- the item's outputs
      const int slot = pi->slot, rows = min(32, toks * a.G - row0);  // the warp's rows
      float l;
      {
        float s0, s1, s2, s3;
        ra_unpair(l2[0], s0, s1);
        ra_unpair(l2[1], s2, s3);
        l = (s0 + s1) + (s2 + s3);
      }
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const uint32_t to_ = lanes + C::kColO + w * D;
      const bool there = lane < rows;
      const size_t at = (((size_t)pi->row + (there ? tok : 0)) * a.Hq + pi->h * a.G + r - tok * a.G) * D;  // the row's outputs
      // 32 columns at a time; gates are loaded two steps ahead: behind the ring's copies a load takes long.
      uint4 gt[2][4];
      // (rows of a sequence without keys are zeros, whatever their gates hold)
      const bool gate = a.gate && pi->keys > 0, gated = gate && slot < 0 && there;
      auto gates = [&](uint4 (&to)[4], int d) {
#pragma unroll
        for (int k = 0; k < 4; ++k) to[k] = ra_ldg128(a.gate + at + d + 8 * k);
      };
      if (gated && !few) {
        gates(gt[0], 0);
        gates(gt[1], 32);
      }
      if (cnt > 0) {
        if (kSub == 1 && cnt > 1 && !(ok = outputs_of(g - 2, 0))) break;
        if (!(ok = outputs_of(g - 1, npv - 1))) break;
        tmem_fence_after();
      }
      if (pi->b1 > pi->edge) {  // values that were none, of edge blocks (a pair's CTAs note their own columns)
        bool special = *(volatile int*)&sh.special[it % C::kRing];
        if (kPair) special = special || ra_ld_pair(&sh.special[it % C::kRing], rank ^ 1);
#pragma unroll 1
        for (int d = 0; d < D && special && cnt > 0; ++d) {
          const int* p = &sh.poison[it % C::kRing][d];
          const int from = kPair && d / C::kVCols != rank ? ra_ld_pair(p, rank ^ 1) : *(const volatile int*)p;
          if (!__any_sync(0xFFFFFFFFu, lim > from)) continue;
          uint32_t y;
          asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\ntcgen05.wait::ld.sync.aligned;" : "=r"(y) : "r"(to_ + d) : "memory");
          if (lim > from) y = 0x7FFFFFFFu;
          __syncwarp();
          asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};\ntcgen05.wait::st.sync.aligned;" ::"r"(to_ + d), "r"(y) : "memory");
        }
      }
      const size_t ps = (size_t)c * 2 + max(slot, 0);
      if (kTiles == 1 && few) {  // the quarters' sums: eight rows a warp
        const uint32_t mine = smem_addr(join_p) + quad * 4096;
        const int row = quad * 8 + (lane >> 2), col = (lane & 3) * 8, t = row * a.g_inv >> 16;
        const bool real = row < rows;
        const size_t to = (((size_t)pi->row + (real ? t : 0)) * a.Hq + pi->h * a.G + (real ? row - t * a.G : 0)) * D + col;
        uint4 gt[2];
        if (gate && slot < 0 && real) gt[0] = ra_ldg128(a.gate + to), gt[1] = ra_ldg128(a.gate + to + 32);
        float(*const quarter)[32][2] = reinterpret_cast<float(*)[32][2]>(sh.quarter);
        quarter[quad][lane][0] = m, quarter[quad][lane][1] = l;
        if (!(ok = meet(0, mpar))) break;
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int x = 0; x < 4; ++x) top = fmaxf(top, quarter[x][lane][0]);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float mx = quarter[x][lane][0];
          sum += (mx == -INFINITY ? 0.0f : ra_ex2(mx - top)) * quarter[x][lane][1];
        }
        const float f = (m == -INFINITY ? 0.0f : ra_ex2(m - top)) * (slot >= 0 ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum);
        m = top, l = sum;
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t y[32];
          __syncwarp();  // the lanes with rows to write come back: the load is the whole warp's
          if (cnt > 0) {
            ra_ld32(to_ + d, y);
            ra_wait32(y);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = 0;
          }
          if (!(ok = meet(0, mpar))) break;  // the last columns have been read
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(y[4 * k + e]) * f;
            sts128(mine + lane * 128 + ((k ^ (lane & 7)) << 4),
                   make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
          }
          if (!(ok = meet(0, mpar))) break;
          float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint4 u = lds128(smem_addr(join_p) + x * 4096 + row * 128 + ((((lane & 3) * 2 + k) ^ (row & 7)) << 4));
              v[4 * k] += __uint_as_float(u.x), v[4 * k + 1] += __uint_as_float(u.y);
              v[4 * k + 2] += __uint_as_float(u.z), v[4 * k + 3] += __uint_as_float(u.w);
            }
          }
          if (real && slot >= 0) {
            float* o = a.part_o + (ps * (D / 4) + (d + col) / 4) * (C::kRows * 4) + row * 4;
            __stcg(reinterpret_cast<float4*>(o), make_float4(v[0], v[1], v[2], v[3]));
            __stcg(reinterpret_cast<float4*>(o + C::kRows * 4), make_float4(v[4], v[5], v[6], v[7]));
          } else if (real) {
            if (gate) {
              ra_gate2(v[0], v[1], gt[0].x);
              ra_gate2(v[2], v[3], gt[0].y);
              ra_gate2(v[4], v[5], gt[0].z);
              ra_gate2(v[6], v[7], gt[0].w);
              gt[0] = gt[1];
              if (d + 64 < D) gt[1] = ra_ldg128(a.gate + to + d + 64);
            }
            *reinterpret_cast<uint4*>(a.out + to + d) =
                make_uint4(ra_bf16x2(v[0], v[1]), ra_bf16x2(v[2], v[3]), ra_bf16x2(v[4], v[5]), ra_bf16x2(v[6], v[7]));
          }
        }
        if (!ok || !(ok = meet(0, mpar))) break;  // before the next item's
      }
#pragma unroll 1
      for (int d = 0; d < D && !idle && !few; d += 32) {
        uint32_t y[32];
        __syncwarp();  // as above
        if (cnt > 0) {
          ra_ld32(to_ + d, y);
          ra_wait32(y);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) y[k] = 0;
        }
        if (slot >= 0) {
          float* o = a.part_o + (ps * (D / 4) + d / 4) * (C::kRows * 4) + r * 4;
          if (there) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              __stcg(reinterpret_cast<uint4*>(o + k * (C::kRows * 4)), make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]));
          }
        } else if (there) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(y[8 * k + e]) * inv;
            if (gated) {
              ra_gate2(v[0], v[1], gt[0][k].x);
              ra_gate2(v[2], v[3], gt[0][k].y);
              ra_gate2(v[4], v[5], gt[0][k].z);
              ra_gate2(v[6], v[7], gt[0][k].w);
            }
            *reinterpret_cast<uint4*>(a.out + at + d + 8 * k) =
                make_uint4(ra_bf16x2(v[0], v[1]), ra_bf16x2(v[2], v[3]), ra_bf16x2(v[4], v[5]), ra_bf16x2(v[6], v[7]));
          }
          if (gated) {
#pragma unroll
            for (int k = 0; k < 4; ++k) gt[0][k] = gt[1][k];
            if (d + 64 < D) gates(gt[1], d + 64);
          }
        }
      }
      if (there && (!few || quad == 0)) {
        if (slot >= 0)
          __stcg(reinterpret_cast<float2*>(a.part_ml + (ps * 256 + r) * 2), make_float2(m, l));
        else if (a.lse)
          a.lse[at / D] = ra_lse(m, l);
      }
      tmem_fence_before();
      if (kPair) {  // the other CTA reads this one's poison
        __syncwarp();
        if (lane == 0) ra_arrive_first(smem_addr(&sh.iempty[it % C::kRing]), rank ^ 1);
      }
      release(it);
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (kPair) ra_pair_sync();  // nothing of the other CTA's is on its way here
  tmem_fence_after();
  if (warp == 1) {
    if constexpr (kPair)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    else
      tmem_dealloc(tmem, 512);
  }
}

template <int D, int kTiles, int kSrc>
cudaError_t launch_one(const RowsArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, int grid, cudaStream_t s) {
  using C = RaCfg<D, kTiles, kSrc>;
  constexpr int kSmem = ra_smem<D, kTiles, kSrc>();
  static_assert(kSmem <= kSmemBytes, "shared memory");
  auto* kern = rows_kernel<D, kTiles, kSrc>;
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !done[dev].load()) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(C::kPair ? grid / 2 * 2 : grid));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = C::kPair ? 2 : 1;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, kmap, vmap);
}

}  // namespace

template <int D, int kTiles>
cudaError_t launch_rows(const RowsArgs& a, int source, const CUtensorMap& kmap, const CUtensorMap& vmap, int grid,
                        cudaStream_t s) {
  switch (source) {
    case kDense: return launch_one<D, kTiles, kDense>(a, kmap, vmap, grid, s);
    case kPaged: return launch_one<D, kTiles, kPaged>(a, kmap, vmap, grid, s);
    default: return launch_one<D, kTiles, kPagedFp8>(a, kmap, vmap, grid, s);
  }
}

}  // namespace vp
