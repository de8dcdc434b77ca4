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
__device__ __forceinline__ void ra_arrive(uint32_t bar) {
  asm volatile("{ .reg .b64 st; mbarrier.arrive.shared::cta.b64 st, [%0]; }" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool ra_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}
// The rest of a bounded wait of a converged warp; false when it ran out here or elsewhere in the CTA.
__device__ __forceinline__ bool ra_wait_slow(uint32_t bar, uint32_t parity, int* abort, int* status) {
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
__device__ __forceinline__ void ra_bulk(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
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
// D(tensor memory) (+)= A B: A in shared memory, or in tensor memory.
__device__ __forceinline__ void ra_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void ra_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void ra_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
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

// v *= sigmoid(g) for eight bf16 gates.  Below zero by half the exponential twice: e^g itself leaves fp32's range long
// before the product does.
__device__ __forceinline__ void ra_gate2(float& v0, float& v1, uint32_t w) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float g[2] = {__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)};
  float* const v[2] = {&v0, &v1};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float h = ra_ex2(-0.5f * kLog2e * fabsf(g[e]));  // NaN stays NaN
    const float den = fmaf(h, h, 1.0f);
    *v[e] = __fdividef(g[e] < 0.0f ? *v[e] * h * h : *v[e], den);
  }
}
__device__ __forceinline__ void ra_gate(float (&v)[8], uint4 w) {
  ra_gate2(v[0], v[1], w.x);
  ra_gate2(v[2], v[3], w.y);
  ra_gate2(v[4], v[5], w.z);
  ra_gate2(v[6], v[7], w.w);
}
// log sum exp from the reference in log2 units and the sum of 2^(t - m).
__device__ __forceinline__ float ra_lse(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// One tile of codes (rows of D bytes, then a scale byte per row) to a bf16 operand tile, by 128 threads.  Eight lanes take 64
// codes of each of two rows, of neighbouring column groups where there are several: reads and writes then meet every bank
// once.  kLook: rows from `left` on and those of `bad` groups of 16 become zeros (weights of zero times what lies there), and
// where poison is given infinite and NaN values do, with their key noted there by column.
template <int D, int BN, bool kLook>
__device__ __forceinline__ void ra_expand(uint32_t src, uint32_t dst, int tid, int left, uint32_t bad, int key0, int* poison) {
  constexpr int kChunks = D / 64, kUnits = BN * D / 16 / 128, kAtOnce = 4;
  const int rsel = tid >> 2 & 1, i = tid & 3;
#pragma unroll 1
  for (int u0 = 0; u0 < kUnits; u0 += kAtOnce) {
    uint4 w[kAtOnce];
    uint32_t e[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int qd = (tid >> 3) + 16 * (u0 + k), row = 2 * (qd / kChunks) + rsel, ch = kChunks > 1 ? (qd % kChunks) ^ rsel : 0;
      w[k] = lds128(src + row * D + ch * 64 + i * 16);
      asm volatile("ld.shared.u8 %0, [%1];" : "=r"(e[k]) : "r"(src + BN * D + row));
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int qd = (tid >> 3) + 16 * (u0 + k), row = 2 * (qd / kChunks) + rsel, ch = kChunks > 1 ? (qd % kChunks) ^ rsel : 0;
      const uint32_t in[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
      // 2^(120 + scale - 127) at once where that is a bf16 value, else in two steps
      const uint32_t f = e[k] > 134 ? 0x7B807B80u : (e[k] + 120) * 0x00800080u;
      uint32_t o[8], nan = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        o[2 * x] = ra_bmul2(ra_code2<0x9180>(in[x]), f);
        o[2 * x + 1] = ra_bmul2(ra_code2<0xB3A2>(in[x]), f);
        nan |= (in[x] & 0x7F7F7F7Fu) + 0x01010101u;
      }
      if (e[k] > 134) {
        const uint32_t f2 = e[k] == 255 ? 0x7FC07FC0u : e[k] * 0x00800080u;
#pragma unroll
        for (int x = 0; x < 8; ++x) o[x] = ra_bmul2(o[x], f2);
      }
      if (nan & 0x80808080u) {  // codes 0x7F
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const uint32_t two = in[x >> 1] >> (x & 1 ? 16 : 0);
          if ((two & 0x7F) == 0x7F) o[x] |= 0x7FC0u;
          if ((two & 0x7F00) == 0x7F00) o[x] |= 0x7FC00000u;
        }
      }
      if (kLook) {
        if (row >= left || (bad >> (row >> 4) & 1)) {
#pragma unroll
          for (int x = 0; x < 8; ++x) o[x] = 0;
        }
        if (poison) {
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const uint32_t z = ra_special(o[x]);
            const int d = ch * 64 + i * 16 + 2 * x;
            if (z & 0x8000u) atomicMin(poison + d, key0 + row), o[x] &= 0xFFFF0000u;
            if (z & 0x80000000u) atomicMin(poison + d + 1, key0 + row), o[x] &= 0x0000FFFFu;
          }
        }
      }
      const uint32_t out = dst + ch * (BN * 128) + row * 128, sw = row & 7;
      sts128(out + (((2 * i) ^ sw) << 4), make_uint4(o[0], o[1], o[2], o[3]));
      sts128(out + (((2 * i + 1) ^ sw) << 4), make_uint4(o[4], o[5], o[6], o[7]));
    }
  }
}

// ------------------------------------------------------------------ work
// A sequence: n new rows from row0 on, which see the L cached positions up to their own.  A bad one (lengths that do not
// fit) has L = 0 and outputs of zero.
struct RaSeq {
  int row0, n, L;
  bool bad;
};
template <int kSrc>
__device__ __forceinline__ RaSeq ra_seq(const RowsArgs& a, int s) {
  RaSeq q;
  int r0 = s, r1 = s + 1;
  if (a.row_start) r0 = __ldg(a.row_start + s), r1 = __ldg(a.row_start + s + 1);
  q.bad = r0 < 0 || r1 > a.M || r1 < r0;
  r0 = max(r0, 0), r1 = min(r1, a.M);
  q.row0 = r0;
  q.n = max(r1 - r0, 0);
  q.L = q.n;
  if (kSrc != kDense) {
    q.L = __ldg(a.kv_len + s);
    q.bad = q.bad || q.L < q.n || q.L > (long long)a.max_pages << a.log_page;
  }
  if (q.bad) q.L = 0;
  return q;
}
// The work is one line: for every sequence, key-value head and item (tok_tile tokens) in turn, the item's keys and
// item_cost.  Its blocks lie at multiples of kBlock keys from the item's start; a CTA owns the blocks that begin
// in its part of the line.
constexpr int kMinKeys = 256;   // of the line per CTA at least

// The line up to item t of one head.
__device__ __forceinline__ long long ra_upto(const RowsArgs& a, const RaSeq& q, int t) {
  if (q.bad) return (long long)t * a.item_cost;
  return (long long)t * (q.L - q.n + a.item_cost) + (long long)a.tok_tile * ((long long)t * (t + 1) / 2);
}
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
  int keys;            // that the last one sees (0: a bad sequence)
  int b0, b1;
  int cnt[2];          // blocks of each tile of 128 rows in this piece
  int edge;            // first block that some token does not see whole
  int slot;            // -1: the whole item; 0, 1: the CTA's first, last part
};

template <int D, int kTiles, int kSrc>
struct RaCfg {
  static constexpr bool kFp8 = kSrc == kPagedFp8;
  static constexpr int kBlock = rows_block(D);
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kThreads = kTiles == 2 ? 512 : 384;
  static constexpr int kTile = kBlock * D * 2;                       // bytes of a block's keys, or values
  static constexpr int kRaw = kBlock * D + 128;                      // the same in codes, and the scales' bytes
  static constexpr int kQ = kTiles == 2 ? kRows * D * 2 : 0;         // one tile's queries lie in tensor memory
  static constexpr int kStages = kFp8 ? (D == 64 ? 6 : 4) : D == 64 ? (kTiles == 2 ? 8 : 10) : kTiles == 2 ? 5 : 6;
  static constexpr int kRawStages = !kFp8 ? 0 : kTiles == 2 ? (D == 64 ? 6 : 2) : D == 64 ? 8 : 5;
  static constexpr int kRing = 3;                                    // items
  // tensor memory: scores (two tiles, or two buffers of the one), outputs, queries
  static constexpr int kColS = kTiles == 2 ? 128 : kBlock;           // from one score buffer to the next
  static constexpr int kColO = 2 * kColS;
  static constexpr int kColQ = kColO + D;                            // one tile
  // registers: what issues or copies keeps few, the softmax warps take the rest of the launch's
  static constexpr int kRegLow = kTiles == 2 ? 64 : 120, kRegHigh = kTiles == 2 ? 192 : 232;
  static_assert(kTiles == 2 ? 8 * kRegLow + 8 * kRegHigh <= 16 * 128 : 8 * kRegLow + 4 * kRegHigh <= 12 * 168, "");
  static_assert(kColO + kTiles * D <= 512 && (kTiles == 2 || kColQ + D / 2 <= 512), "");
};
template <int D, int kTiles, int kSrc>
struct RaShared {
  using C = RaCfg<D, kTiles, kSrc>;
  uint64_t full[C::kStages], ready[C::kStages], empty[C::kStages];
  uint64_t rfull[8], rempty[8];
  uint64_t sfull[2], pfull[2], ofull[2], qfull[2];
  uint64_t ifull[C::kRing], iempty[C::kRing], drain;
  unsigned long long scan[16];
  unsigned long long x0, x1, base;
  RaItem item[C::kRing];
  int poison[C::kRing][D];  // per column: the first key of the item's edge blocks whose value is infinite or NaN
  uint32_t bad[16];         // per block: the groups of 16 keys whose page does not exist
  int s0;
  uint32_t tmem;
  int abort;
};
template <int D, int kTiles, int kSrc>
constexpr int ra_smem() {
  using C = RaCfg<D, kTiles, kSrc>;
  return C::kQ + C::kStages * C::kTile + C::kRawStages * C::kRaw + (int)sizeof(RaShared<D, kTiles, kSrc>);
}

template <int D, int kTiles, int kSrc>
__global__ void __launch_bounds__(RaCfg<D, kTiles, kSrc>::kThreads, 1)
    rows_kernel(const __grid_constant__ RowsArgs a, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
  using C = RaCfg<D, kTiles, kSrc>;
  constexpr int BN = C::kBlock;
  constexpr int kChunks = D / 64;                 // 128-byte column groups of a tile
  constexpr uint32_t kGroup = BN * 128;           // bytes from one to the next
  extern __shared__ __align__(1024) uint8_t dyn[];
  uint8_t* const q_p = dyn;
  uint8_t* const ring_p = q_p + C::kQ;
  uint8_t* const raw_p = ring_p + C::kStages * C::kTile;
  auto& sh = *reinterpret_cast<RaShared<D, kTiles, kSrc>*>(raw_p + C::kRawStages * C::kRaw);
  const uint32_t q_s = smem_addr(q_p), ring = smem_addr(ring_p), raw = smem_addr(raw_p);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x;
#ifdef VP_WAIT_TEST
  // Wait-test hook (workspace word kWsTestSkip): the first CTA leaves out 1 its first scores' commit, 2 a softmax warp's
  // first arrival, 3 its first copies, 4 the first arrival of the warps that prepare values, 5 its first item.
  const int hook = c == 0 ? ((const volatile int*)a.status)[kWsTestSkip / sizeof(int)] : 0;
#else
  constexpr int hook = 0;
#endif

  // -------------------------------------------------------------- the CTA's part of the line
  if (threadIdx.x == 0) {
    a.desc[2 * c] = a.desc[2 * c + 1] = make_int4(0, 0, -1, 0);
    sh.abort = 0;
  }
  {
    const int per = (a.S + C::kThreads - 1) / C::kThreads, s0 = min((int)threadIdx.x * per, a.S), s1 = min(s0 + per, a.S);
    unsigned long long mine = 0;
    for (int s = s0; s < s1; ++s) {
      const RaSeq q = ra_seq<kSrc>(a, s);
      if (q.bad && c == 0) report_unless(a.status, VP_ERR_SHAPE, VP_ERR_TIMEOUT);
      mine += (unsigned long long)ra_line(a, q) * a.Hkv;
    }
    unsigned long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) sh.scan[warp] = upto;
    __syncthreads();
    unsigned long long total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < C::kThreads / 32; ++w) {
      if (w == warp) before = total;
      total += sh.scan[w];
    }
    const unsigned long long most = total / kMinKeys;
    const int ctas = most < 1 ? 1 : most < gridDim.x ? (int)most : (int)gridDim.x;
    if (total == 0 || c >= ctas) return;
    const unsigned long long each = total / ctas, more = total % ctas;
    const unsigned long long x0 = each * c + more * c / ctas, x1 = each * (c + 1) + more * (c + 1) / ctas;
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
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.ready[i], 4);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(&sh.rfull[i], 1);
      mbar_init(&sh.rempty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.sfull[i], 1);
      mbar_init(&sh.pfull[i], 4);
      mbar_init(&sh.ofull[i], 1);
      mbar_init(&sh.qfull[i], 4);
    }
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(&sh.ifull[i], 1);
      mbar_init(&sh.iempty[i], 2 + 4 + 4 * kTiles);  // copying, issuing, value and softmax warps
    }
    mbar_init(&sh.drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&sh.tmem, 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *(volatile uint32_t*)&sh.tmem;

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    const uint32_t b = smem_addr(bar);
    if (__all_sync(0xFFFFFFFFu, ra_try(b, parity))) return true;
    return ra_wait_slow(b, parity, &sh.abort, a.status);
  };
  auto wait2 = [&](uint64_t* bar, uint32_t parity, uint64_t* bar2, uint32_t parity2) -> bool {
    const bool one = ra_try(smem_addr(bar), parity), two = ra_try(smem_addr(bar2), parity2);
    if (__all_sync(0xFFFFFFFFu, one && two)) return true;
    return wait(bar, parity) && wait(bar2, parity2);
  };
  // The it-th item, for every role but the scheduler; null when a wait ran out.
  auto get = [&](int it) -> const RaItem* {
    if (!wait(&sh.ifull[it % C::kRing], (it / C::kRing) & 1)) return nullptr;
    return &sh.item[it % C::kRing];
  };
  auto release = [&](int it) {
    __syncwarp();
    if (lane == 0) ra_arrive(smem_addr(&sh.iempty[it % C::kRing]));
  };

  if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegLow));
    if (warp == 3) {
      // ---------------------------------------------------------- scheduler: the pieces in turn
      const long long x0 = (long long)sh.x0, x1 = (long long)sh.x1;
      long long at = (long long)sh.base;       // the line at the current sequence's (head's, item's) start
      int s = sh.s0, h = 0, t = 0, cached = -1, it = 0;
      int c_row = 0, c_n = 0, c_L = 0, c_bad = 0;  // lane l: sequence cached + l
      bool ok = true, jump = true;
      while (ok && s < a.S && at < x1) {
        if ((s & ~31) != cached) {
          cached = s & ~31;
          c_n = 0;
          if (cached + lane < a.S) {
            const RaSeq q = ra_seq<kSrc>(a, cached + lane);
            c_row = q.row0, c_n = q.n, c_L = q.L, c_bad = q.bad;
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
        q.bad = __shfl_sync(0xFFFFFFFFu, c_bad, s & 31);
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
        const int keys = q.bad ? 0 : q.L - q.n + tok0 + toks, nb = (keys + BN - 1) / BN;
        // blocks whose place on the line lies in [x0, x1); a bad sequence's item by its start
        long long f = x0 - at, e = x1 - at;
        int b0 = f <= 0 ? 0 : (int)min((f + BN - 1) / BN, (long long)nb), b1 = (int)min((e + BN - 1) / BN, (long long)nb);
        const bool mine = nb ? b0 < b1 : f <= 0;
        if (mine) {
          const int slot = it % C::kRing;
          if (it >= C::kRing && !(ok = wait(&sh.iempty[slot], (it / C::kRing - 1) & 1))) break;
          for (int d = lane; d < D; d += 32) sh.poison[slot][d] = 0x7FFFFFFF;
          if (lane == 0) {
            RaItem& i = sh.item[slot];
            i.s = s, i.h = h;
            i.row = q.row0 + tok0;
            i.kv_row = q.row0;
            i.toks = toks;
            i.lim0 = q.bad ? 0 : q.L - q.n + tok0 + 1;
            i.keys = keys;
            i.b0 = b0, i.b1 = b1;
            // the first 128 rows see no further than their last token; the others are there only if there are more
            const int rows = toks * a.G, k0 = q.bad ? 0 : i.lim0 + min(toks - 1, 127 / a.G);
            i.cnt[0] = max(min(b1, (k0 + BN - 1) / BN) - b0, 0);
            i.cnt[1] = kTiles == 2 && rows > 128 ? b1 - b0 : 0;
            i.edge = i.lim0 / BN;
            const bool starts = b0 == 0, ends = b1 == nb;
            i.slot = starts && ends ? -1 : starts ? 1 : 0;
            if (i.slot >= 0) a.desc[2 * c + i.slot] = make_int4(s, h, q.row0 + tok0, rows | (ends ? kPartEnds : 0));
          }
          __syncwarp();
          if (lane == 0 && !(hook == 5 && it == 0)) ra_arrive(smem_addr(&sh.ifull[slot]));
          ++it;
        }
        at += keys + a.item_cost;
        if (++t == items) {
          t = 0;
          if (++h == a.Hkv) h = 0, ++s;
        }
      }
      const int slot = it % C::kRing;
      if (ok && (it < C::kRing || wait(&sh.iempty[slot], (it / C::kRing - 1) & 1))) {
        if (lane == 0) {
          sh.item[slot].s = -1;
          ra_arrive(smem_addr(&sh.ifull[slot]));
        }
      }
      __syncwarp();
    } else if (warp == 0) {
      // ---------------------------------------------------------- copies
      constexpr int kSt = C::kFp8 ? C::kRawStages : C::kStages;
      uint64_t *const full = C::kFp8 ? sh.rfull : sh.full, *const empty = C::kFp8 ? sh.rempty : sh.empty;
      const int P = 1 << a.log_page, box = min(P, BN), npg = BN / box;  // pages of a block, rows of each
      int cur = 0, nxt = 0, cur_s = -1, cur_w = -1, nxt_w = -1;         // lane l: page table entry cur_w + l
      int n = 0, st = 0, g = 0;
      uint32_t par = 1;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const RaItem* pi = get(it);
        if (!pi || pi->s < 0) break;
        const RaItem i = *pi;
        for (int b = i.b0; ok && b < i.b1; ++b, ++g) {
          const int key0 = b * BN;
          int pg = 0;          // of this lane's copy (paged)
          uint32_t bad = 0;    // pages of the block that do not exist, and those with keys to copy
          int have = npg;
          if (kSrc != kDense) {
            const int p0 = key0 >> a.log_page, last = (i.keys - 1) >> a.log_page, w = p0 & ~31;
            if (i.s != cur_s || w != cur_w) {
              const int32_t* tab = a.pages + (size_t)i.s * a.max_pages;
              cur = i.s == cur_s && w == nxt_w ? nxt : w + lane < a.max_pages ? __ldg(tab + w + lane) : 0;
              cur_s = i.s, cur_w = w, nxt_w = w + 32;
              nxt = nxt_w + lane < a.max_pages ? __ldg(tab + nxt_w + lane) : 0;
            }
            const int mine = C::kFp8 || box == BN ? lane : lane / kChunks;
            pg = __shfl_sync(0xFFFFFFFFu, cur, (p0 - w + mine) & 31);
            have = min(npg, last - p0 + 1);
            const int page = __shfl_sync(0xFFFFFFFFu, cur, (p0 - w + lane) & 31);
            const uint32_t wrong = __ballot_sync(0xFFFFFFFFu, lane < have && (page < 0 || page >= a.n_pages));
            const int per = box / 16;  // groups of 16 keys of a page
            if (wrong) {
              for (int k = 0; k < have; ++k)
                if (wrong >> k & 1) bad |= ((1u << per) - 1) << (k * per);
              if (lane == 0) report_unless(a.status, VP_ERR_SHAPE, VP_ERR_TIMEOUT);
            }
            if (lane == 0) sh.bad[g & 15] = bad;
            if (C::kFp8) have = __popc(((1u << have) - 1) & ~wrong);  // copies
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++n) {
            if (!(ok = wait(&empty[st], par))) break;
            const uint32_t bar = smem_addr(&full[st]);
            const bool skip = hook == 3 && n == 0;
            if constexpr (kSrc == kDense) {
              if (ra_elect()) {
                mbar_arrive_expect_tx(&full[st], C::kTile);
                if (!skip) ra_tma_3d(ring + st * C::kTile, kv ? &vmap : &kmap, 0, i.kv_row + key0, i.h * kChunks, bar);
              }
            } else if constexpr (kSrc == kPaged) {
              const uint32_t dst = ring + st * C::kTile;
              const int in_page = key0 & (P - 1), none = a.n_pages * a.Hkv << a.log_page;  // behind the cache: zeros
              const bool real = pg >= 0 && pg < a.n_pages;
              const int y = real ? ((pg * a.Hkv + i.h) << a.log_page) + in_page : none;
              if (lane == 0) mbar_arrive_expect_tx(&full[st], have * box * D * 2);
              __syncwarp();
              if (!skip) {
                if (box == BN) {
                  if (lane == 0) ra_tma_3d(dst, kv ? &vmap : &kmap, 0, y, 0, bar);
                } else if (lane < have * kChunks) {  // a page's column groups apart
                  ra_tma_3d(dst + (lane % kChunks) * kGroup + (lane / kChunks) * box * 128, kv ? &vmap : &kmap, 0, y,
                            lane % kChunks, bar);
                }
              }
            } else {
              const uint32_t dst = raw + st * C::kRaw;
              const int in_page = key0 & (P - 1);
              if (lane == 0) mbar_arrive_expect_tx(&full[st], have * box * (D + 1));
              __syncwarp();
              const int last = (i.keys - 1) >> a.log_page, p0 = key0 >> a.log_page;
              if (!skip && lane < npg && p0 + lane <= last && pg >= 0 && pg < a.n_pages) {
                const int y = ((pg * a.Hkv + i.h) << a.log_page) + in_page;
                ra_tma_2d(dst + lane * box * D, kv ? &vmap : &kmap, 0, y, bar);
                ra_bulk(dst + BN * D + lane * box, (kv ? a.v_scales : a.k_scales) + y, box, bar);
              }
            }
            __syncwarp();
            if (++st == kSt) st = 0, par ^= 1;
          }
        }
        if (ok) release(it);
      }
      // Nothing may be on its way to this CTA's shared memory when it ends: what was issued has landed, whatever ran out.
      for (int i = 0; i < min(n, kSt); ++i) {
        const int e = n - 1 - (n - 1 - i) % kSt;  // the last copy into stage i
        mbar_wait_bounded(&full[e % kSt], (e / kSt) & 1);
      }
      // ... and no commit: a stage's last one frees it
      if (!C::kFp8 && ok)
        for (int i = 0; i < min(n, kSt); ++i) {
          const int e = n - 1 - (n - 1 - i) % kSt;
          if (!wait(&empty[e % kSt], (e / kSt) & 1)) break;
        }
    } else if (warp == 1) {
      // ---------------------------------------------------------- matrix products
      constexpr uint32_t kIdesc = 1u << 4 | 1u << 7 | 1u << 10 | 8u << 24;  // bf16 x bf16 -> fp32, 128 rows
      constexpr uint32_t kIdS = kIdesc | (uint32_t)(BN >> 3) << 17, kIdO = kIdesc | 1u << 16 | (uint32_t)(D >> 3) << 17;
      int st = 0, g = 0;                       // stage; blocks so far (one tile: of the score buffers)
      uint32_t par = 0;
      uint32_t qpar[2] = {0, 0}, ppar[2] = {0, 0};
      bool ok = true, first = true;
      auto scores = [&](int i, int stage) {  // tile i, or buffer i of the one tile
        const uint64_t db = ra_desc_k(ring + stage * C::kTile);
        const uint32_t d = tmem + i * C::kColS;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t kb = db + (uint64_t)((k / 4) * (kGroup >> 4) + (k % 4) * 2);
          if constexpr (kTiles == 2)
            ra_mma_ss(d, ra_desc_k(q_s + i * 128 * D * 2) + (uint64_t)((k / 4) * (16384 >> 4) + (k % 4) * 2), kb, kIdS, k > 0);
          else
            ra_mma_ts(d, tmem + C::kColQ + 8 * k, kb, kIdS, k > 0);
        }
      };
      auto outputs = [&](int i, int o, int stage, bool accumulate) {  // P of score buffer i into output o
        const uint64_t db = ra_desc_mn(ring + stage * C::kTile, kGroup);
        const uint32_t p = tmem + i * C::kColS, d = tmem + C::kColO + o * D;
#pragma unroll
        for (int k = 0; k < BN / 16; ++k) ra_mma_ts(d, p + 8 * k, db + (uint64_t)(k * (2048 >> 4)), kIdO, accumulate || k > 0);
      };
      auto step = [&]() {
        if (++st == C::kStages) st = 0, par ^= 1;
      };
      for (int it = 0; ok; ++it) {
        const RaItem* pi = get(it);
        if (!pi || pi->s < 0) break;
        const int nblk = pi->b1 - pi->b0, cnt0 = pi->cnt[0], cnt1 = pi->cnt[1];
        for (int i = 0; i < kTiles && ok; ++i)
          if ((i ? cnt1 : cnt0) > 0) {
            ok = wait(&sh.qfull[i], qpar[i]);
            qpar[i] ^= 1;
          }
        // Scores of block j + 1 and outputs of block j (the ring's order: keys 0, values 0, keys 1, ...).  With two tiles
        // one's softmax runs beside the other's products, with one its next scores lie in a second buffer.
        for (int j = -1; ok && j < nblk; ++j) {
          const int vs = st;
          const uint32_t vpar = par;
          if (j >= 0) step();
          const int ks = st;
          bool have_v = false, have_k = false;
          if constexpr (kTiles == 1) {
            if (j + 1 < nblk) {
              if (!(ok = wait(&sh.ready[ks], par))) break;
              step();
              tmem_fence_after();
              if (ra_elect()) {
                scores((g + j + 1) & 1, ks);
                if (!(hook == 1 && first)) ra_commit(&sh.sfull[(g + j + 1) & 1]);
                ra_commit(&sh.empty[ks]);
              }
              first = false;
              __syncwarp();
            }
            if (j >= 0) {
              const int buf = (g + j) & 1;
              if (!(ok = wait(&sh.ready[vs], vpar))) break;
              if (!(ok = wait(&sh.pfull[buf], ppar[buf]))) break;
              ppar[buf] ^= 1;
              tmem_fence_after();
              if (ra_elect()) {
                outputs(buf, 0, vs, j > 0);
                ra_commit(&sh.ofull[buf]);
                ra_commit(&sh.empty[vs]);
              }
              __syncwarp();
            }
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int cnt = i ? cnt1 : cnt0;
              if (ok && j >= 0 && j < cnt) {
                if (!have_v) ok = have_v = wait(&sh.ready[vs], vpar);
                ok = ok && wait(&sh.pfull[i], ppar[i]);
                ppar[i] ^= 1;
                tmem_fence_after();
                if (ok && ra_elect()) {
                  outputs(i, i, vs, j > 0);
                  ra_commit(&sh.ofull[i]);
                }
                __syncwarp();
              }
              if (ok && j + 1 < cnt) {
                if (!have_k) ok = have_k = wait(&sh.ready[ks], par);
                tmem_fence_after();
                if (ok && ra_elect()) {
                  scores(i, ks);
                  if (!(hook == 1 && first)) ra_commit(&sh.sfull[i]);
                }
                first = false;
                __syncwarp();
              }
            }
            if (!ok) break;
            // every block is some tile's: the second's where there are more than 128 rows, else the first's
            if (ra_elect()) {
              if (j >= 0) ra_commit(&sh.empty[vs]);
              if (j + 1 < nblk) ra_commit(&sh.empty[ks]);
            }
            __syncwarp();
            if (j + 1 < nblk) step();
          }
        }
        if (!ok) break;
        g += nblk;
        release(it);
      }
      // every product has ended before the tensor memory goes
      if (ra_elect()) ra_commit(&sh.drain);
      __syncwarp();
      mbar_wait_bounded(&sh.drain, 0);
    } else if (warp >= 4) {
      // ---------------------------------------------------------- values that need a look, 8-bit tiles
      const int tid = threadIdx.x - 128;
      int st = 0, g = 0, rst = 0, done = 0;
      uint32_t par = 0, wpar = 1, rpar = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const RaItem* pi = get(it);
        if (!pi || pi->s < 0) break;
        const int b0 = pi->b0, b1 = pi->b1, edge = pi->edge, keys = pi->keys;
        int* const poison = sh.poison[it % C::kRing];
        // The item's queries and gates on their way to L2, ahead of the warps that read them.
        for (int u = tid; u < pi->toks * a.G * kChunks; u += 128) {
          const int row = u / kChunks, t = row * a.g_inv >> 16, hd = pi->h * a.G + row - t * a.G;
          if (it > 0) ra_prefetch(a.q + (size_t)(pi->row + t) * a.ld_q + (size_t)hd * D + u % kChunks * 64);
          if (a.gate) ra_prefetch(a.gate + ((size_t)(pi->row + t) * a.Hq + hd) * D + u % kChunks * 64);
        }
        for (int b = b0; ok && b < b1; ++b, ++g) {
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            const bool look = kv == 1 && b >= edge;
            const int left = keys - b * BN;  // rows of the tile that hold keys
            if constexpr (C::kFp8) {
              if (!(ok = wait(&sh.rfull[rst], rpar))) break;
              if (!(ok = wait(&sh.empty[st], wpar))) break;
              const uint32_t src = raw + rst * C::kRaw, dst = ring + st * C::kTile;
              const uint32_t bad = kv ? sh.bad[g & 15] : 0;
              if (look || bad)
                ra_expand<D, BN, true>(src, dst, tid, left, bad, b * BN, look ? poison : nullptr);
              else
                ra_expand<D, BN, false>(src, dst, tid, left, bad, 0, nullptr);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                if (!(hook == 4 && done == 0 && warp == 4)) ra_arrive(smem_addr(&sh.ready[st]));
                ra_arrive(smem_addr(&sh.rempty[rst]));
              }
              ++done;
              if (++rst == C::kRawStages) rst = 0, rpar ^= 1;
              if (++st == C::kStages) st = 0, wpar ^= 1;
            } else {
              if (!(ok = wait(&sh.full[st], par))) break;
              if (look) {
                // (pages that do not exist were filled with zeros)
                for (int u = tid; u < BN * D / 8; u += 128) {
                  const int ch = u / (BN * 8), row = (u >> 3) % BN, at = u & 7;
                  const uint32_t addr = ring + st * C::kTile + u * 16;
                  if (row >= left) {
                    sts128(addr, make_uint4(0, 0, 0, 0));
                    continue;
                  }
                  const uint4 w = lds128(addr);
                  uint32_t o[4] = {w.x, w.y, w.z, w.w};
                  if (ra_special(o[0]) | ra_special(o[1]) | ra_special(o[2]) | ra_special(o[3])) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                      const uint32_t z = ra_special(o[k]);
                      const int d = ch * 64 + ((at ^ (row & 7)) << 3) + 2 * k, key = b * BN + row;
                      if (z & 0x8000u) atomicMin(poison + d, key), o[k] &= 0xFFFF0000u;
                      if (z & 0x80000000u) atomicMin(poison + d + 1, key), o[k] &= 0x0000FFFFu;
                    }
                    sts128(addr, make_uint4(o[0], o[1], o[2], o[3]));
                  }
                }
                fence_proxy_async_smem();
              }
              __syncwarp();
              if (lane == 0 && !(hook == 4 && done == 0 && warp == 4)) ra_arrive(smem_addr(&sh.ready[st]));
              ++done;
              if (++st == C::kStages) st = 0, par ^= 1;
            }
          }
        }
        if (ok) release(it);
      }
      if (C::kFp8 && ok)  // the stages' last commits have arrived
        for (int i = 0; i < min(done, C::kStages); ++i) {
          const int e = done - 1 - (done - 1 - i) % C::kStages;
          if (!wait(&sh.empty[e % C::kStages], (e / C::kStages) & 1)) break;
        }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegHigh));
    // ------------------------------------------------------------ softmax: a thread per row of tile w
    const int w = (warp - 8) >> 2, quad = warp & 3, rr = quad * 32 + lane, r = w * 128 + rr;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const int tok = r / a.G, head = r - tok * a.G;
    const uint64_t scale_2 = ra_pair(a.scale2, a.scale2);
    int g = 0, npv = 0;  // blocks (one tile: of the score buffers) and outputs so far
    bool ok = true;

    const int first_tok = (w * 128 + quad * 32) / a.G;  // of the warp's rows; a warp without rows passes the scores through
    auto load_q = [&](const RaItem& i) {
      if (first_tok < i.toks) {
        if constexpr (kTiles == 2) {  // a row's lanes together
          constexpr int kLanes = D / 8, kAt = 32 / kLanes;
          uint4 v[kLanes];
#pragma unroll
          for (int k = 0; k < kLanes; ++k) {
            const int row = w * 128 + quad * 32 + k * kAt + lane / kLanes, t = row * a.g_inv >> 16, hd = row - t * a.G;
            v[k] = make_uint4(0, 0, 0, 0);
            if (t < i.toks)
              v[k] = ra_ldg128(a.q + (size_t)(i.row + t) * a.ld_q + (size_t)(i.h * a.G + hd) * D + lane % kLanes * 8);
          }
#pragma unroll
          for (int k = 0; k < kLanes; ++k) {
            const int row = quad * 32 + k * kAt + lane / kLanes, piece = lane % kLanes;
            v[k].x = (v[k].x & a.q_and) ^ a.q_flip, v[k].y = (v[k].y & a.q_and) ^ a.q_flip;
            v[k].z = (v[k].z & a.q_and) ^ a.q_flip, v[k].w = (v[k].w & a.q_and) ^ a.q_flip;
            sts128(q_s + w * 128 * D * 2 + (piece >> 3) * 16384 + row * 128 + (((piece & 7) ^ (row & 7)) << 4), v[k]);
          }
          fence_proxy_async_smem();
        } else {
          const bool there = tok < i.toks;
          const uint16_t* src = a.q + (size_t)(i.row + (there ? tok : 0)) * a.ld_q + (size_t)(i.h * a.G + head) * D;
          uint4 v[D / 8];
#pragma unroll
          for (int k = 0; k < D / 8; ++k) {
            v[k] = make_uint4(0, 0, 0, 0);
            if (there) v[k] = ra_ldg128(src + k * 8);
          }
          __syncwarp();
#pragma unroll
          for (int ch = 0; ch < kChunks; ++ch) {
            uint32_t x[32];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint4 u = v[ch * 8 + k];
              x[4 * k] = (u.x & a.q_and) ^ a.q_flip, x[4 * k + 1] = (u.y & a.q_and) ^ a.q_flip;
              x[4 * k + 2] = (u.z & a.q_and) ^ a.q_flip, x[4 * k + 3] = (u.w & a.q_and) ^ a.q_flip;
            }
            ra_st32(lanes + C::kColQ + ch * 32, x);
          }
          tmem_wait_st();
          tmem_fence_before();
        }
      }
      __syncwarp();
      if (lane == 0) ra_arrive(smem_addr(&sh.qfull[w]));
    };

    // The outputs of block n (one tile), or of this tile's block v, are there.
    auto outputs_of = [&](int n, int v) -> bool {
      return kTiles == 1 ? wait(&sh.ofull[n & 1], n >> 1 & 1) : wait(&sh.ofull[w], v & 1);
    };

    const RaItem* pi = get(0);
    if (pi && pi->s >= 0 && pi->cnt[w] > 0) load_q(*pi);
    for (int it = 0; pi && pi->s >= 0; ++it) {
      const int b0 = pi->b0, cnt = pi->cnt[w], nblk = pi->b1 - b0;
      const int lim = tok < pi->toks ? min(pi->lim0 + tok, pi->keys) : pi->keys;  // keys that this row sees
      const int lim_min = __reduce_min_sync(0xFFFFFFFFu, lim);
      const bool idle = first_tok >= pi->toks;
      float m = -INFINITY, mc = 0.0f;  // reference of the exponents (log2 units), and what is subtracted
      uint64_t l2[2] = {0, 0};         // sums of the weights
      for (int j = 0; j < cnt; ++j) {
        const int buf = kTiles == 2 ? w : (g + j) & 1;
        const uint32_t sp = kTiles == 2 ? (uint32_t)(npv & 1) : (uint32_t)((g + j) >> 1 & 1);
        // Every phase of the outputs' barriers is waited for in turn: a wait tells a phase from the one before it only.  The
        // last outputs on the barrier come before these scores: no time passes for them.
        if (j >= 3 - kTiles)
          ok = kTiles == 1 ? wait2(&sh.sfull[buf], sp, &sh.ofull[buf], (g + j - 2) >> 1 & 1) : wait2(&sh.sfull[buf], sp, &sh.ofull[w], (npv - 1) & 1);
        else
          ok = wait(&sh.sfull[buf], sp);
        if (!ok) break;
        if (idle) {  // no row of the warp is there: whatever the products make of the scores is not read
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) ra_arrive(smem_addr(&sh.pfull[buf]));
          ++npv;
          continue;
        }
        tmem_fence_after();
        const uint32_t ts = lanes + buf * C::kColS;
        uint32_t x[BN];
#pragma unroll
        for (int k = 0; k < BN; k += 32) ra_ld32(ts + k, x + k);
        const int key0 = (b0 + j) * BN;
        const uint32_t bad = kSrc == kDense ? 0 : *(volatile uint32_t*)&sh.bad[(g + j) & 15];
#pragma unroll
        for (int k = 0; k < BN; k += 32) ra_wait32(x + k);
        if (key0 + BN > lim_min || bad) {
          const int sees = lim - key0;
#pragma unroll
          for (int k = 0; k < BN; ++k)
            if (k >= sees || (bad >> (k >> 4) & 1)) x[k] = 0xFF800000u;
        }
        float mx[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = ra_max3(__uint_as_float(x[3 * e]), __uint_as_float(x[3 * e + 1]), __uint_as_float(x[3 * e + 2]));
#pragma unroll
        for (int k = 12; k + 1 < BN; k += 2) mx[k / 2 % 4] = ra_max3(mx[k / 2 % 4], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
        const float top = fmaxf(ra_max3(mx[0], mx[1], mx[2]), mx[3]) * a.scale2;
        // The reference follows the maximum only where that has grown by 2^8: a weight may reach 2^8, which costs bf16
        // nothing, and the outputs are seldom scaled again.
        const bool grow = top > m + 8.0f || (m == -INFINITY && top > m);
        if (j == 0) {
          if (grow) m = top;
        } else if (__any_sync(0xFFFFFFFFu, grow)) {
          const float to = grow ? top : m, f = grow ? ra_ex2(m - to) : 1.0f;
          m = to;
          const uint64_t ff = ra_pair(f, f), zero = 0;
          l2[0] = ra_fma2(l2[0], ff, zero), l2[1] = ra_fma2(l2[1], ff, zero);
          if (kTiles == 1 && !(ok = outputs_of(g + j - 1, 0))) break;
          tmem_fence_after();
          const uint32_t to_ = lanes + C::kColO + w * D;
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            uint32_t y[32];
            ra_ld32(to_ + d, y);
            ra_wait32(y);
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
            ra_st32(to_ + d, y);
          }
        }
        mc = m == -INFINITY ? 0.0f : m;
        const uint64_t mc2 = ra_pair(-mc, -mc);
#pragma unroll
        for (int k = 0; k < BN; k += 32) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float lo, hi;
            ra_unpair(ra_fma2(ra_pair(__uint_as_float(x[k + 2 * e]), __uint_as_float(x[k + 2 * e + 1])), scale_2, mc2), lo, hi);
            lo = ra_ex2(lo), hi = ra_ex2(hi);
            l2[e & 1] = ra_add2(l2[e & 1], ra_pair(lo, hi));
            p[e] = ra_bf16x2(lo, hi);
          }
          ra_st16(ts + k / 2, p);
        }
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0 && !(hook == 2 && it == 0 && j == 0 && warp == 8)) ra_arrive(smem_addr(&sh.pfull[buf]));
        ++npv;
      }
      if (!ok) break;
      g += nblk;
      // the next item's queries, while the last products run
      const RaItem* next = get(it + 1);
      if (!next) break;
      if (next->s >= 0 && next->cnt[w] > 0) load_q(*next);
      // ---- the item's outputs
      const bool there = tok < pi->toks;
      const int slot = pi->slot;
      const bool special = pi->b1 > pi->edge;  // the piece has edge blocks
      const int* const poison = sh.poison[it % C::kRing];
      const size_t orow = (size_t)(pi->row + (there ? tok : 0)) * a.Hq + pi->h * a.G + head;
      uint4 gt[4];  // the gates are loaded a step ahead
      if (a.gate && there && slot < 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) gt[k] = ra_ldg128(a.gate + orow * D + 8 * k);
      }
      if (cnt > 0) {
        if (kTiles == 1 && cnt > 1 && !(ok = outputs_of(g - 2, 0))) break;
        if (!(ok = outputs_of(g - 1, npv - 1))) break;
        tmem_fence_after();
      }
      float s0, s1, s2, s3;
      ra_unpair(l2[0], s0, s1);
      ra_unpair(l2[1], s2, s3);
      const float l = (s0 + s1) + (s2 + s3);
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const uint32_t to_ = lanes + C::kColO + w * D;
      const size_t ps = (size_t)c * 2 + max(slot, 0);
#pragma unroll 1
      for (int d = 0; d < D && !idle; d += 32) {
        uint32_t y[32];
        if (cnt > 0) {
          ra_ld32(to_ + d, y);
          ra_wait32(y);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) y[k] = 0;
        }
        if (special) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (lim > poison[d + k]) y[k] = 0x7FFFFFFFu;
        }
        if (!there) {
        } else if (slot >= 0) {
          float* o = a.part_o + (ps * (D / 4) + d / 4) * (C::kRows * 4) + r * 4;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            __stcg(reinterpret_cast<uint4*>(o + k * (C::kRows * 4)), make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]));
        } else {
          uint16_t* o = a.out + orow * D + d;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(y[8 * k + e]) * inv;
            if (a.gate) {
              ra_gate(v, gt[k]);
              if (d + 32 < D) gt[k] = ra_ldg128(a.gate + orow * D + d + 32 + 8 * k);
            }
            *reinterpret_cast<uint4*>(o + 8 * k) =
                make_uint4(ra_bf16x2(v[0], v[1]), ra_bf16x2(v[2], v[3]), ra_bf16x2(v[4], v[5]), ra_bf16x2(v[6], v[7]));
          }
        }
        __syncwarp();
      }
      if (there) {
        if (slot >= 0)
          __stcg(reinterpret_cast<float2*>(a.part_ml + (ps * 256 + r) * 2), make_float2(m, l));
        else if (a.lse)
          a.lse[orow] = ra_lse(m, l);
      }
      if (cnt > 0) tmem_fence_before();
      release(it);
      pi = next;
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D, int kTiles, int kSrc>
cudaError_t launch_one(const RowsArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, int grid, cudaStream_t s) {
  constexpr int kSmem = ra_smem<D, kTiles, kSrc>();
  static_assert(kSmem <= kSmemBytes, "shared memory");
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !done[dev].load()) {
    e = cudaFuncSetAttribute(rows_kernel<D, kTiles, kSrc>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev].store(true);
  }
  rows_kernel<D, kTiles, kSrc><<<grid, (RaCfg<D, kTiles, kSrc>::kThreads), kSmem, s>>>(a, kmap, vmap);
  return cudaGetLastError();
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
