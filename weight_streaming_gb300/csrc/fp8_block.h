// Block-scaled FP8 (e4m3, one fp32 scale per 128 values): the packed weight layout shared by the
// packer (fp8_quant.cu) and the linear kernel (fp8_linear.cu).
#pragma once
#include <cstddef>
#include <cstdint>

namespace vp {

constexpr int kQBlock = 128;                        // values per scale along K; weight rows per scale
constexpr int kQTileBytes = kQBlock * kQBlock;      // one packed 128 x 128 weight tile
constexpr float kE4m3Max = 448.0f;

// Packed weights: tile (nb, kb) of weight rows 128 nb .. + 127 and columns 128 kb .. + 127 starts at
// (nb * KB + kb) * 16384 and is the shared-memory image of a K-major tensor-core operand with the
// 128-byte swizzle: row r at 128 r, its 16-byte chunk c at chunk c ^ (r & 7).  A tile is one
// contiguous bulk copy; rows past N and columns past K are zero.
__host__ __device__ inline int qblocks(int n) { return (n + kQBlock - 1) / kQBlock; }
__host__ __device__ inline uint32_t qtile_offset(int r, int c) {  // of 16-byte chunk c of row r
  return (uint32_t)(r * kQBlock + ((c ^ (r & 7)) << 4));
}
inline bool q_shape_ok(int N, int K) {
  return N >= 16 && N % 16 == 0 && N <= (1 << 20) && K >= 16 && K % 16 == 0 && K <= 65536 &&
         (long long)N * K < (1LL << 40);
}

}  // namespace vp
