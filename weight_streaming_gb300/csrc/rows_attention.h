// Attention of several new rows per sequence (vp_prompt_attention, vp_paged_attention_rows and its form over an 8-bit
// cache): what the host side (rows_attention.cu) and the kernel's instantiations (rows_attention_*.cu) share.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace vp {

enum RowsSource : int { kDense = 0, kPaged = 1, kPagedFp8 = 2 };

constexpr int kRowsGrid = 152;  // CTAs at most: one per SM

struct RowsArgs {
  const uint16_t *q, *gate;
  uint16_t* out;
  float* lse;
  long long ld_q;
  const int32_t *row_start, *kv_len, *pages;  // row_start NULL: one row per sequence; kv_len NULL: the rows themselves
  const uint8_t *k_scales, *v_scales;         // 8-bit cache: one exponent byte per slot and head
  int S, M, Hq, Hkv, G;
  int n_pages, log_page, max_pages;
  int tok_tile;                // tokens of an item: its rows / G
  int g_inv;                   // 65536 / G, rounded up: r * g_inv >> 16 is r / G for r < 256
  int item_cost;               // what starting and ending an item costs, in keys
  uint32_t polls;              // after which a wait for others' work on an item gives up
  uint32_t q_and, q_flip;      // on the queries' bf16 pairs: the scale's zero and sign
  float scale2;                // |scale| * log2(e), 1 for scale 0
  int4* desc;                  // [grid][2]: s, h, first token (-1: no part), rows | ends << 16 (below)
  float* part_ml;              // [grid][2][256][2]: maximum (log2 units), sum
  float* part_o;               // [grid or pairs][2][D / 4][rows][4]
  int* status;
};

// A part's descriptor word w: its rows, and whether the item ends with it.
constexpr int kPartEnds = 1 << 16;

template <int D, int kTiles>
cudaError_t launch_rows(const RowsArgs& a, int source, const CUtensorMap& kmap, const CUtensorMap& vmap, int grid,
                        cudaStream_t s);

extern template cudaError_t launch_rows<64, 1>(const RowsArgs&, int, const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
extern template cudaError_t launch_rows<64, 2>(const RowsArgs&, int, const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
extern template cudaError_t launch_rows<128, 1>(const RowsArgs&, int, const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
extern template cudaError_t launch_rows<128, 2>(const RowsArgs&, int, const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
extern template cudaError_t launch_rows<256, 2>(const RowsArgs&, int, const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
extern template cudaError_t launch_rows<256, 1>(const RowsArgs&, int, const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);

// Keys of a block, and this CTA's rows and columns of its key and value tiles (the tensor maps' boxes, too): with 256
// columns an item's two tiles lie in a pair of CTAs, which hold half of the keys and half of the values' columns each.
constexpr int rows_block(int D, int tiles) { return D == 256 && tiles == 1 ? 64 : 128; }
constexpr int rows_key_rows(int D, int tiles) { return D == 256 ? 64 : 128; }
constexpr int rows_value_cols(int D, int tiles) { return D == 256 && tiles == 2 ? 128 : D; }

}  // namespace vp
