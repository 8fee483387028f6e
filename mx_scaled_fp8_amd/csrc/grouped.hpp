// What the kernels of the grouped FP8 product share (not part of the ABI).
#pragma once

#include "common.hpp"

namespace mx {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void_t;

constexpr int kStageK = 128;   // K per stage: one 128-byte line of every operand row

// One row tile of an expert.
struct RowTile {
  int32_t expert;
  int32_t first;       // list index of the expert's first row tile
  int32_t count;       // row tiles of the expert
  int32_t row_lo;      // the expert's rows
  int32_t row_hi;
  int32_t pad[3];
};
static_assert(sizeof(RowTile) == 32, "workspace layout");

// 16-byte chunk c of row r of a stage lies at chunk c ^ swz8(r): the 32 rows of an operand read in distinct banks
__device__ __forceinline__ int swz8(int r) { return ((r >> 1) ^ ((r & 1) << 2)) & 7; }

struct GemmArgs {
  const uint8_t* xq;          // [KB, rows, 128] e4m3
  const uint32_t* xs;         // [rows, KB4] scale words, KB4 = KB rounded up to 4
  const uint8_t* w;           // [E, N, K] e4m3
  const void* ws;             // E8M0 [E, N, K/32], or FP32 [E, ceil(N/128), KB]
  uint16_t* out;              // [S, N] BF16
  const RowTile* tiles;       // null: one group of S rows
  const int32_t* row_slot;    // [S] or null: row r reads x row row_slot[r] / k
  DivU32 k_div;
  DivU32 nu_div;              // columns in units (grouped_stream.hip)
  int32_t rows, S, E, N, K, KB;
  int32_t n_tiles;
  int32_t wg_per_xcd;         // compute units of an XCD
};

// The 256 x 256 MXFP8 kernel (grouped_large.hip): K of at least kLargeMinStages stages.
constexpr int kLargeMinStages = 8;
void launch_grouped_large(const GemmArgs& a, hipStream_t stream);

// Row tiles of 32 rows (grouped_stream.hip).
void launch_grouped_stream(bool f32, const GemmArgs& a, hipStream_t stream);

}  // namespace mx
