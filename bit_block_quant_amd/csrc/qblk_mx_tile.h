// qblk_mx_tile.h -- the tile kernel of the microscaled products (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qblk {

struct MxTileArgs {
  const uint8_t* w;
  const uint8_t* ws;
  const uint8_t* xq;  // rows of x_pitch bytes: whole stages of 128 bytes, zeros past k
  const uint8_t* xs;
  void* y;
  float* part;  // split K: partial sums, [split][n][part_pitch(m)]
  int64_t x_pitch;
  int m, k, n, yt, row_tiles, tok_tiles, first_row_tile;
  int stages_per_split;  // a multiple of 4
};

// rows and tokens of each tile shape
struct MxTile {
  int rows, tokens;
};
constexpr MxTile kMxTiles[] = {{256, 256}, {256, 128}, {256, 64}, {128, 128}, {128, 64}, {64, 64}};

// splits > 1 write partial sums
// (sums of e4m3 activations exact to fp32 rounding: shapes 1 and 4)
hipError_t mx_tile_exact(int shape, const MxTileArgs& a, int splits, hipStream_t s);
hipError_t mx_tile(int shape, bool f8, const MxTileArgs& a, int splits, hipStream_t s);

}  // namespace qblk
