// Index arithmetic and kernel choice of the e4m3 products, in plain C++ so that
// they can be walked on the host (tests/test_f8_index.py, tests/f8_choice.py).
#pragma once

#include <cstdint>

namespace qg {

// A lane's load of the scales of stages g .. g + stages - 1 (g < G, in rows of G
// scales) for the row at byte `row` of the resource; an offset past any size
// for a lane without a row.  Of several stages the last ones may lie past the
// row: in the last row that is past the array, so their place goes into the
// vector offset, which every reading of the range check counts, dword by dword.
struct F8ScaleLoad {
  uint32_t voffset;
  int soffset;
};
constexpr F8ScaleLoad f8_scale_load(uint32_t row, int g, int stages) {
  return stages == 1 ? F8ScaleLoad{row, 4 * g} : F8ScaleLoad{row + 4 * (uint32_t)g, 0};
}

// Most tile rows that the experts' joint list holds: `grid` workgroups step
// through rows * tiles_n places in 31 bits, each up to grid / 8 + 1 past the end.
constexpr int f8_most_tile_rows(int tiles_n, int grid) { return (INT32_MAX - grid) / tiles_n; }

// Kernel by the rows of one weight matrix (of the mean expert) and the number
// of tiles, measured on MI355X (us):
//  * the stream kernel up to 16 rows (16 x 11008 x 4096: 15.8, tiles 21.9; one
//    expert's 17 rows read the weights twice, 17 x 4096 x 11008: 23.7, tiles 12.9,
//    17 x 4096 x 4096: 12.0, 12.1), with experts up to a mean of 8, since the
//    larger ones of a mean of 16 read theirs again (64 experts of 4096 x 2752,
//    mean 8: 113, tiles 155; 16 of 1376 x 4096, mean 16: 37.3, tiles 19.9, and
//    tiles ahead there from a mean of 2 on, 20.8 against 17.4);
//  * 64 x 64 tiles, two groups of waves sharing K, while one round of
//    workgroups holds them all (200 x 4096 x 4096: 11.8, one group 13.4), one
//    group beyond (128 x 4096 x 11008: 17.9, two groups 20.9);
//  * 128 x 128 tiles from 256 of them on (512 x 4096 x 11008: 35.8, 64 x 64 tiles
//    46.0);
//  * 256 x 256 tiles, 16-bit outputs of one matrix, where their rounds (one
//    workgroup on a CU) cost less than those of 128 x 128 (two on a CU, a round
//    5/8 as long): 4096 x 4096 x 11008 184 against 199-208, 1024 x 4096 x 11008 57
//    against 60, but 2048 x 4096 x 4096 56 against 38.
// Binary32 outputs take more registers than a 256 x 256 tile leaves, and
// experts' rows seldom fill one (64 experts of 384 rows of 1376 x 4096: 282
// against 258).  R counts rows of no expert too (choices of another GPU's): the
// row counts in use are on the GPU.
enum class F8Kernel { kStream, kTile64TwoGroups, kTile64, kTile128, kTile256 };
constexpr F8Kernel f8_kernel(bool experts, int64_t R, int64_t E, int64_t N, bool wide_out) {
  const int64_t rows = (R + E - 1) / E;   // of one weight matrix
  auto tiles = [&](int64_t s) { return (rows + s - 1) / s * ((N + s - 1) / s) * E; };
  auto rounds = [&](int64_t s, int64_t at_once) { return (tiles(s) + at_once - 1) / at_once; };
  if (rows <= (experts ? 8 : 16)) return F8Kernel::kStream;
  if (tiles(128) < 256) return tiles(64) > 256 ? F8Kernel::kTile64 : F8Kernel::kTile64TwoGroups;
  if (!wide_out && !experts && 8 * rounds(256, 256) < 5 * rounds(128, 512)) return F8Kernel::kTile256;
  return F8Kernel::kTile128;
}

}  // namespace qg
