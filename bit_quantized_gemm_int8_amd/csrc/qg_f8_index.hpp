// Index arithmetic of the e4m3 tile kernels, in plain C++ so that it can be
// walked on the host (tests/test_f8_index.py).
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

}  // namespace qg
