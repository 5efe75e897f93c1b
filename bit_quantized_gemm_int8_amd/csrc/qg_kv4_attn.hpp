// What the two attention kernels of the 4-bit cache share: which sequence and
// rows a workgroup has, and which cached positions those rows can see.
//
// The rows of a sequence and kv head h are its n tokens times the G = Hq / H
// query heads of h, row = token * G + head.  A tile is up to ROWS of them.
#pragma once

#include "qg_kv4.hpp"

#include <algorithm>

// a lambda that is called more than once is still part of the kernel: its captures stay in registers
#define QG_INLINE __attribute__((always_inline))

namespace qg {

// Exact division of 0 <= n < 2^31 by a divisor that the host knows:
// n / d = (n * mag) >> (31 + sh), mag = ceil(2^(31 + sh) / d), sh = ceil(log2 d).
// A division proper costs some 40 instructions at the start of every workgroup.
struct Kv4Div {
  int d, sh;
  u32 mag;
  __device__ __forceinline__ int operator()(int n) const { return (int)(((uint64_t)(u32)n * mag) >> (31 + sh)); }
};
inline Kv4Div kv4_div(int64_t d) {
  Kv4Div v{(int)d, 0, 0};
  while (((int64_t)1 << v.sh) < d) ++v.sh;
  v.mag = (u32)((((uint64_t)1 << (31 + v.sh)) + (uint64_t)d - 1) / (uint64_t)d);
  return v;
}
// What the attention kernels divide by: kv heads, query heads of one, and without
// offsets a sequence's tokens and tiles.
struct Kv4Divs {
  Kv4Div H, G, tiles;
  int n;
};
inline Kv4Divs kv4_divs(const Kv4Seqs& s, int G, int rows) {
  const int64_t n = s.offsets == nullptr ? s.T / s.B : 0;
  return {kv4_div(s.H), kv4_div(G), kv4_div(std::max<int64_t>((n * G + rows - 1) / rows, 1)), (int)n};
}

struct Kv4Tile {
  int b;          // sequence, -1: no such tile
  int token0, n;  // its first row of the call, and its tokens
  int row0;       // the tile's first row
};

// Up to this many sequences with offsets are taken longest first.
constexpr int kKv4Sorted = 32;

// Tile `idx` among the sequences with min_rows <= n G <= max_rows, ROWS rows each.
// All lanes of a wave call it with the same arguments; the result is uniform.
// Workgroups differ in length and the longest should not start last: the last rows of a
// sequence, which see most, come first (600 tokens of two prompts of 1500, 8 heads of
// 256: 45 us, in the rows' order 48), and up to kKv4Sorted sequences with offsets in the
// order of their lengths (9 of 1148 to 4001 positions, 8 heads of 256: 139 us, in the
// order of the call 147).  More would cost a decode step's start more than it gives.
template <int ROWS>
__device__ __forceinline__ Kv4Tile kv4_tile(const Kv4Seqs& s, const Kv4Divs& by, int64_t min_rows,
                                            int64_t max_rows, int idx) {
  if (s.offsets == nullptr) {
    const int b = by.tiles(idx);
    return {b < s.B ? b : -1, b * by.n, by.n, (by.tiles.d - 1 - (idx - b * by.tiles.d)) * ROWS};
  }
  const int G = by.G.d;
  const int lane = threadIdx.x & 63;
  if (s.B <= kKv4Sorted) {
    int first = 0, n = 0, len = 0;
    if (lane < s.B) {
      first = min(max(s.offsets[lane], 0), s.T);
      n = min(max(s.offsets[lane + 1], first), s.T) - first;
      len = s.lengths[lane];
    }
    const int64_t rows = (int64_t)n * G;
    const int tiles = rows >= min_rows && rows <= max_rows ? (int)((rows + ROWS - 1) / ROWS) : 0;
    int before = 0;   // tiles of the sequences ahead of the lane's
    for (int j = 0; j < s.B; ++j) {
      const int l = __builtin_amdgcn_readlane(len, j), t = __builtin_amdgcn_readlane(tiles, j);
      before += l > len || (l == len && j < lane) ? t : 0;
    }
    const uint64_t here = __ballot(idx >= before && idx - before < tiles);
    if (here == 0) return {-1, 0, 0, 0};
    const int l = __ffsll((unsigned long long)here) - 1;
    const int tile = __builtin_amdgcn_readlane(before + tiles, l) - 1 - idx;
    return {l, __builtin_amdgcn_readlane(first, l), __builtin_amdgcn_readlane(n, l), tile * ROWS};
  }
  int64_t base = 0;
  for (int b0 = 0; b0 < s.B; b0 += 64) {
    int first = 0, n = 0;
    if (b0 + lane < s.B) {
      first = min(max(s.offsets[b0 + lane], 0), s.T);
      n = min(max(s.offsets[b0 + lane + 1], first), s.T) - first;
    }
    const int64_t rows = (int64_t)n * G;
    const int tiles = rows >= min_rows && rows <= max_rows ? (int)((rows + ROWS - 1) / ROWS) : 0;
    int64_t upto = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t below = __shfl_up(upto, o, kWave);
      if (lane >= o) upto += below;
    }
    const uint64_t behind = __ballot(base + upto > idx);
    if (behind != 0) {
      const int l = __ffsll((unsigned long long)behind) - 1;
      const int64_t before = base + __shfl(upto, l, kWave) - __shfl(tiles, l, kWave);
      return {__builtin_amdgcn_readfirstlane(b0 + l), __builtin_amdgcn_readfirstlane(__shfl(first, l, kWave)),
              __builtin_amdgcn_readfirstlane(__shfl(n, l, kWave)),
              __builtin_amdgcn_readfirstlane((int)(idx - before)) * ROWS};
    }
    base += __shfl(upto, 63, kWave);
  }
  return {-1, 0, 0, 0};
}

// The cached positions that rows at positions p0 .. p1 can see, in tiles of
// STEP: tiles 0 .. first - 1 hold first positions that stay visible, the next
// ones are tiles skip + first, ... of the cache.
struct Kv4Span {
  int tiles, first, skip;
  __device__ __forceinline__ int tile(int u) const { return u < first ? u : u + skip; }
};

template <int STEP>
__device__ __forceinline__ Kv4Span kv4_span(int p0, int p1, int window, int sinks, int capacity) {
  const int end = min(p1 + 1, capacity);
  if (end <= 0) return {0, 0, 0};
  const int all = (end + STEP - 1) / STEP;
  if (window <= 0) return {all, 0, 0};
  const int low = max(p0 - window + 1, 0) / STEP;   // first tile of the window
  if (low >= all) {                                 // the cache ends ahead of the window
    const int first = min((min(sinks, end) + STEP - 1) / STEP, all);
    return {first, first, 0};
  }
  const int first = min((sinks + STEP - 1) / STEP, low);
  return {first + all - low, first, low - first};
}

// Position of row `row` of a tile's sequence (kPast: the row does not exist).
constexpr int kKv4Past = -0x40000000;

// Rows of a workgroup of the prompt kernel.
constexpr int kKv4ManyRows = 256;

}  // namespace qg
