// Attention of many query rows over the 4-bit paged KV cache (qg_kv4.hpp):
// prompts and chunks of them, heads of 64 and 128 channels.  The mathematics is
// that of attn_kv4.hip; here the codes of 64 positions become binary16 values once
// for all 256 rows of a workgroup.
//
// A value (q - z) s has 11 significant bits.  Scaled by a power of two that takes s
// to [2^-18, 2^-8) it is exact in binary16, and since a nibble masked out of a code
// word is the binary16 subnormal n 2^-24, one packed fma makes two values,
// n 2^-24 (s 2^24) - z s.  The power of two comes from the first tile's largest
// scale (that one goes to [2^-13, 2^-12)); a position whose scale does not fit takes
// its own, and the tile's weights are made in a general form that knows the factor.
//
// Both products have the query rows as columns, so that a lane has one query row
// throughout: scores^T = K Q^T, outputs^T = V^T P^T, with the scores' registers
// the second product's operand as they are (positions in the order of the lane).
// A tile that all rows see, with no odd scales, costs one fma, one exponential, one
// addition and half a conversion for each score; the weights' common factor changes
// only where a row's sum of a tile passes 2^14.
//
// Two halves of the workgroup, one wave of each on every SIMD, take turns: while one
// has the matrix cores (outputs of the last tile, scores of this one, and between
// the products part of the unpacking of a later tile) the other unpacks the rest and
// makes weights.
//
// 4096 tokens of 32 heads of 128 channels, 137 GFLOP: 148 to 157 us on different GPUs,
// 0.9 PFLOP/s (a large matrix product reaches 1.24).  A turn takes some 2400 cycles; its 32 products take
// 1150, issued 45 to 50 cycles apart beside the other wave's vector instructions.  None
// of the parts bounds it alone: of 153 us, without the exponentials 138 are left, with half
// the products 135.
#include "qg_decode.hpp"
#include "qg_kv4_attn.hpp"

#include <algorithm>
#include <type_traits>

namespace qg {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));

constexpr int kTile = 64;      // positions of a tile
constexpr int kManyWaves = kKv4ManyRows / 32;
constexpr int kVBufs = 3;      // tiles of values at hand (two of keys)
constexpr float kLow = -3.402823466e38f;
constexpr float kUnset = 1e30f;
// A sum outside of these in the exponent of the outputs keeps its own; within, an
// exponential is zero below 2^-86 of the largest.
constexpr float kApartLow = 0x1p-40f, kApartHigh = 0x1p60f;
constexpr u32 kHidden = 0xFFFFFFFFu;   // group word of a position that no row sees

__device__ __forceinline__ int float_exp(u32 bits) { return (int)((bits >> 23) & 255u) - 127; }

// A group's scale as the unpacked values have it, times 2^24: s 2^(15 - e), or with
// its own exponent in the place of e where that leaves [2^6, 2^16).  A group of zeros
// and one that is NaN have zero codes and zero points: any finite scale will do.
struct Kv4Fit {
  float v;
  bool odd;
};
__device__ __forceinline__ Kv4Fit kv4_fit(u32 word, float f /* 2^(15 - e) */) {
  const float a = __uint_as_float(word & 0xFFFF0000u) * f;
  const bool odd = __float_as_uint(a) - 0x42800000u >= 0x47800000u - 0x42800000u;   // 2^6 <= a < 2^16
  return {odd ? __uint_as_float((word & 0x007F0000u) | 0x47000000u) : a, odd};
}
// two values in binary16
__device__ __forceinline__ u32 pair_of(float a, float b) { return __builtin_bit_cast(u32, v2h{(_Float16)a, (_Float16)b}); }
__device__ __forceinline__ u32 mul2(u32 a, u32 b) {
  return __builtin_bit_cast(u32, __builtin_bit_cast(v2h, a) * __builtin_bit_cast(v2h, b));
}
constexpr u32 kSixteenth2 = 0x2C002C00u;   // 2^-4 twice

// f(0), f(1), ... with constants for arguments
template <int N, int I = 0, typename F>
__device__ __forceinline__ void for_each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>());
    for_each<N, I + 1>(f);
  }
}

}  // namespace

struct Kv4ManyArgs {
  Kv4Seqs s;
  Kv4Attend a;
  int G, tiles, splits;
  Kv4Divs by;
  Kv4Div by_splits;
  int64_t min_rows;   // sequences of fewer rows are another kernel's
  float *part_o, *part_ml;
};

template <int DT, int D>
__global__ __launch_bounds__(64 * kManyWaves, 2) void k_kv4_attend_many(Kv4ManyArgs p) {
  constexpr int NW = kManyWaves, NT = 64 * NW, kRows = kKv4ManyRows, kC = D / 8;   // code words of a position
  constexpr int kSt = D / 16;        // steps of the first product
  constexpr int kDt = D / 32;        // channel tiles of the second
  // values: [tile % bufs][position / 32][step][half][channel], keys: [tile % 2][position / 32]
  // [word][position % 32], 16 bytes each; group words and flags of tiles
  extern __shared__ __align__(16) char lds[];
  v4i* const vbuf = (v4i*)lds;
  v4i* const kbuf = vbuf + kVBufs * kTile * kC;
  u32(*const kraw)[kTile] = (u32(*)[kTile])(kbuf + 2 * kTile * kC);   // [4]
  u32(*const vraw)[kTile] = kraw + 4;
  int* const flags = (int*)(vraw + 4);                                // [8], then the largest scales
  float(*const own)[kTile] = (float(*)[kTile])(flags + 16) + 2 * (threadIdx.x >> 6);   // [2] of each wave

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = p.s.H;
  const int from = p.by_splits((int)blockIdx.x), split = blockIdx.x - from * p.splits;
  const int tile_n = p.by.H(from), h = from - tile_n * H;
  const Kv4Tile t = kv4_tile<kRows>(p.s, p.by, p.min_rows, (int64_t)1 << 40, tile_n);
  const int64_t part = (int64_t)blockIdx.x * kRows;
  if (t.b < 0) return;
  const int rows = min(t.n * p.G - t.row0, kRows);
  const int first = max(p.s.lengths[t.b], -0x3FFFFFFF) - t.n;   // n <= 2^30: no overflow
  const int p0 = first + p.by.G(t.row0), p1 = first + p.by.G(t.row0 + rows - 1);
  const int shift = p.s.shift, S = 1 << shift, W = p.s.W, window = p.a.window, sinks = p.a.sinks;
  const int capacity = (int)min((int64_t)W << shift, (int64_t)0x40000000);
  const Kv4Span span = kv4_span<kTile>(p0, p1, window, sinks, capacity);
  const int per = (span.tiles + p.splits - 1) / p.splits, first_tile = split * per;
  const int n_tiles = min(per, span.tiles - first_tile);   // of this split
  if (n_tiles <= 0 && p.splits > 1) {   // the join leaves it out
    if (tid < kRows) *(v2f*)(p.part_ml + (part + tid) * 2) = v2f{kUnset, 0.f};
    return;
  }
  const int32_t* table = p.s.table + (int64_t)t.b * W;
  const int page_words = (int)kv4_words(S, D);

  // ---- this wave's 32 rows: one a lane, both halves of the wave alike --------
  const int c = lane & 31, half = lane >> 5;
  const int row = t.row0 + 32 * wave + c;
  const bool there = 32 * wave + c < rows;
  const int row_token = p.by.G(row);
  const int pos = there ? first + row_token : kKv4Past;
  const bool alive = 32 * wave < rows;                               // the wave has rows
  const int last_row = min(32 * wave + 31, rows - 1);
  const int wp0 = first + p.by.G(t.row0 + 32 * wave), wp1 = first + p.by.G(t.row0 + last_row);
  // ---- loads of tiles ------------------------------------------------------------
  // The first half of the workgroup brings the keys, the other half the values.
  // Load n of a tile: key codes of position n % 64, words 4 (n / 64) ..; value codes
  // of positions 4 (n / kC) .., word n % kC.
  constexpr int NH = NT / 2, kN = kTile * kC / 4, kL = (kN + NH - 1) / NH;
  const bool keys = wave < NW / 2;
  const int htid = keys ? tid : tid - NH;
  const char* const pool = (const char*)(p.s.pages + (int64_t)h * page_words);
  const u32 page_step = (u32)H * (u32)page_words * 4u;   // < 2^32: 1024 heads of 256 positions of 136 bytes
  const int inside = S < kTile ? S - 1 : kTile - 1;      // bits of a position that the thread holds
  int off[kL], wat[kL];                                  // position in the tile; where its values go
  const char *code_at[kL], *word_at[kL];                 // of page 0
#pragma unroll
  for (int i = 0; i < kL; ++i) {
    const int n = (htid + i * NH) % kN;   // threads past the tile repeat it
    off[i] = keys ? n % kTile : n / kC * 4;
    code_at[i] = pool + ((off[i] & inside) * (D / 2) + (keys ? n / kTile * 16 : S * (D / 2) + n % kC * 16));
    word_at[i] = pool + (S * D + (keys ? 0 : 4 * S) + (off[i] & inside) * 4);
    if (keys) {
      wat[i] = ((off[i] >> 5) * kC + n / kTile * 4) * 32 + (off[i] & 31);
    } else {
      // of 32 positions: quads 4 step + half and 4 step + 2 + half side by side; channel
      // 8 w + j at place 8 j + w (64 channels) or 16 j + w
      const int quad = n / kC, qq = quad & 7;
      wat[i] = 2 * ((((quad >> 3) * 2 + (qq >> 2)) * 2 + (qq & 1)) * D + n % kC) + (qq >> 1 & 1);
    }
  }
  int id[kL], page_of[kL];   // page of the thread's position; of it, in the tile
#pragma unroll
  for (int i = 0; i < kL; ++i) page_of[i] = S < kTile ? off[i] >> shift : 0;
  v4i code[kL], word[kL];   // word: of one position (keys) or four
  bool page_ok[kL];
  auto fetch_ids = [&](int tile) QG_INLINE {
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      id[i] = table[min(((tile * kTile) >> shift) + page_of[i], W - 1)];   // past the table: any page, the capacity hides it
    }
  };
  auto fetch = [&](int tile) QG_INLINE {
    const u32 slot0 = (u32)(tile * kTile) & (u32)(S - 1);
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      page_ok[i] = (u32)id[i] < (u32)p.s.P;
      const uint64_t page = (uint64_t)(page_ok[i] ? (u32)id[i] : 0u) * page_step;
      code[i] = ld16(code_at[i] + page + slot0 * (D / 2));
      if (keys) word[i][0] = *(const int*)(word_at[i] + page + slot0 * 4);
      else word[i] = ld16(word_at[i] + page + slot0 * 4);
    }
  };
  auto tile_at = [&](int u) QG_INLINE { return span.tile(first_tile + min(u, n_tiles - 1)); };
  // The first tile's codes come in behind the queries, while those are scaled.
  if (n_tiles > 0) fetch_ids(tile_at(0));
  v4i qw[kSt];
  {
    const int r = there ? row : t.row0, token = p.by.G(r);
    const int64_t at = (int64_t)(t.token0 + token) * p.a.q_stride + (int64_t)(h * p.G + r - token * p.G) * D;
#pragma unroll
    for (int j = 0; j < kSt; ++j) qw[j] = ld16((const uint16_t*)p.a.q + at + 16 * j + 8 * half);
  }
  if (n_tiles > 0) {
    fetch(tile_at(0));
    fetch_ids(tile_at(1));
  }
  v8h q[kSt];
  const float to_log2 = p.a.scale * 1.44269504088896f;
  int unit;   // scores in base 2 are to_log2 2^unit times those of the scaled queries and keys
  {
    float x[kSt][8], top = 0.f;
#pragma unroll
    for (int j = 0; j < kSt; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const u32 u = there ? ((u32)qw[j][e >> 1] >> (16 * (e & 1))) & 0xFFFFu : 0u;
        x[j][e] = DT == BF16 ? bf16_bits_to_f32(u) : f16_bits_to_f32((uint16_t)u);
        top = fmaxf(top, fabsf(x[j][e]));
      }
    }
    top = fmaxf(top, __shfl_xor(top, 32, kWave));
    const int e = top > 0.f && top < __builtin_inff() ? 14 - ilogbf(top) : 0;
    constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};   // of the unpacked codes
#pragma unroll
    for (int j = 0; j < kSt; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) q[j][i] = (_Float16)ldexpf(x[j][order[i]], e);
    unit = 9 - e;
  }
  v16f o[kDt];
#pragma unroll
  for (int j = 0; j < kDt; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[j][e] = 0.f;
  // Exponents added to the scores, for the outputs' weights and for their sum l.  They are
  // one but where value scales have moved the outputs' so far that l leaves kApartLow .. kApartHigh in it.
  float l = 0.f, sh = there ? kUnset : -kUnset, shl = sh;
  bool apart = false;   // some row's differ: the wave's tiles take the general form

  // positions of a tile that some row sees, or that lie between such
  auto seen_from = [&](int tile) QG_INLINE {
    const int t0 = tile * kTile;
    return window > 0 && t0 >= sinks ? max(p0 - window + 1 - t0, 0) : 0;
  };
  auto seen_to = [&](int tile) QG_INLINE { return min(p1 + 1, capacity) - tile * kTile; };
  float kf = 0.f, vf_ = 0.f;   // 2^(15 - e) of keys and values
  // The thread's codes -> values of a tile, number u.  True where a scale is odd.
  const auto fma2 = [](u32 n, u32 s, u32 z) QG_INLINE {
    return __builtin_bit_cast(int, __builtin_elementwise_fma(__builtin_bit_cast(v2h, n), __builtin_bit_cast(v2h, s),
                                                             __builtin_bit_cast(v2h, z)));
  };
  // In pieces, piece k of kPieces: some for the places between the products, the rest
  // for the turn behind them, ahead of the weights (all of them between the products:
  // 160 us for a prompt of 4096 tokens of 32 heads, so 157; the products' turn is the
  // longer one).  Words 0 and 1 of the keys are read ahead of that turn's barrier.
  constexpr int kPieces = 4 * kDt + 2 * kSt;
  u32 s24[kL][2], s20[kL][2], zz[kL][2];   // constants: of the keys' position, or of the values' two pairs
  float sv[kL][4];
  bool odd = false;
  // Positions that no row sees, or of no page, ahead of the unpacking: their words are
  // marked (and read as a scale that is odd).
  auto mark = [&](auto role, int tile) QG_INLINE {
    constexpr bool KEYS = decltype(role)::value;
    const int low = seen_from(tile), high = seen_to(tile);
    bool pages = true;
#pragma unroll
    for (int i = 0; i < kL; ++i) pages &= page_ok[i];
    if (low <= 0 && high >= kTile && __all(pages)) return;
#pragma unroll
    for (int i = 0; i < kL; ++i)
#pragma unroll
      for (int e = 0; e < (KEYS ? 1 : 4); ++e)
        if (!(page_ok[i] & (off[i] + e >= low) & (off[i] + e < high))) word[i][e] = (int)kHidden;
  };
  auto fit_key = [&](int i, int u) QG_INLINE {
    const u32 w = (u32)word[i][0];
    const Kv4Fit fit = kv4_fit(w, kf);
    odd |= fit.odd;
    kraw[u & 3][off[i]] = w;
    s24[i][0] = pair_of(fit.v, fit.v);
    s20[i][0] = mul2(s24[i][0], kSixteenth2);
    zz[i][0] = mul2(s24[i][0], (w & 15u) * 0x10001u) ^ 0x80008000u;   // z is z 2^-24 as it stands
  };
  auto word_of_key = [&](int i, int j, int u) QG_INLINE {
    const u32 x = (u32)code[i][j], hi = x >> 8;
    (kbuf + (u & 1) * kTile * kC)[wat[i] + 32 * j] =
        v4i{fma2(x & 0x000F000Fu, s24[i][0], zz[i][0]), fma2(x & 0x00F000F0u, s20[i][0], zz[i][0]),
            fma2(hi & 0x000F000Fu, s24[i][0], zz[i][0]), fma2(hi & 0x00F000F0u, s20[i][0], zz[i][0])};
  };
  auto fit_value = [&](int i, int e) QG_INLINE {
    const Kv4Fit fit = kv4_fit((u32)word[i][e], vf_);
    odd |= fit.odd;
    sv[i][e] = fit.v;
    if (e & 1) {
      const int t = e >> 1;
      s24[i][t] = pair_of(sv[i][e - 1], sv[i][e]);
      s20[i][t] = mul2(s24[i][t], kSixteenth2);
      zz[i][t] = mul2(s24[i][t], ((u32)word[i][e - 1] & 15u) | (((u32)word[i][e] & 15u) << 16)) ^ 0x80008000u;
    }
  };
  // channel 4 hf + j of the values' word, at four positions
  auto channel_of_value = [&](int i, int hf, int j, int vb_at) QG_INLINE {
    v2i* const vb = (v2i*)(vbuf + vb_at * kTile * kC);
    constexpr int kStep = D == 64 ? 8 : 16;
    const u32 sel = hf ? 0x07060302u : 0x05040100u, mask = j & 1 ? 0x00F000F0u : 0x000F000Fu;
    const u32 x = __builtin_amdgcn_perm((u32)code[i][1], (u32)code[i][0], sel);
    const u32 y = __builtin_amdgcn_perm((u32)code[i][3], (u32)code[i][2], sel);
    vb[wat[i] + 2 * kStep * (4 * hf + j)] =
        v2i{fma2((j & 2 ? x >> 8 : x) & mask, j & 1 ? s20[i][0] : s24[i][0], zz[i][0]),
            fma2((j & 2 ? y >> 8 : y) & mask, j & 1 ? s20[i][1] : s24[i][1], zz[i][1])};
  };
  constexpr int kWhole = 0, kBetween = 1, kBehind = 2;   // which pieces: all, those between the products, the others
  constexpr int kKeysBetween = 3, kValuesBetween = 4;    // of 5 and 12
  auto piece = [&](auto role, auto which, auto at, int vb_at, int u) QG_INLINE {
    constexpr bool KEYS = decltype(role)::value;
    constexpr int k = decltype(at)::value, WHICH = decltype(which)::value;
    constexpr auto now = [](int w) { return WHICH == kWhole || (w < (KEYS ? kKeysBetween : kValuesBetween)) == (WHICH == kBetween); };
    if constexpr (KEYS) {
      // a fit, then its four words, two places apart
      constexpr int kEvery = kPieces / (5 * kL);
      if constexpr (k % kEvery == 0 && k / kEvery < 5 * kL) {
        constexpr int i = k / kEvery / 5, w = k / kEvery % 5;
        if constexpr (!now(w)) return;
        else if constexpr (w == 0) fit_key(i, u);
        else word_of_key(i, w - 1, u);
      }
    } else {
      // four fits, then eight channels
      constexpr int kEvery = kPieces / (12 * kL);
      if constexpr (k % kEvery == 0 && k / kEvery < 12 * kL) {
        constexpr int i = k / kEvery / 12, w = k / kEvery % 12;
        if constexpr (!now(w)) {
          return;
        } else if constexpr (w < 4) {
          fit_value(i, w);
          if constexpr (w == 3) *(v4i*)&vraw[u & 3][off[i]] = word[i];
        } else {
          channel_of_value(i, (w - 4) / 4, (w - 4) % 4, vb_at);
        }
      }
    }
  };
  auto unpack = [&](auto role, int tile, int vb_at, int u) QG_INLINE {
    mark(role, tile);
    odd = false;
    for_each<kPieces>([&](auto k) QG_INLINE { piece(role, std::integral_constant<int, kWhole>(), k, vb_at, u); });
  };

  // ---- the products of a tile ------------------------------------------------------
  v16f s[2];     // scores of the tile at hand
  v8h pf[2][2];  // weights of the one before it
#pragma unroll
  for (int i = 0; i < 4; ++i) pf[i >> 1][i & 1] = v8h{};
  auto outputs = [&](int vb_at) QG_INLINE {
    const v4i* const vb = vbuf + vb_at * kTile * kC + half * D + c;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < 2 * kDt; ++t)
        o[t % kDt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
            __builtin_bit_cast(v8h, vb[i * kC * 32 + 2 * (t / kDt) * D + 32 * (t % kDt)]), pf[i][t / kDt], o[t % kDt], 0, 0, 0);
  };

  // Outputs of the last tile and scores of this one with the unpacking of a later one
  // between the products.  Operands are read kAhead products ahead; the order is
  // pinned, since the compiler's own reads each operand right before its product
  // and waits for it (3300 cycles for the 32 products' 1024).
  constexpr int kAhead = 6;
  v4i ring[kAhead];
  const v4i *vb = vbuf, *kb = kbuf;
  auto read = [&](auto at) QG_INLINE {
    constexpr int k = decltype(at)::value;
    if constexpr (k < kPieces && k % 2 == 0) {
      constexpr int i = k / 2 / (2 * kDt), t = k / 2 % (2 * kDt);
      ring[k % kAhead] = vb[i * kC * 32 + 2 * (t / kDt) * D + 32 * (t % kDt)];
    } else if constexpr (k < kPieces) {
      constexpr int i = k / 2 & 1, j = k / 4;
      ring[k % kAhead] = kb[(i * kC + 2 * j) * 32];
    }
  };
  // The first operands of tile u's turn, ahead of the barrier in front of it.
  auto read_ahead = [&](int vlast, int u) QG_INLINE {
    vb = vbuf + vlast * kTile * kC + half * D + c;
    kb = kbuf + (u & 1) * kTile * kC + half * 32 + c;
    for_each<kAhead - 1>([&](auto k) QG_INLINE { read(k); });
  };
  auto fused = [&](auto role, int vb_at, int u) QG_INLINE {
    odd = false;
    __builtin_amdgcn_sched_barrier(0);
    for_each<kPieces>([&](auto at) QG_INLINE {
      constexpr int k = decltype(at)::value;
      read(std::integral_constant<int, k + kAhead - 1>());
      const v8h x = __builtin_bit_cast(v8h, ring[k % kAhead]);
      if constexpr (k % 2 == 0) {
        constexpr int i = k / 2 / (2 * kDt), t = k / 2 % (2 * kDt);
        o[t % kDt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, pf[i][t / kDt], o[t % kDt], 0, 0, 0);
      } else {
        constexpr int i = k / 2 & 1, j = k / 4;
        const v16f zero = {};
        s[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, q[j], j ? s[i] : zero, 0, 0, 0);
      }
      piece(role, std::integral_constant<int, kBetween>(), at, vb_at, u + 1);
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  // ---- scores of a tile to weights -------------------------------------------------
  // With x the scores in base 2 and e the exponents of the values' powers of two, the
  // weights are exp2(x + e - ev + sh) for one sh of a row, which falls where their sum
  // would pass 2^14, outputs with it, and l the sum of exp2(x + shl):
  // out = 2^(9 + ev + shl - sh) o / l.
  int ek = 0, ev = 0;   // exponents of the common powers of two
  float ct = 0.f;
  // The row's sh down to `to`, where that is below it, and the outputs with it.
  auto lower = [&](float to) QG_INLINE {
    const float by = to < sh ? __builtin_amdgcn_exp2f(to - sh) : 1.f;   // 0 for a row's first tile
    sh = fminf(sh, to);
#pragma unroll
    for (int j = 0; j < kDt; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[j][e] *= by;
  };
  auto both = [](float v) QG_INLINE { return fmaxf(v, __shfl_xor(v, 32, kWave)); };
  auto weights = [&](int tile, int u, bool all, bool odd) QG_INLINE {
    const int t0 = tile * kTile + 4 * half;
    const u32 reach = window > 0 ? (u32)window : 0x7FFFFFFFu;
    float by = ct;
    if (odd) {
      // any position may be out of sight, of no page, or of another power of two:
      // a lane finds its position's exponents, for all lanes to read
      {
        const u32 wk = kraw[u & 3][lane], wv = vraw[u & 3][lane];
        const float ke = (float)float_exp(wk), ve = (float)float_exp(wv);   // 128: not finite
        const float nan = __builtin_nanf("");
        own[0][lane] = wk == kHidden ? kUnset : ke == 128.f ? nan : kv4_fit(wk, kf).odd ? ke : (float)ek;
        own[1][lane] = ve == 128.f ? nan : kv4_fit(wv, vf_).odd ? ve - (float)ev : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const v4f f = *(const v4f*)&own[0][32 * i + 8 * a + 4 * half];
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int at = t0 + 32 * i + 8 * a + b, e = 4 * a + b;
            const bool seen = !(f[b] == kUnset) & (((u32)(pos - at) < reach) | ((at < sinks) & (at <= pos)));
            // (a NaN's integer is 0)
            s[i][e] = seen ? ldexpf(__builtin_fmaf(s[i][e], to_log2, f[b] * 0.f), unit + (int)f[b]) : -__builtin_inff();
          }
          __builtin_amdgcn_sched_barrier(0);   // few exponents at a time: registers
        }
      // the sum of the exponentials here, since the values' powers of two differ
      float top = kLow;
#pragma unroll
      for (int e = 0; e < 32; ++e) top = fmaxf(top, s[e >> 4][e & 15]);
      if (__any(top + shl > 60.f)) {
        const float was = shl;
        top = both(top);
        shl = fminf(was, -floorf(top) - fabsf(top) * 0x1p-21f);
        l *= __builtin_amdgcn_exp2f(shl - was);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const v4f f = *(const v4f*)&own[1][32 * i + 8 * a + 4 * half];
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int e = 4 * a + b;
            l += __builtin_amdgcn_exp2f(s[i][e] + shl);
            s[i][e] = s[i][e] == -__builtin_inff() ? s[i][e] : s[i][e] + f[b];   // whatever lies out of sight
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      by = 1.f;
    } else if (!all) {
      // some position is outside a row's window
      const int back = pos - t0;
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const u32 d = (u32)(back - (32 * (e >> 4) + 8 * (e % 16 / 4) + e % 4));
        s[e >> 4][e & 15] = d < reach ? s[e >> 4][e & 15] * ct : -__builtin_inff();
      }
      by = 1.f;
    }
    // The second round's sums pass: sh is then below minus the largest score, by more
    // than rounding takes from either.
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
      float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][e], by, sh));
          part[e & 3] += w[e];
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) pf[i][e >> 3][e & 7] = (_Float16)w[e];
      }
      const float sum = (part[0] + part[1]) + (part[2] + part[3]);
      if (round > 0 || !__any(sum > 0x1p14f)) {   // a NaN stays one
        if (!odd) l += sum;
        break;
      }
      float top = kLow;
#pragma unroll
      for (int e = 0; e < 32; ++e) top = fmaxf(top, s[e >> 4][e & 15] * by);
      top = both(top);
      const float was = sh;
      lower(-floorf(top) - fabsf(top) * 0x1p-21f);
      if (!odd) {
        l *= __builtin_amdgcn_exp2f(sh - was);
        shl = sh;
      }
    }
    if (odd && __any(shl != sh)) {
      const float other = l * __builtin_amdgcn_exp2f(sh - shl), most = both(other);
      apart = __any(((most < kApartLow) | (most > kApartHigh)) & (both(l) > 0.f));
      if (!apart) {
        l = other;
        shl = sh;
      }
    }
  };

  if (n_tiles > 0) {
    // the first tile, and from its largest scales the common powers of two
    if (tid < 8) flags[tid] = 0;
    // the values ahead of the first tile's, which zero weights meet
    for (int i = tid; i < kTile * kC; i += NT) vbuf[(kVBufs - 1) * kTile * kC + i] = v4i{0, 0, 0, 0};
    float most = 0.f;
    const int low = seen_from(tile_at(0)), high = seen_to(tile_at(0));
#pragma unroll
    for (int i = 0; i < kL; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (keys && e > 0) continue;
        const float v = kv4_scale((u32)word[i][e]);
        if (page_ok[i] & (off[i] + e >= low) & (off[i] + e < high) & (v < __builtin_inff())) most = fmaxf(most, v);
      }
    most = wave_max_nonneg(most);
    float* const tops = (float*)(flags + 8);
    if (lane == 0) tops[wave] = most;
    __syncthreads();
    float top_k = 0.f, top_v = 0.f;
#pragma unroll
    for (int w = 0; w < NW / 2; ++w) {
      top_k = fmaxf(top_k, tops[w]);
      top_v = fmaxf(top_v, tops[NW / 2 + w]);
    }
    // room for scales 16 times as large and 64 times as small; where all are zero, for
    // scales in [2^-7, 2^3): 4096 tokens of 32 heads behind 64 zeros 178 us, and 413 where every
    // later scale is odd, 158 without zeros
    const auto common = [](float top) QG_INLINE {
      const int e = __builtin_amdgcn_readfirstlane(float_exp(__float_as_uint(top)));
      return e > -127 ? min(max(e, -100), 100) + 4 : 2;
    };
    ek = common(top_k);
    ev = common(top_v);
    kf = ldexpf(1.f, 15 - ek);
    vf_ = ldexpf(1.f, 15 - ev);
    ct = ldexpf(to_log2, unit + ek);
    if (keys) unpack(std::true_type(), tile_at(0), 0, 0);
    else unpack(std::false_type(), tile_at(0), 0, 0);
    if (__any(odd)) flags[0] = 1;
    fetch(tile_at(1));
    fetch_ids(tile_at(2));
    __syncthreads();
  }
  // In turn 2 u the first half has the products of tile u, in turn 2 u + 1 its
  // weights; the second half runs one turn behind.  Keys of tile u + 1 are written by
  // the first half in turns 2 u and 2 u + 1, into the buffer that the second half read
  // last in turn 2 u - 1; values of tile u + 1 by the second half in turn 2 u + 2 (their
  // group words in turn 2 u + 1), into that of tile u - 2, which was read last in turn
  // 2 u - 1.  The first half needs the values in turn 2 u + 4.
  // Every turn has both products, so that the outputs stay in one place: where the
  // wave sees nothing of a tile its weights are zeros (and the values are finite).
  int vnow = 0;   // buffer of the tile's values
  // Tiles of this wave by their first position: from act0 on (or below sinks0) some
  // row sees something; between all0 and all1 every row sees everything.
  const int act0 = window > 0 ? wp0 - window + 2 - kTile : -0x7FFFFFFF, sinks0 = window > 0 ? sinks : 0;
  const int all0 = window > 0 ? wp1 - window + 1 : 0, all1 = wp0 - kTile + 1;
  const int act1 = alive ? wp1 : -1;
  auto loop = [&](auto role) QG_INLINE {
    constexpr bool KEYS = decltype(role)::value;
    if constexpr (!KEYS) lds_barrier();
    int now = tile_at(0), next = tile_at(1), third = tile_at(2);
    read_ahead(kVBufs - 1, 0);
#pragma unroll 1
    for (int u = 0; u < n_tiles; ++u) {
      const int t0 = now * kTile, fourth = tile_at(u + 3);
      const int vnext = vnow == kVBufs - 1 ? 0 : vnow + 1;
      mark(role, next);
      __builtin_amdgcn_s_setprio(1);
      const int flag = flags[u & 7];   // complete since the last turn
      fused(role, vnext, u);
      __builtin_amdgcn_s_setprio(0);
      if (__any(odd)) flags[(u + 1) & 7] = 1;
      if (KEYS && wave == 0) flags[(u + 4) & 7] = 0;
      const bool is_odd = __builtin_amdgcn_readfirstlane(flag) != 0;
      lds_barrier();
      for_each<kPieces>([&](auto k) QG_INLINE { piece(role, std::integral_constant<int, kBehind>(), k, vnext, u + 1); });
      fetch(third);   // the codes are used: the next ones
      fetch_ids(fourth);
      __builtin_amdgcn_sched_barrier(0);
      const bool all = t0 >= all0 && t0 <= all1;
      if (t0 <= act1 && (t0 >= act0 || t0 < sinks0)) {
        // first positions that stay visible take the general form
        weights(now, u, all, is_odd || apart || (!all && t0 < sinks0));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) pf[i >> 1][i & 1] = v8h{};
      }
      now = next;
      next = third;
      third = fourth;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the pieces are written, long since
      read_ahead(vnow, u + 1);
      vnow = vnext;
      asm volatile("s_barrier" ::: "memory");
    }
    if constexpr (KEYS) lds_barrier();
  };
  if (keys) loop(std::true_type());
  else loop(std::false_type());
  if (n_tiles > 0) outputs(vnow == 0 ? kVBufs - 1 : vnow - 1);

  // ---- outputs: lane (c, half) has, of row c, eight runs of 8 channels ---------------
  l += __shfl_xor(l, 32, kWave);
  if (!there) return;
  const int64_t to = ((int64_t)(t.token0 + row_token) * p.a.Hq + h * p.G + row - row_token * p.G) * D;
  const bool whole = p.splits == 1;
  // parts: [32 rows][D / 8][row][8], so that the lanes of a store are neighbours
  const int64_t to_part = (part + 32 * wave) * D + 8 * c;
  // 8 channels of the output, or of this split's
  auto store = [&](int d, const float (&x)[8]) QG_INLINE {
    if (whole) {
      kv4_store8<DT>(p.a.out, to + d, x);
    } else {
      *(v4f*)(p.part_o + to_part + 32 * d) = v4f{x[0], x[1], x[2], x[3]};
      *(v4f*)(p.part_o + to_part + 32 * d + 4) = v4f{x[4], x[5], x[6], x[7]};
    }
  };
  if (!whole && half == 0) *(v2f*)(p.part_ml + (part + 32 * wave + c) * 2) = v2f{shl, l};
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  // 2^(9 + ev) in the unit of l; the whole powers behind the rest, which may not hold them
  const float gap = shl - sh, more = fmaxf(floorf(gap), -1000.f);
  const float f = inv * __builtin_amdgcn_exp2f(gap - more);
  const int up = 9 + ev + (int)more;
  if constexpr (D == 64) {
    // place 32 j + 8 a + 4 half + b holds channel 8 (place % 8) + place / 8
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int a = 0; a < 4; ++a) x[4 * j + a] = ldexpf(o[j][4 * a + b] * f, up);
      store(32 * half + 8 * b, x);
    }
  } else {
    // place 32 j + 8 a + 4 half + b holds channel 8 (place % 16) + place / 16
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[2 * j] = ldexpf(o[j][4 * a + b] * f, up);
          x[2 * j + 1] = ldexpf(o[j][4 * (a + 2) + b] * f, up);
        }
        store(64 * a + 32 * half + 8 * b, x);
      }
  }
}

namespace {

template <int D>
constexpr int many_lds() { return (kVBufs + 2) * kTile * (D / 8) * 16 + 8 * kTile * 4 + 16 * 4 + 8 * 2 * kTile * 4; }

template <int DT>
hipError_t many_t(const Kv4ManyArgs& p, hipStream_t st) {
  const unsigned grid = (unsigned)((int64_t)p.tiles * p.s.H * p.splits);
  if (p.a.D == 64) k_kv4_attend_many<DT, 64><<<grid, 64 * kManyWaves, many_lds<64>(), st>>>(p);
  else k_kv4_attend_many<DT, 128><<<grid, 64 * kManyWaves, many_lds<128>(), st>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_many(const Kv4Seqs& s, const Kv4Attend& a, int dtype, int64_t min_rows, int64_t tiles,
                           int splits, float* part_o, float* part_ml, hipStream_t st) {
  const Kv4ManyArgs p{s, a, a.Hq / s.H, (int)tiles, splits, kv4_divs(s, a.Hq / s.H, kKv4ManyRows), kv4_div(splits),
                      min_rows, part_o, part_ml};
  return dtype == F16 ? many_t<F16>(p, st) : many_t<BF16>(p, st);
}

}  // namespace qg
