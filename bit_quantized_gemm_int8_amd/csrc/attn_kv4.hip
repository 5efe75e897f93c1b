// Attention of a few query rows over the 4-bit paged KV cache (qg_kv4.hpp).
//
//   x_t = scale (q . k_t),  o = sum_t exp(x_t) v_t / sum_t exp(x_t)
// with k_t = (n_t - z_t) s_t and v_t alike, over the positions a row can see.
// The codes n go to the matrix cores as they are:
//   q . k_t = s_t (sum_d q_d n_td - z_t sum_d q_d)
//   o       = (sum_t (p_t s_t) n_t - sum_t (p_t s_t) z_t) / sum_t p_t
// A nibble masked out of a code word is a binary16 subnormal, n 2^-20 at bits 4 to 7
// of its half, which gfx950's matrix cores take exactly: unpacking costs an AND and at
// most a shift for two codes.  (At bits 0 to 3 they do not: an operand n 2^-24 counts
// with the exponent of 2^-14 when the products are aligned, and sums of 32 came out up
// to 1.6e-5 of their terms too small, against 1.3e-7 for n 2^-20.)  Queries are
// scaled to binary16's upper range by a power of two of their row: exact down to 2^-28 of
// the row's largest element, and off by up to 2^-39 of that below, where binary16 is
// subnormal.  The weights p s are rounded to binary16 (half a step:
// 2^-11), the codes' sum and the zero points' sum taking the same rounded weights,
// both through the matrix cores.  Binary16 outputs, whose own rounding is no larger, get
// what the rounding left over in a second product (2^-22).  Softmax and sums: binary32.
//
// Layout.  A wave takes 32 positions a step.  Both products have the query rows
// as columns, so that a lane has one query row throughout: a lane's scores, 4
// neighbouring positions in each half of the step, are the operand that the second
// product needs, with the positions in that order.  Value codes of 4 positions of a
// word are neighbours in the cache for the same reason.  No lane exchange per
// step: the softmax's weights are exp2(x + sh) for an sh of the row that falls only where
// they pass 2^9, outputs and sum with it.  The outputs' weights p s are in a power of two
// of their own for each row and value group, so that neither the sum nor the other group
// loses bits to scales far from those before them.
//
// What bounds it.  Many sequences: memory (64 requests of up to 16384 positions, 8 kv
// heads of 128, 680 MB: 131 us, 5.2 TB/s).  One: latency, offsets, page table, codes and
// the join in turn (4096 positions of 32 heads 12.7 us, a call of one page's positions
// 6).  Heads of 256 with many rows: the vector unit, since the codes are unpacked again
// for each 16 rows (137 us for 60 GFLOP.  With a kernel that took 141, tiles of 32 rows
// took 220, all registers of a wave and more, and one wave a SIMD; waves that share 32
// rows, with weights and queries in LDS, keep in step and took 151).
#include "qg_kv4_attn.hpp"

#include <algorithm>

namespace qg {

namespace {

constexpr int kStep = 32;            // positions of a wave's step
constexpr int kAttnWaves = 4, kAttnWavesLong = 8;   // of a workgroup
constexpr float kLowest = -3.402823466e38f, kUnset = 1e30f;
constexpr u32 kNibbles = 0x00F000F0u;

typedef int v2i __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float max16(float v) {   // over the four lanes of one column
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
}
__device__ __forceinline__ float sum16(float v) {
  v += __shfl_xor(v, 16, kWave);
  return v + __shfl_xor(v, 32, kWave);
}

}  // namespace

struct Kv4FewArgs {
  Kv4Seqs s;
  Kv4Attend a;
  int G, splits;
  Kv4Divs by;
  Kv4Div by_splits;
  int64_t min_rows, max_rows;   // sequences of other numbers of rows are another kernel's
  float* part_o;
  float* part_ml;
};

// Workspace of a call with several splits: outputs [tile][split][row][D] (of the prompt
// kernel [tile][split][row / 32][D / 8][row % 32][8]) and (sh, sum) [tile][split][row],
// binary32, where tile counts row tiles times kv heads; a split's outputs are over its
// own sum, so that they are in range wherever its values are.

// Steps of split `split` of a tile with `tiles` steps.
__device__ __forceinline__ int kv4_per_split(int tiles, const Kv4Div& splits) {
  return max(splits((int)(tiles + splits.d - 1)), kAttnWaves);
}

// Positions of a tile's first row's sequence and of the tile's first and last row.
template <int ROWS>
__device__ __forceinline__ void kv4_positions(const Kv4FewArgs& p, const Kv4Tile& t, int& p0, int& p1,
                                              int& first, int& rows) {
  rows = min(t.n * p.G - t.row0, ROWS);
  first = max(p.s.lengths[t.b], -0x3FFFFFFF) - t.n;   // n <= 2^30: no overflow
  p0 = first + p.by.G(t.row0);
  p1 = first + p.by.G(t.row0 + rows - 1);
}

// ONCE: a sequence's rows are one tile, so that its cache is read once: past the
// caches (64 requests of up to 16384 positions, 8 kv heads: 131 us against 146; where
// many tiles read the same pages it costs 8%).
template <int DT, int D, int RT, bool ONCE, int NW = kAttnWaves>
__global__ __launch_bounds__(64 * NW, D * RT == 64 ? 4 : D == 128 && RT == 1 ? 3 : 2) void k_kv4_attend_few(Kv4FewArgs p) {
  constexpr int kRows = 16 * RT, kGd = kv4_groups(D), kKw = D / 32, kTd = D / 16;   // key words, channel tiles
  constexpr bool kTwice = DT == F16;   // weights in two parts
  // outputs of the waves, 16 rows and up to 128 channels at a time
  constexpr int kCols = D < 128 ? D : 128;
  __shared__ float red[NW][16][kCols + 4];
  __shared__ float stat[NW][kRows][2];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int th = p.by_splits((int)blockIdx.x), split = blockIdx.x - th * p.splits;
  const int tile_n = p.by.H(th), h = th - tile_n * p.s.H;
  const Kv4Tile t = kv4_tile<kRows>(p.s, p.by, p.min_rows, p.max_rows, tile_n);
  if (t.b < 0) return;
  int p0, p1, first, rows;
  kv4_positions<kRows>(p, t, p0, p1, first, rows);
  const int shift = p.s.shift, S = 1 << shift, W = p.s.W, window = p.a.window, sinks = p.a.sinks;
  const int capacity = (int)min((int64_t)W << shift, (int64_t)0x40000000);
  const Kv4Span span = kv4_span<kStep>(p0, p1, window, sinks, capacity);
  const int per = kv4_per_split(span.tiles, p.by_splits);
  const int u0 = split * per, u1 = min(u0 + per, span.tiles);
  if (u0 >= u1 && p.splits > 1) {   // a split without steps: the join leaves it out
    if (threadIdx.x < kRows) *(v2f*)(p.part_ml + (((int64_t)th * p.splits + split) * kRows + threadIdx.x) * 2) = v2f{kUnset, 0.f};
    return;
  }
  const int32_t* const table = p.s.table + (int64_t)t.b * W;
  const int page_words = (int)kv4_words(S, D);
  const char* const pool = (const char*)(p.s.pages + (int64_t)h * page_words);
  const uint32_t page_step = (uint32_t)p.s.H * (uint32_t)page_words * 4u;   // < 2^32: 1024 heads of 256 positions of 272 bytes

  // ---- codes and group words of a step, as a lane holds them -------------------
  const int c = lane & 15, g = lane >> 4;
  const u32 off_k = c * (D / 2) + g * (D == 64 ? 8 : 16);
  const u32 off_v = (g * (D / 8) + (D == 64 ? c >> 1 : c)) * 16;
  const u32 off_p = 16 * g;
  int kc[2][kKw];
  v4i vc[2][kGd], kp[2][kGd], vp[2][kGd];
  int id[2], id_next[2];
  const char* at[2];
  // pages of the halves of step u; any where there is none
  auto fetch_ids = [&](int u) QG_INLINE {
    const int tile = span.tile(min(u, u1 - 1));
#pragma unroll
    for (int i = 0; i < 2; ++i) id_next[i] = __builtin_amdgcn_readfirstlane(table[min((tile * kStep + 16 * i) >> shift, W - 1)]);
  };
  auto load_keys = [&](int u) QG_INLINE {
    const int tile = span.tile(min(u, u1 - 1));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      id[i] = id_next[i];
      const u32 slot = (u32)(tile * kStep + 16 * i) & (u32)(S - 1);
      at[i] = pool + (uint64_t)((u32)id[i] < (u32)p.s.P ? (u32)id[i] : 0u) * page_step;
      const char* const kb = at[i] + slot * (D / 2);
      const char* const pb = at[i] + (S * D + slot * 4);
#pragma unroll
      for (int gd = 0; gd < kGd; ++gd) {
        if constexpr (D == 64) {
          const v2i a = *(const v2i*)(kb + off_k);
          kc[i][0] = a[0];
          kc[i][1] = a[1];
        } else {
          const v4i a = ONCE ? ld16_stream(kb + (off_k + 64 * gd)) : ld16(kb + (off_k + 64 * gd));
#pragma unroll
          for (int j = 0; j < 4; ++j) kc[i][4 * gd + j] = a[j];
        }
        kp[i][gd] = ld16(pb + gd * 4 * S + off_p);
      }
    }
  };
  auto load_values = [&](int u) QG_INLINE {   // of the pages that load_keys took
    const int tile = span.tile(min(u, u1 - 1));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32 slot = (u32)(tile * kStep + 16 * i) & (u32)(S - 1);
      const char* const vb = at[i] + (S + slot) * (D / 2);
      const char* const pb = at[i] + (S * D + (kGd * S + slot) * 4);
#pragma unroll
      for (int gd = 0; gd < kGd; ++gd) {
        vc[i][gd] = ONCE ? ld16_stream(vb + (off_v + 256 * gd)) : ld16(vb + (off_v + 256 * gd));
        vp[i][gd] = ld16(pb + gd * 4 * S + off_p);
      }
    }
  };

  // ---- queries -------------------------------------------------------------------
  // A lane's words in the order of the unpacked codes (nibbles 0 4 1 5 2 6 3 7), and
  // their sum.
  int pos[RT];
  v8h q[RT][kKw];
  float cc[RT], qs[RT][kGd];
  v4i qw[RT][kKw];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const bool there = 16 * r + c < rows;
    const int row = t.row0 + (there ? 16 * r + c : 0), token = p.by.G(row);
    pos[r] = there ? first + token : kKv4Past;
    const uint16_t* const from = (const uint16_t*)p.a.q + (int64_t)(t.token0 + token) * p.a.q_stride +
                                 (int64_t)(h * p.G + row - token * p.G) * D;
#pragma unroll
    for (int j = 0; j < kKw; ++j) {
      const int d = D == 64 ? 16 * g + 8 * j : 128 * (j / 4) + 32 * g + 8 * (j % 4);
      qw[r][j] = ld16(from + d);
      if (!there) qw[r][j] = v4i{0, 0, 0, 0};
    }
  }
  // the first step's codes come in meanwhile
  const int n_steps = u1 - u0;   // of the workgroup, at least 1 where there is anything to load
  int u = u0 + wave;
  if (n_steps > 0) {
    fetch_ids(u);
    load_keys(u);
    load_values(u);
    fetch_ids(u + NW);
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    float x[kKw][8], top = 0.f;
#pragma unroll
    for (int j = 0; j < kKw; ++j) {
      const v4i a = qw[r][j];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const u32 v = ((u32)a[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
        x[j][e] = DT == BF16 ? bf16_bits_to_f32(v) : f16_bits_to_f32((uint16_t)v);
        top = fmaxf(top, fabsf(x[j][e]));
      }
    }
    top = max16(top);
    // top 2^e in [2^14, 2^15); not for zero rows and infinities
    // (subnormal tops fall short of it)
    const int e2 = top > 0.f && top < __builtin_inff() ? 141 - (int)(__float_as_uint(top) >> 23) : 0;
#pragma unroll
    for (int gd = 0; gd < kGd; ++gd) qs[r][gd] = 0.f;
#pragma unroll
    for (int j = 0; j < kKw; ++j) {
      constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        q[r][j][i] = (_Float16)ldexpf(x[j][order[i]], e2);
        sum += (float)q[r][j][i];   // the zero points meet the queries that the codes meet
      }
      qs[r][j / 4] += sum;
    }
    // scores in units of 2^(e2 - 20), exponents in base 2
#pragma unroll
    for (int gd = 0; gd < kGd; ++gd) qs[r][gd] = sum16(qs[r][gd]) * 0x1p-20f;
    cc[r] = ldexpf(p.a.scale * 1.44269504088896f, 20 - e2);
  }

  // outputs: rows = channels, columns = query rows; sums of the zero points
  v4f o[RT][kTd], oz[RT][kGd];
  // l: sum of exp2(x + sh); outputs: sums of exp2(x + sh) s unit
  float l[RT], sh[RT], unit[RT][kGd];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
#pragma unroll
    for (int j = 0; j < kTd; ++j) o[r][j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int gd = 0; gd < kGd; ++gd) {
      oz[r][gd] = v4f{0.f, 0.f, 0.f, 0.f};
      unit[r][gd] = 1.f;
    }
    l[r] = 0.f;
    sh[r] = kUnset;
  }

#pragma unroll 1
  for (; u < u1; u += NW) {
    const int tile = span.tile(u), t0 = tile * kStep;
    const bool ok0 = (u32)id[0] < (u32)p.s.P, ok1 = (u32)id[1] < (u32)p.s.P;
    const bool full = ok0 && ok1 && t0 + kStep - 1 <= p0 && t0 + kStep <= capacity &&
                      (window <= 0 || t0 > p1 - window || t0 + kStep <= sinks);
    // scores: rows = positions, columns = query rows
    float y[RT][2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v8h kf[kKw];
#pragma unroll
      for (int j = 0; j < kKw; ++j) {
        const u32 w = (u32)kc[i][j];
        kf[j] = __builtin_bit_cast(v8h, v4i{(int)(w << 4 & kNibbles), (int)(w & kNibbles), (int)(w >> 4 & kNibbles),
                                            (int)(w >> 8 & kNibbles)});
      }
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int gd = 0; gd < kGd; ++gd) {
          constexpr int kPer = kKw / kGd;
          v4f a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            a = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[kPer * gd + j], q[r][kPer * gd + j], a, 0, 0, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const u32 w = (u32)kp[i][gd][e];
            const float v = __builtin_fmaf(-(float)(w & 15u), qs[r][gd], a[e]) * kv4_scale(w);
            y[r][i][e] = gd ? y[r][i][e] + v : v;
          }
        }
    }
    float vs[kGd][2][4];
    u32 zf[kGd][2][2];
#pragma unroll
    for (int gd = 0; gd < kGd; ++gd)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) vs[gd][i][e] = kv4_scale((u32)vp[i][gd][e]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          zf[gd][i][e] = (((u32)vp[i][gd][2 * e] & 15u) | (((u32)vp[i][gd][2 * e + 1] & 15u) << 16)) << 4;
      }
    load_keys(u + NW);
    // weights
    v8h pf[RT][kGd], pl[RT][kGd];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[r][i][e] *= cc[r];
      float sv[kGd][2][4], most = 0.f;   // the scales in the row's units
#pragma unroll
      for (int gd = 0; gd < kGd; ++gd)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) sv[gd][i][e] = vs[gd][i][e] * unit[r][gd];
      if (!full) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = t0 + 16 * i + 4 * g + e;
            const bool seen = (i ? ok1 : ok0) & (j <= pos[r]) & (j < capacity) & ((window <= 0) | (j > pos[r] - window) | (j < sinks));
            y[r][i][e] = seen ? y[r][i][e] : -__builtin_inff();
#pragma unroll
            for (int gd = 0; gd < kGd; ++gd) sv[gd][i][e] = seen ? sv[gd][i][e] : 0.f;   // whatever lies out of sight
          }
      }
#pragma unroll
      for (int gd = 0; gd < kGd; ++gd)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) most = fmaxf(most, sv[gd][i][e]);
      float w[kGd][2][4];
#pragma unroll 1
      for (int round = 0; round < 2; ++round) {   // the second round's weights pass
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = __builtin_amdgcn_exp2f(y[r][i][e] + sh[r]);
            sum += x;
#pragma unroll
            for (int gd = 0; gd < kGd; ++gd) w[gd][i][e] = x * sv[gd][i][e];
          }
        // binary16 holds 2^9 2^6; a NaN stays one
        if (round > 0 || !__any(most > 0x1p6f || sum > 0x1p9f)) {
          l[r] += sum;
          break;
        }
        // The row's sh to where its largest exponential is near 1, by more than rounding
        // takes from a score, and each unit to where the group's largest weight is.  Neither
        // the sum nor the outputs ever grow by it.  Whole numbers, so that the outputs'
        // exponent keeps its place as long as their weights do.
        float top = kLowest;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, y[r][i][e]);
        top = max16(top);
        const float was = sh[r];
        sh[r] = fminf(was, -floorf(top) - ceilf(fabsf(top) * 0x1p-21f));
        l[r] *= __builtin_amdgcn_exp2f(sh[r] - was);   // 0 for a row's first weights
#pragma unroll
        for (int gd = 0; gd < kGd; ++gd) {
          float most_w = kLowest;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float yy = y[r][i][e];
              if (yy > -__builtin_inff()) most_w = fmaxf(most_w, yy + __builtin_amdgcn_logf(vs[gd][i][e]));
            }
          most_w = max16(most_w);
          const float had = (float)((int)(__float_as_uint(unit[r][gd]) >> 23) - 127);
          const float to = floorf(fminf(-floorf(most_w) - fabsf(most_w) * 0x1p-21f - sh[r], had + (was - sh[r])));
          // of scales up to 2^124.1, and exponentials up to 2^9, at least 2^-126 will do
          const float now = fminf(fmaxf(to, -126.f), 126.f);
          const float by = __builtin_amdgcn_exp2f((sh[r] - was) + (now - had));
          unit[r][gd] = ldexpf(1.f, (int)now);
          constexpr int kPer = kTd / kGd;
#pragma unroll
          for (int j = 0; j < kPer; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][gd * kPer + j][e] *= by;
          oz[r][gd][0] *= by;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // no infinity, which an exponential of zero would make a NaN
              const float v = vs[gd][i][e] * unit[r][gd];
              sv[gd][i][e] = y[r][i][e] == -__builtin_inff() ? 0.f : v > 0x1p127f ? 0x1p127f : v;
            }
        }
      }
#pragma unroll
      for (int gd = 0; gd < kGd; ++gd) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const _Float16 hi = (_Float16)w[gd][i][e];
            pf[r][gd][4 * i + e] = hi;
            if constexpr (kTwice) pl[r][gd][4 * i + e] = (_Float16)(w[gd][i][e] - (float)hi);
          }
      }
    }
    // values: rows = channels, columns = query rows
#pragma unroll
    for (int gd = 0; gd < kGd; ++gd) {
      const v8h z = __builtin_bit_cast(v8h, v4i{(int)zf[gd][0][0], (int)zf[gd][0][1], (int)zf[gd][1][0], (int)zf[gd][1][1]});
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        oz[r][gd] = __builtin_amdgcn_mfma_f32_16x16x32_f16(z, pf[r][gd], oz[r][gd], 0, 0, 0);
        if constexpr (kTwice) oz[r][gd] = __builtin_amdgcn_mfma_f32_16x16x32_f16(z, pl[r][gd], oz[r][gd], 0, 0, 0);
      }
      constexpr int kHalves = D == 64 ? 1 : 2;
#pragma unroll
      for (int half = 0; half < kHalves; ++half) {
        u32 x[4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const u32 sel = D == 64 ? ((c & 1) ? 0x07060302u : 0x05040100u) : half ? 0x07060302u : 0x05040100u;
            x[2 * i + e] = __builtin_amdgcn_perm((u32)vc[i][gd][2 * e + 1], (u32)vc[i][gd][2 * e], sel);
          }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v4i vf;
#pragma unroll
          for (int e = 0; e < 4; ++e) vf[e] = (int)((j == 0 ? x[e] << 4 : x[e] >> (4 * (j - 1))) & kNibbles);
          const int td = 8 * gd + 4 * half + j;
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            o[r][td] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, vf), pf[r][gd], o[r][td], 0, 0, 0);
            if constexpr (kTwice)
              o[r][td] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, vf), pl[r][gd], o[r][td], 0, 0, 0);
          }
        }
      }
    }
    load_values(u + NW);
    fetch_ids(u + 2 * NW);
  }

  // ---- join the waves: the smallest sh of each row, sums, outputs in its unit -------
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const float sum = sum16(l[r]);
    if (g == 0) {
      stat[wave][16 * r + c][0] = sh[r];
      stat[wave][16 * r + c][1] = sum;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    float low = kUnset, sum = 0.f;
#pragma unroll
    for (int v = 0; v < NW; ++v) low = fminf(low, stat[v][16 * r + c][0]);
#pragma unroll
    for (int v = 0; v < NW; ++v)
      sum += stat[v][16 * r + c][1] * __builtin_amdgcn_exp2f(low - stat[v][16 * r + c][0]);
    const float mine = __builtin_amdgcn_exp2f(low - sh[r]);
    const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
#pragma unroll
    for (int gd = 0; gd < kGd; ++gd) {
      const float f = mine * inv, back = 1.f / unit[r][gd];   // unit: a power of two
      constexpr int kPer = kTd / kGd;
      if (r || gd) __syncthreads();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // channel row 4 g + e of the tiles: channels 8 (4 g + e) + j, or of 64 channels
        // 8 ((4 g + e) / 2) + 4 ((4 g + e) % 2) + j
        float* const to = &red[wave][c][kPer * (4 * g + e)];
#pragma unroll
        for (int j = 0; j < kPer; j += 4) {
          v4f x;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x[k] = (o[r][gd * kPer + j + k][e] - oz[r][gd][0]) * 0x1p20f * f * back;
          *(v4f*)(to + j) = x;
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 16 * kCols / 8; i += 64 * NW) {
        const int row = i / (kCols / 8), col = 8 * (i % (kCols / 8));
        if (16 * r + row >= rows) continue;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = red[0][row][col + e];
#pragma unroll
          for (int v = 1; v < NW; ++v) x[e] += red[v][row][col + e];
        }
        const int d = kCols * gd + col;
        if (p.splits > 1) {
          float* const to = p.part_o + (((int64_t)th * p.splits + split) * kRows + 16 * r + row) * D + d;
          *(v4f*)to = v4f{x[0], x[1], x[2], x[3]};
          *(v4f*)(to + 4) = v4f{x[4], x[5], x[6], x[7]};
        } else {
          const int qr = t.row0 + 16 * r + row, token = p.by.G(qr);
          kv4_store8<DT>(p.a.out, ((int64_t)(t.token0 + token) * p.a.Hq + h * p.G + qr - token * p.G) * D + d, x);
        }
      }
    }
    if (p.splits > 1 && wave == 0 && g == 0) {
      float* const to = p.part_ml + (((int64_t)th * p.splits + split) * kRows + 16 * r + c) * 2;
      to[0] = low;
      to[1] = sum;
    }
  }
}

// Join the splits of a tile, by their shares in the sum.  SUB lanes take the splits
// of 8 channels of a row in turn, so that their loads are under way together.
template <int DT, int D, int ROWS, int SUB>
__global__ __launch_bounds__(256) void k_kv4_attend_join(Kv4FewArgs p, int rows_most, Kv4Div parts) {
  const int th = parts((int)blockIdx.x), part = blockIdx.x - th * parts.d;
  const int tile_n = p.by.H(th), h = th - tile_n * p.s.H;
  const Kv4Tile t = kv4_tile<ROWS>(p.s, p.by, p.min_rows, p.max_rows, tile_n);
  if (t.b < 0) return;
  const int rows = min(t.n * p.G - t.row0, rows_most);
  const int item = part * (256 / SUB) + (int)threadIdx.x / SUB, sub = threadIdx.x & (SUB - 1);
  // neighbouring threads have neighbours of the parts
  constexpr bool kMany = ROWS == kKv4ManyRows;
  const int row = kMany ? item / (4 * D) * 32 + (item & 31) : item / (D / 8);
  const int chunk = kMany ? (item >> 5) % (D / 8) : item % (D / 8), d = 8 * chunk;
  if (row >= rows) return;   // the lanes of an item alike
  const float* const ml = p.part_ml + ((int64_t)th * p.splits * ROWS + row) * 2;
  const float* const po = p.part_o + (int64_t)th * p.splits * ROWS * D +
                          (kMany ? (row >> 5) * 32 * D + 32 * d + 8 * (row & 31) : row * D + d);
  // The lane's first splits stay while the sums are joined, the others come kMore at a time,
  // so that their loads are under way together (one request of 65536 positions and one kv head
  // of 128, 256 splits: 19 us, one at a time 23).
  constexpr int kFirst = SUB == 4 ? 4 : 2, kMore = 4;
  const auto sums = [&](int v) QG_INLINE { return *(const v2f*)(ml + (int64_t)min(v, p.splits - 1) * ROWS * 2); };
  const auto outputs = [&](int v, int half) QG_INLINE {
    return *(const v4f*)(po + (int64_t)min(v, p.splits - 1) * ROWS * D + 4 * half);
  };
  v2f two[kFirst];
  v4f a[kFirst], b[kFirst];
#pragma unroll
  for (int i = 0; i < kFirst; ++i) {
    two[i] = sums(sub + i * SUB);
    a[i] = outputs(sub + i * SUB, 0);
    b[i] = outputs(sub + i * SUB, 1);
  }
  float low = kUnset, l = 0.f, x[8];
  const auto join = [&](float sh, float sum) QG_INLINE {
    const float to = fminf(low, sh);
    l = l * __builtin_amdgcn_exp2f(to - low) + sum * __builtin_amdgcn_exp2f(to - sh);
    low = to;
  };
#pragma unroll
  for (int i = 0; i < kFirst; ++i)
    if (sub + i * SUB < p.splits) join(two[i][0], two[i][1]);
  for (int v = sub + kFirst * SUB; v < p.splits; v += kMore * SUB) {
    v2f t[kMore];
#pragma unroll
    for (int i = 0; i < kMore; ++i) t[i] = sums(v + i * SUB);
#pragma unroll
    for (int i = 0; i < kMore; ++i)
      if (v + i * SUB < p.splits) join(t[i][0], t[i][1]);
  }
#pragma unroll
  for (int o = 1; o < SUB; o <<= 1) join(__shfl_xor(low, o, kWave), __shfl_xor(l, o, kWave));
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 0.f;
  const auto add = [&](int v, const v2f& t, const v4f& a, const v4f& b) QG_INLINE {
    // no steps, or nothing in the row's sight: no outputs there.  Scores that are all NaN
    // leave sh unset too, and their sum NaN.
    if (v >= p.splits || (t[0] == kUnset && t[1] == 0.f)) return;
    const float f = t[1] * __builtin_amdgcn_exp2f(low - t[0]) * inv;   // 1 at most
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] += a[e] * f;
      x[4 + e] += b[e] * f;
    }
  };
#pragma unroll
  for (int i = 0; i < kFirst; ++i) add(sub + i * SUB, two[i], a[i], b[i]);
  for (int v = sub + kFirst * SUB; v < p.splits; v += kMore * SUB) {
    v2f t[kMore];
    v4f a2[kMore], b2[kMore];
#pragma unroll
    for (int i = 0; i < kMore; ++i) {
      t[i] = sums(v + i * SUB);
      a2[i] = outputs(v + i * SUB, 0);
      b2[i] = outputs(v + i * SUB, 1);
    }
#pragma unroll
    for (int i = 0; i < kMore; ++i) add(v + i * SUB, t[i], a2[i], b2[i]);
  }
#pragma unroll
  for (int o = 1; o < SUB; o <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] += __shfl_xor(x[e], o, kWave);
  if (sub != 0) return;
  const int qr = t.row0 + row, token = p.by.G(qr);
  kv4_store8<DT>(p.a.out, ((int64_t)(t.token0 + token) * p.a.Hq + h * p.G + qr - token * p.G) * D + d, x);
}

// ---- launch -------------------------------------------------------------------

namespace {

// Sequences of up to kFewRows rows are this file's, longer ones the prompt
// kernel's.  Without offsets the call's sequences are alike; with them the GPU
// tells, so that both kernels are launched where either may have some.  With 64 rows
// this kernel is never the slower one (heads of 128, us, this kernel and the other: one
// request of 8192 positions and 8 kv heads 16 and 26, 32 of 4096 positions 107 and 107),
// with 192 it is from 32 requests times kv heads on (4 of 4096 and 8 kv heads 47 and 39, 32
// kv heads 149 and 79).  With 128 it goes by the call: one of 2048 positions 14 and 25, 4
// of 4096 with 8 kv heads 36 and 34, with 32 104 and 68.
constexpr int64_t kFewRows = 128;

// With offsets, sequences of few rows among longer ones have whole tiles of the
// prompt kernel where the tiles find room side by side and no row sees more than
// this: the second kernel and its join cost more.  A chunk of 1500 tokens and two
// tokens of two other requests, 16 heads, a window of 2048 positions: 53 us, with both
// kernels 70.  A prompt beside 1 to 19 single tokens that see 512 to 4096 positions, 32
// heads on 8: up to 29% less (650 tokens at the end of 4096 positions and 19 single ones
// 130 and 184), but where the prompt is short and the single ones many and long, which
// the host cannot tell (300 tokens by themselves and 8 single ones of 4096 positions 63 and
// 54, the worst of those measured 104 and 84).
constexpr int64_t kOneSight = 4096;

struct AttendPlan {
  int64_t few_tiles, many_tiles;   // tiles of a kv head, 0: no launch
  int few_rows;                    // rows of a tile of the former
  int few_splits, many_splits;     // of the cached positions
  int64_t few_part, many_part;     // floats of their parts
  bool one;                        // the latter's sequences may be of any length
  bool fits;
};

AttendPlan attend_plan(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t capacity, bool uniform) {
  AttendPlan a = {};
  const int64_t G = Hq / H, rows = T * G;
  const auto up = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  const bool wide = D == 256;   // all rows here
  const bool long_ones = rows / B > kFewRows;   // on average
  a.one = !uniform && !wide && long_ones && capacity <= kOneSight && (rows / kKv4ManyRows + B) * H <= 256;
  const bool few = wide || !(uniform ? long_ones : a.one), many = !wide && (uniform ? long_ones : rows > kFewRows);
  if (few) {
    // 32 rows a tile where that makes one tile of two, on average: 64 requests of 4 tokens
    // of 8 query heads a kv head and 8192 positions 180 us, with 16 rows 192; 8 tokens each
    // of 8 requests 37 and 36, 5 tokens of one of 16384 positions 13.7 and 12.5.
    a.few_rows = D < 256 && rows > 16 * B && rows <= 32 * B ? 32 : 16;
    if (uniform) a.few_tiles = B * up(rows / B, a.few_rows);
    else a.few_tiles = std::min(std::min(rows, rows / a.few_rows + B), wide ? rows : B * up(kFewRows, a.few_rows));
    // Splits of the cached positions.  A workgroup on each CU, of 256 positions or more
    // (one request's 4096 positions of 32 heads in 8 parts: 13 us, whole 28; 8 requests of
    // 2047 and 2 heads in parts of 256 12 us, of 512 14); four on each where that leaves
    // 2048 positions or more, for sequences of uneven lengths (64 of up to 16384: 131 us,
    // without 154).  Joining costs some 4 us of it.
    const int64_t all = a.few_tiles * H;
    a.few_splits = (int)std::max<int64_t>({1, std::min(up(256, all), capacity / 256), std::min(up(2048, all), capacity / 2048)});
    a.few_part = a.few_splits > 1 ? all * a.few_splits * a.few_rows * (D + 2) : 0;
  }
  if (many) {
    a.many_tiles = uniform ? B * up(rows / B, kKv4ManyRows) : rows / kKv4ManyRows + (a.one ? B : std::min(B, rows / (kFewRows + 1)));
    const int64_t all = a.many_tiles * H;
    // a workgroup on each CU, of 512 positions or more (a chunk of 1500 tokens of 16 heads,
    // a window of 2048 positions: 60 us in two parts, 83 whole)
    a.many_splits = (int)std::max<int64_t>(1, std::min(256 / all, capacity / 512));
    a.many_part = a.many_splits > 1 ? all * a.many_splits * kKv4ManyRows * (D + 2) : 0;
  }
  // a launch holds fewer than 2^32 threads; a join has up to 16 for 8 channels of a row
  const auto fits = [&](int64_t tiles, int splits, int64_t threads, int64_t joins) {
    return tiles * H * std::max<int64_t>(splits * threads, splits > 1 ? joins * (D / 8) + 256 : 0) < (int64_t)1 << 32;
  };
  a.fits = fits(a.few_tiles, std::max(a.few_splits, 1), 64 * kAttnWaves, 16 * a.few_rows) &&
           fits(a.many_tiles, std::max(a.many_splits, 1), 2 * kKv4ManyRows, 4 * kKv4ManyRows);
  return a;
}

}  // namespace

int64_t kv4_attend_workspace(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t D,
                             int64_t capacity, bool uniform) {
  // A call's window may let its rows see less, which leaves fewer splits and may leave one kernel.
  const AttendPlan a = attend_plan(T, B, Hq, H, D, capacity, uniform);
  const AttendPlan b = attend_plan(T, B, Hq, H, D, std::min(capacity, kOneSight), uniform);
  if (!a.fits || !b.fits) return -1;
  return std::max({a.few_part, a.many_part, b.few_part, b.many_part}) * 4;   // one kernel after the other
}

template <int DT, int D, int ROWS, int SUB>
static void join_t(const Kv4FewArgs& p, int64_t tiles, hipStream_t st) {
  // workgroups of 256 / SUB items of 8 channels; without offsets the rows of a tile are known
  const int64_t rows = p.s.offsets == nullptr ? std::min<int64_t>(ROWS, (int64_t)p.by.n * p.G) : ROWS;
  const Kv4Div parts = kv4_div(((ROWS == kKv4ManyRows ? (rows + 31) / 32 * 32 : rows) * (D / 8) * SUB + 255) / 256);
  k_kv4_attend_join<DT, D, ROWS, SUB><<<(unsigned)(tiles * parts.d), 256, 0, st>>>(p, (int)rows, parts);
}

// A thread takes up to 4 splits by itself (2 splits of 6000 rows: 7 us, with 4 lanes
// to each item 14), more are shared out.
template <int DT, int D>
static void join_many(const Kv4FewArgs& p, int64_t tiles, hipStream_t st) {
  if (p.splits <= 4) join_t<DT, D, kKv4ManyRows, 1>(p, tiles, st);
  else join_t<DT, D, kKv4ManyRows, 4>(p, tiles, st);
}

template <int DT, int D, int RT>
static hipError_t few_t(Kv4FewArgs p, int64_t tiles, int64_t sight, hipStream_t st) {
  const unsigned grid = (unsigned)(tiles * p.splits);
  const bool once = p.by.n > 0 && (int64_t)p.by.n * p.G <= 16 * RT;
  if constexpr (RT == 1 && D < 256) {
    // With a workgroup or less on each CU and a long way to go, two waves on each SIMD
    // (32 requests of 8 kv heads, a window of 1024 positions 13.4 us, with four waves 16.2;
    // 16 of 4096 positions 20.4 and 23.8).  Short ways and joins lose by it (5 drafted
    // tokens of 8 requests of 2047 positions 12.9 and 11.6), and with more workgroups two
    // waves are there already (64 requests of up to 16384 positions 153 and 131).
    if (grid <= 256 && sight / p.splits >= 1024) {
      if (once) k_kv4_attend_few<DT, D, RT, true, kAttnWavesLong><<<grid, 64 * kAttnWavesLong, 0, st>>>(p);
      else k_kv4_attend_few<DT, D, RT, false, kAttnWavesLong><<<grid, 64 * kAttnWavesLong, 0, st>>>(p);
      if (p.splits > 1) join_t<DT, D, 16 * RT, 16>(p, tiles, st);
      return hipGetLastError();
    }
  }
  if (once) k_kv4_attend_few<DT, D, RT, true><<<grid, 64 * kAttnWaves, 0, st>>>(p);
  else k_kv4_attend_few<DT, D, RT, false><<<grid, 64 * kAttnWaves, 0, st>>>(p);
  if (p.splits > 1) join_t<DT, D, 16 * RT, 16>(p, tiles, st);
  return hipGetLastError();
}

template <int DT>
static hipError_t few_d(const Kv4FewArgs& p, int D, int rows, int64_t tiles, int64_t sight, hipStream_t st) {
  if (D == 256) return few_t<DT, 256, 1>(p, tiles, sight, st);
  if (rows == 16) return D == 64 ? few_t<DT, 64, 1>(p, tiles, sight, st) : few_t<DT, 128, 1>(p, tiles, sight, st);
  return D == 64 ? few_t<DT, 64, 2>(p, tiles, sight, st) : few_t<DT, 128, 2>(p, tiles, sight, st);
}

hipError_t launch_kv4_attend(const Kv4Seqs& s, const Kv4Attend& a, int dtype, hipStream_t st) {
  // A window bounds what the rows of a sequence see: fewer splits than the workspace is for.
  const int64_t capacity = (int64_t)s.W << s.shift;
  const int64_t seen = a.window > 0 ? std::min<int64_t>(capacity, (int64_t)a.window + a.sinks + kFewRows + 2 * kStep) : capacity;
  const AttendPlan plan = attend_plan(s.T, s.B, a.Hq, s.H, a.D, seen, s.offsets == nullptr);
  Kv4FewArgs p;
  p.s = s;
  p.a = a;
  p.G = a.Hq / s.H;
  p.part_o = (float*)a.workspace;
  if (plan.many_tiles > 0) {
    const int64_t tiles = plan.many_tiles * s.H;
    p.min_rows = s.offsets == nullptr || plan.one ? 1 : kFewRows + 1;
    p.max_rows = (int64_t)1 << 40;
    p.splits = plan.many_splits;
    p.part_ml = p.part_o + tiles * p.splits * kKv4ManyRows * a.D;
    hipError_t e = launch_kv4_many(s, a, dtype, p.min_rows, plan.many_tiles, p.splits, p.part_o, p.part_ml, st);
    if (e == hipSuccess && p.splits > 1) {
      p.by = kv4_divs(s, p.G, kKv4ManyRows);
      if (dtype == F16) a.D == 64 ? join_many<F16, 64>(p, tiles, st) : join_many<F16, 128>(p, tiles, st);
      else a.D == 64 ? join_many<BF16, 64>(p, tiles, st) : join_many<BF16, 128>(p, tiles, st);
      e = hipGetLastError();
    }
    if (e != hipSuccess || plan.few_tiles == 0) return e;
  }
  p.min_rows = 1;
  p.max_rows = s.offsets != nullptr && a.D < 256 ? kFewRows : (int64_t)1 << 40;
  p.splits = plan.few_splits;
  p.by = kv4_divs(s, p.G, plan.few_rows);
  p.by_splits = kv4_div(p.splits);
  const int64_t tiles = plan.few_tiles * s.H;
  p.part_ml = p.part_o + tiles * p.splits * plan.few_rows * a.D;
  return dtype == F16 ? few_d<F16>(p, a.D, plan.few_rows, tiles, seen, st)
                      : few_d<BF16>(p, a.D, plan.few_rows, tiles, seen, st);
}

}  // namespace qg
