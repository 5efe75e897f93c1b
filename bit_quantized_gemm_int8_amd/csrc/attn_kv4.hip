// Attention of a few query rows over the 4-bit paged KV cache (qg_kv4.hpp).
//
//   x_t = scale (q . k_t),  o = sum_t exp(x_t) v_t / sum_t exp(x_t)
// with k_t = (n_t - z_t) s_t and v_t alike, over the positions a row can see.
// The codes n go to the matrix cores as they are:
//   q . k_t = s_t (sum_d q_d n_td - z_t sum_d q_d)
//   o       = (sum_t (p_t s_t) n_t - sum_t (p_t s_t) z_t) / sum_t p_t
// A nibble masked out of a code word is a binary16 subnormal, n 2^-24 (or
// n 2^-20 one nibble up), which gfx950's matrix cores take exactly: unpacking
// costs one AND for two codes.  Queries are scaled to binary16's upper range by
// a power of two of their row, exactly for bfloat16 and binary16 inputs; the
// weights p s are scaled by a power of two of their row and rounded to binary16
// (half a step: 2^-11), the codes' sum and the zero points' sum taking the same
// rounded weights, both through the matrix cores.  Softmax and sums: binary32.
//
// Layout.  A wave takes 32 positions a step: the scores' product has positions
// as rows and query rows as columns, so that a lane holds 4 neighbouring
// positions of one query row for each half of the step -- which is the operand
// the second product needs, with the positions in that order.  Value codes of 4
// positions of a word are neighbours in the cache for the same reason.  No
// lane exchange per step: the running maximum is a bound that is raised only
// where a score passes it by 2^8.
#include "qg_kv4_attn.hpp"

#include <algorithm>

namespace qg {

namespace {

constexpr int kStep = 32;            // positions of a wave's step
constexpr int kAttnWaves = 4;
constexpr float kLowest = -3.402823466e38f;

typedef int v2i __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float max16(float v) {   // over the four lanes of one column
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
}
__device__ __forceinline__ float sum16(float v) {
  v += __shfl_xor(v, 16, kWave);
  return v + __shfl_xor(v, 32, kWave);
}

// One step's codes and group words, as a lane holds them.
template <int D>
struct Kv4Step {
  static constexpr int kGd = kv4_groups(D), kKw = D / 32;   // key words of a position
  int k[2][kKw];
  v4i v[2][kGd];
  v4i kp[2][kGd], vp[2][kGd];
};

}  // namespace

// Workspace of a call with several splits: outputs [tile][split][row][D] and
// (maximum, sum) [tile][split][row], binary32, where tile counts row tiles
// times kv heads.

template <int DT, int D, int RT>
struct Kv4Few {
  static constexpr int kRows = 16 * RT, kGd = kv4_groups(D), kKw = D / 32, kTd = D / 16;
  typedef Kv4Step<D> Step;

  // uniform
  Kv4Seqs s;
  const int32_t* table;   // the sequence's
  int h, page_words, window, sinks, capacity;
  int p0, p1;             // positions of the tile's first and last row
  Kv4Span span;
  // per lane
  int c, g;
  u32 off_k, off_v, off_p;
  int pos[RT];            // position of the lane's query row
  v8h q[RT][kKw];
  float cc[RT], qs[RT][kGd];
  v4f o[RT][kTd], oz[RT][kGd];
  float m[RT], l[RT], rinv[RT][kGd], lim[RT][kGd];

  // Pages of the two halves of cache tile `tile` (-1: none).
  __device__ __forceinline__ void ids(int tile, int (&id)[2]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int pi = (tile * kStep + 16 * i) >> s.shift;
      int v = -1;
      if (pi < s.W) v = table[pi];
      v = __builtin_amdgcn_readfirstlane(v);
      id[i] = (u32)v < (u32)s.P ? v : -1;
    }
  }

  __device__ __forceinline__ void load(int tile, const int (&id)[2], Step& t) const {
    const int S = 1 << s.shift;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int slot = (tile * kStep + 16 * i) & (S - 1);
      const char* page = (const char*)(s.pages + ((int64_t)max(id[i], 0) * s.H + h) * page_words);
      const char* kb = page + slot * (D / 2);
      const char* vb = kb + S * (D / 2);
      const char* pb = page + S * D + slot * 4;
#pragma unroll
      for (int gd = 0; gd < kGd; ++gd) {
        if constexpr (D == 64) {
          const v2i a = *(const v2i*)(kb + off_k);
          t.k[i][0] = a[0];
          t.k[i][1] = a[1];
        } else {
          const v4i a = ld16(kb + off_k + 64 * gd);
#pragma unroll
          for (int j = 0; j < 4; ++j) t.k[i][4 * gd + j] = a[j];
        }
        t.v[i][gd] = ld16(vb + off_v + 256 * gd);
        t.kp[i][gd] = ld16(pb + off_p + gd * 4 * S);
        t.vp[i][gd] = ld16(pb + off_p + (kGd + gd) * 4 * S);
      }
    }
  }

  __device__ __forceinline__ void start() {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
      for (int j = 0; j < kTd; ++j) o[r][j] = v4f{0.f, 0.f, 0.f, 0.f};
      m[r] = kLowest;
      l[r] = 0.f;
#pragma unroll
      for (int gd = 0; gd < kGd; ++gd) {
        oz[r][gd] = v4f{0.f, 0.f, 0.f, 0.f};
        rinv[r][gd] = 0.f;
        lim[r][gd] = 0.f;
      }
    }
  }

  // A query row: its lane's words in the order of the unpacked codes (nibbles
  // 0 4 1 5 2 6 3 7, the second of each byte 16 times as large), their sum.
  __device__ __forceinline__ void query(int r, const void* base, int64_t at, bool there, float scale) {
    float x[kKw][8];
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < kKw; ++j) {
      const int d = D == 64 ? 16 * g + 8 * j : 128 * (j / 4) + 32 * g + 8 * (j % 4);
      const v4i a = there ? ld16((const uint16_t*)base + at + d) : v4i{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const u32 u = ((u32)a[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
        x[j][e] = DT == BF16 ? bf16_bits_to_f32(u) : f16_bits_to_f32((uint16_t)u);
        top = fmaxf(top, fabsf(x[j][e]));
      }
    }
    top = max16(top);
    // top 2^e in [2^14, 2^15); not for zero rows and infinities
    const int e = top > 0.f && top < __builtin_inff() ? 14 - (ilogbf(top)) : 0;
#pragma unroll
    for (int gd = 0; gd < kGd; ++gd) qs[r][gd] = 0.f;
#pragma unroll
    for (int j = 0; j < kKw; ++j) {
      constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};
      v8h w;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = ldexpf(x[j][order[i]], e);
        sum += v;
        w[i] = (_Float16)((i & 2) ? v * 0.0625f : v);
      }
      q[r][j] = w;
      qs[r][j / 4] += sum;
    }
    // scores in units of 2^(e - 24), exponents in base 2
#pragma unroll
    for (int gd = 0; gd < kGd; ++gd) qs[r][gd] = sum16(qs[r][gd]) * 0x1p-24f;
    cc[r] = ldexpf(scale * 1.44269504088896f, 24 - e);
  }

  // One step.  EDGE: some position is out of some row's sight.
  template <bool EDGE>
  __device__ __forceinline__ void step(int tile, const int (&id)[2], const Step& t) {
    // scores: rows = positions, columns = query rows
    float y[RT][2][4];
    float sv[kGd][2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v8h kf[kKw];
#pragma unroll
      for (int j = 0; j < kKw; ++j) {
        const u32 w = (u32)t.k[i][j], hi = w >> 8;
        kf[j] = __builtin_bit_cast(v8h, v4i{(int)(w & 0x000F000Fu), (int)(w & 0x00F000F0u),
                                            (int)(hi & 0x000F000Fu), (int)(hi & 0x00F000F0u)});
      }
#pragma unroll
      for (int gd = 0; gd < kGd; ++gd)
#pragma unroll
        for (int e = 0; e < 4; ++e) sv[gd][i][e] = kv4_scale((u32)t.vp[i][gd][e]);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
#pragma unroll
        for (int gd = 0; gd < kGd; ++gd) {
          constexpr int kPer = kKw / kGd;
          v4f a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            a = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[kPer * gd + j], q[r][kPer * gd + j], a, 0, 0, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const u32 w = (u32)t.kp[i][gd][e];
            const float u = __builtin_fmaf(-(float)(w & 15u), qs[r][gd], a[e]) * kv4_scale(w);
            y[r][i][e] = gd ? y[r][i][e] + u : u;
          }
        }
        if constexpr (EDGE) {
          const int t0 = tile * kStep + 16 * i + 4 * g;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int p = t0 + e;
            const bool seen = id[i] >= 0 && p <= pos[r] && p < capacity &&
                              (window <= 0 || p > pos[r] - window || p < sinks);
            if (!seen) y[r][i][e] = -__builtin_inff();
          }
        }
      }
    }
    // weights
    v8h pf[RT][kGd];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float top = kLowest;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[r][i][e] = EDGE && y[r][i][e] == -__builtin_inff() ? -__builtin_inff() : y[r][i][e] * cc[r];
          top = fmaxf(top, y[r][i][e]);
        }
      float alpha = 1.f;
      if (__any(top > m[r] + 8.f)) {   // the bound rises: all lanes of a column agree
        const float mn = fmaxf(m[r], max16(top));
        alpha = __builtin_amdgcn_exp2f(m[r] - mn);
        m[r] = mn;
        l[r] *= alpha;
#pragma unroll
        for (int gd = 0; gd < kGd; ++gd) lim[r][gd] = -1.f;
      }
      float p[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[i][e] = __builtin_amdgcn_exp2f(y[r][i][e] - m[r]);
          l[r] += p[i][e];
        }
#pragma unroll
      for (int gd = 0; gd < kGd; ++gd) {
        float w[2][4], most = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[i][e] = p[i][e] * sv[gd][i][e];
            if (EDGE && y[r][i][e] == -__builtin_inff()) w[i][e] = 0.f;   // whatever scale lies there
            most = fmaxf(most, w[i][e]);
          }
        if (__any(most > lim[r][gd])) {   // another power of two for the row's weights
          const bool set = rinv[r][gd] > 0.f;
          const float ref = set ? alpha / rinv[r][gd] : 0.f;
          const float big = fminf(fmaxf(fmaxf(max16(most), ref), 0x1p-100f), 0x1p100f);
          const float f = __uint_as_float(0x7F000000u - (__float_as_uint(big) & 0x7F800000u));  // 2^-floor(log2 big)
          const bool some = fmaxf(max16(most), ref) > 0.f;
          const float by = set ? f * ref : 1.f;
          rinv[r][gd] = some ? f : 0.f;
          lim[r][gd] = some ? 0x1p12f / f : 0.f;
          float rows[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) rows[e] = __shfl(by, 4 * g + e, kWave);
#pragma unroll
          for (int j = 0; j < kTd / kGd; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][gd * (kTd / kGd) + j][e] *= rows[e];
#pragma unroll
          for (int e = 0; e < 4; ++e) oz[r][gd][e] *= rows[e];
        }
        v8h pk;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) pk[4 * i + e] = (_Float16)(w[i][e] * rinv[r][gd]);
        pf[r][gd] = pk;
      }
    }
    // values: rows = query rows, columns = channels, 8 c + j of the lane's word
#pragma unroll
    for (int gd = 0; gd < kGd; ++gd) {
      v4i zf;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          zf[2 * i + e] = (int)(((u32)t.vp[i][gd][2 * e] & 15u) | (((u32)t.vp[i][gd][2 * e + 1] & 15u) << 16));
#pragma unroll
      for (int r = 0; r < RT; ++r)
        oz[r][gd] = __builtin_amdgcn_mfma_f32_16x16x32_f16(pf[r][gd], __builtin_bit_cast(v8h, zf), oz[r][gd], 0, 0, 0);
      constexpr int kHalves = D == 64 ? 1 : 2;
#pragma unroll
      for (int half = 0; half < kHalves; ++half) {
        u32 x[4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const u32 sel = D == 64 ? ((c & 1) ? 0x07060302u : 0x05040100u) : half ? 0x07060302u : 0x05040100u;
            x[2 * i + e] = __builtin_amdgcn_perm((u32)t.v[i][gd][2 * e + 1], (u32)t.v[i][gd][2 * e], sel);
          }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32 mask = (j & 1) ? 0x00F000F0u : 0x000F000Fu;
          v4i vf;
#pragma unroll
          for (int e = 0; e < 4; ++e) vf[e] = (int)((j & 2 ? x[e] >> 8 : x[e]) & mask);
          const int td = 8 * gd + 4 * half + j;
#pragma unroll
          for (int r = 0; r < RT; ++r)
            o[r][td] = __builtin_amdgcn_mfma_f32_16x16x32_f16(pf[r][gd], __builtin_bit_cast(v8h, vf), o[r][td], 0, 0, 0);
        }
      }
    }
  }

  __device__ __forceinline__ void run_step(int tile, const int (&id)[2], const Step& t) {
    const int a = tile * kStep;
    const bool full = id[0] >= 0 && id[1] >= 0 && a + kStep - 1 <= p0 && a + kStep <= capacity &&
                      (window <= 0 || a > p1 - window || a + kStep <= sinks);
    if (full) step<false>(tile, id, t);
    else step<true>(tile, id, t);
  }

  // Steps u, u + stride, ... below end, the next one's loads ahead of each.
  __device__ __forceinline__ void run(int u, int end, int stride) {
    if (u >= end) return;
    Step a, b;
    int ia[2], ib[2];
    ids(span.tile(u), ia);
    load(span.tile(u), ia, a);
    while (true) {
      const int ub = min(u + stride, end - 1);
      ids(span.tile(ub), ib);
      load(span.tile(ub), ib, b);
      run_step(span.tile(u), ia, a);
      u += stride;
      if (u >= end) break;
      const int ua = min(u + stride, end - 1);
      ids(span.tile(ua), ia);
      load(span.tile(ua), ia, a);
      run_step(span.tile(u), ib, b);
      u += stride;
      if (u >= end) break;
    }
  }
};

struct Kv4FewArgs {
  Kv4Seqs s;
  Kv4Attend a;
  int G, splits;
  int64_t max_rows;   // sequences of more rows are another kernel's
  float* part_o;
  float* part_ml;
};

// Steps of split `split` of a tile with `tiles` steps.
__device__ __forceinline__ int kv4_per_split(int tiles, int splits) {
  return max((tiles + splits - 1) / splits, kAttnWaves);
}

// What both kernels below derive from a workgroup's tile.
template <int ROWS>
__device__ __forceinline__ void kv4_positions(const Kv4FewArgs& p, const Kv4Tile& t, int& p0, int& p1,
                                              int& len, int& rows) {
  rows = min(t.n * p.G - t.row0, ROWS);
  len = min(p.s.lengths[t.b], 0x3FFFFFFF);
  const int first = max(len, -0x3FFFFFFF) - t.n;   // n <= 2^30: no overflow
  len = first;
  p0 = first + t.row0 / p.G;
  p1 = first + (t.row0 + rows - 1) / p.G;
}

template <int DT, int D, int RT>
__global__ __launch_bounds__(64 * kAttnWaves) void k_kv4_attend_few(Kv4FewArgs p) {
  typedef Kv4Few<DT, D, RT> W;
  constexpr int kRows = W::kRows, kTd = W::kTd;
  // outputs of three waves, 16 rows and up to 128 channels at a time
  constexpr int kCols = D < 128 ? D : 128;
  __shared__ float red[kAttnWaves][16][kCols + 4];
  __shared__ float stat[kAttnWaves][kRows][2];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int split = blockIdx.x % p.splits;
  const int th = blockIdx.x / p.splits;
  const int h = th % p.s.H;
  const Kv4Tile t = kv4_tile<kRows>(p.s, p.G, 1, p.max_rows, th / p.s.H);
  if (t.b < 0) return;
  W w;
  int first, rows;
  kv4_positions<kRows>(p, t, w.p0, w.p1, first, rows);
  w.s = p.s;
  w.h = h;
  w.table = p.s.table + (int64_t)t.b * p.s.W;
  w.page_words = (int)kv4_words(1 << p.s.shift, D);
  w.window = p.a.window;
  w.sinks = p.a.sinks;
  w.capacity = (int)min((int64_t)p.s.W << p.s.shift, (int64_t)0x40000000);
  w.span = kv4_span<kStep>(w.p0, w.p1, w.window, w.sinks, w.capacity);
  const int per = kv4_per_split(w.span.tiles, p.splits);
  const int u0 = split * per, u1 = min(u0 + per, w.span.tiles);
  if (u0 >= u1 && (p.splits > 1 || split > 0)) return;   // a split without steps: the join leaves it out
  w.c = lane & 15;
  w.g = lane >> 4;
  w.off_k = w.c * (D / 2) + w.g * (D == 64 ? 8 : 16);
  w.off_v = (w.g * (D / 8) + (D == 64 ? w.c >> 1 : w.c)) * 16;
  w.off_p = 16 * w.g;
  w.start();
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = t.row0 + 16 * r + w.c;
    const bool there = 16 * r + w.c < rows;
    w.pos[r] = there ? first + row / p.G : kKv4Past;
    w.query(r, p.a.q, (int64_t)(t.token0 + row / p.G) * p.a.q_stride + (int64_t)(h * p.G + row % p.G) * D,
            there, p.a.scale);
  }
  w.run(u0 + wave, u1, kAttnWaves);

  // Join the waves: maximum and sum of each row, then the outputs in common units.
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const float l = sum16(w.l[r]);
    if (w.g == 0) {
      stat[wave][16 * r + w.c][0] = w.m[r];
      stat[wave][16 * r + w.c][1] = l;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    // the lane's column: its factor to the common maximum and out of the weights' units
    float m = kLowest, l = 0.f;
#pragma unroll
    for (int v = 0; v < kAttnWaves; ++v) m = fmaxf(m, stat[v][16 * r + w.c][0]);
#pragma unroll
    for (int v = 0; v < kAttnWaves; ++v)
      l += stat[v][16 * r + w.c][1] * __builtin_amdgcn_exp2f(stat[v][16 * r + w.c][0] - m);
    const float mine = __builtin_amdgcn_exp2f(w.m[r] - m);
    const float inv = p.splits > 1 ? 1.f : l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
    for (int gd = 0; gd < W::kGd; ++gd) {
      const float back = w.rinv[r][gd] > 0.f ? mine / w.rinv[r][gd] * inv : 0.f;
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = __shfl(back, 4 * w.g + e, kWave);
      constexpr int kPer = kTd / W::kGd;
      if (r || gd) __syncthreads();
#pragma unroll
      for (int j = 0; j < kPer; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = (w.o[r][gd * kPer + j][e] * ((j & 1) ? 0x1p20f : 0x1p24f) - w.oz[r][gd][e] * 0x1p24f) * f[e];
          const int col = D == 64 ? 8 * (w.c >> 1) + 4 * (w.c & 1) + j : 8 * w.c + j;
          red[wave][4 * w.g + e][col] = x;
        }
      __syncthreads();
      for (int i = threadIdx.x; i < 16 * kCols / 8; i += 64 * kAttnWaves) {
        const int row = i / (kCols / 8), col = 8 * (i % (kCols / 8));
        if (16 * r + row >= rows) continue;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = red[0][row][col + e];
#pragma unroll
          for (int v = 1; v < kAttnWaves; ++v) x[e] += red[v][row][col + e];
        }
        const int d = kCols * gd + col;
        if (p.splits > 1) {
          float* to = p.part_o + (((int64_t)th * p.splits + split) * kRows + 16 * r + row) * D + d;
          *(v4f*)to = v4f{x[0], x[1], x[2], x[3]};
          *(v4f*)(to + 4) = v4f{x[4], x[5], x[6], x[7]};
        } else {
          const int qr = t.row0 + 16 * r + row;
          kv4_store8<DT>(p.a.out, ((int64_t)(t.token0 + qr / p.G) * p.a.Hq + h * p.G + qr % p.G) * D + d, x);
        }
      }
    }
    if (p.splits > 1 && wave == 0 && w.g == 0) {
      float* to = p.part_ml + (((int64_t)th * p.splits + split) * kRows + 16 * r + w.c) * 2;
      to[0] = m;
      to[1] = l;
    }
  }
}

// Join the splits of a tile: weights 2^(m_i - m) of each split's outputs and sums.
template <int DT, int D, int ROWS>
__global__ __launch_bounds__(256) void k_kv4_attend_join(Kv4FewArgs p) {
  const int th = blockIdx.x, h = th % p.s.H;
  const Kv4Tile t = kv4_tile<ROWS>(p.s, p.G, 1, p.max_rows, th / p.s.H);
  if (t.b < 0) return;
  int p0, p1, first, rows;
  kv4_positions<ROWS>(p, t, p0, p1, first, rows);
  const int capacity = (int)min((int64_t)p.s.W << p.s.shift, (int64_t)0x40000000);
  const Kv4Span span = kv4_span<kStep>(p0, p1, p.a.window, p.a.sinks, capacity);
  const int per = kv4_per_split(span.tiles, p.splits), used = (span.tiles + per - 1) / per;
  for (int i = threadIdx.x; i < rows * (D / 8); i += 256) {
    const int row = i / (D / 8), d = 8 * (i % (D / 8));
    const float* ml = p.part_ml + ((int64_t)th * p.splits * ROWS + row) * 2;
    const float* po = p.part_o + ((int64_t)th * p.splits * ROWS + row) * D + d;
    float m = kLowest, l = 0.f, x[8];
    for (int v = 0; v < used; ++v) m = fmaxf(m, ml[(int64_t)v * ROWS * 2]);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    for (int v = 0; v < used; ++v) {
      const float f = __builtin_amdgcn_exp2f(ml[(int64_t)v * ROWS * 2] - m);
      l += f * ml[(int64_t)v * ROWS * 2 + 1];
      const v4f a = *(const v4f*)(po + (int64_t)v * ROWS * D), b = *(const v4f*)(po + (int64_t)v * ROWS * D + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] += f * a[e];
        x[4 + e] += f * b[e];
      }
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= inv;
    const int qr = t.row0 + row;
    kv4_store8<DT>(p.a.out, ((int64_t)(t.token0 + qr / p.G) * p.a.Hq + h * p.G + qr % p.G) * D + d, x);
  }
}

// ---- launch -------------------------------------------------------------------

namespace {

// Sequences of up to kFewRows rows are this file's, longer ones the prompt
// kernel's.  Without offsets the call's sequences are alike; with them the GPU
// tells, so that both kernels are launched where either may have some.
constexpr int64_t kFewRows = 64;

struct AttendPlan {
  int64_t few_tiles, many_tiles;   // tiles of a kv head, 0: no launch
  int few_rows, many_rows;         // rows of a tile
  int splits;
  bool fits;
};

AttendPlan attend_plan(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t capacity, bool uniform) {
  AttendPlan a = {};
  const int64_t G = Hq / H, rows = T * G;
  const auto up = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  const auto tiles = [&](int64_t tile, int64_t most) {
    // of sequences with at most `most` rows each, `rows` together
    if (uniform) return B * up(rows / B, tile);
    return std::min(std::min(rows, rows / tile + B), most == 0 ? rows : B * up(most, tile));
  };
  const bool wide = D == 256;   // all rows here
  const bool few = wide || !uniform || rows / B <= kFewRows, many = !wide && (uniform ? !few : rows > kFewRows);
  if (few) {
    // 16 rows a tile where a sequence has no more on average, else 32
    a.few_rows = D < 256 && rows > 16 * B ? 32 : 16;
    a.few_tiles = tiles(a.few_rows, wide ? 0 : kFewRows);
    // splits of the cached positions: enough workgroups for the GPU, at least 256 positions each
    const int64_t want = up(2048, a.few_tiles * H);
    a.splits = (int)std::max<int64_t>(1, std::min(want, capacity / 256));
  }
  if (many) {
    const auto of = [&](int64_t tile) {
      return uniform ? tiles(tile, 0) : rows / tile + std::min(B, rows / (kFewRows + 1));
    };
    a.many_rows = D < 256 && of(256) * H >= 512 ? 256 : 128;
    a.many_tiles = of(a.many_rows);
  }
  // a launch holds fewer than 2^32 threads
  a.fits = a.few_tiles * H * std::max(a.splits, 1) < (int64_t)1 << 24 && a.many_tiles * H < (int64_t)1 << 23;
  return a;
}

}  // namespace

int64_t kv4_attend_workspace(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t D,
                             int64_t capacity, bool uniform) {
  const AttendPlan a = attend_plan(T, B, Hq, H, D, capacity, uniform);
  if (!a.fits) return -1;
  return a.splits > 1 ? a.few_tiles * H * a.splits * a.few_rows * (D + 2) * 4 : 0;
}

template <int DT, int D, int RT>
static hipError_t few_t(Kv4FewArgs p, int64_t tiles, hipStream_t st) {
  k_kv4_attend_few<DT, D, RT><<<(unsigned)(tiles * p.splits), 64 * kAttnWaves, 0, st>>>(p);
  if (p.splits > 1) k_kv4_attend_join<DT, D, 16 * RT><<<(unsigned)tiles, 256, 0, st>>>(p);
  return hipGetLastError();
}

template <int DT>
static hipError_t few_d(const Kv4FewArgs& p, int D, int rows, int64_t tiles, hipStream_t st) {
  if (D == 256) return few_t<DT, 256, 1>(p, tiles, st);
  if (rows == 16) return D == 64 ? few_t<DT, 64, 1>(p, tiles, st) : few_t<DT, 128, 1>(p, tiles, st);
  return D == 64 ? few_t<DT, 64, 2>(p, tiles, st) : few_t<DT, 128, 2>(p, tiles, st);
}

hipError_t launch_kv4_attend(const Kv4Seqs& s, const Kv4Attend& a, int dtype, hipStream_t st) {
  const AttendPlan plan =
      attend_plan(s.T, s.B, a.Hq, s.H, a.D, (int64_t)s.W << s.shift, s.offsets == nullptr);
  if (plan.many_tiles > 0) {
    const hipError_t e = launch_kv4_many(s, a, dtype, s.offsets == nullptr ? 1 : kFewRows + 1, plan.many_rows,
                                         plan.many_tiles, st);
    if (e != hipSuccess || plan.few_tiles == 0) return e;
  }
  Kv4FewArgs p;
  p.s = s;
  p.a = a;
  p.G = a.Hq / s.H;
  p.max_rows = plan.many_tiles > 0 || s.offsets != nullptr && a.D < 256 ? kFewRows : (int64_t)1 << 40;
  p.splits = plan.splits;
  const int64_t tiles = plan.few_tiles * s.H;
  p.part_o = (float*)a.workspace;
  p.part_ml = p.part_o + tiles * p.splits * plan.few_rows * a.D;
  return dtype == F16 ? few_d<F16>(p, a.D, plan.few_rows, tiles, st) : few_d<BF16>(p, a.D, plan.few_rows, tiles, st);
}

}  // namespace qg
