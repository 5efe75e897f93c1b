// Attention of many query rows over the 4-bit paged KV cache (qg_kv4.hpp):
// prompts and chunks of them.  The mathematics is that of attn_kv4.hip; here the
// codes of 64 positions become binary16 values once for all rows of a workgroup.
//
// A value (q - z) s has 11 significant bits.  Scaled by the power of two that
// takes the tile's largest scale to [2^-9, 2^-8) it is exact in binary16 as long
// as its own scale is no less than 2^-9 of that; and since a nibble masked out of
// a code word is the binary16 subnormal n 2^-24, one packed fma makes two values,
// n 2^-24 (s 2^24) - z s.  Positions with a smaller scale take their own power of
// two, and a factor for the scores (keys) or weights (values) that the step's
// general form applies.
//
// Both products have the query rows as columns, so that a lane has one query row
// throughout: scores^T = K Q^T, outputs^T = V^T P^T, with the scores' registers
// the second product's operand as they are (positions in the order of the lane).
// Running bound and power of two of the weights as in attn_kv4.hip.  A step whose
// positions all rows of a wave see, with no odd scales, takes the short form: one
// fma, one exponential, one addition and half a conversion for each score, and a
// check of the sums that sends what passed the bound to the general form.
#include "qg_kv4_attn.hpp"

#include <algorithm>

namespace qg {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef int v2i __attribute__((ext_vector_type(2)));

constexpr int kTile = 64;      // positions of a tile
constexpr float kLow = -3.402823466e38f;

// What a tile's positions need besides their codes.
template <int Gd>
struct Kv4Marks {
  // keys: 16 n 2^-24 and n 2^-24 to values, and -z s, each twice (two channels)
  v4i key[kTile][Gd];
  // values: the same for single positions
  _Float16 s24[Gd][kTile], s20[Gd][kTile], z[Gd][kTile];
  float fk[kTile];             // factor of the scores, -1: no page
  float fv[Gd][kTile];         // factor of the weights
  float ek, ev[Gd];            // powers of two of the tile's keys and values (exponents)
  int odd[1 + Gd];             // some factor is not 1
};

__device__ __forceinline__ int float_exp(float x) { return (int)((__float_as_uint(x) >> 23) & 255u) - 127; }

}  // namespace

struct Kv4ManyArgs {
  Kv4Seqs s;
  Kv4Attend a;
  int G, tiles;
  int64_t min_rows;   // sequences of fewer rows are another kernel's
};

template <int DT, int D, int NW>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void k_kv4_attend_many(Kv4ManyArgs p) {
  constexpr int NT = 64 * NW, kRows = 32 * NW, kGd = kv4_groups(D), kC = D / 8;   // code words of a position
  constexpr int kSt = D / 16;        // steps of the first product
  constexpr int kDt = D / 32;        // channel tiles of the second
  constexpr int kKl = (kTile * kC / 4 + NT - 1) / NT;   // 16-byte loads of key codes of a thread
  constexpr int kVl = (kTile / 4 * kC + NT - 1) / NT;   // and of value codes
  // [2][position / 32][word][position % 32] and [2][position / 32][step][half][channel], 16 bytes each
  extern __shared__ __align__(16) char lds[];
  v4i* const kbuf = (v4i*)lds;
  v4i* const vbuf = kbuf + 2 * kTile * kC;
  Kv4Marks<kGd>* const marks = (Kv4Marks<kGd>*)(vbuf + 2 * kTile * kC);

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = p.s.H;
  const int h = blockIdx.x % H;
  // the rows that see most first
  const Kv4Tile t = kv4_tile<kRows>(p.s, p.G, p.min_rows, (int64_t)1 << 40, p.tiles - 1 - (int)(blockIdx.x / H));
  if (t.b < 0) return;
  const int rows = min(t.n * p.G - t.row0, kRows);
  const int len = min(max(p.s.lengths[t.b], -0x3FFFFFFF), 0x3FFFFFFF);
  const int first = len - t.n;
  const int p0 = first + t.row0 / p.G, p1 = first + (t.row0 + rows - 1) / p.G;
  const int shift = p.s.shift, S = 1 << shift, W = p.s.W, window = p.a.window, sinks = p.a.sinks;
  const int capacity = (int)min((int64_t)W << shift, (int64_t)0x40000000);
  const Kv4Span span = kv4_span<kTile>(p0, p1, window, sinks, capacity);
  const int32_t* table = p.s.table + (int64_t)t.b * W;
  const int page_words = (int)kv4_words(S, D);

  // ---- this wave's 32 rows: one a lane, both halves of the wave alike --------
  const int c = lane & 31, half = lane >> 5;
  const int row = t.row0 + 32 * wave + c;
  const bool there = 32 * wave + c < rows;
  const int pos = there ? first + row / p.G : kKv4Past;
  const bool alive = 32 * wave < rows;                               // the wave has rows
  const int last_row = min(32 * wave + 31, rows - 1);
  const int wp0 = first + (t.row0 + 32 * wave) / p.G, wp1 = first + (t.row0 + last_row) / p.G;
  v8h q[kSt];
  float cc;
  {
    float x[kSt][8], top = 0.f;
    const int64_t at = (int64_t)(t.token0 + row / p.G) * p.a.q_stride + (int64_t)(h * p.G + row % p.G) * D;
#pragma unroll
    for (int j = 0; j < kSt; ++j) {
      const v4i a = there ? ld16((const uint16_t*)p.a.q + at + 16 * j + 8 * half) : v4i{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const u32 u = ((u32)a[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
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
    cc = ldexpf(p.a.scale * 1.44269504088896f, 9 - e);
  }
  v16f o[kDt];
#pragma unroll
  for (int j = 0; j < kDt; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[j][e] = 0.f;
  float m = kLow, l = 0.f, rinv[kGd], lim[kGd];
#pragma unroll
  for (int g = 0; g < kGd; ++g) rinv[g] = lim[g] = 0.f;

  // ---- loads of later tiles ----------------------------------------------------
  // key codes: thread i of a tile has position i % 64 and words 4 (i / 64) ..;
  // value codes: four positions 4 (i / kC) .. and word i % kC
  const int n_tiles = span.tiles;
  auto page_id = [&](int tile, int off) {
    const int pi = (tile * kTile + off) >> shift;
    return pi < W ? table[pi] : -1;
  };
  auto page_of = [&](int id) {
    return (const char*)(p.s.pages + ((int64_t)((u32)id < (u32)p.s.P ? id : 0) * H + h) * page_words);
  };
  int kid[kKl], vid[kVl], mid = -1;
  v4i kc[kKl], vc[kVl];
  u32 mw[kGd];
  const bool mark_k = wave == 0, mark_v = wave >= 1 && wave <= kGd;   // who makes the marks
  auto fetch_ids = [&](int u) {
    const int tile = span.tile(min(u, n_tiles - 1));
#pragma unroll
    for (int i = 0; i < kKl; ++i) kid[i] = page_id(tile, (tid + i * NT) % kTile);
#pragma unroll
    for (int i = 0; i < kVl; ++i) vid[i] = page_id(tile, (tid + i * NT) / kC * 4 % kTile);
  };
  auto fetch_codes = [&](int u) {
    const int tile = span.tile(min(u, n_tiles - 1));
#pragma unroll
    for (int i = 0; i < kKl; ++i) {
      const int n = tid + i * NT, off = n % kTile;
      if (kTile * kC / 4 % NT == 0 || n < kTile * kC / 4)
        kc[i] = ld16(page_of(kid[i]) + ((tile * kTile + off) & (S - 1)) * (D / 2) + n / kTile * 16);
    }
#pragma unroll
    for (int i = 0; i < kVl; ++i) {
      const int n = tid + i * NT, off = n / kC * 4;
      if (kTile / 4 * kC % NT == 0 || n < kTile / 4 * kC)
        vc[i] = ld16(page_of(vid[i]) + S * (D / 2) + ((tile * kTile + off) & (S - 1)) * (D / 2) + n % kC * 16);
    }
  };
  auto fetch_mark_id = [&](int u) {
    if (mark_k || mark_v) mid = page_id(span.tile(min(u, n_tiles - 1)), lane);
  };
  int mid_now = -1;   // page of the words in mw
  auto fetch_words = [&](int u) {
    mid_now = mid;
    if (!(mark_k || mark_v)) return;
    const int slot = (span.tile(min(u, n_tiles - 1)) * kTile + lane) & (S - 1);
    const u32* g = (const u32*)page_of(mid) + S * (D / 4) + slot;
    if (mark_k) {
#pragma unroll
      for (int i = 0; i < kGd; ++i) mw[i] = g[i * S];
    } else {
      mw[0] = g[(kGd + wave - 1) * S];
    }
  };
  // The marks of tile u from the words in mw.
  auto mark = [&](int u) {
    if (!(mark_k || mark_v)) return;
    Kv4Marks<kGd>& out = marks[u % 3];
    const int at = span.tile(min(u, n_tiles - 1)) * kTile + lane;
    const bool page = (u32)mid_now < (u32)p.s.P && at < capacity;
    const bool some = page && at <= p1 && (window <= 0 || at > p0 - window || at < sinks);   // some row sees it
    float s[kGd];
    u32 z[kGd];
    bool nan = false;
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < kGd; ++i) {
      s[i] = 0.f;
      z[i] = 0;
      if (i > 0 && !mark_k) continue;
      const float v = some ? kv4_scale(mw[i]) : 0.f;
      const bool bad = !(v < __builtin_inff());
      nan |= bad;
      s[i] = bad ? 0.f : v;
      z[i] = some ? mw[i] & 15u : 0u;
      mine = fmaxf(mine, s[i]);
    }
    const float top = wave_max_nonneg(mine);
    // scales below 2^-9 of the largest by their own power of two
    const bool own = mine > 0.f && mine * 512.f < top;
    const int et = float_exp(fmaxf(top, 0x1p-126f)), e = own ? float_exp(fmaxf(mine, 0x1p-126f)) : et;
    const float f = own ? ldexpf(1.f, e - et) : 1.f;
    const bool odd = __any(own || nan || !page);
    if (mark_k) {
#pragma unroll
      for (int i = 0; i < kGd; ++i) {
        const float v = nan ? __builtin_nanf("") : ldexpf(s[i], -e - 9);
        const u32 a = f32_to_f16_bits(v * 0x1p24f), b = f32_to_f16_bits(v * 0x1p20f), d = f32_to_f16_bits(-(float)z[i] * v);
        out.key[lane][i] = v4i{(int)(a * 0x10001u), (int)(b * 0x10001u), (int)(d * 0x10001u), 0};
      }
      out.fk[lane] = page ? f : -1.f;
      if (lane == 0) {
        out.ek = (float)et;
        out.odd[0] = odd;
      }
    } else {
      const int g = wave - 1;
      const float v = ldexpf(s[0], -e - 9);
      out.s24[g][lane] = (_Float16)(v * 0x1p24f);
      out.s20[g][lane] = (_Float16)(v * 0x1p20f);
      out.z[g][lane] = (_Float16)(-(float)z[0] * v);
      out.fv[g][lane] = nan ? __builtin_nanf("") : f;
      if (lane == 0) {
        out.ev[g] = (float)et;
        out.odd[1 + g] = odd;
      }
    }
  };
  // Codes in kc, vc -> values of tile u.
  auto unpack = [&](int u) {
    const Kv4Marks<kGd>& mk = marks[u % 3];
    v4i* const kb = kbuf + (u & 1) * kTile * kC;
    v2i* const vb = (v2i*)(vbuf + (u & 1) * kTile * kC);
    const auto fma2 = [](u32 n, u32 s, u32 z) {
      return __builtin_bit_cast(int, __builtin_elementwise_fma(__builtin_bit_cast(v2h, n), __builtin_bit_cast(v2h, s),
                                                               __builtin_bit_cast(v2h, z)));
    };
#pragma unroll
    for (int i = 0; i < kKl; ++i) {
      const int n = tid + i * NT, off = n % kTile, w0 = n / kTile * 4;
      if (kTile * kC / 4 % NT != 0 && n >= kTile * kC / 4) continue;
      const v4i par = mk.key[off][kGd > 1 ? w0 / 16 : 0];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32 w = (u32)kc[i][j], hi = w >> 8;
        kb[((off >> 5) * kC + w0 + j) * 32 + (off & 31)] =
            v4i{fma2(w & 0x000F000Fu, par[0], par[2]), fma2(w & 0x00F000F0u, par[1], par[2]),
                fma2(hi & 0x000F000Fu, par[0], par[2]), fma2(hi & 0x00F000F0u, par[1], par[2])};
      }
    }
#pragma unroll
    for (int i = 0; i < kVl; ++i) {
      const int n = tid + i * NT, quad = n / kC, word = n % kC;
      if (kTile / 4 * kC % NT != 0 && n >= kTile / 4 * kC) continue;
      const int g = kGd > 1 ? word / 16 : 0;
      const v2i a = *(const v2i*)&mk.s24[g][4 * quad], b = *(const v2i*)&mk.s20[g][4 * quad], d = *(const v2i*)&mk.z[g][4 * quad];
      // of 32 positions: quads 4 step + half and 4 step + 2 + half side by side
      const int qq = quad & 7;
      v2i* const to = vb + 2 * (((((quad >> 3) * 2 + (qq >> 2)) * 2 + (qq & 1)) * D + word % 16) + (kGd > 1 ? g * 128 : 0)) + (qq >> 1 & 1);
      constexpr int kStep = D == 64 ? 8 : 16;   // channel 8 w + j at place kStep j + w of its 64 or 128
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const u32 sel = hf ? 0x07060302u : 0x05040100u;
        const u32 x = __builtin_amdgcn_perm((u32)vc[i][1], (u32)vc[i][0], sel);
        const u32 y = __builtin_amdgcn_perm((u32)vc[i][3], (u32)vc[i][2], sel);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32 mask = j & 1 ? 0x00F000F0u : 0x000F000Fu;
          const v2i sc = j & 1 ? b : a;
          to[2 * kStep * (4 * hf + j)] = v2i{fma2((j & 2 ? x >> 8 : x) & mask, sc[0], d[0]), fma2((j & 2 ? y >> 8 : y) & mask, sc[1], d[1])};
        }
      }
    }
  };

  // ---- one half tile of 32 positions ------------------------------------------------
  auto half_tile = [&](int u, int sub, const Kv4Marks<kGd>& mk, bool simple) {
    const v4i* const kb = kbuf + (u & 1) * kTile * kC + sub * kC * 32;
    v16f s;
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = 0.f;
#pragma unroll
    for (int j = 0; j < kSt; ++j)
      s = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, kb[(2 * j + half) * 32 + c]), q[j], s, 0, 0, 0);
    const float ct = ldexpf(cc, (int)mk.ek);
    v8h pf[kGd][2];
    bool done = false;
    if (simple) {
      float rs[kGd];   // exponent of the weights' unit
      bool fits = true;
#pragma unroll
      for (int g = 0; g < kGd; ++g) {
        rs[g] = mk.ev[g] + (float)float_exp(rinv[g]);
        fits &= rinv[g] > 0.f && fabsf(rs[g]) <= 60.f;
      }
      if (__all(fits || !there)) {   // columns of no row may hold anything
        const float shift0 = rs[0] - m;
        float w[16], sum = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], ct, shift0));
          sum += w[e];
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) pf[0][e >> 3][e & 7] = (_Float16)w[e];
        bool small = sum <= 0x1p14f;
        if constexpr (kGd > 1) {
          const float more = __builtin_amdgcn_exp2f(rs[kGd - 1] - rs[0]);
          small &= sum * more <= 0x1p14f;
#pragma unroll
          for (int e = 0; e < 16; ++e) pf[kGd - 1][e >> 3][e & 7] = (_Float16)(w[e] * more);
        }
        done = __all(small || !there);
        if (done) l += sum * __builtin_amdgcn_exp2f(-rs[0]);
      }
    }
    if (!done) {
      float top = kLow;
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const v4f f = *(const v4f*)&mk.fk[32 * sub + 8 * a + 4 * half];
        const int t0 = span.tile(u) * kTile + 32 * sub + 8 * a + 4 * half;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int at = t0 + b;
          const bool seen = f[b] >= 0.f && at <= pos && (window <= 0 || at > pos - window || at < sinks);
          s[4 * a + b] = seen ? s[4 * a + b] * ct * f[b] : -__builtin_inff();
          top = fmaxf(top, s[4 * a + b]);
        }
      }
      float alpha = 1.f;
      if (__any(top > m + 8.f)) {
        const float mn = fmaxf(m, fmaxf(top, __shfl_xor(top, 32, kWave)));
        alpha = __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= alpha;
#pragma unroll
        for (int g = 0; g < kGd; ++g) lim[g] = -1.f;
      }
      float w[kGd][16];
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int e = 4 * a + b;
          const bool seen = s[e] != -__builtin_inff();
          const float pe = __builtin_amdgcn_exp2f(s[e] - m);
          l += pe;
#pragma unroll
          for (int g = 0; g < kGd; ++g) {
            const float f = mk.fv[g][32 * sub + 8 * a + 4 * half + b];
            w[g][e] = seen ? pe * f : 0.f;
          }
        }
#pragma unroll
      for (int g = 0; g < kGd; ++g) {
        const float tev = ldexpf(1.f, (int)mk.ev[g]);
        float most = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          w[g][e] *= tev;
          most = fmaxf(most, w[g][e]);
        }
        if (__any(most > lim[g])) {
          const bool set = rinv[g] > 0.f;
          const float ref = set ? alpha / rinv[g] : 0.f;
          const float all = fmaxf(fmaxf(most, __shfl_xor(most, 32, kWave)), ref);
          const float big = fminf(fmaxf(all, 0x1p-100f), 0x1p100f);
          const float f = __uint_as_float(0x7F000000u - (__float_as_uint(big) & 0x7F800000u));
          const float by = set ? f * ref : 1.f;
          rinv[g] = all > 0.f ? f : 0.f;
          lim[g] = all > 0.f ? 0x1p12f / f : 0.f;
#pragma unroll
          for (int j = 0; j < kDt / kGd; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[g * (kDt / kGd) + j][e] *= by;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) pf[g][e >> 3][e & 7] = (_Float16)(w[g][e] * rinv[g]);
      }
    }
    const v4i* const vb = vbuf + (u & 1) * kTile * kC + sub * kC * 32;
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int j = 0; j < kDt; ++j) {
        const v8h v = __builtin_bit_cast(v8h, vb[(2 * st + half) * D + 32 * j + c]);
        o[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, pf[kGd > 1 ? j / (kDt / kGd) : 0][st], o[j], 0, 0, 0);
      }
  };

  if (n_tiles > 0) {
    fetch_ids(0);
    fetch_mark_id(0);
    fetch_codes(0);
    fetch_words(0);
    fetch_mark_id(1);
    mark(0);
    fetch_words(1);
    fetch_mark_id(2);
    __syncthreads();
    unpack(0);
    mark(1);
    fetch_ids(1);
    fetch_codes(1);
    fetch_ids(2);
    fetch_words(2);
    fetch_mark_id(3);
    __syncthreads();
  }
  for (int u = 0; u < n_tiles; ++u) {
    if (u + 1 < n_tiles) {
      unpack(u + 1);
      mark(u + 2);
      fetch_codes(u + 2);
      fetch_ids(u + 3);
      fetch_words(u + 3);
      fetch_mark_id(u + 4);
    }
    const int t0 = span.tile(u) * kTile;
    // something of the tile is in some row's sight
    if (alive && t0 <= wp1 && (window <= 0 || t0 + kTile - 1 > wp0 - window || t0 < sinks)) {
      const Kv4Marks<kGd>& mk = marks[u % 3];
      bool odd = false;
#pragma unroll
      for (int i = 0; i < 1 + kGd; ++i) odd |= mk.odd[i] != 0;
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const int a = t0 + 32 * sub;
        const bool simple = !odd && a + 31 <= wp0 && (window <= 0 || a > wp1 - window || a + 32 <= sinks);
        half_tile(u, sub, mk, __builtin_amdgcn_readfirstlane(simple));
      }
    }
    __syncthreads();
  }

  // ---- outputs: lane (c, half) has, of row c, eight runs of 8 channels ---------------
  l += __shfl_xor(l, 32, kWave);
  if (!there) return;
  const int64_t to = ((int64_t)(t.token0 + row / p.G) * p.a.Hq + h * p.G + row % p.G) * D;
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
  for (int g = 0; g < kGd; ++g) {
    const float f = rinv[g] > 0.f ? 512.f / rinv[g] * inv : 0.f;
    constexpr int kPer = kDt / kGd;   // channel tiles of a group: 4, or 2 of 64 channels
    if constexpr (D == 64) {
      // place 32 j + 8 a + 4 half + b holds channel 8 (place % 8) + place / 8
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int a = 0; a < 4; ++a) x[4 * j + a] = o[j][4 * a + b] * f;
        kv4_store8<DT>(p.a.out, to + 32 * half + 8 * b, x);
      }
    } else {
      // place 32 j + 8 a + 4 half + b holds channel 8 (place % 16) + place / 16
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          float x[8];
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            x[2 * j] = o[kPer * g + j][4 * a + b] * f;
            x[2 * j + 1] = o[kPer * g + j][4 * (a + 2) + b] * f;
          }
          kv4_store8<DT>(p.a.out, to + 128 * g + 64 * a + 32 * half + 8 * b, x);
        }
    }
  }
}

namespace {

template <int D>
constexpr int many_lds() { return 2 * 2 * kTile * (D / 8) * 16 + 3 * (int)sizeof(Kv4Marks<kv4_groups(D)>); }

template <int DT, int D, int NW>
hipError_t many_t(Kv4ManyArgs p, hipStream_t st) {
  constexpr int bytes = many_lds<D>();
  static_assert(bytes <= 160 * 1024, "");
  k_kv4_attend_many<DT, D, NW><<<(unsigned)(p.tiles * p.s.H), 64 * NW, bytes, st>>>(p);
  return hipGetLastError();
}

template <int DT, int NW>
hipError_t many_d(const Kv4ManyArgs& p, hipStream_t st) {
  switch (p.a.D) {
    case 64: return many_t<DT, 64, NW>(p, st);
    case 128: return many_t<DT, 128, NW>(p, st);
    default: return many_t<DT, 256, 4>(p, st);
  }
}

}  // namespace

hipError_t launch_kv4_many(const Kv4Seqs& s, const Kv4Attend& a, int dtype, int64_t min_rows, int rows,
                           int64_t tiles, hipStream_t st) {
  const Kv4ManyArgs p{s, a, a.Hq / s.H, (int)tiles, min_rows};
  if (rows == 256) return dtype == F16 ? many_d<F16, 8>(p, st) : many_d<BF16, 8>(p, st);
  return dtype == F16 ? many_d<F16, 4>(p, st) : many_d<BF16, 4>(p, st);
}

}  // namespace qg
