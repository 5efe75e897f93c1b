// Filling and reading the 4-bit paged KV cache (layout: qg_kv4.hpp).
//
// Appending.  A token's keys are rotated by its position, (a, b) -> (a c - b s,
// b c + a s) for pairs of channels, and keys and values become 4-bit codes per
// group of channels:
//   lo = min(0, min x), hi = max(0, max x), t = (hi - lo) / 15,
//   s = t rounded up to 7 significant bits, z = rne(-lo / s),
//   q = clamp(rne(x / s) + z, 0, 15).
// Zero lies in every range, so 0 <= z <= 15 and a zero stays exactly zero.
// s >= t keeps 15 steps enough; the 7 bits cost at most 1.6% of the step.
#include "qg_kv4.hpp"

#include <algorithm>

namespace qg {

namespace {

// Rotation of channel pairs: each product and each sum rounded by itself, so
// that the codes behind it do not hang on how the compiler joins them.
__device__ __forceinline__ void kv4_turn(float& a, float& b, float c, float s) {
#pragma clang fp contract(off)
  const float ac = a * c, bs = b * s, bc = b * c, as = a * s;
  a = ac - bs;
  b = bc + as;
}

// Channel group [lo, hi] -> its word and the reciprocal of its scale.
__device__ __forceinline__ u32 kv4_group(float lo, float hi, float& s, float& r) {
  const float t = (hi - lo) / 15.f;
  s = __uint_as_float((__float_as_uint(t) + 0x1FFFFu) & ~0x1FFFFu);
  r = 0.f;
  if (!(s < __builtin_inff())) {   // an infinity, a NaN, or a range past binary32
    s = 0.f;
    return kKv4Nan;
  }
  if (!(s >= 0x1p-126f)) {   // subnormal scales count as zero: no kernel has to know them
    s = 0.f;
    return 0u;
  }
  r = 1.f / s;
  const float z = fminf(rintf(-lo / s), 15.f);
  return __float_as_uint(s) | (u32)z;
}

// 8 codes as a word.  The quotient x / s is within (-15.5, 15.5); its nearest
// integer comes from x r unless that lies within 2^-15 of a tie, and from the
// correctly rounded division there (as in sym_code_t, whose bound on the two's
// distance holds here too): one test for the 8.
__device__ __forceinline__ u32 kv4_codes(const float (&x)[8], float s, float r, u32 word) {
  if (!(s >= 0x1p-126f)) return 0u;   // a scale of zero, or the mark of a group without one
  const float z = (float)(word & 15u);
  float t[8], far = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = x[e] * r;
    t[e] = rintf(a);
    far = fmaxf(far, fabsf(a - t[e]));
  }
  if (!(far <= kCodeTie)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = rintf(x[e] / s);
  }
  u32 out = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) out |= (u32)__builtin_amdgcn_fmed3f(t[e] + z, 0.f, 15.f) << (4 * e);
  return out;
}

}  // namespace

// A workgroup takes one token and up to 256 / (D / 16) of its heads, queries first, then
// keys, then values: D / 16 neighbouring threads a head, each with two chunks of 8
// channels, the two that a rotation by halves pairs up.  Bound by memory: what it reads
// and writes once.  4096 tokens of 32 heads of 128 channels and as many kv heads,
// binary16, 151 MB: 38 us, 4.0 TB/s; one token of 16 sequences 4.5 us, a launch's
// latency.  (Four positions of a block of value codes a workgroup, which stores them
// side by side: 39, and 133 against 142 for 16384 tokens; but where sequences begin inside
// a block, or have fewer tokens, 190 against 143, and 43 against 24 for 4096 single ones.)
template <int DT, int D>
__global__ __launch_bounds__(256) void k_kv4_append(Kv4Seqs s, Kv4Append a, int parts) {
  constexpr int kL = D / 16, kGd = kv4_groups(D);
  const int part = blockIdx.x % parts, row = blockIdx.x / parts;
  const int hh = part * (int)(blockDim.x / kL) + (int)threadIdx.x / kL, l = (int)threadIdx.x % kL;
  if (hh >= a.Hq + 2 * s.H) return;   // whole groups of kL lanes: the exchanges stay complete
  const bool is_q = hh < a.Hq, is_k = !is_q && hh < a.Hq + s.H;
  const int h = is_q ? hh : is_k ? hh - a.Hq : hh - a.Hq - s.H;
  const Kv4Row at = kv4_row(s, row);
  if (at.b < 0) return;   // rows of no sequence stay as they are
  const bool known = a.rot == 0 || (at.pos >= 0 && at.pos < a.table_rows);
  int slot = 0;
  int32_t* page = nullptr;
  if (!is_q) {
    page = known ? kv4_page(s, at.b, at.pos, h, D, slot) : nullptr;
    if (page == nullptr) return;   // the kL lanes of a head alike
  }
  const int rc = a.rot >> 4;   // chunks of a half of the rotated channels
  const int c0 = l < rc ? l : 2 * rc + (l - rc), c1 = l < rc ? l + rc : c0 + (kL - rc);
  const void* const src = is_q ? a.q : is_k ? a.k : a.v;
  const int64_t from = row * (is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride) + (int64_t)h * D;
  float x0[8], x1[8];
  kv4_load8<DT>(src, from + 8 * c0, x0);
  kv4_load8<DT>(src, from + 8 * c1, x1);
  if ((is_q || is_k) && l < rc) {
    const int64_t tab = known ? at.pos * (a.rot >> 1) : 0;
    if (a.interleaved) {   // angle i turns channels 2 i and 2 i + 1
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        kv4_turn(x0[2 * e], x0[2 * e + 1], a.cos[tab + 4 * c0 + e], a.sin[tab + 4 * c0 + e]);
        kv4_turn(x1[2 * e], x1[2 * e + 1], a.cos[tab + 4 * c1 + e], a.sin[tab + 4 * c1 + e]);
      }
    } else {               // angle i turns channels i and i + rot / 2
#pragma unroll
      for (int e = 0; e < 8; ++e) kv4_turn(x0[e], x1[e], a.cos[tab + 8 * c0 + e], a.sin[tab + 8 * c0 + e]);
    }
  }
  if (is_q) {
    if (!known) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x0[e] = x1[e] = 0.f;
    }
    const int64_t o = ((int64_t)row * a.Hq + h) * D;
    kv4_store8<DT>(a.q_out, o + 8 * c0, x0);
    kv4_store8<DT>(a.q_out, o + 8 * c1, x1);
    return;
  }
  // range of each group, zero included; a value that is not finite makes it infinite
  const int g0 = c0 >> 4, g1 = c1 >> 4;
  float lo[kGd], hi[kGd];
#pragma unroll
  for (int g = 0; g < kGd; ++g) lo[g] = hi[g] = 0.f;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    float mn = 0.f, mx = 0.f, odd = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = t ? x1[e] : x0[e];
      mn = fminf(mn, v);
      mx = fmaxf(mx, v);
      odd = __builtin_fmaf(v, 0.f, odd);
    }
    if (odd != 0.f) mx = __builtin_inff();
    const int g = t ? g1 : g0;
#pragma unroll
    for (int i = 0; i < kGd; ++i) {
      lo[i] = g == i ? fminf(lo[i], mn) : lo[i];
      hi[i] = g == i ? fmaxf(hi[i], mx) : hi[i];
    }
  }
  float sc[kGd], re[kGd];
  u32 word[kGd];
#pragma unroll
  for (int g = 0; g < kGd; ++g) {
#pragma unroll
    for (int o = 1; o < kL; o <<= 1) {
      lo[g] = fminf(lo[g], __shfl_xor(lo[g], o, kWave));
      hi[g] = fmaxf(hi[g], __shfl_xor(hi[g], o, kWave));
    }
    word[g] = kv4_group(lo[g], hi[g], sc[g], re[g]);
  }
  const u32 q0 = kv4_codes(x0, g0 ? sc[kGd - 1] : sc[0], g0 ? re[kGd - 1] : re[0], g0 ? word[kGd - 1] : word[0]);
  const u32 q1 = kv4_codes(x1, g1 ? sc[kGd - 1] : sc[0], g1 ? re[kGd - 1] : re[0], g1 ? word[kGd - 1] : word[0]);
  const int S = 1 << s.shift, step = is_k ? 1 : 4;
  int32_t* const codes = is_k ? page + slot * (D / 8) : page + S * (D / 8) + (slot >> 2) * (D / 2) + (slot & 3);
  codes[c0 * step] = (int32_t)q0;
  codes[c1 * step] = (int32_t)q1;
  if (l < kGd) page[S * (D / 4) + (is_k ? 0 : kGd * S) + l * S + slot] = (int32_t)(l ? word[kGd - 1] : word[0]);
}

// Rows that a workgroup reads back where a call has many.
constexpr int kQuad = 4;

// Whether rows row .. row + 3 are the four positions of one block of value codes.
// (offsets may be wrong: rows past the call's do not count, whatever they say)
__device__ __forceinline__ bool kv4_quad(const Kv4Seqs& s, const Kv4Row& at, int row) {
  return at.b >= 0 && row + kQuad <= s.T && row + kQuad <= at.end && (at.pos & (kQuad - 1)) == 0;
}

// N rows of one chunk of 8 channels of one head.
template <int DT, int D, int N>
__device__ __forceinline__ void kv4_dequant_rows(const Kv4Seqs& s, void* out, int row, const Kv4Row& at,
                                                 int h, int is_v, int c) {
  constexpr int kC = D / 8, kGd = kv4_groups(D);
  const int S = 1 << s.shift;
  int slot = 0;
  const int32_t* const page = kv4_page(s, at.b, at.pos, h, D, slot);
  u32 w[N], p[N];
#pragma unroll
  for (int n = 0; n < N; ++n) w[n] = p[n] = 0;   // zeros where the position has no page
  if (page != nullptr) {
    const int32_t* const par = page + S * (D / 4) + (is_v ? kGd * S : 0) + (c >> 4) * S + slot;
    const int32_t* const codes = is_v ? page + S * kC + (slot >> 2) * (D / 2) + 4 * c + (slot & 3) : page + slot * kC + c;
    if constexpr (N == kQuad) {
      const v4i pw = ld16(par);
      if (is_v) {
        const v4i cw = ld16(codes);
#pragma unroll
        for (int n = 0; n < N; ++n) w[n] = (u32)cw[n];
      } else {
#pragma unroll
        for (int n = 0; n < N; ++n) w[n] = (u32)codes[n * kC];
      }
#pragma unroll
      for (int n = 0; n < N; ++n) p[n] = (u32)pw[n];
    } else {
      w[0] = (u32)*codes;
      p[0] = (u32)*par;
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const float sc = kv4_scale(p[n]);
    const int z = (int)(p[n] & 15u);
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)((int)((w[n] >> (4 * e)) & 15u) - z) * sc;
    kv4_store8<DT>(out, ((int64_t)(row + n) * s.H + h) * D + 8 * c, x);
  }
}

// Values of the cached positions of the call's rows, [T][H][D] each: ROWS rows and
// up to 256 chunks of 8 channels of keys or values a workgroup.  (q - z) s is exact
// in binary32.  Bound by memory: 65536 positions of 8 heads of 128 channels to
// binary16, 340 MB, 67 us, 5.1 TB/s, what a large copy reaches.
template <int DT, int D, int ROWS>
__global__ __launch_bounds__(256) void k_kv4_dequant(Kv4Seqs s, void* __restrict__ k,
                                                     void* __restrict__ v, int parts) {
  constexpr int kC = D / 8;
  const int part = blockIdx.x % parts, row = blockIdx.x / parts * ROWS;
  const int at_c = part * (int)blockDim.x + (int)threadIdx.x;
  if (at_c >= 2 * s.H * kC) return;
  const int c = at_c % kC, hv = at_c / kC, is_v = hv >= s.H, h = is_v ? hv - s.H : hv;
  void* const out = is_v ? v : k;
  const Kv4Row at = kv4_row(s, row);
  if constexpr (ROWS == kQuad) {
    if (kv4_quad(s, at, row)) return kv4_dequant_rows<DT, D, kQuad>(s, out, row, at, h, is_v, c);
    for (int r = 0; r < kQuad; ++r) {
      if (row + r >= s.T) return;
      const Kv4Row one = kv4_row(s, row + r);
      if (one.b >= 0) kv4_dequant_rows<DT, D, 1>(s, out, row + r, one, h, is_v, c);
    }
  } else {
    if (at.b >= 0) kv4_dequant_rows<DT, D, 1>(s, out, row, at, h, is_v, c);   // rows of no sequence stay as they are
  }
}

// Threads and workgroups of one row of `items` threads: workgroups as even as whole
// waves and whole heads (`head` threads, a divisor of 64) allow.
static void kv4_split(int64_t items, int& threads, int& parts) {
  parts = (int)((items + 255) / 256);
  threads = (int)(((items + parts - 1) / parts + 63) / 64 * 64);
}

// Reading back: four rows a workgroup where there are enough workgroups to fill the GPU
// several times over, since their value codes and group words are then 16 bytes side by side.
// One row against four: 65536 rows of 8 heads 84 us and 66, alike from an odd position on; 500
// rows 3.1 and 3.5.  Not where sequences have fewer rows than four on average, which
// would come after one another (4096 single ones by offsets 12.0 and 14.5).
static bool kv4_quads(const Kv4Seqs& s, int parts) {
  return (int64_t)s.T * parts >= 4096 && s.T / s.B >= kQuad;
}

template <int DT, int D>
static hipError_t kv4_append_t(const Kv4Seqs& s, const Kv4Append& a, hipStream_t st) {
  int threads, parts;
  kv4_split((int64_t)(a.Hq + 2 * s.H) * (D / 16), threads, parts);
  k_kv4_append<DT, D><<<(unsigned)((int64_t)s.T * parts), threads, 0, st>>>(s, a, parts);
  return hipGetLastError();
}

template <int DT>
static hipError_t kv4_append_d(const Kv4Seqs& s, const Kv4Append& a, hipStream_t st) {
  switch (a.D) {
    case 64: return kv4_append_t<DT, 64>(s, a, st);
    case 128: return kv4_append_t<DT, 128>(s, a, st);
    default: return kv4_append_t<DT, 256>(s, a, st);
  }
}

hipError_t launch_kv4_append(const Kv4Seqs& s, const Kv4Append& a, int dtype, hipStream_t st) {
  switch (dtype) {
    case F32: return kv4_append_d<F32>(s, a, st);
    case F16: return kv4_append_d<F16>(s, a, st);
    default: return kv4_append_d<BF16>(s, a, st);
  }
}

template <int DT, int D>
static hipError_t kv4_dequant_t(const Kv4Seqs& s, void* k, void* v, hipStream_t st) {
  int threads, parts;
  kv4_split((int64_t)2 * s.H * (D / 8), threads, parts);
  if (kv4_quads(s, parts))
    k_kv4_dequant<DT, D, kQuad><<<(unsigned)(((int64_t)s.T + kQuad - 1) / kQuad * parts), threads, 0, st>>>(s, k, v, parts);
  else
    k_kv4_dequant<DT, D, 1><<<(unsigned)((int64_t)s.T * parts), threads, 0, st>>>(s, k, v, parts);
  return hipGetLastError();
}

template <int DT>
static hipError_t kv4_dequant_d(const Kv4Seqs& s, int D, void* k, void* v, hipStream_t st) {
  switch (D) {
    case 64: return kv4_dequant_t<DT, 64>(s, k, v, st);
    case 128: return kv4_dequant_t<DT, 128>(s, k, v, st);
    default: return kv4_dequant_t<DT, 256>(s, k, v, st);
  }
}

hipError_t launch_kv4_dequant(const Kv4Seqs& s, int D, void* k, void* v, int out_dtype,
                              hipStream_t st) {
  switch (out_dtype) {
    case F32: return kv4_dequant_d<F32>(s, D, k, v, st);
    case F16: return kv4_dequant_d<F16>(s, D, k, v, st);
    default: return kv4_dequant_d<BF16>(s, D, k, v, st);
  }
}

}  // namespace qg
