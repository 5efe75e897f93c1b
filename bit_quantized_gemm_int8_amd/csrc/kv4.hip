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
// distance holds here too).
__device__ __forceinline__ u32 kv4_codes(const float (&x)[8], float s, float r, u32 word) {
  if (!(s >= 0x1p-126f)) {   // subnormal scales count as zero: no kernel has to know them
    s = 0.f;
    return 0u;
  }
  const float z = (float)(word & 15u);
  u32 out = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = x[e] * r;
    float t = rintf(a);
    if (!(fabsf(a - t) <= kCodeTie)) t = rintf(x[e] / s);
    out |= (u32)__builtin_amdgcn_fmed3f(t + z, 0.f, 15.f) << (4 * e);
  }
  return out;
}

}  // namespace

// One row (token) of one head: D / 16 neighbouring threads with two chunks of 8
// channels each, the two that a rotation by halves pairs up.  A workgroup takes
// one token and up to 256 / (D / 16) of its heads, queries first, then keys,
// then values.
template <int DT, int D>
__global__ __launch_bounds__(256) void k_kv4_append(Kv4Seqs s, Kv4Append a, int parts) {
  constexpr int kL = D / 16, kGd = kv4_groups(D);
  const int row = blockIdx.x / parts, part = blockIdx.x - row * parts;
  const int heads = a.Hq + 2 * s.H;
  const int hh = part * (int)(blockDim.x / kL) + (int)threadIdx.x / kL, l = (int)threadIdx.x % kL;
  if (hh >= heads) return;   // whole groups of kL lanes: the exchanges below stay complete
  const Kv4Row at = kv4_row(s, row);
  if (at.b < 0) return;      // rows of no sequence stay as they are
  const int rc = a.rot >> 4;   // chunks of a half of the rotated channels
  const int c0 = l < rc ? l : 2 * rc + (l - rc), c1 = l < rc ? l + rc : c0 + (kL - rc);
  const bool known = a.rot == 0 || (at.pos >= 0 && at.pos < a.table_rows);
  const bool is_q = hh < a.Hq, is_k = !is_q && hh < a.Hq + s.H;
  const int h = is_q ? hh : is_k ? hh - a.Hq : hh - a.Hq - s.H;
  const void* src = is_q ? a.q : is_k ? a.k : a.v;
  const int64_t base = row * (is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride) + (int64_t)h * D;
  int slot = 0;
  int32_t* page = nullptr;
  if (!is_q) {
    page = known ? kv4_page(s, at.b, at.pos, h, D, slot) : nullptr;
    if (page == nullptr) return;   // the kL lanes of a head alike
  }
  float x0[8], x1[8];
  kv4_load8<DT>(src, base + 8 * c0, x0);
  kv4_load8<DT>(src, base + 8 * c1, x1);
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
    const int g = (t ? c1 : c0) >> 4;
#pragma unroll
    for (int i = 0; i < kGd; ++i) {
      lo[i] = g == i ? fminf(lo[i], mn) : lo[i];
      hi[i] = g == i ? fmaxf(hi[i], mx) : hi[i];
    }
  }
  float sc[kGd], rc_[kGd];
  u32 word[kGd];
#pragma unroll
  for (int g = 0; g < kGd; ++g) {
#pragma unroll
    for (int o = 1; o < kL; o <<= 1) {
      lo[g] = fminf(lo[g], __shfl_xor(lo[g], o, kWave));
      hi[g] = fmaxf(hi[g], __shfl_xor(hi[g], o, kWave));
    }
    word[g] = kv4_group(lo[g], hi[g], sc[g], rc_[g]);
  }
  const int S = 1 << s.shift, g0 = c0 >> 4, g1 = c1 >> 4;
  const u32 q0 = kv4_codes(x0, g0 ? sc[kGd - 1] : sc[0], g0 ? rc_[kGd - 1] : rc_[0], g0 ? word[kGd - 1] : word[0]);
  const u32 q1 = kv4_codes(x1, g1 ? sc[kGd - 1] : sc[0], g1 ? rc_[kGd - 1] : rc_[0], g1 ? word[kGd - 1] : word[0]);
  int32_t* codes = is_k ? page + (int64_t)slot * (D / 8)
                        : page + S * (D / 8) + (slot >> 2) * (D / 2) + (slot & 3);
  const int step = is_k ? 1 : 4;
  codes[c0 * step] = (int32_t)q0;
  codes[c1 * step] = (int32_t)q1;
  int32_t* par = page + S * (D / 4) + (is_k ? 0 : kGd * S) + slot;
  if (l < kGd) par[l * S] = (int32_t)(kGd > 1 && l ? word[kGd - 1] : word[0]);
}

// Values of the cached positions of the call's rows, [T][H][D] each: one thread
// for 8 channels of keys or values; (q - z) s is exact in binary32.
template <int DT, int D>
__global__ __launch_bounds__(256) void k_kv4_dequant(Kv4Seqs s, void* __restrict__ k,
                                                     void* __restrict__ v, int parts) {
  constexpr int kC = D / 8;
  const int row = blockIdx.x / parts, part = blockIdx.x - row * parts;
  const int i = part * (int)blockDim.x + (int)threadIdx.x;
  if (i >= 2 * s.H * kC) return;
  const Kv4Row at = kv4_row(s, row);
  if (at.b < 0) return;
  const int c = i % kC, hv = i / kC, is_v = hv >= s.H, h = is_v ? hv - s.H : hv;
  const int S = 1 << s.shift;
  int slot = 0;
  const int32_t* page = kv4_page(s, at.b, at.pos, h, D, slot);
  float x[8];
  if (page == nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
  } else {
    const u32 w = is_v ? page[S * kC + (slot >> 2) * (D / 2) + 4 * c + (slot & 3)]
                       : page[slot * kC + c];
    const u32 p = page[S * (D / 4) + (is_v ? kv4_groups(D) * S : 0) + (c >> 4) * S + slot];
    const float sc = kv4_scale(p);
    const int z = (int)(p & 15u);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)((int)((w >> (4 * e)) & 15u) - z) * sc;
  }
  kv4_store8<DT>(is_v ? v : k, ((int64_t)row * s.H + h) * D + 8 * c, x);
}

// Threads and workgroups of one row of `items` threads.
static void kv4_split(int64_t items, int& threads, int& parts) {
  threads = (int)std::min<int64_t>(256, (items + 63) / 64 * 64);
  parts = (int)((items + threads - 1) / threads);
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
  k_kv4_dequant<DT, D><<<(unsigned)((int64_t)s.T * parts), threads, 0, st>>>(s, k, v, parts);
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
