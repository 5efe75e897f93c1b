// The 4-bit paged KV cache: layout, group code, and where a call's rows lie.
//
// pages [P][H][words] int32.  The words of one head of a page of S positions:
//   key codes    [S][D / 8]       code of channel 8 i + j in bits 4 j of word i
//   value codes  [S / 4][D / 8][4]  the same words, four positions side by side
//   key groups   [Gd][S]          scale and zero point of each position and group
//   value groups [Gd][S]
// Groups are min(D, 128) channels, Gd = max(1, D / 128).  Value codes of four
// positions are neighbours because a lane of the attention kernels feeds the
// matrix cores with four positions of one channel word: one 16-byte load.
//
// A group's word: the scale s, a binary32 with 7 significant bits, in the upper
// half, the zero point z in the low 4 bits; a code q stands for (q - z) s.
// (q - z) s then has at most 11 significant bits: it is exact in binary16, up
// to a power of two, so a matrix core can take it as an operand.
#pragma once

#include "qg_device.hpp"
#include "qg_launch.hpp"

namespace qg {

constexpr u32 kKv4Nan = 0x7FC00000u;   // group word of values that are not all finite

__device__ __forceinline__ float kv4_scale(u32 w) { return __uint_as_float(w & 0xFFFF0000u); }

// Words of one head of a page.
__host__ __device__ constexpr int kv4_groups(int D) { return D > 128 ? D / 128 : 1; }
__host__ __device__ constexpr int64_t kv4_words(int S, int D) {
  return (int64_t)S * (D / 4 + 2 * kv4_groups(D));
}

// 8 consecutive channels as binary32.
template <int DT>
__device__ __forceinline__ void kv4_load8(const void* p, int64_t at, float (&v)[8]) {
  if constexpr (DT == F32) {
    const v4i a = ld16((const float*)p + at), b = ld16((const float*)p + at + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = __int_as_float(a[e]);
      v[4 + e] = __int_as_float(b[e]);
    }
  } else {
    const v4i a = ld16((const uint16_t*)p + at);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const u32 u = ((u32)a[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
      v[e] = DT == BF16 ? bf16_bits_to_f32(u) : f16_bits_to_f32((uint16_t)u);
    }
  }
}

// binary32 to bfloat16, nearest even, a NaN staying one.
__device__ __forceinline__ uint16_t kv4_bf16(float f) {
  return f != f ? (uint16_t)0x7FC0u : f32_to_bf16_bits(f);
}

template <int DT>
__device__ __forceinline__ void kv4_store8(void* p, int64_t at, const float (&v)[8]) {
  if constexpr (DT == F32) {
    v4i a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = __float_as_int(v[e]);
      b[e] = __float_as_int(v[4 + e]);
    }
    st16((float*)p + at, a);
    st16((float*)p + at + 4, b);
  } else {
    v4i a;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const u32 lo = DT == BF16 ? kv4_bf16(v[2 * e]) : f32_to_f16_bits(v[2 * e]);
      const u32 hi = DT == BF16 ? kv4_bf16(v[2 * e + 1]) : f32_to_f16_bits(v[2 * e + 1]);
      a[e] = (int)(lo | (hi << 16));
    }
    st16((uint16_t*)p + at, a);
  }
}

// The sequence of row `row` of a call and the row's position, -1 where the
// row belongs to no sequence.  offsets NULL: n_uniform rows for each.
// Reads offsets at 0 .. B only, whatever they hold.
struct Kv4Row {
  int b;
  int64_t pos;
  int64_t end;   // first row behind the sequence's
};

__device__ __forceinline__ Kv4Row kv4_row(const Kv4Seqs& s, int row) {
  int b;
  int64_t end;
  if (s.offsets == nullptr) {
    const int n = s.T / s.B;
    b = row / n;
    end = (int64_t)(b + 1) * n;
  } else {
    int lo = 0, hi = s.B;   // the first b whose rows end behind `row`
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s.offsets[mid + 1] <= row) lo = mid + 1;
      else hi = mid;
    }
    b = lo;
    if (b >= s.B || row < s.offsets[b]) return {-1, -1, 0};
    end = s.offsets[b + 1];
  }
  return {b, (int64_t)s.lengths[b] - end + row, end};
}

// First word of position pos of sequence b in head h, and its slot; NULL
// where the position is outside the page table or its page outside the pool.
__device__ __forceinline__ int32_t* kv4_page(const Kv4Seqs& s, int b, int64_t pos, int h, int D,
                                             int& slot) {
  if (pos < 0 || pos >= ((int64_t)s.W << s.shift)) return nullptr;
  const int id = s.table[(int64_t)b * s.W + (pos >> s.shift)];
  if ((u32)id >= (u32)s.P) return nullptr;
  slot = (int)(pos & ((1 << s.shift) - 1));
  return s.pages + ((int64_t)id * s.H + h) * kv4_words(1 << s.shift, D);
}

}  // namespace qg
