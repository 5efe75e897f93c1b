// 8-bit float (e4m3: 4 exponent bits, bias 7, 3 mantissa bits, no infinities,
// largest finite value 448) pieces shared by the block-scaled kernels.
//
// A slice of up to 128 inputs (of one token, or a 128 x 128 block of a weight
// matrix) has s = max|x| / 448 and codes e4m3(x / s): the binary32 quotient,
// correctly rounded, then rounded to the nearest e4m3 value, halves to even.
#pragma once

#include "qg_device.hpp"

namespace qg {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr int kF8Block = 128;
constexpr float kF8Max = 448.f;

// Two codes in the low 16 bits (hi = false) or the high 16 bits (hi = true)
// of a word; the quotients are clamped first, since a subnormal s can come
// out so far below max|x| / 448 that a quotient passes 464, the last value
// that still rounds to 448.
template <bool HI>
__device__ __forceinline__ int f8_pair(float a, float b, int old) {
  a = __builtin_amdgcn_fmed3f(a, -kF8Max, kF8Max);
  b = __builtin_amdgcn_fmed3f(b, -kF8Max, kF8Max);
  return __builtin_amdgcn_cvt_pk_fp8_f32(a, b, old, HI);
}

// Eight codes (two words) as binary16 values: exact, since e4m3 values have 4
// significant bits and lie within 2^-9 .. 448.
__device__ __forceinline__ v8h f8_to_f16x8(int lo, int hi) {
  const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false);
  const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true);
  const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false);
  const v2h d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true);
  return v8h{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Outputs, rounded to nearest even.  bfloat16 by the conversion instruction,
// which keeps every NaN a NaN.
template <typename OutT>
__device__ __forceinline__ OutT round_to(float v) {
  return (OutT)v;
}
template <>
__device__ __forceinline__ uint16_t round_to<uint16_t>(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

}  // namespace qg
