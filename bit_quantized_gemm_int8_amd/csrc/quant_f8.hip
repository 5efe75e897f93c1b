// e4m3 quantizers with one binary32 scale for each 128 inputs of a token
// (activations) or for each 128 x 128 block (weights); see qg_f8.hpp for the
// rounding.
//
// Both are bound by memory: an input is read once and its code written once.
#include "qg_f8.hpp"
#include "qg_launch.hpp"

namespace qg {

// Sixteen consecutive inputs as binary32 (exact widening).
template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&v)[16]);
template <>
__device__ __forceinline__ void load16<float>(const float* p, float (&v)[16]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const v4i w = ld16(p + 4 * c);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * c + i] = __int_as_float(w[i]);
  }
}
template <>
__device__ __forceinline__ void load16<uint16_t>(const uint16_t* p, float (&v)[16]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const v4i w = ld16(p + 8 * c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[8 * c + 2 * i] = bf16_bits_to_f32((u32)w[i] & 0xffffu);
      v[8 * c + 2 * i + 1] = __uint_as_float((u32)w[i] & 0xffff0000u);
    }
  }
}
template <>
__device__ __forceinline__ void load16<_Float16>(const _Float16* p, float (&v)[16]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const v8h w = __builtin_bit_cast(v8h, ld16(p + 8 * c));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[8 * c + i] = (float)w[i];
  }
}

// Magnitudes are compared as bit patterns, which order like the values they
// stand for and put NaN above infinity: a NaN is not lost in the maximum.
__device__ __forceinline__ int mag_bits(float v) { return __float_as_int(v) & 0x7fffffff; }

// Max over each aligned group of 8 lanes.
__device__ __forceinline__ int max_lanes8(int x) {
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, false));    // quad_perm [1,0,3,2]
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, false));    // quad_perm [2,3,0,1]
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, false));   // row_half_mirror
  return x;
}

// The codes of 16 inputs; zeros where the scale is 0 or not finite.
__device__ __forceinline__ v4i codes16(const float (&v)[16], float s) {
  v4i q = {0, 0, 0, 0};
  if (s > 0.f && s < __builtin_inff()) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[i] = f8_pair<false>(v[4 * i] / s, v[4 * i + 1] / s, 0);
      q[i] = f8_pair<true>(v[4 * i + 2] / s, v[4 * i + 3] / s, q[i]);
    }
  }
  return q;
}

// A group of 128 inputs lies with 8 consecutive lanes, 16 inputs each, so a
// group needs no memory but registers and three DPP steps.  Where K is a
// multiple of 128 (WHOLE) group i is simply the i-th run of 128 inputs.
constexpr int kQuantF8Threads = 256;

template <typename T, bool WHOLE>
__global__ __launch_bounds__(kQuantF8Threads) void k_quant_f8_rows(const T* __restrict__ x,
                                                                   int64_t groups, int K, int G,
                                                                   uint8_t* __restrict__ xq,
                                                                   float* __restrict__ xs) {
  const int64_t gi = (int64_t)blockIdx.x * (kQuantF8Threads / 8) + (threadIdx.x >> 3);
  const int c = threadIdx.x & 7;
  if (gi >= groups) return;   // the 8 lanes of a group leave together
  int64_t at;
  bool in = true;
  if constexpr (WHOLE) {
    at = gi * kF8Block + 16 * c;
  } else {
    const int64_t m = gi / G;
    const int k = (int)(gi - m * G) * kF8Block + 16 * c;
    in = k < K;               // K is a multiple of 16: a lane is in or out
    at = m * K + k;
  }
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.f;
  if (in) load16<T>(x + at, v);
  int a = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = max(a, mag_bits(v[i]));
  const float s = __int_as_float(max_lanes8(a)) / kF8Max;
  if (in) st16(xq + at, codes16(v, s));
  if (c == 0) xs[gi] = s;
}

template <typename T>
static hipError_t quant_f8_rows_t(const T* x, int64_t M, int64_t K, uint8_t* xq, float* xs,
                                  hipStream_t st) {
  const int64_t G = (K + kF8Block - 1) / kF8Block, groups = M * G;
  const int per = kQuantF8Threads / 8;
  const dim3 grid((unsigned)((groups + per - 1) / per)), block(kQuantF8Threads);
  if (K % kF8Block == 0)
    k_quant_f8_rows<T, true><<<grid, block, 0, st>>>(x, groups, (int)K, (int)G, xq, xs);
  else
    k_quant_f8_rows<T, false><<<grid, block, 0, st>>>(x, groups, (int)K, (int)G, xq, xs);
  return hipGetLastError();
}

hipError_t launch_quant_f8_rows(const void* x, int x_dtype, int64_t M, int64_t K, uint8_t* xq,
                                float* xs, hipStream_t st) {
  switch (x_dtype) {
    case F32: return quant_f8_rows_t((const float*)x, M, K, xq, xs, st);
    case F16: return quant_f8_rows_t((const _Float16*)x, M, K, xq, xs, st);
    default: return quant_f8_rows_t((const uint16_t*)x, M, K, xq, xs, st);
  }
}

// ---------------------------------------------------------------------------
// Weights: one workgroup per 128 x 128 block.  w is [K][N], the codes are
// [N][K], so the block is read along n, held in registers over the block's
// maximum, and turned through LDS: a thread owns 16 consecutive k of 4
// columns, writes each column's 16 codes as one chunk, and rows of 128 codes
// leave as whole lines.
// ---------------------------------------------------------------------------
constexpr int kQuantF8WThreads = 256;

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(_Float16 v) { return (float)v; }
__device__ __forceinline__ float widen(uint16_t v) { return bf16_bits_to_f32(v); }

template <typename T> struct Vec4;
template <> struct Vec4<float> { typedef v4f type; };
template <> struct Vec4<_Float16> { typedef _Float16 type __attribute__((ext_vector_type(4))); };
template <> struct Vec4<uint16_t> { typedef uint16_t type __attribute__((ext_vector_type(4))); };

template <typename T>
__global__ __launch_bounds__(kQuantF8WThreads) void k_quant_f8_weight(
    const T* __restrict__ w, int K, int N, int G, int B, int vec, uint8_t* __restrict__ wq,
    float* __restrict__ ws) {
  __shared__ __attribute__((aligned(16))) int8_t tile[kF8Block * kF8Block];
  __shared__ int red[kQuantF8WThreads / kWave];
  static_assert(kQuantF8WThreads == 4 * kWave, "four waves meet in red");
  const int64_t blk = blockIdx.x;                    // (expert, n block, k block)
  const int g = (int)(blk % G);
  const int64_t eb = blk / G;
  const int b = (int)(eb % B);
  const int64_t e = eb / B;
  const int tid = threadIdx.x;
  const int n0 = b * kF8Block + 4 * (tid & 31), k0 = g * kF8Block + 16 * (tid >> 5);
  const T* src = w + (e * K + k0) * N + n0;
  float v[4][16];
#pragma unroll
  for (int p = 0; p < 16; ++p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i][p] = 0.f;
    if (k0 < K) {                                    // K is a multiple of 16
      if (vec) {
        if (n0 < N) {                                // N is a multiple of 4
          const typename Vec4<T>::type t = *reinterpret_cast<const typename Vec4<T>::type*>(src + (int64_t)p * N);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i][p] = widen((T)t[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n0 + i < N) v[i][p] = widen(src[(int64_t)p * N + i]);
      }
    }
  }
  int a = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int p = 0; p < 16; ++p) a = max(a, mag_bits(v[i][p]));
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) a = max(a, __shfl_xor(a, d, kWave));
  if ((tid & 63) == 0) red[tid >> 6] = a;
  __syncthreads();
  a = max(max(red[0], red[1]), max(red[2], red[3]));
  const float s = __int_as_float(a) / kF8Max;
  // chunk c of row r sits at slot c ^ ((r >> 2) & 7): the 32 lanes of a write
  // hold rows 4 apart, so every 8 of them hit 8 different chunk slots
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * (tid & 31) + i, c = tid >> 5;
    st16(tile + r * kF8Block + ((c ^ ((r >> 2) & 7)) << 4), codes16(v[i], s));
  }
  __syncthreads();
  if (tid == 0) ws[(e * B + b) * G + g] = s;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int r = 32 * p + (tid >> 3), c = tid & 7;
    const int n = b * kF8Block + r, k = g * kF8Block + 16 * c;
    if (n < N && k < K)
      st16(wq + (e * N + n) * (int64_t)K + k, ld16(tile + r * kF8Block + ((c ^ ((r >> 2) & 7)) << 4)));
  }
}

template <typename T>
static hipError_t quant_f8_weight_t(const T* w, int64_t E, int64_t K, int64_t N, uint8_t* wq,
                                    float* ws, hipStream_t st) {
  const int64_t G = (K + kF8Block - 1) / kF8Block, B = (N + kF8Block - 1) / kF8Block;
  const int vec = N % 4 == 0;   // then every row of 4 columns is aligned to its vector
  k_quant_f8_weight<T><<<dim3((unsigned)(E * B * G)), dim3(kQuantF8WThreads), 0, st>>>(
      w, (int)K, (int)N, (int)G, (int)B, vec, wq, ws);
  return hipGetLastError();
}

hipError_t launch_quant_f8_weight(const void* w, int w_dtype, int64_t E, int64_t K, int64_t N,
                                  uint8_t* wq, float* ws, hipStream_t st) {
  switch (w_dtype) {
    case F32: return quant_f8_weight_t((const float*)w, E, K, N, wq, ws, st);
    case F16: return quant_f8_weight_t((const _Float16*)w, E, K, N, wq, ws, st);
    default: return quant_f8_weight_t((const uint16_t*)w, E, K, N, wq, ws, st);
  }
}

}  // namespace qg
