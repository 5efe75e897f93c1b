// Expert routing around the experts' products: which experts each token goes
// to and with what weight (route), which row of the products belongs to which
// token and expert (plan), and the weighted sum of a token's rows (combine).
#include "qg_f8.hpp"
#include "qg_launch.hpp"

namespace qg {

__device__ __forceinline__ float logit_f32(float v) { return v; }
__device__ __forceinline__ float logit_f32(_Float16 v) { return (float)v; }
__device__ __forceinline__ float logit_f32(uint16_t v) { return bf16_bits_to_f32(v); }

// ---------------------------------------------------------------------------
// Route: one wave per token, expert e = 64 i + lane in register i.
//
// The choice compares score + bias in binary64: scores of different experts
// differ by less than their binary32 errors now and then, and then the order
// would hang on the order of the sums.  Equal values go to the lowest expert.
// A closed expert (logit -inf or NaN, or a bias that makes the value -inf or
// NaN) has the value -inf and is never chosen.
// ---------------------------------------------------------------------------
constexpr int kRouteWaves = 4;
constexpr int kRouteMaxExperts = 1024;

template <int EPL, typename T>
__global__ __launch_bounds__(64 * kRouteWaves) void k_route(
    const T* __restrict__ logits, const float* __restrict__ bias, int64_t tokens, int E,
    int groups, int top_groups, int k, int sigmoid, int renormalize, float scale,
    int32_t* __restrict__ expert, float* __restrict__ weight) {
  __shared__ double values[kRouteWaves][64 * EPL];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (t >= tokens) return;     // no barrier below: the waves are independent
  const double ninf = -__builtin_inf();
  const T* row = logits + t * E;

  float x[EPL];
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = 64 * i + lane;
    float v = e < E ? logit_f32(row[e]) : -__builtin_inff();
    v = v > -__builtin_inff() ? fminf(v, 3.402823466e38f) : -__builtin_inff();   // NaN is closed
    x[i] = v;
    top = fmaxf(top, v);
  }
  double p[EPL], c[EPL];
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] = 1.0 / (1.0 + exp(-(double)x[i]));
  } else {
    top = wave_max(top);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      p[i] = x[i] > -__builtin_inff() ? exp((double)x[i] - (double)top) : 0.0;
      sum += p[i];
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, kWave);
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] = sum > 0.0 ? p[i] / sum : 0.0;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = 64 * i + lane;
    c[i] = bias && e < E ? p[i] + (double)bias[e] : p[i];
    if (!(x[i] > -__builtin_inff()) || !(c[i] > ninf)) c[i] = ninf;
  }

  if (groups > 1) {
    // lane g < groups: the sum of its group's two largest values
    const int size = E / groups;
    double* v = values[wave];
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[64 * i + lane] = c[i];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    double a = ninf, b = ninf;
    if (lane < groups)
      for (int i = 0; i < size; ++i) {
        const double u = v[lane * size + i];
        b = fmax(b, fmin(a, u));
        a = fmax(a, u);
      }
    const double value = b > ninf ? a + b : a;
    int rank = 0;
    for (int g = 0; g < groups; ++g) {
      const double o = __shfl(value, g, kWave);
      rank += o > value || (o == value && g < lane);
    }
    const uint64_t kept = __ballot(lane < groups && rank < top_groups);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = 64 * i + lane;
      if (e < E && !((kept >> (e / size)) & 1)) c[i] = ninf;
    }
  }

  // k times the largest value that is left; lane j keeps choice j
  double mine = 0.0, total = 0.0;
  int chosen = -1;
  for (int s = 0; s < k; ++s) {
    double best = ninf, score = 0.0;
    int at = kRouteMaxExperts;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (c[i] > best) best = c[i], at = 64 * i + lane, score = p[i];
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
      const double ob = __shfl_xor(best, d, kWave), os = __shfl_xor(score, d, kWave);
      const int oa = __shfl_xor(at, d, kWave);
      if (ob > best || (ob == best && oa < at)) best = ob, at = oa, score = os;
    }
    if (!(best > ninf)) break;   // uniform: nothing is left
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (at == 64 * i + lane) c[i] = ninf;
    total += score;
    if (lane == s) chosen = at, mine = score;
  }
  if (lane < k) {
    if (renormalize) mine = total > 0.0 ? mine / total : 0.0;
    expert[t * k + lane] = chosen;
    weight[t * k + lane] = (float)(mine * (double)scale);
  }
}

template <typename T>
static hipError_t route_t(const T* logits, const float* bias, int64_t tokens, int E, int groups,
                          int top_groups, int k, int sigmoid, int renormalize, float scale,
                          int32_t* expert, float* weight, hipStream_t st) {
  const dim3 grid((unsigned)((tokens + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
#define QG_ROUTE(EPL) k_route<EPL, T><<<grid, block, 0, st>>>(logits, bias, tokens, E, groups, top_groups, k, sigmoid, renormalize, scale, expert, weight)
  if (E <= 64) QG_ROUTE(1);
  else if (E <= 128) QG_ROUTE(2);
  else if (E <= 256) QG_ROUTE(4);
  else if (E <= 512) QG_ROUTE(8);
  else QG_ROUTE(16);
#undef QG_ROUTE
  return hipGetLastError();
}

hipError_t launch_route(const void* logits, int dtype, const float* bias, int64_t tokens,
                        int64_t E, int64_t groups, int64_t top_groups, int64_t k, int sigmoid,
                        int renormalize, float scale, int32_t* expert, float* weight,
                        hipStream_t st) {
  const int e = (int)E, g = (int)groups, tg = (int)top_groups, kk = (int)k;
  switch (dtype) {
    case F32: return route_t((const float*)logits, bias, tokens, e, g, tg, kk, sigmoid, renormalize, scale, expert, weight, st);
    case F16: return route_t((const _Float16*)logits, bias, tokens, e, g, tg, kk, sigmoid, renormalize, scale, expert, weight, st);
    default: return route_t((const uint16_t*)logits, bias, tokens, e, g, tg, kk, sigmoid, renormalize, scale, expert, weight, st);
  }
}

// ---------------------------------------------------------------------------
// Plan: a stable sort of the choices by expert in one launch without
// workspace or atomics.  Workgroup e reads all choices twice: once to count
// those of lower experts (where its rows start) and its own in each wave's
// run, once to place its own in order.  Workgroup E does the same for the
// entries that are no expert.
// ---------------------------------------------------------------------------
constexpr int kPlanWaves = 8;

__global__ __launch_bounds__(64 * kPlanWaves) void k_plan(const int32_t* __restrict__ expert,
                                                          int n, int k, int E, int vec,
                                                          int32_t* __restrict__ offsets,
                                                          int32_t* __restrict__ row_token,
                                                          int32_t* __restrict__ slot) {
  __shared__ int below[kPlanWaves], own[kPlanWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const u32 me = blockIdx.x;   // E: entries outside 0 .. E-1
  // four consecutive entries a lane; every wave a contiguous run of them
  const int steps = (n + 255) / 256, per = (steps + kPlanWaves - 1) / kPlanWaves;
  const int s0 = wave * per, s1 = min(s0 + per, steps);
  auto fetch = [&](int s, u32 (&id)[4]) {
    const int at = s * 256 + 4 * lane;
    if (vec && at + 4 <= n) {
      const v4i v = ld16(expert + at);
#pragma unroll
      for (int q = 0; q < 4; ++q) id[q] = (u32)v[q] < (u32)E ? (u32)v[q] : (u32)E;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const u32 v = at + q < n ? (u32)expert[at + q] : 0xffffffffu;
        id[q] = at + q < n ? (v < (u32)E ? v : (u32)E) : 0xffffffffu;
      }
    }
  };
  int less = 0, mine = 0;
  for (int s = s0; s < s1; ++s) {
    u32 id[4];
    fetch(s, id);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      less += id[q] < me;
      mine += id[q] == me;
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    less += __shfl_xor(less, d, kWave);
    mine += __shfl_xor(mine, d, kWave);
  }
  if (lane == 0) below[wave] = less, own[wave] = mine;
  __syncthreads();
  int start = 0, pos = 0;
  for (int w = 0; w < kPlanWaves; ++w) {
    start += below[w];
    pos += w < wave ? own[w] : 0;
  }
  pos += start;
  if (threadIdx.x == 0) offsets[me] = start;
  const uint64_t before = (1ull << lane) - 1;
  for (int s = s0; s < s1; ++s) {
    u32 id[4];
    fetch(s, id);
    int ahead = 0, all = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint64_t b = __ballot(id[q] == me);
      ahead += __popcll(b & before);
      all += __popcll(b);
    }
    if (all == 0) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (id[q] == me) {
        const int at = s * 256 + 4 * lane + q, to = pos + ahead++;
        slot[at] = me < (u32)E ? to : -1;
        row_token[to] = me < (u32)E ? at / k : -1;
      }
    pos += all;
  }
}

hipError_t launch_plan(const int32_t* expert, int64_t T, int64_t k, int64_t E, int32_t* offsets,
                       int32_t* row_token, int32_t* slot, hipStream_t st) {
  k_plan<<<dim3((unsigned)(E + 1)), dim3(64 * kPlanWaves), 0, st>>>(
      expert, (int)(T * k), (int)k, (int)E, (uintptr_t)expert % 16 == 0, offsets, row_token, slot);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Combine: y[t] = sum_j weight[t,j] rows[slot[t,j]], in the order of j, in
// binary32.  A thread owns 16 bytes of a row; a token's slots and weights
// are the same for its whole workgroup.  Bound by reading the rows.
// ---------------------------------------------------------------------------
constexpr int kCombineThreads = 256;

template <typename T, typename OutT, bool VEC>
__global__ __launch_bounds__(kCombineThreads) void k_combine(
    const T* __restrict__ rows, const int32_t* __restrict__ slot, const float* __restrict__ weight,
    int k, int64_t R, int N, int chunks, OutT* __restrict__ y) {
  constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;
  const int64_t t = blockIdx.x / chunks;
  const int n = ((int)(blockIdx.x % chunks) * kCombineThreads + (int)threadIdx.x) * V;
  if (n >= N) return;
  typedef T vec __attribute__((ext_vector_type(V)));
  typedef OutT ovec __attribute__((ext_vector_type(V)));
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  for (int j = 0; j < k; ++j) {
    const int64_t r = slot[t * k + j];
    if (r < 0 || r >= R) continue;
    const float w = weight[t * k + j];
    if constexpr (VEC) {
      const vec v = *reinterpret_cast<const vec*>(rows + r * N + n);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(w, logit_f32((T)v[i]), acc[i]);
    } else {
      acc[0] = fmaf(w, logit_f32(rows[r * N + n]), acc[0]);
    }
  }
  if constexpr (VEC) {
    ovec o;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = Out<OutT>::cvt(acc[i]);
    *reinterpret_cast<ovec*>(y + t * N + n) = o;
  } else {
    y[t * N + n] = Out<OutT>::cvt(acc[0]);
  }
}

template <typename T, typename OutT>
static hipError_t combine_to(const T* rows, const int32_t* slot, const float* weight, int64_t tokens,
                             int k, int64_t R, int N, OutT* y, hipStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  // whole vectors where every row of both sides is aligned to them
  const bool whole = N % V == 0 && (uintptr_t)rows % 16 == 0 && (uintptr_t)y % (V * sizeof(OutT)) == 0;
  const int v = whole ? V : 1;
  const int chunks = (N + kCombineThreads * v - 1) / (kCombineThreads * v);
  const dim3 grid((unsigned)(tokens * chunks)), block(kCombineThreads);
  if (v > 1) k_combine<T, OutT, true><<<grid, block, 0, st>>>(rows, slot, weight, k, R, N, chunks, y);
  else k_combine<T, OutT, false><<<grid, block, 0, st>>>(rows, slot, weight, k, R, N, chunks, y);
  return hipGetLastError();
}

template <typename T>
static hipError_t combine_t(const T* rows, const int32_t* slot, const float* weight, int64_t tokens,
                            int k, int64_t R, int N, void* y, int y_dtype, hipStream_t st) {
  switch (y_dtype) {
    case F32: return combine_to(rows, slot, weight, tokens, k, R, N, (float*)y, st);
    case F16: return combine_to(rows, slot, weight, tokens, k, R, N, (_Float16*)y, st);
    default: return combine_to(rows, slot, weight, tokens, k, R, N, (uint16_t*)y, st);
  }
}

hipError_t launch_combine(const void* rows, int dtype, const int32_t* slot, const float* weight,
                          int64_t tokens, int64_t k, int64_t R, int64_t N, void* y, int y_dtype,
                          hipStream_t st) {
  switch (dtype) {
    case F32: return combine_t((const float*)rows, slot, weight, tokens, (int)k, R, (int)N, y, y_dtype, st);
    case F16: return combine_t((const _Float16*)rows, slot, weight, tokens, (int)k, R, (int)N, y, y_dtype, st);
    default: return combine_t((const uint16_t*)rows, slot, weight, tokens, (int)k, R, (int)N, y, y_dtype, st);
  }
}

}  // namespace qg
