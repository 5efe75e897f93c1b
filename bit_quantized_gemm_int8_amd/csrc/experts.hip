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
// The choice is defined by score + bias in binary64, equal values to the lowest
// expert: scores of different experts differ by less than their binary32 errors
// now and then, and the order would hang on the arithmetic.  A closed expert
// (logit -inf or NaN, or a bias that makes the value -inf or NaN) has the value
// -inf and is never chosen.
//
// Binary64 for all of a token's experts costs more than reading them (16384
// tokens, 256 experts, 8 choices: 105 us against 9 as below), so the wave
// chooses by binary32 values first and checks that every two neighbours in the
// order it finds, the first value not chosen among them, are further apart than
// their errors (or have the same logit and bias, and then the same value in any
// arithmetic); only otherwise it takes binary64.  Without bias and groups the
// score rises with the logit, and logits are compared as they are.
// ---------------------------------------------------------------------------
constexpr int kRouteWaves = 4;
constexpr int kRouteMaxExperts = 1024;
constexpr float kInf = __builtin_inff();

struct RouteArgs {
  const float* bias;
  int E, groups, top_groups, k, sigmoid, renormalize;
  float scale;
};

// The definition: logits x (closed ones -inf) of one token, the largest `top`.
template <int EPL>
__device__ __noinline__ void route_exact(const float* xs, float top, const RouteArgs& a,
                                         double* values, int32_t* expert, float* weight) {
  const int lane = threadIdx.x & 63;
  const double ninf = -__builtin_inf();
  float x[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) x[i] = xs[i];
  double p[EPL], c[EPL];
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] = 1.0 / (1.0 + exp(-(double)x[i]));
  } else {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      p[i] = x[i] > -kInf ? exp((double)x[i] - (double)top) : 0.0;
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
    c[i] = a.bias && e < a.E ? p[i] + (double)a.bias[e] : p[i];
    if (!(x[i] > -kInf) || !(c[i] > ninf)) c[i] = ninf;
  }

  if (a.groups > 1) {
    // lane g < groups: the sum of its group's two largest values
    const int size = a.E / a.groups;
#pragma unroll
    for (int i = 0; i < EPL; ++i) values[64 * i + lane] = c[i];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    double u = ninf, v = ninf;
    if (lane < a.groups)
      for (int i = 0; i < size; ++i) {
        const double w = values[lane * size + i];
        v = fmax(v, fmin(u, w));
        u = fmax(u, w);
      }
    const double value = v > ninf ? u + v : u;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double o = __shfl(value, g, kWave);
      rank += o > value || (o == value && g < lane);
    }
    const uint64_t kept = __ballot(lane < a.groups && rank < a.top_groups);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = 64 * i + lane;
      if (e < a.E && !((kept >> (e / size)) & 1)) c[i] = ninf;
    }
  }

  // k times the largest value that is left; lane j keeps choice j
  double mine = 0.0, total = 0.0;
  int chosen = -1;
  for (int s = 0; s < a.k; ++s) {
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
  if (lane < a.k) {
    if (a.renormalize) mine = total > 0.0 ? mine / total : 0.0;
    expert[lane] = chosen;
    weight[lane] = (float)(mine * (double)a.scale);
  }
}

// Floats as integers of the same order (-0 is taken out first); closed: kClosed.
constexpr int kClosed = (int)0x80000000;
__device__ __forceinline__ int order_key(float v) {
  const int b = __float_as_int(v + 0.f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float key_value(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }

// Max of integers over a wave: rotations within rows of 16 lanes, then the four
// rows' values read into scalars.  The result is uniform.
__device__ __forceinline__ int wave_max_int(int x) {
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x121, 0xF, 0xF, false));   // row_ror:1
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x122, 0xF, 0xF, false));   // row_ror:2
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x124, 0xF, 0xF, false));   // row_ror:4
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x128, 0xF, 0xF, false));   // row_ror:8
  return max(max(__builtin_amdgcn_readlane(x, 0), __builtin_amdgcn_readlane(x, 16)),
             max(__builtin_amdgcn_readlane(x, 32), __builtin_amdgcn_readlane(x, 48)));
}

// Bound on the binary32 error of a score p = e^d / sum or 1 / (1 + e^-d): the
// argument of the exponential is off by 2^-23 of itself at most (difference and
// product with log2 e), the exponential, the sum (a tree over at most 16 + 6
// values, 2^-24 each) and the quotient by less than 40 * 2^-24 in all.
__device__ __forceinline__ float score_error(float p, float d) {
  return p * ((1.5f * fabsf(d) + 20.f) * 0x1p-23f) + 0x1p-120f;
}

template <int EPL, typename T>
__global__ __launch_bounds__(64 * kRouteWaves) void k_route(const T* __restrict__ logits,
                                                            int64_t tokens, RouteArgs a,
                                                            int32_t* __restrict__ expert,
                                                            float* __restrict__ weight) {
  __shared__ double values[kRouteWaves][64 * EPL];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (t >= tokens) return;     // no barrier below: the waves are independent
  const T* row = logits + t * a.E;
  expert += t * a.k;
  weight += t * a.k;

  float x[EPL];
  int most = kClosed;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = 64 * i + lane;
    const float v = e < a.E ? logit_f32(row[e]) : -kInf;
    x[i] = v > -kInf ? fminf(v, 3.402823466e38f) : -kInf;   // NaN is closed
    most = max(most, x[i] > -kInf ? order_key(x[i]) : kClosed);
  }
  most = wave_max_int(most);
  const float top = most == kClosed ? -kInf : key_value(most);

  const bool plain = !a.bias && a.groups == 1;
  auto score = [&](float v, float total) {   // of an open logit
    return a.sigmoid ? 1.f / (1.f + __expf(-v)) : __expf(v - top) / total;
  };
  float total = 1.f;
  if (!a.sigmoid && !(plain && a.renormalize)) {
    total = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) total += x[i] > -kInf ? __expf(x[i] - top) : 0.f;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) total += __shfl_xor(total, d, kWave);
  }
  int key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = 64 * i + lane;
    float c = x[i];
    if (!plain && c > -kInf) {
      c = score(c, total);
      if (a.bias) c += a.bias[e];
    }
    key[i] = c > -kInf ? order_key(c) : kClosed;
  }

  bool sure = true;
  if (a.groups > 1) {
    // lane g < groups: the sum of its group's two largest values, and a bound
    // on the sum's error: that of a score of 1 at the far end of the logits
    const int size = a.E / a.groups;
    int* v = reinterpret_cast<int*>(values[wave]);
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[64 * i + lane] = key[i];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    int u = kClosed, w = kClosed;
    if (lane < a.groups) {
      // each lane starts at another place of its group: fewer bank conflicts
      int at = lane % size;
      for (int i = 0; i < size; ++i) {
        const int o = v[lane * size + at];
        w = max(w, min(u, o));
        u = max(u, o);
        at = at + 1 == size ? 0 : at + 1;
      }
    }
    float value = u == kClosed ? -kInf : key_value(u);
    float off = u == kClosed ? 0.f : fabsf(value) * 0x1p-22f;
    if (w != kClosed) {
      const float second = key_value(w);
      off += fabsf(second) * 0x1p-22f;
      value += second;
    }
    // p (1.5 |d| + 20) 2^-23 is at most 1.5 / e + 20 of 2^-23 for each of the two
    off += 2.f * 21.f * 0x1p-23f;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const float o = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(value), g));
      rank += o > value || (o == value && g < lane);
    }
    const bool in = lane < a.groups && rank < a.top_groups;
    const uint64_t kept = __ballot(in);
    // the kept values' lower ends against the others' upper ends; closed groups
    // are last in any arithmetic
    const int low = wave_max_int(in && value > -kInf ? order_key(off - value) : kClosed);
    const int high = wave_max_int(lane < a.groups && !in && value > -kInf ? order_key(value + off) : kClosed);
    if (high != kClosed && !(-key_value(low) > key_value(high))) sure = false;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = 64 * i + lane;
      if (e < a.E && !((kept >> (e / size)) & 1)) key[i] = kClosed;
    }
  }

  // k times the largest value that is left, and once more to see how near the
  // first value not chosen is; lane j keeps choice j
  int chosen = -1, before = kClosed, before_e = 0, count = 0;
  float cx = 0.f, before_x = 0.f;
  for (int s = 0; s <= a.k && sure; ++s) {
    int best = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) best = max(best, key[i]);
    best = wave_max_int(best);
    if (best == kClosed) break;
    int e = -1;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint64_t who = __ballot(key[i] == best);
      if (e < 0 && who) {
        const int l = __builtin_ctzll(who);
        e = 64 * i + l;
        v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x[i]), l));
        if (lane == l) key[i] = kClosed;
      }
    }
    if (s > 0) {
      const float hi = key_value(before), lo = key_value(best), gap = hi - lo;
      bool apart;
      if (plain) {
        // scores rise with the logits: apart in binary64 unless the logits are
        // within a few of its steps, or the scores round to 0 or 1
        apart = a.sigmoid ? gap * __expf(-fmaxf(hi, 0.f)) > 0x1p-44f && lo > -600.f
                          : gap > 0x1p-44f && lo - top > -600.f;
      } else {
        const float pa = score(before_x, total), pb = score(v, total);
        const float da = a.sigmoid ? before_x : before_x - top, db = a.sigmoid ? v : v - top;
        apart = gap > score_error(pa, da) + score_error(pb, db) + (fabsf(hi) + fabsf(lo)) * 0x1p-22f;
      }
      if (!apart) sure = v == before_x && (!a.bias || a.bias[e] == a.bias[before_e]);
    }
    before = best;
    before_e = e;
    before_x = v;
    if (s < a.k) {
      if (lane == s) chosen = e, cx = v;
      ++count;
    }
  }
  if (!sure) {
    route_exact<EPL>(x, top, a, values[wave], expert, weight);
    return;
  }
  // The chosen scores in binary64 (one a lane).  Renormalised softmax needs no
  // sum over the other experts.
  double mine = 0.0;
  if (lane < count) mine = a.sigmoid ? 1.0 / (1.0 + exp(-(double)cx)) : exp((double)cx - (double)top);
  if (a.renormalize) {
    double sum = mine;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, kWave);
    mine = sum > 0.0 ? mine / sum : 0.0;
  } else if (!a.sigmoid) {
    mine = lane < count ? mine / (double)total : 0.0;   // (no expert open: no sum)
  }
  if (lane < a.k) {
    expert[lane] = chosen;
    weight[lane] = (float)(mine * (double)a.scale);
  }
}

template <typename T>
static hipError_t route_t(const T* logits, const float* bias, int64_t tokens, int E, int groups,
                          int top_groups, int k, int sigmoid, int renormalize, float scale,
                          int32_t* expert, float* weight, hipStream_t st) {
  const dim3 grid((unsigned)((tokens + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
  const RouteArgs a{bias, E, groups, top_groups, k, sigmoid, renormalize, scale};
#define QG_ROUTE(EPL) k_route<EPL, T><<<grid, block, 0, st>>>(logits, tokens, a, expert, weight)
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
