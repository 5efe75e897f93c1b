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
// tokens, 256 experts, 8 choices: 105 us against 13.8 as below), so the wave
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

// A logit as it counts: closed (-inf) for NaN, the largest finite value for +inf.
template <typename T>
__device__ __forceinline__ float logit_at(const T* row, int e) {
  const float v = logit_f32(row[e]);
  return v > -kInf ? fminf(v, 3.402823466e38f) : -kInf;
}

// The definition, for one token by a whole wave.
template <int EPL, typename T>
__device__ void route_exact(const T* row, const RouteArgs& a, double* values, int32_t* expert,
                            float* weight) {
  const int lane = threadIdx.x & 63;
  const double ninf = -__builtin_inf();
  float x[EPL], top = -kInf;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = 64 * i + lane;
    x[i] = e < a.E ? logit_at(row, e) : -kInf;
    top = fmaxf(top, x[i]);
  }
  top = wave_max(top);
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

// Max over the LPT lanes of a token, in all of them.
template <int LPT>
__device__ __forceinline__ int token_max(int x) {
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x121, 0xF, 0xF, false));   // row_ror:1
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x122, 0xF, 0xF, false));   // row_ror:2
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x124, 0xF, 0xF, false));   // row_ror:4
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x128, 0xF, 0xF, false));   // row_ror:8
  if constexpr (LPT == 64)
    x = max(max(__builtin_amdgcn_readlane(x, 0), __builtin_amdgcn_readlane(x, 16)),
            max(__builtin_amdgcn_readlane(x, 32), __builtin_amdgcn_readlane(x, 48)));
  return x;
}

// LPT lanes a token (16, or 64 where a token needs more registers or choices
// than 16 lanes have), expert e = LPT i + its lane in register i: the
// instructions of a choice serve 64 / LPT tokens (16384 tokens, 256 experts:
// 32 us with 64 lanes, 13.8 with 16).
template <int LPT, int EPL, typename T>
__global__ __launch_bounds__(64 * kRouteWaves) void k_route(const T* __restrict__ logits,
                                                            int64_t tokens, RouteArgs a,
                                                            int32_t* __restrict__ expert,
                                                            float* __restrict__ weight) {
  constexpr int TPW = 64 / LPT, EPW = (LPT * EPL + 63) / 64;   // tokens a wave; values a lane of route_exact
  __shared__ __attribute__((aligned(8))) int values[kRouteWaves][TPW * LPT * EPL > 128 * EPW ? TPW * LPT * EPL : 128 * EPW];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane % LPT;
  const int64_t t0 = ((int64_t)blockIdx.x * kRouteWaves + wave) * TPW;
  if (t0 >= tokens) return;    // no barrier below: the waves are independent
  const int64_t t = t0 + lane / LPT;
  const bool here = t < tokens;      // (a token past the end takes part, closed)
  const T* row = logits + t * a.E;

  float x[EPL];
  int most = kClosed;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = LPT * i + l;
    x[i] = here && e < a.E ? logit_at(row, e) : -kInf;
    most = max(most, x[i] > -kInf ? order_key(x[i]) : kClosed);
  }
  most = token_max<LPT>(most);
  const float top = most == kClosed ? 0.f : key_value(most);

  // Binary32 values and a bound on their errors.  A score e^d / sum is off by
  // at most p (1.5 |d| + 20) 2^-23: the argument of the exponential by 2^-23 of
  // itself (difference and product with log2 e), the exponential, the sum (a
  // tree over EPL and 6 more, 2^-24 each) and the quotient by less than 40 *
  // 2^-24; e^d |d| <= 1 / e and p <= 1 / sum make that 21 2^-23 / sum.  A score
  // 1 / (1 + e^-d) has no sum, and p (1 - p) |d| < 0.3: 4.5 * 2^-23.
  const bool plain = !a.bias && a.groups == 1;
  float total = 1.f;
  if (!a.sigmoid && !plain) {
    total = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) total += x[i] > -kInf ? __expf(x[i] - top) : 0.f;
#pragma unroll
    for (int d = LPT / 2; d >= 1; d >>= 1) total += __shfl_xor(total, d, kWave);
  }
  const float err = a.sigmoid ? 4.5f * 0x1p-23f : 21.f * 0x1p-23f / fmaxf(total, 1.f);
  // Weights are binary64 scores, rounded once, whether the choice takes binary64
  // or not: softmax that is not renormalised sums all exponentials in it (16384
  // tokens, 256 experts: 18.6 us; 13.9 with `total`, whose error, up to 40 * 2^-24
  // of a weight, then shows).
  double sum64 = 1.0;
  if (!a.sigmoid && !a.renormalize) {
    sum64 = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum64 += x[i] > -kInf ? exp((double)x[i] - (double)top) : 0.0;
#pragma unroll
    for (int d = LPT / 2; d >= 1; d >>= 1) sum64 += __shfl_xor(sum64, d, kWave);
  }
  int key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = LPT * i + l;
    float c = x[i];
    if (!plain && c > -kInf) {
      c = a.sigmoid ? 1.f / (1.f + __expf(-c)) : __expf(c - top) / total;
      if (a.bias) c += a.bias[e];
    }
    key[i] = c > -kInf ? order_key(c) : kClosed;
  }

  bool sure = true;
  if (a.groups > 1) {
    // lane l < groups of a token: the sum of its group's two largest values
    const int size = a.E / a.groups;
    int* v = values[wave] + lane / LPT * (LPT * EPL);
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[LPT * i + l] = key[i];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    int u = kClosed, w = kClosed;
    if (l < a.groups) {
      // each lane starts at another place of its group: fewer bank conflicts
      int at = l % size;
      for (int i = 0; i < size; ++i) {
        const int o = v[l * size + at];
        w = max(w, min(u, o));
        u = max(u, o);
        at = at + 1 == size ? 0 : at + 1;
      }
    }
    float value = u == kClosed ? -kInf : key_value(u);
    // a value is off by its score's error and a rounding, the sum by another
    float off = 2.f * err;
    if (u != kClosed) {
      const float second = w == kClosed ? 0.f : key_value(w);
      off += (fabsf(value) + fabsf(second)) * 0x1p-22f;
      value += second;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const float o = __shfl(value, lane - l + g, kWave);
      rank += o > value || (o == value && g < l);
    }
    const bool in = l < a.groups && rank < a.top_groups;
    const uint64_t kept = __ballot(in) >> (lane - l);
    // the kept values' lower ends against the others' upper ends; closed groups
    // are last in any arithmetic
    const int low = token_max<LPT>(in && value > -kInf ? order_key(off - value) : kClosed);
    const int high = token_max<LPT>(l < a.groups && !in && value > -kInf ? order_key(value + off) : kClosed);
    if (high != kClosed && !(-key_value(low) > key_value(high))) sure = false;
    // e / size as a product: e < 2^10 and the factor is less than one too large
    const u32 by = ((1u << 20) + size - 1) / size;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = LPT * i + l;
      if (!(e < a.E && ((kept >> ((e * by) >> 20)) & 1))) key[i] = kClosed;
    }
  }

  // k times the largest value that is left, the lowest expert of equal ones,
  // and once more to see how near the first value not chosen is; lane j keeps
  // choice j
  int chosen = -1, before = kClosed, before_e = 0;
  for (int s = 0; s <= a.k; ++s) {
    int m = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = max(m, key[i]);
    const int best = token_max<LPT>(m);
    if (!__any(best != kClosed)) break;
    int e = kRouteMaxExperts;
#pragma unroll
    for (int i = EPL - 1; i >= 0; --i) e = key[i] == best ? LPT * i + l : e;
    e = -token_max<LPT>(-e);
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = e - l == LPT * i ? kClosed : key[i];
    if (s > 0 && best != kClosed) {
      const float hi = key_value(before), lo = key_value(best), gap = hi - lo;
      bool apart;
      if (plain)
        // scores rise with the logits: apart in binary64 unless the logits are
        // within a few of its steps, or the scores round to 0 or 1
        apart = a.sigmoid ? gap * __expf(-fmaxf(hi, 0.f)) > 0x1p-44f && lo > -600.f
                          : gap > 0x1p-44f && lo - top > -600.f;
      else
        apart = gap > 2.f * err + (fabsf(hi) + fabsf(lo)) * 0x1p-22f;
      if (!apart)
        sure = sure && logit_at(row, e) == logit_at(row, before_e) && (!a.bias || a.bias[e] == a.bias[before_e]);
    }
    before = best;
    before_e = e;
    if (l == s && s < a.k && best != kClosed) chosen = e;
  }

  // The chosen scores in binary64 (one a lane).  Renormalised softmax needs no
  // sum over the other experts.
  double mine = 0.0;
  if (chosen >= 0) {
    const double d = (double)logit_at(row, chosen);
    mine = a.sigmoid ? 1.0 / (1.0 + exp(-d)) : exp(d - (double)top);
  }
  if (a.renormalize) {
    double sum = mine;
#pragma unroll
    for (int d = LPT / 2; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, kWave);
    mine = sum > 0.0 ? mine / sum : 0.0;
  } else if (!a.sigmoid && chosen >= 0) {
    mine /= sum64;
  }
  if (here && l < a.k) {
    expert[t * a.k + l] = chosen;
    weight[t * a.k + l] = (float)(mine * (double)a.scale);
  }
  // tokens whose order the binary32 values leave open
  for (uint64_t open = __ballot(here && !sure && l == 0); open; open &= open - 1) {
    const int64_t o = t0 + __builtin_ctzll(open) / LPT;
    route_exact<EPW>(logits + o * a.E, a, reinterpret_cast<double*>(values[wave]), expert + o * a.k, weight + o * a.k);
  }
}

template <typename T>
static hipError_t route_t(const T* logits, const float* bias, int64_t tokens, int E, int groups,
                          int top_groups, int k, int sigmoid, int renormalize, float scale,
                          int32_t* expert, float* weight, hipStream_t st) {
  const RouteArgs a{bias, E, groups, top_groups, k, sigmoid, renormalize, scale};
  auto go = [&](auto kernel, int tokens_per_wave) {
    const int64_t per = kRouteWaves * tokens_per_wave;
    kernel<<<dim3((unsigned)((tokens + per - 1) / per)), dim3(64 * kRouteWaves), 0, st>>>(logits, tokens, a, expert, weight);
  };
  if (E <= 256 && k <= 16 && groups <= 16) {
    if (E <= 16) go(k_route<16, 1, T>, 4);
    else if (E <= 64) go(k_route<16, 4, T>, 4);
    else if (E <= 128) go(k_route<16, 8, T>, 4);
    else go(k_route<16, 16, T>, 4);
  } else {
    if (E <= 256) go(k_route<64, 4, T>, 1);
    else if (E <= 512) go(k_route<64, 8, T>, 1);
    else go(k_route<64, 16, T>, 1);
  }
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
// Plan: a stable sort of the choices by expert in one launch, without
// workspace; counts are integers, so their order does not matter, and places
// follow from counts and lane order alone.
//
// Few choices (up to 4096): workgroup e reads them all, counts those of lower
// experts (where its rows start) and its own, and places its own in order.
// Workgroup E does the same for the entries that are no expert.
// ---------------------------------------------------------------------------
template <int WAVES, int kPlanBatch>
__global__ __launch_bounds__(64 * WAVES) void k_plan(const int32_t* __restrict__ expert, int n,
                                                     int k, int E, int vec,
                                                     int32_t* __restrict__ offsets,
                                                     int32_t* __restrict__ row_token,
                                                     int32_t* __restrict__ slot) {
  __shared__ int below[WAVES], own[WAVES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const u32 me = blockIdx.x;   // E: entries outside 0 .. E-1
  // four consecutive entries a lane; every wave a contiguous run of at most
  // kPlanBatch steps, whose loads are all issued before the first is used
  const int steps = (n + 255) / 256, per = (steps + WAVES - 1) / WAVES;
  const int s0 = wave * per, s1 = min(s0 + per, steps);
  struct Batch {
    u32 id[kPlanBatch][4];     // past n: no one's (0xffffffff)
  };
  auto fetch = [&](int b, Batch& v) {
#pragma unroll
    for (int q = 0; q < kPlanBatch; ++q) {
      const int at = (b + q) * 256 + 4 * lane;
      if (vec && b + q < s1 && at + 4 <= n) {
        const v4i w = ld16(expert + at);
#pragma unroll
        for (int c = 0; c < 4; ++c) v.id[q][c] = (u32)w[c];
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) v.id[q][c] = b + q < s1 && at + c < n ? (u32)expert[at + c] : 0xffffffffu;
      }
    }
#pragma unroll
    for (int q = 0; q < kPlanBatch; ++q)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        v.id[q][c] = b + q < s1 && (b + q) * 256 + 4 * lane + c < n ? min(v.id[q][c], (u32)E) : 0xffffffffu;
  };
  Batch v;
  int less = 0, mine = 0;
  fetch(s0, v);
#pragma unroll
  for (int q = 0; q < kPlanBatch; ++q)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      less += v.id[q][c] < me;
      mine += v.id[q][c] == me;
    }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    less += __shfl_xor(less, d, kWave);
    mine += __shfl_xor(mine, d, kWave);
  }
  if (lane == 0) below[wave] = less, own[wave] = mine;
  __syncthreads();
  int start = 0, pos = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    start += below[w];
    pos += w < wave ? own[w] : 0;
  }
  pos += start;
  if (threadIdx.x == 0) offsets[me] = start;
  const uint64_t before = (1ull << lane) - 1;
#pragma unroll
  for (int q = 0; q < kPlanBatch; ++q) {
    uint64_t who[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) who[c] = __ballot(v.id[q][c] == me);
    if (!(who[0] | who[1] | who[2] | who[3])) continue;
    int ahead = 0, all = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      ahead += __popcll(who[c] & before);
      all += __popcll(who[c]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (v.id[q][c] == me) {
        const int at = (s0 + q) * 256 + 4 * lane + c, to = pos + ahead++;
        slot[at] = me < (u32)E ? to : -1;
        row_token[to] = me < (u32)E ? (int)((u32)at / (u32)k) : -1;
      }
    pos += all;
  }
}

// Many choices: a workgroup owns a segment of `chunks` chunks of 1024 R of them,
// and counts all choices by expert in LDS, those ahead of its segment apart.
// A wave's 64 R choices of a chunk are ranked among equals by ballots over the
// bits of the expert; the counts of the waves before it, of the chunks and of
// the segments before give the row.  Slots leave as whole lines from one XCD
// and the rows of an expert in runs (a workgroup for each expert, scattering
// its slots over lines that other XCDs write too: 45 us for 131072 choices of
// 256 experts, 14.5 so).  Every workgroup reads all choices, so there are at
// most as many as CUs, and the time grows with the choices (2^20: 112 us, 2^22:
// 0.46 ms, 2^25: 4.0 ms; a workgroup for each chunk: 27.8 ms).
constexpr int kPlanWaves = 16;
constexpr int kPlanBuckets = kRouteMaxExperts + 1;   // the last: no expert
constexpr int64_t kPlanSegments = 256;

template <int R>
__global__ __launch_bounds__(64 * kPlanWaves) void k_plan_segments(
    const int32_t* __restrict__ expert, int n, int k, int E, int chunks, int vec,
    int32_t* __restrict__ offsets, int32_t* __restrict__ row_token, int32_t* __restrict__ slot) {
  __shared__ int ahead[kPlanBuckets], rest[kPlanBuckets], base[kPlanWaves][kPlanBuckets];
  __shared__ int sums[kPlanWaves];
  constexpr int kThreads = 64 * kPlanWaves;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // consecutive segments on one XCD, so that the runs they write meet in its L2
  const int per = gridDim.x / 8, rem = gridDim.x % 8, xcd = blockIdx.x % 8;
  const int64_t seg = (int64_t)(xcd * per + min(xcd, rem) + (int)blockIdx.x / 8) * chunks * (kThreads * R);
  auto clear_base = [&] {
    for (int e = tid; e <= E; e += kThreads)
      for (int w = 0; w < kPlanWaves; ++w) base[w][e] = 0;
  };
  for (int e = tid; e <= E; e += kThreads) ahead[e] = rest[e] = 0;
  clear_base();
  __syncthreads();
  auto bucket = [&](int id) { return (u32)id < (u32)E ? id : E; };
  // segments start at multiples of 4, so four consecutive entries lie on one
  // side of seg
  for (int64_t at = 4 * tid; at < n; at += 4 * kThreads) {
    int* const to = at < seg ? ahead : rest;
    if (vec && at + 4 <= n) {
      const v4i v = ld16(expert + at);
#pragma unroll
      for (int c = 0; c < 4; ++c) atomicAdd(&to[bucket(v[c])], 1);
    } else {
      for (int c = 0; c < 4 && at + c < n; ++c) atomicAdd(&to[bucket(expert[at + c])], 1);
    }
  }
  const int bits = 32 - __builtin_clz((u32)E);       // of 0 .. E
  int64_t first = seg;                               // of the chunk
  for (int chunk = 0;;) {
    // ranks of this wave's choices among its own of the same expert
    int id[R], rank[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t at = first + (wave * R + r) * 64 + lane;
      const bool in = at < n;
      id[r] = in ? bucket(expert[at]) : 0;
      uint64_t same = __ballot(in);
      for (int b = 0; b < bits; ++b) {
        const uint64_t one = __ballot((id[r] >> b) & 1);
        same &= (id[r] >> b) & 1 ? one : ~one;
      }
      const int mine = __popcll(same & ((1ull << lane) - 1));
      // one wave's LDS accesses execute in order
      rank[r] = in ? base[wave][id[r]] + mine : -1;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (in && mine == 0) base[wave][id[r]] += __popcll(same);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    __syncthreads();
    if (chunk == 0) {
      // ahead becomes the first row of the segment's choices of each bucket: a
      // scan over the totals; a thread has one bucket, and the last thread the
      // one past 1023 too
      const int total = tid <= E ? ahead[tid] + rest[tid] : 0;
      int run = total;
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) {
        const int t = __shfl_up(run, d, kWave);
        if (lane >= d) run += t;
      }
      if (lane == 63) sums[wave] = run;
      __syncthreads();
      int start = run - total;
      for (int w = 0; w < wave; ++w) start += sums[w];
      auto begin = [&](int e, int from) {
        if (blockIdx.x == 0) offsets[e] = from;
        ahead[e] += from;
      };
      if (tid <= E) begin(tid, start);
      if (tid == kThreads - 1 && E == kThreads) begin(E, start + total);
    }
    // (a bucket's thread is the same here and above)
    auto spread = [&](int e) {
      int from = ahead[e];
      for (int w = 0; w < kPlanWaves; ++w) {
        const int c = base[w][e];
        base[w][e] = from;
        from += c;
      }
      ahead[e] = from;
    };
    if (tid <= E) spread(tid);
    if (tid == kThreads - 1 && E == kThreads) spread(E);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (rank[r] < 0) continue;
      const int at = (int)(first + (wave * R + r) * 64 + lane), to = base[wave][id[r]] + rank[r];
      slot[at] = id[r] < E ? to : -1;
      row_token[to] = id[r] < E ? (int)((u32)at / (u32)k) : -1;
    }
    first += kThreads * R;
    if (++chunk == chunks || first >= n) break;      // alike for the whole workgroup
    __syncthreads();
    clear_base();
    __syncthreads();
  }
}

hipError_t launch_plan(const int32_t* expert, int64_t T, int64_t k, int64_t E, int32_t* offsets,
                       int32_t* row_token, int32_t* slot, hipStream_t st) {
  const int n = (int)(T * k), vec = (uintptr_t)expert % 16 == 0;
  if (n <= 4096) {
    const dim3 grid((unsigned)(E + 1)), block(256);
    if (n <= 1024) k_plan<4, 1><<<grid, block, 0, st>>>(expert, n, (int)k, (int)E, vec, offsets, row_token, slot);
    else k_plan<4, 4><<<grid, block, 0, st>>>(expert, n, (int)k, (int)E, vec, offsets, row_token, slot);
  } else {
    // every workgroup reads all choices: longer segments where there are many
    const dim3 block(64 * kPlanWaves);
    if (n <= 131072) {
      k_plan_segments<2><<<dim3((unsigned)((n + 2047) / 2048)), block, 0, st>>>(expert, n, (int)k, (int)E, 1, vec, offsets, row_token, slot);
    } else {
      const int64_t all = (n + (int64_t)16383) / 16384, chunks = (all + kPlanSegments - 1) / kPlanSegments;
      k_plan_segments<16><<<dim3((unsigned)((all + chunks - 1) / chunks)), block, 0, st>>>(expert, n, (int)k, (int)E, (int)chunks, vec, offsets, row_token, slot);
    }
  }
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
    for (int i = 0; i < V; ++i) o[i] = round_to<OutT>(acc[i]);
    *reinterpret_cast<ovec*>(y + t * N + n) = o;
  } else {
    y[t * N + n] = round_to<OutT>(acc[0]);
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
