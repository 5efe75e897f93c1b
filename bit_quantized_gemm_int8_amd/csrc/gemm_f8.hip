// Products of e4m3 codes with a binary32 scale for each 128 inputs of a token
// and for each 128 x 128 block of the weights:
//   y[m,n] = sum_g xs[m,g] ws[n/128,g] sum_{k in g} xq[m,k] wq[n,k]
// alone, or with a weight matrix of its own for each run of rows (experts:
// rows offsets[e] .. offsets[e+1] - 1 meet expert e's weights, and row r may
// take its codes from token row_token[r]).
//
// Two kernels:
//  * stream (few rows for each weight matrix): bound by the weight bytes.
//    16 weight rows per wave read as whole lines (qg_decode.hpp), the codes
//    widened to binary16 in registers (exact) for the 16-bit matrix cores.
//  * tile (many rows): bound by the matrix cores.  Stages of 128 k, one scale
//    block, come into LDS by DMA.  The matrix core's sum over a stage starts
//    at zero and is scaled into binary32 accumulators.
//
// What the matrix cores add up.  A product of two e4m3 codes has 8
// significant bits.  The 16-bit matrix instructions keep them all and sum in
// binary32.  The 8-bit ones (twice the rate) take products 8 at a time, by
// consecutive k of one lane's operand, align the 8 to the largest exponent
// among them and drop what lies below 2^-13 of it; only the sums of 8 are
// added in binary32 (seen on MI355X by single small products next to a large
// one).  So a product loses less than 2^-13 of the largest of its 8: about
// 1.5e-5 of the result's size for normal data, 6e-5 with outlier channels,
// at most 7 * 2^-13 * sum of the largest of each 8.  16-bit outputs, whose
// own rounding is 2^-9 or 2^-12, take the 8-bit instructions in the tile
// kernel; binary32 outputs and everything in the stream kernel, where the
// matrix cores wait for memory anyway, take the exact products.
#include <algorithm>
#include <type_traits>

#include "qg_decode.hpp"
#include "qg_f8.hpp"
#include "qg_launch.hpp"

namespace qg {

// Rows of one call: `offsets` null is the plain product (one weight matrix,
// all M rows); else E + 1 row offsets, which are read by the kernel and
// clamped to 0 .. R, an end below its start to the start, so that no value can
// lead out of range.
struct F8Rows {
  const int32_t* offsets;
  const int32_t* token;   // row -> row of xq, or null: the row itself
  int64_t T;              // rows of xq
  int R;                  // rows of y
};

__device__ __forceinline__ void f8_expert_rows(const F8Rows& fr, int e, int& lo, int& hi) {
  lo = min(max(fr.offsets[e], 0), fr.R);
  hi = min(max(fr.offsets[e + 1], lo), fr.R);
}

// The row of xq that row r of y is made from; -1: none (r past the run, or a
// token that does not exist: its row is computed as zeros).
__device__ __forceinline__ int64_t f8_source(const F8Rows& fr, int r, int hi) {
  if (r >= hi) return -1;
  const int64_t t = fr.token ? (int64_t)fr.token[r] : (int64_t)r;
  return t >= 0 && t < fr.T ? t : -1;
}

// ---------------------------------------------------------------------------
// Stream kernel.  A workgroup of NB x KS waves owns NB blocks of 16 weight
// rows and up to 16 MT token rows.  K is walked in phases of PU = KS UPW
// units of 128: the token codes and scales of a phase are staged in LDS once
// for all waves (two buffers, one barrier a phase, the next phase's loads in
// flight), wave (blk, ks) takes units ks UPW .. of the phase, and the KS
// partial sums of a block meet in LDS in a fixed order.
//
// Weight rows are the matrix core's first operand, so a lane's accumulators
// are 4 consecutive outputs of one token and the scale of a unit is one
// value per lane.
// ---------------------------------------------------------------------------
template <int MT, int NB, int KS, int UPW, typename OutT, bool EXPERTS>
__global__ __launch_bounds__(64 * NB * KS) void k_f8_stream(
    const uint8_t* __restrict__ xq, const float* __restrict__ xs, const uint8_t* __restrict__ wq,
    const float* __restrict__ ws, F8Rows fr, int N, int K, OutT* __restrict__ y, int vec) {
  constexpr int kThreads = 64 * NB * KS, kRows = 16 * MT;
  constexpr int PU = KS * UPW, PB = kUnitBytes * PU, kRowChunks = PB / 16;
  constexpr int kPitch = PB + 16;                  // an odd number of chunks: no bank conflicts
  constexpr int CPT = (kRows * kRowChunks + kThreads - 1) / kThreads;
  static_assert(kRows * kRowChunks % kThreads == 0, "whole rounds of chunks");
  constexpr int SPT = (kRows * PU + kThreads - 1) / kThreads;
  __shared__ __attribute__((aligned(16))) int8_t xbuf[2][kRows * kPitch];
  __shared__ float xsbuf[2][PU * kRows];
  __shared__ __attribute__((aligned(16))) int8_t tiles[NB * KS][kTileBytes];
  __shared__ __attribute__((aligned(16))) v4f red[KS > 1 ? KS - 1 : 1][NB][MT][64];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int blk = wave / KS, ks = wave % KS;
  const int r = lane & 15, j = lane >> 4;
  const int G = (K + kF8Block - 1) / kF8Block, B = (N + kF8Block - 1) / kF8Block;
  const int groups_n = ((N + 15) / 16 + NB - 1) / NB;
  const int e = EXPERTS ? blockIdx.x / groups_n : 0;
  const int n_base = 16 * ((EXPERTS ? blockIdx.x % groups_n : blockIdx.x) * NB + blk);
  int lo = 0, hi = fr.R;
  if constexpr (EXPERTS) f8_expert_rows(fr, e, lo, hi);

  const int rows_n = min(max(N - n_base, 0), 16);
  const rsrc_t wr = make_rsrc_uniform(wq + ((int64_t)e * N + min(n_base, N - 1)) * K, (u32)(rows_n * K));
  const float* wsr = ws + ((int64_t)e * B + min(n_base / kF8Block, B - 1)) * G;
  const UnitLanes ul = unit_lanes(lane, K);
  const int phases = (G + PU - 1) / PU;
  int8_t* tile = tiles[wave];

  struct Batch {
    v4i w[UPW][2], x[CPT];
    float s[SPT];
  };

  for (int m0 = lo; m0 < hi; m0 += kRows) {
    // the row and chunk of each of this thread's staging loads are the same
    // in every phase
    const uint8_t* xp[CPT];
    const float* sp[SPT];
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int64_t t = f8_source(fr, m0 + (tid + c * kThreads) / kRowChunks, hi);
      xp[c] = t < 0 ? nullptr : xq + t * K;
    }
#pragma unroll
    for (int c = 0; c < SPT; ++c) {
      const int i = tid + c * kThreads;
      const int64_t t = i < kRows * PU ? f8_source(fr, m0 + i / PU, hi) : -1;
      sp[c] = t < 0 ? nullptr : xs + t * G;
    }
    auto load = [&](Batch& bt, int p) {
#pragma unroll
      for (int v = 0; v < UPW; ++v) unit_load(bt.w[v], wr, ul, p * PU + ks * UPW + v, true, K);
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        const int kb = p * PB + ((tid + c * kThreads) % kRowChunks) * 16;
        bt.x[c] = xp[c] && kb < K ? ld16(xp[c] + kb) : v4i{0, 0, 0, 0};
      }
#pragma unroll
      for (int c = 0; c < SPT; ++c) {
        const int g = p * PU + (tid + c * kThreads) % PU;
        bt.s[c] = sp[c] && g < G ? sp[c][g] : 0.f;
      }
      __builtin_amdgcn_sched_barrier(0);
    };

    v4f acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
    auto process = [&](const Batch& bt, int p) {
      int8_t* buf = xbuf[p & 1];
      float* sbuf = xsbuf[p & 1];
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        const int chunk = tid + c * kThreads;
        st16(buf + (chunk / kRowChunks) * kPitch + (chunk % kRowChunks) * 16, bt.x[c]);
      }
#pragma unroll
      for (int c = 0; c < SPT; ++c) {
        const int i = tid + c * kThreads;
        if (i < kRows * PU) sbuf[(i % PU) * kRows + i / PU] = bt.s[c];
      }
      // Phase p is complete once every wave is here; the buffer that phase
      // p + 1 overwrites was last read at phase p - 1, before this barrier.
      lds_barrier();
#pragma unroll
      for (int v = 0; v < UPW; ++v) {
        const int u = ks * UPW + v;
        const float sw = wsr[min(p * PU + u, G - 1)];
        v4i f[2];
        unit_transpose(tile, bt.w[v], ul, f);
        v8h wf[4];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          wf[2 * s] = f8_to_f16x8(f[s][0], f[s][1]);
          wf[2 * s + 1] = f8_to_f16x8(f[s][2], f[s][3]);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          v4f d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            // past K both operands are zero
            const v4i a = ld16(buf + (16 * t + r) * kPitch + kUnitBytes * u + 64 * s + 16 * j);
            d = __builtin_amdgcn_mfma_f32_16x16x32_f16(wf[2 * s], f8_to_f16x8(a[0], a[1]), d, 0, 0, 0);
            d = __builtin_amdgcn_mfma_f32_16x16x32_f16(wf[2 * s + 1], f8_to_f16x8(a[2], a[3]), d, 0, 0, 0);
          }
          const float sc = sbuf[u * kRows + 16 * t + r] * sw;
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(d[i], sc, acc[t][i]);
        }
      }
    };

    Batch b0, b1;
    load(b0, 0);
    // every wave runs the same number of phases, so all reach every barrier;
    // a phase past the end is loaded as zeros
    for (int p = 0; p < phases; p += 2) {
      load(b1, p + 1);
      process(b0, p);
      load(b0, p + 2);
      process(b1, p + 1);
    }

    if constexpr (KS > 1) {
      if (ks > 0) {
#pragma unroll
        for (int t = 0; t < MT; ++t) red[ks - 1][blk][t][lane] = acc[t];
      }
      lds_barrier();
      if (ks == 0) {
#pragma unroll
        for (int o = 0; o < KS - 1; ++o)
#pragma unroll
          for (int t = 0; t < MT; ++t) acc[t] += red[o][blk][t][lane];
      }
    }
    if (ks == 0) {
      const int n = n_base + 4 * j;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int m = m0 + 16 * t + r;
        if (m >= hi) continue;
        OutT* dst = y + (int64_t)m * N + n;
        if (vec && n + 4 <= N) {
          typedef OutT o4 __attribute__((ext_vector_type(4)));
          *reinterpret_cast<o4*>(dst) = o4{Out<OutT>::cvt(acc[t][0]), Out<OutT>::cvt(acc[t][1]),
                                           Out<OutT>::cvt(acc[t][2]), Out<OutT>::cvt(acc[t][3])};
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + i < N) dst[i] = Out<OutT>::cvt(acc[t][i]);
        }
      }
    }
    // the next run of rows overwrites phase buffers and partial sums that
    // other waves may still read
    if constexpr (EXPERTS) lds_barrier();
  }
}

template <int MT, int NB, int KS, typename OutT>
static void launch_f8_stream_nb(const uint8_t* xq, const float* xs, const uint8_t* wq,
                                const float* ws, const F8Rows& fr, int64_t E, int N, int K,
                                OutT* y, int vec, hipStream_t st) {
  constexpr int UPW = MT == 1 ? 2 : 1;
  const int64_t groups_n = ((N + 15) / 16 + NB - 1) / NB;
  const dim3 block(64 * NB * KS);
  if (fr.offsets)
    k_f8_stream<MT, NB, KS, UPW, OutT, true><<<dim3((unsigned)(E * groups_n)), block, 0, st>>>(
        xq, xs, wq, ws, fr, N, K, y, vec);
  else
    k_f8_stream<MT, NB, KS, UPW, OutT, false><<<dim3((unsigned)groups_n), block, 0, st>>>(
        xq, xs, wq, ws, fr, N, K, y, vec);
}

template <int MT, typename OutT>
static void launch_f8_stream(const uint8_t* xq, const float* xs, const uint8_t* wq,
                             const float* ws, const F8Rows& fr, int64_t E, int N, int K, OutT* y,
                             int vec, hipStream_t st) {
  const int64_t blocks = E * ((N + 15) / 16);
  if (blocks <= 256) launch_f8_stream_nb<MT, 1, MT <= 2 ? 8 : 4, OutT>(xq, xs, wq, ws, fr, E, N, K, y, vec, st);
  else if (blocks <= 768) launch_f8_stream_nb<MT, 2, 4, OutT>(xq, xs, wq, ws, fr, E, N, K, y, vec, st);
  else launch_f8_stream_nb<MT, 4, 2, OutT>(xq, xs, wq, ws, fr, E, N, K, y, vec, st);
}

// ---------------------------------------------------------------------------
// Tile kernel: BM x BN outputs per workgroup of WM x WN waves, each wave
// 32 MI x 32 NJ outputs of 32x32 matrix instructions.  A stage is the 128 k
// of one scale block: BM token rows and BN weight rows of 128 bytes, and the
// BM token scales, all by buffer-to-LDS DMA into one of two stage buffers
// while the other is multiplied.  Chunks are XOR-swizzled as in the int8 tile
// kernel: row r's chunk c at slot c ^ ((r >> 1) & 7), so that 16 rows reading
// one chunk hit 16 different bank groups.
//
// The weights are the first operand, so a lane's 16 accumulators of a block
// belong to one token (lane & 31) and share one scale, xs ws.
// ---------------------------------------------------------------------------
constexpr int kF8Stage = 128;   // bytes of a row in a stage = one scale block

template <int BM, int BN>
constexpr int f8_stage_bytes() { return (BM + BN) * kF8Stage + 4 * BM; }

// Tile of a workgroup: rows m0 .. < hi of y (m0 + BM may pass hi), columns n0 ..
struct F8Tile {
  int e, m0, hi, n0;
};

template <int BM, int BN, int WM, int WN, bool EXACT, typename OutT, bool EXPERTS>
__device__ __forceinline__ void f8_tile(int8_t* lds, const uint8_t* __restrict__ xq,
                                        const float* __restrict__ xs,
                                        const uint8_t* __restrict__ wq,
                                        const float* __restrict__ ws, const F8Rows& fr,
                                        const F8Tile& at, int N, int K, OutT* __restrict__ y,
                                        int vec) {
  constexpr int NW = WM * WN, MI = BM / WM / 32, NJ = BN / WN / 32;
  constexpr int kStage = f8_stage_bytes<BM, BN>();
  constexpr int kLoadsA = BM / 8, kLoadsB = BN / 8;      // 1 KB loads of 8 rows
  constexpr int LA = kLoadsA / NW, LB = kLoadsB / NW;    // of each wave
  constexpr int LS = BM / 64;                            // scale loads: 64 rows each
  static_assert(LA * NW == kLoadsA && LB * NW == kLoadsB && LS <= NW, "whole loads per wave");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int row_a = wm * 32 * MI, row_b = wn * 32 * NJ;
  const int G = (K + kF8Block - 1) / kF8Block, B = (N + kF8Block - 1) / kF8Block;

  // Token rows come from one resource: of this tile's rows where they follow
  // each other, else of all of xq (whose size the host keeps under 2 GiB).
  const bool gather = EXPERTS && fr.token != nullptr;
  const int64_t row0 = gather ? 0 : at.m0;
  const int rows_x = gather ? (int)fr.T : (int)min((int64_t)BM, min((int64_t)at.hi, fr.T) - at.m0);
  const rsrc_t ar = make_rsrc_uniform(xq + row0 * K, (u32)(max(rows_x, 0) * K));
  const rsrc_t sr = make_rsrc_uniform(xs + row0 * G, (u32)(max(rows_x, 0) * G * 4));
  const rsrc_t br = make_rsrc_uniform(wq + ((int64_t)at.e * N + at.n0) * K,
                                      (u32)(min(BN, N - at.n0) * K));
  const float* wsr = ws + ((int64_t)at.e * B + min((at.n0 + row_b) / kF8Block, B - 1)) * G;

  // Byte offset of this lane's row for each of its loads (kOOB: no row).
  const int lrow = lane >> 3, slot = lane & 7;
  u32 offa[LA];
  int cha[LA];
#pragma unroll
  for (int i = 0; i < LA; ++i) {
    const int row = 8 * (wave * LA + i) + lrow;
    cha[i] = 16 * (slot ^ ((row >> 1) & 7));
    if (EXPERTS) {
      const int64_t t = f8_source(fr, at.m0 + row, at.hi);
      offa[i] = t < 0 ? kOOB : (u32)((t - row0) * K);
    } else {
      offa[i] = row < rows_x ? (u32)(row * K) : kOOB;
    }
  }
  u32 offs = kOOB;
  if (wave < LS) {
    const int row = 64 * wave + lane;
    if (EXPERTS) {
      const int64_t t = f8_source(fr, at.m0 + row, at.hi);
      offs = t < 0 ? kOOB : (u32)((t - row0) * G * 4);
    } else {
      offs = row < rows_x ? (u32)(row * G * 4) : kOOB;
    }
  }
  // One load of a stage: i < LA token rows, then weight rows, then scales.
  auto dma = [&](int8_t* buf, int g, int i) {
    if (i < LA) {
      const int k = g * kF8Stage + cha[i];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, QG_LDS(buf + (wave * LA + i) * 1024), 16,
                                               k < K && offa[i] != kOOB ? offa[i] + k : kOOB, 0, 0, 0);
    } else if (i < LA + LB) {
      const int q = wave * LB + i - LA, row = 8 * q + lrow;
      const int k = g * kF8Stage + 16 * (slot ^ ((row >> 1) & 7));
      // rows past N lie behind the resource's end
      __builtin_amdgcn_raw_ptr_buffer_load_lds(br, QG_LDS(buf + BM * kF8Stage + q * 1024), 16,
                                               k < K ? (u32)(row * K + k) : kOOB, 0, 0, 0);
    } else if (wave < LS) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(sr, QG_LDS(buf + (BM + BN) * kF8Stage + wave * 256), 4,
                                               g < G && offs != kOOB ? offs + 4 * g : kOOB, 0, 0, 0);
    }
  };
  constexpr int kLoads = LA + LB + 1;

  v16f acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) acc[i][jj] = v16f{};

  const int l31 = lane & 31, half = lane >> 5;
  // The four chunks of a row that a lane holds: 4 (of 8) 16-byte chunks; both
  // operands split k alike, so any fixed split will do.
  auto frag = [&](const int8_t* base, int row, v4i (&f)[4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int ch = 4 * half + c;
      f[c] = ld16(base + row * kF8Stage + ((ch ^ ((row >> 1) & 7)) << 4));
    }
  };
  auto multiply = [&](const int8_t* buf, int8_t* next, int g) {
    v4i bf[NJ][4];
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) frag(buf + BM * kF8Stage, row_b + 32 * jj + l31, bf[jj]);
    const float* sc = reinterpret_cast<const float*>(buf + (BM + BN) * kF8Stage);
    const float sw = wsr[min(g, G - 1)];
    v4i af[2][4];
    frag(buf, row_a + l31, af[0]);
    constexpr int kEvery = (kLoads + MI * NJ - 1) / (MI * NJ);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (i + 1 < MI) frag(buf, row_a + 32 * (i + 1) + l31, af[(i + 1) & 1]);
      const v4i (&a)[4] = af[i & 1];
      const float s = sc[row_a + 32 * i + l31] * sw;
#pragma unroll
      for (int jj = 0; jj < NJ; ++jj) {
        __builtin_amdgcn_sched_barrier(0);
        v16f d = {};
        const v4i (&b)[4] = bf[jj];
        if constexpr (EXACT) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            d = __builtin_amdgcn_mfma_f32_32x32x16_f16(f8_to_f16x8(b[c][0], b[c][1]), f8_to_f16x8(a[c][0], a[c][1]), d, 0, 0, 0);
            d = __builtin_amdgcn_mfma_f32_32x32x16_f16(f8_to_f16x8(b[c][2], b[c][3]), f8_to_f16x8(a[c][2], a[c][3]), d, 0, 0, 0);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 4; c += 2) {
            const v8i bb = {b[c][0], b[c][1], b[c][2], b[c][3], b[c + 1][0], b[c + 1][1], b[c + 1][2], b[c + 1][3]};
            const v8i aa = {a[c][0], a[c][1], a[c][2], a[c][3], a[c + 1][0], a[c + 1][1], a[c + 1][2], a[c + 1][3]};
            d = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bb, aa, d, 0, 0, 0, 0, 0, 0);
          }
        }
        // this wave's loads of the next stage, spread over the products
#pragma unroll
        for (int l = 0; l < kEvery; ++l) {
          const int ld = (i * NJ + jj) * kEvery + l;
          if (ld < kLoads) dma(next, g + 1, ld);
        }
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][jj][q] = fmaf(d[q], s, acc[i][jj][q]);
      }
    }
  };
  // This wave's loads have landed and all waves are done with the buffer that
  // the next loads overwrite.
  auto sync = [] { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

#pragma unroll
  for (int i = 0; i < kLoads; ++i) dma(lds, 0, i);
  for (int g = 0; g < G; g += 2) {
    // a stage past G is loaded as zeros and adds nothing (one at most)
    sync();
    multiply(lds, lds + kStage, g);
    sync();
    multiply(lds + kStage, lds, g + 1);
  }
  sync();   // the last (zero) loads have landed before LDS is used again

  // Lane l holds token row 32 i + (l & 31); register q of block (i, jj) output
  // column 32 jj + 8 (q >> 2) + 4 (l >> 5) + (q & 3).
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = at.m0 + row_a + 32 * i + l31;
    if (m >= at.hi) continue;
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = at.n0 + row_b + 32 * jj + 8 * q + 4 * half;
        OutT* dst = y + (int64_t)m * N + n;
        if (vec && n + 4 <= N) {
          typedef OutT o4 __attribute__((ext_vector_type(4)));
          *reinterpret_cast<o4*>(dst) =
              o4{Out<OutT>::cvt(acc[i][jj][4 * q]), Out<OutT>::cvt(acc[i][jj][4 * q + 1]),
                 Out<OutT>::cvt(acc[i][jj][4 * q + 2]), Out<OutT>::cvt(acc[i][jj][4 * q + 3])};
        } else {
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (n + t < N) dst[t] = Out<OutT>::cvt(acc[i][jj][4 * q + t]);
        }
      }
  }
}

template <int BM, int BN, int WM, int WN, bool EXACT, typename OutT>
__global__ __launch_bounds__(64 * WM * WN) void k_f8_tile(
    const uint8_t* __restrict__ xq, const float* __restrict__ xs, const uint8_t* __restrict__ wq,
    const float* __restrict__ ws, F8Rows fr, int N, int K, OutT* __restrict__ y, int vec) {
  __shared__ __attribute__((aligned(16))) int8_t lds[2 * f8_stage_bytes<BM, BN>()];
  const int M = fr.R;
  // Consecutive workgroups go to the 8 XCDs in turn: renumber so that each
  // XCD walks a contiguous run of tiles, in column-major groups of 4 tile
  // rows, whose tiles share token and weight rows in that XCD's L2.
  const int tiles_m = (M + BM - 1) / BM, tiles_n = (N + BN - 1) / BN, total = tiles_m * tiles_n;
  const int per = total / 8, rem = total % 8, xcd = blockIdx.x % 8;
  const int bid = xcd * per + min(xcd, rem) + blockIdx.x / 8;
  constexpr int GROUP = 4;
  const int group = bid / (GROUP * tiles_n), first = group * GROUP;
  const int gsize = min(tiles_m - first, GROUP), in = bid - group * GROUP * tiles_n;
  const F8Tile at{0, (first + in % gsize) * BM, M, in / gsize * BN};
  f8_tile<BM, BN, WM, WN, EXACT, OutT, false>(lds, xq, xs, wq, ws, fr, at, N, K, y, vec);
}

// The experts' tiles.  The row counts are on the GPU only, so every workgroup
// counts the tiles of all experts first (a scan over E in LDS), then takes
// tiles of the joint list: XCD x the x-th eighth of it, so that an expert's
// weights stay in one L2.
constexpr int kF8MaxExperts = 1024;

template <int BM, int BN, int WM, int WN, bool EXACT, typename OutT>
__global__ __launch_bounds__(64 * WM * WN) void k_f8_tile_experts(
    const uint8_t* __restrict__ xq, const float* __restrict__ xs, const uint8_t* __restrict__ wq,
    const float* __restrict__ ws, F8Rows fr, int E, int N, int K, OutT* __restrict__ y, int vec) {
  __shared__ __attribute__((aligned(16))) int8_t lds[2 * f8_stage_bytes<BM, BN>()];
  __shared__ int first[kF8MaxExperts + 1];   // tile rows ahead of each expert
  const int tiles_n = (N + BN - 1) / BN;
  if (threadIdx.x < kWave) {
    // each lane counts a run of experts, the lanes' sums are scanned; offsets
    // that do not rise can name rows many times over, so the count saturates
    const int64_t most = 0x7fffffff / tiles_n;
    const int per = (E + kWave - 1) / kWave, e0 = threadIdx.x * per;
    int64_t sum = 0;
    for (int e = e0; e < min(e0 + per, E); ++e) {
      int lo, hi;
      f8_expert_rows(fr, e, lo, hi);
      sum += (hi - lo + BM - 1) / BM;
    }
    int64_t run = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int64_t t = __shfl_up(run, d, kWave);
      if ((int)threadIdx.x >= d) run += t;
    }
    run -= sum;
    for (int e = e0; e < min(e0 + per, E); ++e) {
      int lo, hi;
      f8_expert_rows(fr, e, lo, hi);
      first[e] = (int)min(run, most);
      run += (hi - lo + BM - 1) / BM;
    }
    if (threadIdx.x == kWave - 1) first[E] = (int)min(run, most);
  }
  __syncthreads();
  const int total = first[E] * tiles_n;
  const int per = total / 8, rem = total % 8, xcd = blockIdx.x % 8;
  const int begin = xcd * per + min(xcd, rem), end = begin + per + (xcd < rem);
  for (int t = begin + blockIdx.x / 8; t < end; t += gridDim.x / 8) {
    // the last expert whose first tile is at or before t
    int a = 0, b = E - 1;
    while (a < b) {
      const int mid = (a + b + 1) / 2;
      if (first[mid] * tiles_n <= t) a = mid;
      else b = mid - 1;
    }
    int lo, hi;
    f8_expert_rows(fr, a, lo, hi);
    const int rows = first[a + 1] - first[a], in = t - first[a] * tiles_n;
    const F8Tile at{a, lo + in % rows * BM, hi, in / rows * BN};
    f8_tile<BM, BN, WM, WN, EXACT, OutT, true>(lds, xq, xs, wq, ws, fr, at, N, K, y, vec);
  }
}

template <int BM, int BN, int WM, int WN, typename OutT>
static void launch_f8_tile(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                           const F8Rows& fr, int64_t E, int N, int K, OutT* y, int vec,
                           hipStream_t st) {
  constexpr bool EXACT = std::is_same<OutT, float>::value;
  constexpr int kLds = 2 * f8_stage_bytes<BM, BN>() + 4 * (kF8MaxExperts + 1);
  const dim3 block(64 * WM * WN);
  const int64_t tiles_n = (N + BN - 1) / BN;
  if (fr.offsets) {
    // as many workgroups as can be resident, a multiple of the 8 XCDs
    const int64_t most = ((int64_t)fr.R + BM - 1) / BM + E;
    const int64_t grid = std::min<int64_t>(256 * (int64_t)(kLdsBytesPerCU / kLds), (most * tiles_n + 7) / 8 * 8);
    k_f8_tile_experts<BM, BN, WM, WN, EXACT, OutT><<<dim3((unsigned)grid), block, 0, st>>>(
        xq, xs, wq, ws, fr, (int)E, N, K, y, vec);
  } else {
    const int64_t tiles = ((int64_t)fr.R + BM - 1) / BM * tiles_n;
    k_f8_tile<BM, BN, WM, WN, EXACT, OutT><<<dim3((unsigned)tiles), block, 0, st>>>(
        xq, xs, wq, ws, fr, N, K, y, vec);
  }
}

template <typename OutT>
static hipError_t gemm_f8_t(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                            const F8Rows& fr, int64_t E, int N, int K, OutT* y, hipStream_t st) {
  const int64_t rows = fr.offsets ? (fr.R + E - 1) / E : fr.R;   // of one weight matrix
  // 4 consecutive outputs as one store where every row is aligned to it
  const int vec = N % 4 == 0 && (uintptr_t)y % (4 * sizeof(OutT)) == 0;
  if (rows <= 16) {
    launch_f8_stream<1, OutT>(xq, xs, wq, ws, fr, E, N, K, y, vec, st);
  } else if (rows <= 32) {
    launch_f8_stream<2, OutT>(xq, xs, wq, ws, fr, E, N, K, y, vec, st);
  } else if (rows <= 64) {
    launch_f8_stream<4, OutT>(xq, xs, wq, ws, fr, E, N, K, y, vec, st);
  } else {
    const int64_t mid = ((rows + 127) / 128) * ((N + 127) / 128) * E;
    if (mid >= 256) launch_f8_tile<128, 128, 2, 2, OutT>(xq, xs, wq, ws, fr, E, N, K, y, vec, st);
    else launch_f8_tile<64, 64, 2, 2, OutT>(xq, xs, wq, ws, fr, E, N, K, y, vec, st);
  }
  return hipGetLastError();
}

hipError_t launch_gemm_f8(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                          const int32_t* offsets, const int32_t* row_token, int64_t T, int64_t R,
                          int64_t E, int64_t N, int64_t K, void* y, int y_dtype, hipStream_t st) {
  const F8Rows fr{offsets, row_token, T, (int)R};
  const int n = (int)N, k = (int)K;
  switch (y_dtype) {
    case F32: return gemm_f8_t<float>(xq, xs, wq, ws, fr, E, n, k, (float*)y, st);
    case F16: return gemm_f8_t<_Float16>(xq, xs, wq, ws, fr, E, n, k, (_Float16*)y, st);
    default: return gemm_f8_t<uint16_t>(xq, xs, wq, ws, fr, E, n, k, (uint16_t*)y, st);
  }
}

}  // namespace qg
