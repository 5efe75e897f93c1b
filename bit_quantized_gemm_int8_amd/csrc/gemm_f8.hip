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
//  * tile (many rows): bound by the way from L2 into LDS and by the matrix
//    cores together on 256 x 256 tiles (4096 x 4096 x 11008: 184 us, a copy
//    without the loads of later stages 144, one without the matrix instructions
//    144), by the former on 128 x 128 (24576 rows over 64 experts of 1376 x 4096:
//    258 us, 147 and 241).  Stages of 128 k, one scale block, come by DMA.  The
//    matrix core's sum over a stage starts at zero and is scaled into binary32
//    accumulators.
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
#include "qg_f8_index.hpp"
#include "qg_launch.hpp"

namespace qg {

// Rows of one call: `offsets` null is the plain product (one weight matrix,
// all M rows); else E + 1 row offsets, which are read by the kernel and
// clamped to 0 .. R, an end below its start to the start, so that no value can
// lead out of range.
struct F8Rows {
  const int32_t* offsets;
  const int32_t* token;   // row -> row of xq, or null: the row itself
  int T;                  // rows of xq
  int R;                  // rows of y
};

__device__ __forceinline__ void f8_expert_rows(const F8Rows& fr, int e, int& lo, int& hi) {
  lo = min(max(fr.offsets[e], 0), fr.R);
  hi = min(max(fr.offsets[e + 1], lo), fr.R);
}

// The row of xq that row r of y is made from; -1: none (r past the run, or a
// token that does not exist: its row is computed as zeros).
__device__ __forceinline__ int f8_source(const F8Rows& fr, int r, int hi) {
  if (r >= hi) return -1;
  const int t = fr.token ? fr.token[r] : r;
  return t >= 0 && t < fr.T ? t : -1;
}

// ---------------------------------------------------------------------------
// Stream kernel.  A workgroup of NB x KS waves owns NB blocks of 16 weight
// rows and up to 16 token rows (at a time).  K is walked in phases of PU = KS UPW
// units of 128: the token codes and scales of a phase are staged in LDS once
// for all waves (two buffers, one barrier a phase, the next phase's loads in
// flight), wave (blk, ks) takes units ks UPW .. of the phase, and the KS
// partial sums of a block meet in LDS in a fixed order.
//
// Weight rows are the matrix core's first operand, so a lane's accumulators
// are 4 consecutive outputs of one token and the scale of a unit is one
// value per lane.
// ---------------------------------------------------------------------------
template <int NB, int KS, int UPW, typename OutT, bool EXPERTS>
__global__ __launch_bounds__(64 * NB * KS) void k_f8_stream(
    const uint8_t* __restrict__ xq, const float* __restrict__ xs, const uint8_t* __restrict__ wq,
    const float* __restrict__ ws, F8Rows fr, int N, int K, OutT* __restrict__ y, int vec) {
  constexpr int kThreads = 64 * NB * KS, kRows = 16;
  constexpr int PU = KS * UPW, PB = kUnitBytes * PU, kRowChunks = PB / 16;
  constexpr int kPitch = PB + 16;                  // an odd number of chunks: no bank conflicts
  constexpr int CPT = (kRows * kRowChunks + kThreads - 1) / kThreads;
  static_assert(kRows * kRowChunks % kThreads == 0, "whole rounds of chunks");
  constexpr int SPT = (kRows * PU + kThreads - 1) / kThreads;
  __shared__ __attribute__((aligned(16))) int8_t xbuf[2][kRows * kPitch];
  __shared__ float xsbuf[2][PU * kRows];
  __shared__ __attribute__((aligned(16))) int8_t tiles[NB * KS][kTileBytes];
  __shared__ __attribute__((aligned(16))) v4f red[KS > 1 ? KS - 1 : 1][NB][64];

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
      const int t = f8_source(fr, m0 + (tid + c * kThreads) / kRowChunks, hi);
      xp[c] = t < 0 ? nullptr : xq + (int64_t)t * K;
    }
#pragma unroll
    for (int c = 0; c < SPT; ++c) {
      const int i = tid + c * kThreads;
      const int t = i < kRows * PU ? f8_source(fr, m0 + i / PU, hi) : -1;
      sp[c] = t < 0 ? nullptr : xs + (int64_t)t * G;
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

    v4f acc = {0.f, 0.f, 0.f, 0.f};
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
        v4f d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          // past K both operands are zero
          const v4i a = ld16(buf + r * kPitch + kUnitBytes * u + 64 * s + 16 * j);
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(wf[2 * s], f8_to_f16x8(a[0], a[1]), d, 0, 0, 0);
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(wf[2 * s + 1], f8_to_f16x8(a[2], a[3]), d, 0, 0, 0);
        }
        const float sc = sbuf[u * kRows + r] * sw;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(d[i], sc, acc[i]);
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
      if (ks > 0) red[ks - 1][blk][lane] = acc;
      lds_barrier();
      if (ks == 0) {
#pragma unroll
        for (int o = 0; o < KS - 1; ++o) acc += red[o][blk][lane];
      }
    }
    const int m = m0 + r, n = n_base + 4 * j;
    if (ks == 0 && m < hi) {
      OutT* dst = y + (int64_t)m * N + n;
      if (vec && n + 4 <= N) {
        typedef OutT o4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<o4*>(dst) = o4{round_to<OutT>(acc[0]), round_to<OutT>(acc[1]),
                                         round_to<OutT>(acc[2]), round_to<OutT>(acc[3])};
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < N) dst[i] = round_to<OutT>(acc[i]);
      }
    }
    // the next run of rows overwrites phase buffers and partial sums that
    // other waves may still read
    if constexpr (EXPERTS) lds_barrier();
  }
}

template <int NB, int KS, typename OutT>
static void launch_f8_stream_nb(const uint8_t* xq, const float* xs, const uint8_t* wq,
                                const float* ws, const F8Rows& fr, int64_t E, int N, int K,
                                OutT* y, int vec, hipStream_t st) {
  constexpr int UPW = 2;
  const int64_t groups_n = ((N + 15) / 16 + NB - 1) / NB;
  const dim3 block(64 * NB * KS);
  if (fr.offsets)
    k_f8_stream<NB, KS, UPW, OutT, true><<<dim3((unsigned)(E * groups_n)), block, 0, st>>>(
        xq, xs, wq, ws, fr, N, K, y, vec);
  else
    k_f8_stream<NB, KS, UPW, OutT, false><<<dim3((unsigned)groups_n), block, 0, st>>>(
        xq, xs, wq, ws, fr, N, K, y, vec);
}

template <typename OutT>
static void launch_f8_stream(const uint8_t* xq, const float* xs, const uint8_t* wq,
                             const float* ws, const F8Rows& fr, int64_t E, int N, int K, OutT* y,
                             int vec, hipStream_t st) {
  // Blocks of 16 weight rows: one a workgroup with its K in 8 parts while that
  // gives every CU at most one (1 x 11008 x 4096: 12.8 us, two blocks in 4
  // parts 15.5, four in 2 23.6), two up to 600 blocks, four beyond, which stage
  // the token rows less often (8 x 4096 x 11008, 688 blocks: 12.2, two a workgroup
  // 13.8; 96 rows over 64 experts of 4096 x 2752: 91.2 against 96.8).
  const int64_t blocks = E * ((N + 15) / 16);
  if (blocks <= 256) launch_f8_stream_nb<1, 8>(xq, xs, wq, ws, fr, E, N, K, y, vec, st);
  else if (blocks <= 600) launch_f8_stream_nb<2, 4>(xq, xs, wq, ws, fr, E, N, K, y, vec, st);
  else launch_f8_stream_nb<4, 2>(xq, xs, wq, ws, fr, E, N, K, y, vec, st);
}

// ---------------------------------------------------------------------------
// Tile kernel: BM x BN outputs per workgroup of WM x WN waves, each wave
// 32 MI x 32 NJ outputs of 32x32 matrix instructions.  A stage is the 128 k
// of one scale block: BM token rows and BN weight rows of 128 bytes, and the
// scales, all by buffer-to-LDS DMA into a ring of NB buffers, NB - 1 stages
// ahead of the products.  Chunks are XOR-swizzled as in the int8 tile
// kernel: row r's chunk c at slot c ^ ((r >> 1) & 7), so that 16 rows reading
// one chunk hit 16 different bank groups.
//
// The weights are the first operand, so a lane's 16 accumulators of a block
// belong to one token (lane & 31) and share one scale, xs ws.
// ---------------------------------------------------------------------------
constexpr int kF8Stage = 128;   // bytes of a row in a stage = one scale block

// Scales come SG stages at a time, SG of them for each token row and then for
// each column block of the tile (a run of 64 lanes): a row's scales of one stage
// are 4 bytes of a line, and a request for them costs L2 as much as one for 128
// bytes of codes, a third of all requests with SG = 1.  4 for 128 x 128 tiles:
// 24576 rows over 64 experts of 4096 x 2752 417 us, 444 with 1; 1024 x 4096 x
// 4096 28.3, 30.5; of 31 plain shapes of 256 .. 512 tiles those of K = 11008 take
// 7% less on average and at most 0.2% more, those of K = 4096 between 7% less and
// 11% more (768 x 4096 x 5504: 33.4, 30.0; 512 x 4096 x 11008: 35.4, 32.5), as
// much on average; shapes of equal tile counts and widths lie on both sides, so
// no rule on sizes divides them.  A 256 x 256 tile has no registers left for it
// (4096 x 4096 x 11008: 221 us, 181 with 1), and rings deeper than two stages
// count loads.
template <int BM>
constexpr int f8_scale_stages(int NB) { return NB == 2 && BM <= 128 ? 4 : 1; }
// LDS of a group of waves: NB buffers of token and weight rows, then the ring
// of scales (two blocks of SG stages, or one for each stage).
template <int BM, int BN>
constexpr int f8_rows_bytes() { return (BM + BN) * kF8Stage; }
template <int BM>
constexpr int f8_scales_bytes(int NB) { return f8_scale_stages<BM>(NB) * (4 * BM + 256); }
template <int BM, int BN, int NB>
constexpr int f8_ring_bytes() { return NB * (f8_rows_bytes<BM, BN>() + f8_scales_bytes<BM>(NB)); }

// Direct loads into LDS, 16 and 4 bytes a lane at lds (wave-uniform) + 16 or
// 4 lane, at byte voff + soff of the resource; out of range reads zeros.
__device__ __forceinline__ void f8_dma16(rsrc_t r, int8_t* lds, u32 voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, QG_LDS(lds), 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void f8_dma4(rsrc_t r, int8_t* lds, u32 voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, QG_LDS(lds), 4, voff, soff, 0, 0);
}

// Tile of a workgroup: rows m0 .. < hi of y (m0 + BM may pass hi), columns n0 ..
struct F8Tile {
  int e, m0, hi, n0;
};

template <int BM, int BN, int WM, int WN, int KS, int NB, bool EXACT, typename OutT, bool EXPERTS, typename Next>
__device__ __forceinline__ void f8_tiles(int8_t* lds0, const uint8_t* __restrict__ xq,
                                         const float* __restrict__ xs,
                                         const uint8_t* __restrict__ wq,
                                         const float* __restrict__ ws, const F8Rows& fr, int N,
                                         int K, OutT* __restrict__ y, int vec, Next next_tile) {
  constexpr int NW = WM * WN, MI = BM / WM / 32, NJ = BN / WN / 32;
  constexpr int kStage = f8_rows_bytes<BM, BN>(), SG = f8_scale_stages<BM>(NB), kScales = f8_scales_bytes<BM>(NB);
  static_assert(SG == 1 || KS == 1, "blocks of scales are counted in stages");
  constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;      // 1 KB loads of 8 rows, of each wave
  static_assert(LA * NW * 8 == BM && LB * NW * 8 == BN && BM < 64 * NW && BM % 64 == 0,
                "whole loads per wave");
  const int lane = threadIdx.x & 63;
  // KS groups of waves share a tile: group kg multiplies stages kg, kg + KS, ..
  // out of a ring of its own, and the sums meet at the end
  const int kg = __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * NW));
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % NW);
  int8_t* const lds = lds0 + kg * f8_ring_bytes<BM, BN, NB>();
  int8_t* const slds = lds + NB * kStage;
  const int wm = wave / WN, wn = wave % WN;
  const int row_a = wm * 32 * MI, row_b = wn * 32 * NJ;
  const int G = (K + kF8Block - 1) / kF8Block, B = (N + kF8Block - 1) / kF8Block;
  const bool gather = EXPERTS && fr.token != nullptr;

  // ---- loads of a tile's stages ----
  // Byte offset of this lane's chunk of stage 0 for each of its loads (kOOB: no
  // row), the scale's likewise.  A stage adds 128 bytes as a scalar offset; in
  // the last stage the chunks past K are masked.
  const int lrow = lane >> 3, slot = lane & 7;
  u32 offa[LA], offb[LB], offs;
  rsrc_t ar, sr, br;
#pragma unroll
  for (int i = 0; i < LB; ++i) {   // rows past N lie behind the resource's end
    const int row = 8 * (wave * LB + i) + lrow;
    offb[i] = (u32)(row * K) + 16 * (slot ^ ((row >> 1) & 7));
  }
  // The rows of xq this lane's loads of a tile take, and that of its scale;
  // -1: none.  Wave w < BM / 64 loads token scales, the others (all alike) the
  // weight scales.
  struct Rows {
    int a[LA], s;
  };
  auto rows_of = [&](const F8Tile& at) {
    Rows r;
#pragma unroll
    for (int i = 0; i < LA; ++i) r.a[i] = f8_source(fr, at.m0 + 8 * (wave * LA + i) + lrow, at.hi);
    const int row = 64 * wave + lane;
    r.s = row < BM ? f8_source(fr, at.m0 + row, at.hi) : -1;
    return r;
  };
  auto aim = [&](const F8Tile& at, const Rows& r) {
    // Token rows come from one resource: of this tile's rows where they follow
    // each other, else of all of xq (whose size the host keeps under 2 GiB).
    // (A row that does not exist has a vector offset past any size.)
    const int row0 = gather ? 0 : at.m0;
    const int rows_x = gather ? fr.T : min(BM, at.hi - at.m0);
    ar = make_rsrc_uniform(xq + (int64_t)row0 * K, (u32)(rows_x * K));
    br = make_rsrc_uniform(wq + ((int64_t)at.e * N + at.n0) * K, (u32)(min(BN, N - at.n0) * K));
#pragma unroll
    for (int i = 0; i < LA; ++i)
      offa[i] = r.a[i] < 0 ? kOOB : (u32)((r.a[i] - row0) * K) + 16 * (slot ^ (((8 * (wave * LA + i) + lrow) >> 1) & 7));
    if (wave < BM / 64) {
      sr = make_rsrc_uniform(xs + (int64_t)row0 * G, (u32)(rows_x * G * 4));
      offs = r.s < 0 ? kOOB : (u32)((r.s - row0) * G * 4);
    } else {
      const int b0 = at.n0 / kF8Block, blocks = min((BN + kF8Block - 1) / kF8Block, B - b0);
      sr = make_rsrc_uniform(ws + ((int64_t)at.e * B + b0) * G, (u32)(blocks * G * 4));
      offs = lane < blocks ? (u32)(lane * G * 4) : kOOB;
    }
  };
  // One load of stage g: i < LA token rows, then weight rows, then scales.
  // in.row[b]: whether the lane's chunk of a load with q % 2 == b lies within K
  // (never past the last stage, whose successor is loaded as zeros).
  struct StageIn {
    bool row[2], scale;
  };
  auto stage_in = [&](int g) {
    StageIn in;
#pragma unroll
    for (int b = 0; b < 2; ++b) in.row[b] = g * kF8Stage + 16 * (slot ^ ((4 * b + (lrow >> 1)) & 7)) < K;
    in.scale = g < G;
    return in;
  };
  auto dma = [&](int8_t* buf, int g, int i, const StageIn& in) {
    if (i < LA) {
      const int q = wave * LA + i;
      f8_dma16(ar, buf + q * 1024, in.row[LA % 2 ? q & 1 : i & 1] ? offa[i] : kOOB, g * kF8Stage);
    } else if (i < LA + LB) {
      const int q = wave * LB + i - LA;
      f8_dma16(br, buf + BM * kF8Stage + q * 1024, in.row[LB % 2 ? q & 1 : (i - LA) & 1] ? offb[i - LA] : kOOB, g * kF8Stage);
    } else if (g % SG == 0) {
      const F8ScaleLoad at = f8_scale_load(in.scale ? offs : kOOB, g, SG);
      if constexpr (SG == 1) f8_dma4(sr, slds + (buf - lds) / kStage * kScales + min(wave, BM / 64) * 256, at.voffset, at.soffset);
      else f8_dma16(sr, slds + (g / SG & 1) * kScales + min(wave, BM / 64) * (64 * 4 * SG), at.voffset, at.soffset);
    }
  };
  constexpr int kLoads = LA + LB + 1;
  // ---- products of a stage ----
  const int l31 = lane & 31, half = lane >> 5;
  // A lane holds 4 of a row's 8 chunks; both operands split k alike, so any
  // fixed split will do.  The swizzle depends on the row's low bits only, so
  // the slots are the same for every 32-row block.
  int cslot[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) cslot[c] = l31 * kF8Stage + (((4 * half + c) ^ ((l31 >> 1) & 7)) << 4);
  auto frag = [&](const int8_t* base, v4i (&f)[4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) f[c] = ld16(base + cslot[c]);
  };
  v16f acc[MI][NJ];
  // The product of a 32 x 32 block over the stage is a chain of its own that
  // starts at zero; it is scaled into the accumulators one step later, so the
  // vector ALU works on one block while the matrix core is at the next.  The
  // last block's turn comes in the next stage.
  constexpr int kSteps = MI * NJ;
  static_assert(kSteps % 2 == 0 || kSteps == 1, "the two products in flight alternate");
  v16f d[2];
  float sprev;
  auto scale_in = [&](int t, const v16f& p, float sc) {
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[t / NJ][t % NJ][q] = fmaf(p[q], sc, acc[t / NJ][t % NJ][q]);
    // keeps the sums here, next to the following block's products: the
    // compiler would gather them at the end and hold every product until then
    asm volatile("" : "+v"(acc[t / NJ][t % NJ]));
  };
  auto multiply = [&](const int8_t* buf, int8_t* ahead, int g) {
    v4i bf[NJ][4], af[2][4];
    float sx[MI];
    frag(buf + row_a * kF8Stage, af[0]);
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) frag(buf + BM * kF8Stage + (row_b + 32 * jj) * kF8Stage, bf[jj]);
    const float* sc = reinterpret_cast<const float*>(slds + (SG == 1 ? (int)(buf - lds) / kStage : g / SG & 1) * kScales) + g % SG;
#pragma unroll
    for (int i = 0; i < MI; ++i) sx[i] = sc[SG * (row_a + 32 * i + l31)];
    const StageIn in = stage_in(g + KS * (NB - 1));
    const float sw = sc[SG * (BM + row_b / kF8Block)];
    constexpr int kEvery = (kLoads + kSteps - 1) / kSteps;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      const int i = t / NJ, jj = t % NJ;
      if (jj == 0 && i + 1 < MI) frag(buf + (row_a + 32 * (i + 1)) * kF8Stage, af[(i + 1) & 1]);
      const v4i (&a)[4] = af[i & 1];
      const v4i (&b)[4] = bf[jj];
      v16f p = {};
      if constexpr (EXACT) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          p = __builtin_amdgcn_mfma_f32_32x32x16_f16(f8_to_f16x8(b[c][0], b[c][1]), f8_to_f16x8(a[c][0], a[c][1]), p, 0, 0, 0);
          p = __builtin_amdgcn_mfma_f32_32x32x16_f16(f8_to_f16x8(b[c][2], b[c][3]), f8_to_f16x8(a[c][2], a[c][3]), p, 0, 0, 0);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          const v8i bb = {b[c][0], b[c][1], b[c][2], b[c][3], b[c + 1][0], b[c + 1][1], b[c + 1][2], b[c + 1][3]};
          const v8i aa = {a[c][0], a[c][1], a[c][2], a[c][3], a[c + 1][0], a[c + 1][1], a[c + 1][2], a[c + 1][3]};
          p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bb, aa, p, 0, 0, 0, 0, 0, 0);
        }
      }
      // this wave's loads of a later stage, ahead of its last products
#pragma unroll
      for (int l = 0; l < kEvery; ++l)
        if (t * kEvery + l < kLoads) dma(ahead, g + KS * (NB - 1), t * kEvery + l, in);
      if constexpr (kSteps == 1) {
        scale_in(0, d[0], sprev);
        d[0] = p;
      } else {
        scale_in((t + kSteps - 1) % kSteps, d[(t + 1) & 1], sprev);
        d[t & 1] = p;
      }
      sprev = sx[i] * sw;
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // This wave's loads have landed, its LDS reads are done, and so are all
  // other waves'.  (Stages are awaited by sync_stage, which leaves the loads of
  // the stages after it under way: vmcnt counts in order.)
  auto sync = [] { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

  // ---- outputs of a tile ----
  // Lane l holds token row 32 i + (l & 31); register q of block (i, jj) output
  // column 32 jj + 8 (q >> 2) + 4 (l >> 5) + (q & 3).  Stored from there, a wave
  // would touch 32 rows with 16 bytes each, so where rows of y are 16-byte
  // aligned (vec 2) the outputs are turned in LDS, JP column blocks (up to 128
  // bytes of a row) at a time, and leave as 16-byte chunks of consecutive lanes
  // (4096 x 4096 x 11008: 212 us with the direct stores, 184 so).
  typedef OutT o4 __attribute__((ext_vector_type(4)));
  constexpr int E = (int)sizeof(OutT);
  constexpr int kRegion = (EXPERTS || KS > 1 ? 1 : NB) * kStage;   // experts: the others hold the next tile's loads
  constexpr int JP = NJ % 2 == 0 && 64 * E <= 128 && NW * 32 * MI * 64 * E <= kRegion ? 2 : 1;
  constexpr int RB = JP * 32 * E, CH = RB / 16;
  constexpr int IP = NW * 32 * MI * RB <= kRegion ? MI : MI % 2 == 0 ? MI / 2 : 1;   // row blocks at a time
  constexpr int kStoresPerPass = 32 * IP * CH / 64, kStores = MI / IP * (NJ / JP) * kStoresPerPass;
  constexpr int kUnder = (NB - 2) * kLoads;              // loads of the later stages
  static_assert(kUnder + (EXPERTS ? kStores : 0) <= 63, "vmcnt counts to 63");
  static_assert(NW * 32 * IP * RB <= kRegion, "a region of LDS for each wave");
  auto four = [&](int i, int jj, int q) {
    return o4{round_to<OutT>(acc[i][jj][4 * q]), round_to<OutT>(acc[i][jj][4 * q + 1]),
              round_to<OutT>(acc[i][jj][4 * q + 2]), round_to<OutT>(acc[i][jj][4 * q + 3])};
  };
  auto store_lines = [&](const F8Tile& at, int8_t* region) {
    int8_t* reg = region + wave * (32 * IP * RB);
    // rows past the run and columns past N go out of the resource's range:
    // every store is issued, so their number is known to the next wait.
    // Non-temporal: outputs would push operands out of L2 (4096 x 4096 x 11008:
    // 202 us with the default policy, 184 so)
    const rsrc_t yr = make_rsrc_uniform(y + (int64_t)at.m0 * N, (u32)((at.hi - at.m0 < BM ? at.hi - at.m0 : BM) * N * E));
#pragma unroll
    for (int ps = 0; ps < MI / IP * (NJ / JP); ++ps) {
      const int ip = ps / (NJ / JP) * IP, jp = ps % (NJ / JP) * JP;
#pragma unroll
      for (int jj = 0; jj < JP; ++jj)
#pragma unroll
        for (int i = 0; i < IP; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int row = 32 * i + l31, byte = E * (32 * jj + 8 * q + 4 * half);
            *reinterpret_cast<o4*>(reg + row * RB + (((byte >> 4) ^ (row & (CH - 1))) << 4) + (byte & 15)) = four(ip + i, jp + jj, q);
          }
      // one wave's LDS accesses execute in order; the statement keeps the
      // compiler from reordering them
      asm volatile("" ::: "memory");
#pragma unroll
      for (int it = 0; it < kStoresPerPass; ++it) {
        const int row = it * (64 / CH) + lane / CH, ch = lane % CH;
        const int n = at.n0 + row_b + 32 * jp + ch * (16 / E);
        const v4i v = ld16(reg + row * RB + ((ch ^ (row & (CH - 1))) << 4));
        __builtin_amdgcn_raw_buffer_store_b128(v, yr, n < N ? (u32)(((row_a + 32 * ip + row) * N + n) * E) : kOOB, 0, kAuxNonTemporal);
      }
      asm volatile("" ::: "memory");
    }
  };
  auto store_direct = [&](const F8Tile& at) {
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
            *reinterpret_cast<o4*>(dst) = four(i, jj, q);
          } else {
#pragma unroll
            for (int t = 0; t < 4; ++t)
              if (n + t < N) dst[t] = round_to<OutT>(acc[i][jj][4 * q + t]);
          }
        }
    }
  };

  // ---- the tiles ----
  // The first stages of the next tile are loaded ahead of a tile's stores, and
  // the next tile waits for those loads only, not for the stores behind them.
  auto sync_stage = [&](bool stores) {
    if (EXPERTS && stores)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kUnder + kStores) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kUnder) : "memory");
  };
  auto buffer = [&](int b) { return lds + (b >= NB ? b - NB : b) * kStage; };
  F8Tile at, next;
  if (!next_tile(at)) return;
  int sb = 0;                        // buffer of the tile's first stage
  aim(at, rows_of(at));
  auto first_stages = [&](int b) {
#pragma unroll
    for (int g = 0; g < NB - 1; ++g) {
      const StageIn in = stage_in(kg + KS * g);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) dma(buffer(b + g), kg + KS * g, i, in);
    }
  };
  first_stages(0);
  bool stored = false;               // kStores stores were issued behind the first stages' loads
  for (;;) {
    const bool more = next_tile(next);
    Rows rn;
    if (EXPERTS && more) rn = rows_of(next);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int jj = 0; jj < NJ; ++jj) acc[i][jj] = v16f{};
    d[0] = d[1] = v16f{};
    sprev = 0.f;
    int b = sb;                      // buffer of stage g; the one before it is free
    // (every group runs the same number of stages; one past G is all zeros)
    for (int g = 0; g < (G + KS - 1) / KS; ++g) {
      sync_stage(stored && g < NB - 1);
      multiply(buffer(b), buffer(b + NB - 1), kg + KS * g);
      b = b + 1 == NB ? 0 : b + 1;
    }
    scale_in(kSteps - 1, d[(kSteps - 1) & 1], sprev);
    sync();   // the stage buffers are free
    if (EXPERTS && more) {
      aim(next, rn);
      first_stages(b);
    }
    if constexpr (KS > 1) {
      // the other groups hand their sums to group 0, which adds them in order
      constexpr int kSums = 4096;     // 16 sums of 64 lanes
      static_assert(NW * MI * NJ * kSums <= kStage, "a wave's sums in its ring's free buffer");
      auto part = [&](int k, int i, int jj, int c) {
        int8_t* free = buffer(b + NB - 1) + (k - kg) * f8_ring_bytes<BM, BN, NB>();
        return free + ((wave * MI + i) * NJ + jj) * kSums + c * 1024 + 16 * lane;
      };
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int jj = 0; jj < NJ; ++jj)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (kg > 0)
              *reinterpret_cast<v4f*>(part(kg, i, jj, c)) = v4f{acc[i][jj][4 * c], acc[i][jj][4 * c + 1], acc[i][jj][4 * c + 2], acc[i][jj][4 * c + 3]};
      lds_barrier();
      if (kg == 0) {
#pragma unroll
        for (int k = 1; k < KS; ++k)
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int jj = 0; jj < NJ; ++jj)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const v4f o = *reinterpret_cast<const v4f*>(part(k, i, jj, c));
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][jj][4 * c + q] += o[q];
              }
      }
    }
    if (kg == 0) {
      if (vec > 1) store_lines(at, EXPERTS || KS > 1 ? buffer(b + NB - 1) : lds);
      else store_direct(at);
    }
    if (!EXPERTS || !more) return;
    at = next;
    sb = b;
    stored = vec > 1 && kg == 0;
  }
}

template <int BM, int BN, int WM, int WN, int KS, int NB, bool EXACT, typename OutT>
__global__ __launch_bounds__(64 * WM * WN * KS, 2) void k_f8_tile(
    const uint8_t* __restrict__ xq, const float* __restrict__ xs, const uint8_t* __restrict__ wq,
    const float* __restrict__ ws, F8Rows fr, int N, int K, OutT* __restrict__ y, int vec) {
  __shared__ __attribute__((aligned(16))) int8_t lds[KS * f8_ring_bytes<BM, BN, NB>()];
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
  int left = 1;
  f8_tiles<BM, BN, WM, WN, KS, NB, EXACT, OutT, false>(lds, xq, xs, wq, ws, fr, N, K, y, vec, [&](F8Tile& t) {
    t = F8Tile{0, (first + in % gsize) * BM, M, in / gsize * BN};
    return left-- > 0;
  });
}

// The experts' tiles.  The row counts are on the GPU only, so every workgroup
// counts the tiles of all experts first (a scan over E in LDS), then takes
// tiles of the joint list: XCD x the x-th eighth of it, so that an expert's
// weights stay in one L2.
constexpr int kF8MaxExperts = 1024;

template <int BM, int BN, int WM, int WN, int KS, int NB, bool EXACT, typename OutT>
__global__ __launch_bounds__(64 * WM * WN * KS, 2) void k_f8_tile_experts(
    const uint8_t* __restrict__ xq, const float* __restrict__ xs, const uint8_t* __restrict__ wq,
    const float* __restrict__ ws, F8Rows fr, int E, int N, int K, OutT* __restrict__ y, int vec) {
  __shared__ __attribute__((aligned(16))) int8_t lds[KS * f8_ring_bytes<BM, BN, NB>()];
  // tile rows ahead of each expert, and its number of rows
  __shared__ int first[kF8MaxExperts + 1], count[kF8MaxExperts];
  const int tiles_n = (N + BN - 1) / BN;
  if (threadIdx.x < kWave) {
    // each lane counts a run of experts, the lanes' sums are scanned; offsets
    // that do not rise can name rows many times over, so the count saturates
    const int64_t most = f8_most_tile_rows(tiles_n, gridDim.x);
    const int per = (E + kWave - 1) / kWave, e0 = threadIdx.x * per;
    int64_t sum = 0;
    for (int e = e0; e < min(e0 + per, E); ++e) {
      int lo, hi;
      f8_expert_rows(fr, e, lo, hi);
      count[e] = hi - lo;
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
      first[e] = (int)min(run, most);
      run += (count[e] + BM - 1) / BM;
    }
    if (threadIdx.x == kWave - 1) first[E] = (int)min(run, most);
  }
  __syncthreads();
  const int total = first[E] * tiles_n;
  const int per = total / 8, rem = total % 8, xcd = blockIdx.x % 8;
  const int begin = xcd * per + min(xcd, rem), end = begin + per + (xcd < rem);
  // With several tile rows an expert, the two workgroups that share a CU (the
  // first and second half of an XCD's) take neighbours, which read the same
  // weight rows (64 experts of 384 rows: 258 us, 260 without; with one tile row
  // there is nothing to share and the order of the list is better, 16 experts
  // of 64 rows: 22.3 us against 23.2).
  const int slots = gridDim.x / 8, at = blockIdx.x / 8, half = (slots + 1) / 2;
  int t = begin + (fr.R <= (int64_t)E * BM ? at : at < half ? 2 * at : 2 * (at - half) + 1);
  f8_tiles<BM, BN, WM, WN, KS, NB, EXACT, OutT, true>(lds, xq, xs, wq, ws, fr, N, K, y, vec, [&](F8Tile& to) {
    if (t >= end) return false;
    // the last expert whose first tile is at or before t
    int a = 0, b = E - 1;
    while (a < b) {
      const int mid = (a + b + 1) / 2;
      if (first[mid] * tiles_n <= t) a = mid;
      else b = mid - 1;
    }
    a = __builtin_amdgcn_readfirstlane(a);
    const int lo = min(max(fr.offsets[a], 0), fr.R), hi = lo + __builtin_amdgcn_readfirstlane(count[a]);
    const int in = t - __builtin_amdgcn_readfirstlane(first[a]) * tiles_n, rows = (hi - lo + BM - 1) / BM;
    to = F8Tile{a, lo + in % rows * BM, hi, in / rows * BN};
    t += gridDim.x / 8;
    return true;
  });
}

template <int BM, int BN, int WM, int WN, int KS, int NB, typename OutT>
static void launch_f8_tile(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                           const F8Rows& fr, int N, int K, OutT* y, int vec, hipStream_t st) {
  const int64_t tiles = ((int64_t)fr.R + BM - 1) / BM * ((N + BN - 1) / BN);
  k_f8_tile<BM, BN, WM, WN, KS, NB, std::is_same<OutT, float>::value, OutT>
      <<<dim3((unsigned)tiles), dim3(64 * WM * WN * KS), 0, st>>>(xq, xs, wq, ws, fr, N, K, y, vec);
}

template <int BM, int BN, int WM, int WN, int KS, int NB, typename OutT>
static void launch_f8_tile(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                           const F8Rows& fr, int64_t E, int N, int K, OutT* y, int vec,
                           hipStream_t st) {
  if (!fr.offsets)
    return launch_f8_tile<BM, BN, WM, WN, KS, NB>(xq, xs, wq, ws, fr, N, K, y, vec, st);
  // as many workgroups as can be resident, a multiple of the 8 XCDs
  constexpr int kLds = KS * f8_ring_bytes<BM, BN, NB>() + 8 * kF8MaxExperts + 4;
  const int64_t most = (((int64_t)fr.R + BM - 1) / BM + E) * ((N + BN - 1) / BN);
  const int64_t grid = std::min<int64_t>(256 * (int64_t)(kLdsBytesPerCU / kLds), (most + 7) / 8 * 8);
  k_f8_tile_experts<BM, BN, WM, WN, KS, NB, std::is_same<OutT, float>::value, OutT>
      <<<dim3((unsigned)grid), dim3(64 * WM * WN * KS), 0, st>>>(xq, xs, wq, ws, fr, (int)E, N, K, y, vec);
}

template <typename OutT>
static hipError_t gemm_f8_t(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                            const F8Rows& fr, int64_t E, int N, int K, OutT* y, hipStream_t st) {
  // how wide a store every row of y is aligned to: 2: 16 bytes (and a tile's
  // rows within reach of 32-bit offsets), 1: 4 outputs
  const int vec = (uintptr_t)y % 16 == 0 && N * sizeof(OutT) % 16 == 0 && N <= (1 << 20) ? 2
                  : (uintptr_t)y % (4 * sizeof(OutT)) == 0 && N % 4 == 0 ? 1 : 0;
  switch (f8_kernel(fr.offsets != nullptr, fr.R, E, N, sizeof(OutT) > 2)) {
    case F8Kernel::kStream: launch_f8_stream(xq, xs, wq, ws, fr, E, N, K, y, vec, st); break;
    case F8Kernel::kTile64TwoGroups: launch_f8_tile<64, 64, 2, 2, 2, 3>(xq, xs, wq, ws, fr, E, N, K, y, vec, st); break;
    case F8Kernel::kTile64: launch_f8_tile<64, 64, 2, 2, 1, 3>(xq, xs, wq, ws, fr, E, N, K, y, vec, st); break;
    case F8Kernel::kTile128: launch_f8_tile<128, 128, 2, 2, 1, 2>(xq, xs, wq, ws, fr, E, N, K, y, vec, st); break;
    case F8Kernel::kTile256:
      if constexpr (sizeof(OutT) == 2) launch_f8_tile<256, 256, 2, 4, 1, 2>(xq, xs, wq, ws, fr, N, K, y, vec, st);
      break;
  }
  return hipGetLastError();
}

hipError_t launch_gemm_f8(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                          const int32_t* offsets, const int32_t* row_token, int64_t T, int64_t R,
                          int64_t E, int64_t N, int64_t K, void* y, int y_dtype, hipStream_t st) {
  const F8Rows fr{offsets, row_token, (int)T, (int)R};
  const int n = (int)N, k = (int)K;
  switch (y_dtype) {
    case F32: return gemm_f8_t<float>(xq, xs, wq, ws, fr, E, n, k, (float*)y, st);
    case F16: return gemm_f8_t<_Float16>(xq, xs, wq, ws, fr, E, n, k, (_Float16*)y, st);
    default: return gemm_f8_t<uint16_t>(xq, xs, wq, ws, fr, E, n, k, (uint16_t*)y, st);
  }
}

}  // namespace qg
