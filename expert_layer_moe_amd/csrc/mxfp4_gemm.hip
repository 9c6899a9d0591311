// Matrix product of 4-bit codes (e2m1) in blocks of 32 under powers of two (e8m0):
//   out[m][n] = sum over blocks b of 2^(sa[m][b] + sb[n][b] - 254)
//               (sum over k in b of a[m][k] b[n][k])
// One MFMA (16 x 16 x 128) takes four blocks of either operand with their scale
// codes, and adds their sum to the accumulator: on this matrix unit products and
// sums of e2m1 codes under their scales are exact, but for one rounding to fp32 of
// accumulator and sum together (measured, with scales up to 2^60 apart), so fp32
// results need nothing else than bf16 ones.  A scale code of 255 gives NaN.
//
// The weights are the MFMA's A operand and the token rows its B operand: a lane's
// four sums are four columns of one token.  Lane (r, g) = (l % 16, l / 16) holds 32
// codes, one block, of row r of either: 16 bytes, a piece.  Which four of a row's
// blocks an MFMA takes, and in which order, is free as long as both operands agree.
#include "moe_common.h"
#include "moe_gemm_tile.h"
#include "moe_kernels.h"

#include <algorithm>

namespace moe {
namespace {

constexpr int kBlock = 32;     // values of a block, 16 bytes: a piece
constexpr int kRow = 128;      // bytes of a step of a row: 8 pieces, 256 values
constexpr uint32_t kOne = 127; // scale code of 1, for pieces past the end

__device__ __forceinline__ i32x8 operand(u32x4 p) {
  return __builtin_shufflevector(__builtin_bit_cast(i32x4, p), __builtin_bit_cast(i32x4, p), 0, 1, 2,
                                 3, -1, -1, -1, -1);
}
// D(16x16, fp32) += A(16x128) * B(128x16) under byte W of wscale and byte A of
// ascale: lane l has row l % 16 of A, column l % 16 of B, and D[4 (l / 16) + i][l % 16].
template <int W, int A>
__device__ __forceinline__ floatx4 mfma(u32x4 w, uint32_t wscale, u32x4 a, uint32_t ascale, floatx4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w), operand(a), c, 4, 4, W,
                                                          (int)wscale, A, (int)ascale);
}

// Two or four scale codes from any byte address on.
__device__ __forceinline__ uint32_t load_u16(const uint8_t* p) {
  uint16_t v;
  __builtin_memcpy(&v, p, 2);
  return v;
}
__device__ __forceinline__ u32x4 load_u128(const uint8_t* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// ---- few rows --------------------------------------------------------------------
// One block per 16 columns and 16 MT rows; its 8 waves split the steps of K and
// meet in LDS.  Bound by reading the weights: they stream through rings in LDS,
// whole 128-byte lines of 8 rows a load; the token rows and all scales, from L2,
// through registers.  In a step lane group g takes pieces 2 g and 2 g + 1, whose
// scale codes lie side by side.
//
// Rows and columns past the end read the last ones, unstored.  The last step, if
// it ends inside, is a wave's of its own: pieces past the end are zeros under 1.
template <int MT, bool ONCE>
struct Rows {
  static constexpr int W = 8, kSets = 4, kAhead = kSets - 1;
  static constexpr int kEntry = 16 * kRow;
  static constexpr int kLoads = 2 + 1 + 3 * MT;   // of a step, in flight
  __amdgpu_buffer_rsrc_t wbuf, abuf;
  const uint8_t *wsc, *asc[MT];   // this lane's scale codes of step 0
  uint32_t wrow[2], arow[MT];
  u32x4 a[kSets][MT][2];
  uint32_t sa[kSets][MT], sw[kSets];
  floatx4 acc[MT];

  __device__ __forceinline__ void issue(uint8_t* __restrict__ to, int step, int set) {
    const uint32_t k0 = step * kRow;
#pragma unroll
    for (int p = 0; p < 2; ++p) to_lds16<ONCE>(wbuf, wrow[p], k0, to + 1024 * p);
    sw[set] = load_u16(wsc + step * 8);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      a[set][t][0] = load16(abuf, arow[t], k0);
      a[set][t][1] = load16(abuf, arow[t] + 16, k0);
      sa[set][t] = load_u16(asc[t] + step * 8);
    }
  }
  // The step in set i and `cur`.
  __device__ __forceinline__ void multiply(const uint8_t* __restrict__ cur, int lane, int i) {
    const int r = lane % 16, g = lane / 16;
    const u32x4 w0 = ld16(cur + r * kRow + 16 * (2 * g ^ r / 2)),
                w1 = ld16(cur + r * kRow + 16 * ((2 * g + 1) ^ r / 2));
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      acc[t] = mfma<0, 0>(w0, sw[i], a[i][t][0], sa[i][t], acc[t]);
      acc[t] = mfma<1, 1>(w1, sw[i], a[i][t][1], sa[i][t], acc[t]);
    }
  }
};

template <int MT, bool F32, bool ONCE>
__global__ __launch_bounds__(8 * kWave) __attribute__((amdgpu_waves_per_eu(4)))
void mx_gemm_rows_kernel(MxGemm p) {
  using RW = Rows<MT, ONCE>;
  constexpr int W = RW::W;
  __shared__ __attribute__((aligned(16))) uint8_t ring[W][RW::kSets * RW::kEntry];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int r = lane % 16, g = lane / 16;
  const int blocks_n = (p.N + 15) / 16;
  const int n0 = (int)(block_index() % blocks_n) * 16, m0 = (int)(block_index() / blocks_n) * (16 * MT);
  if (m0 >= p.M) return;
  const int nb = p.K / kBlock, steps = nb / 8;   // (whole steps)
  RW rw;
  rw.wbuf = buffer_at(p.b + (size_t)n0 * p.ldb);
  rw.abuf = buffer_at(p.a + (size_t)m0 * p.lda);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int row = 8 * q + lane / 8;
    rw.wrow[q] = (uint32_t)min(row, p.N - 1 - n0) * (uint32_t)p.ldb + 16 * (lane % 8 ^ row / 2);
  }
  const int wr = min(r, p.N - 1 - n0);
  rw.wsc = p.sb + (size_t)(n0 + wr) * p.ldsb + 2 * g;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const uint32_t m = min(16 * t + r, p.M - 1 - m0);
    rw.arow[t] = m * (uint32_t)p.lda + 32 * g;
    rw.asc[t] = p.sa + (size_t)(m0 + m) * p.ldsa + 2 * g;
    rw.acc[t] = floatx4{0.f, 0.f, 0.f, 0.f};
  }
  const int b0 = (int)((long long)steps * wave / W), n = (int)((long long)steps * (wave + 1) / W) - b0;
  uint8_t* mine = ring[wave];
  for (int j = 0; j < n; j += RW::kSets) {
#pragma unroll
    for (int i = 0; i < RW::kSets; ++i)
      if (j + i < n) rw.issue(mine + i * RW::kEntry, b0 + j + i, i);
    wait_loads<0>();
#pragma unroll
    for (int i = 0; i < RW::kSets; ++i)
      if (j + i < n) rw.multiply(mine + i * RW::kEntry, lane, i);
    wait_loads<0>();
  }
  if (const int left = nb - 8 * steps; left != 0 && wave == W - 1) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int piece = 2 * g + h;
      const bool in = piece < left;
      const uint32_t k0 = steps * kRow;
      const u32x4 zero = {0u, 0u, 0u, 0u};
      const u32x4 w = in ? load16(rw.wbuf, wr * (uint32_t)p.ldb + 16 * piece, k0) : zero;
      const uint32_t sw = in ? rw.wsc[steps * 8 + h] : kOne;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const u32x4 a = in ? load16(rw.abuf, rw.arow[t] + 16 * h, k0) : zero;
        const uint32_t sa = in ? rw.asc[t][steps * 8 + h] : kOne;
        rw.acc[t] = mfma<0, 0>(w, sw, a, sa, rw.acc[t]);
      }
    }
  }
  floatx4* red = reinterpret_cast<floatx4*>(mine);
#pragma unroll
  for (int t = 0; t < MT; ++t) red[t * kWave + lane] = rw.acc[t];
  __syncthreads();
  for (int t = wave; t < MT; t += W) {
    floatx4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const floatx4 v = reinterpret_cast<const floatx4*>(ring[w])[t * kWave + lane];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += v[i];
    }
    const int m = m0 + 16 * t + r;
    if (m < p.M) store4<F32>(p.out, p.ldo, p.N, m, n0 + 4 * g, s);
  }
}

// ---- tiles ---------------------------------------------------------------------------
// BM token rows x BN weight rows per block; wave (wm, wn) of WM x WN computes
// 16 TM rows x 16 TN columns.  Steps of K of both operands go from memory straight
// to LDS (16 bytes a lane, no registers) into S stages, S - 1 of them ahead of the
// one that is multiplied: rows of 128 bytes whose piece c lies at place c ^ (row / 2
// % 8), so that the 16 rows of an operand read fall on all banks once.  Rows past
// the end read the last one, unstored; pieces past the end are zeros under 1.
//
// MFMA q = 0, 1 of a step takes piece 4 q + g in lane group g.  Scale codes go
// through registers to LDS, two steps' at a time, so that the four that a lane needs
// lie in one word: of the 16 codes of a row, g, 4 + g, 8 + g and 12 + g; a lane's
// rows of its wave's tiles lie side by side.
template <int TM, int TN, int WM, int WN, int S>
struct Tile {
  static constexpr int W = WM * WN, BM = 16 * TM * WM, BN = 16 * TN * WN;
  static constexpr int LA = BM / 8 / W, LB = BN / 8 / W;   // loads of 8 rows per wave and stage
  static constexpr int kBytes = (BM + BN) * kRow;          // of a stage
  static constexpr int kLoads = LA + LB;                   // a wave's loads of a stage
  static constexpr int kThreads = W * kWave;
  static constexpr int LS = (BM + BN + kThreads - 1) / kThreads;   // rows of scale codes of a thread
  static constexpr int kScales = (BM + BN) * 16;           // bytes of two steps' scale codes
  static_assert(LA * 8 * W == BM && LB * 8 * W == BN, "whole loads");

  int nb;
  __amdgpu_buffer_rsrc_t abuf, bbuf;         // from the tile's first row on
  uint32_t aoff[LA], boff[LB];               // this lane's rows and pieces
  int piece;                                 // of a row's 8, the same in all its rows
  const uint8_t* src[LS];                    // this thread's rows of scale codes
  uint32_t dst[LS], apart[LS];               // and their places: of group 0, between groups
  u32x4 sc[LS];

  // Loads step `step` into a stage.
  __device__ __forceinline__ void load(uint8_t* __restrict__ stage, int step, int wave, int lane) {
    uint8_t* to = stage + wave * 8 * kRow;
    const uint32_t k0 = step * kRow;
    const bool in = 8 * step + piece < nb;
    if (8 * step + 8 > nb && !in) {
#pragma unroll
      for (int j = 0; j < LA + LB; ++j)
        *reinterpret_cast<u32x4*>(to + j * W * 8 * kRow + 16 * lane) = u32x4{0u, 0u, 0u, 0u};
    }
    if (in) {
#pragma unroll
      for (int j = 0; j < LA; ++j) to_lds16(abuf, aoff[j], k0, to + j * W * 8 * kRow);
#pragma unroll
      for (int j = 0; j < LB; ++j) to_lds16(bbuf, boff[j], k0, to + (LA + j) * W * 8 * kRow);
    }
  }

  // The scale codes of steps 2 pair and 2 pair + 1.
  __device__ __forceinline__ void load_scales(int pair) {
#pragma unroll
    for (int i = 0; i < LS; ++i) {
      if (16 * pair + 16 <= nb) {
        sc[i] = load_u128(src[i] + 16 * pair);
      } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t v = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int at = 16 * pair + 4 * w + b;
            v |= (at < nb ? (uint32_t)src[i][at] : kOne) << 8 * b;
          }
          sc[i][w] = v;
        }
      }
    }
  }
  // Byte g of every word into word g, and out.
  __device__ __forceinline__ void store_scales(uint8_t* __restrict__ to) const {
#pragma unroll
    for (int i = 0; i < LS; ++i) {
      if (dst[i] == ~0u) continue;
      const u32x4 v = sc[i];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t sel = 0x0c0c0000u | (uint32_t)(4 + g) << 8 | (uint32_t)g;   // {v1, v0} byte g
        const uint32_t lo = __builtin_amdgcn_perm(v[1], v[0], sel), hi = __builtin_amdgcn_perm(v[3], v[2], sel);
        *reinterpret_cast<uint32_t*>(to + dst[i] + g * apart[i]) = lo | hi << 16;
      }
    }
  }
  template <int H>
  __device__ __forceinline__ void step(const uint8_t* __restrict__ cur, int wave, int lane,
                                       const uint32_t (&sa)[TM], const uint32_t (&sw)[TN],
                                       floatx4 (&acc)[TM][TN]) {
    const int r = lane % 16, g = lane / 16;
    const int sw0 = 16 * (g ^ (r / 2)), sw1 = sw0 ^ 64;   // places of pieces g, g + 4 of row r
    const uint8_t* at = cur + (wave / WN * 16 * TM + r) * kRow;
    const uint8_t* bt = cur + (BM + wave % WN * 16 * TN + r) * kRow;
    u32x4 w0[TN], w1[TN];
#pragma unroll
    for (int q = 0; q < TN; ++q) {
      w0[q] = ld16(bt + q * 16 * kRow + sw0);
      w1[q] = ld16(bt + q * 16 * kRow + sw1);
    }
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      const u32x4 a0 = ld16(at + t * 16 * kRow + sw0), a1 = ld16(at + t * 16 * kRow + sw1);
#pragma unroll
      for (int q = 0; q < TN; ++q) acc[t][q] = mfma<2 * H, 2 * H>(w0[q], sw[q], a0, sa[t], acc[t][q]);
#pragma unroll
      for (int q = 0; q < TN; ++q)
        acc[t][q] = mfma<2 * H + 1, 2 * H + 1>(w1[q], sw[q], a1, sa[t], acc[t][q]);
    }
  }
};

template <int N>
__device__ __forceinline__ void read_words(const uint8_t* from, uint32_t (&to)[N]) {
  __builtin_memcpy(to, __builtin_assume_aligned(from, N % 4 == 0 ? 16 : 4 * N), 4 * N);
}

template <int TM, int TN, int WM, int WN, int S, bool F32>
__global__ __launch_bounds__(WM * WN * kWave) __attribute__((amdgpu_waves_per_eu(TM * TN >= 64 ? 1 : 2)))
void mx_gemm_tile_kernel(MxGemm p, int tiles_m, int tiles_n) {
  using T = Tile<TM, TN, WM, WN, S>;
  constexpr int W = T::W, BM = T::BM, BN = T::BN;
  __shared__ __attribute__((aligned(16))) uint8_t lds[S * T::kBytes + 2 * T::kScales];
  uint8_t* scales = lds + S * T::kBytes;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int wm = wave / WN, wn = wave % WN;
  int tm, tn;
  if (!tile_of_block(tiles_m, tiles_n, tm, tn)) return;
  const int m0 = tm * BM, n0 = tn * BN;
  const int nb = p.K / kBlock, steps = (nb + 7) / 8;

  T tl;
  tl.nb = nb;
  tl.abuf = buffer_at(p.a + (size_t)m0 * p.lda);
  tl.bbuf = buffer_at(p.b + (size_t)n0 * p.ldb);
  tl.piece = (lane % 8) ^ ((wave * 4 + lane / 16) % 8);
#pragma unroll
  for (int j = 0; j < T::LA; ++j)
    tl.aoff[j] = (uint32_t)min((j * W + wave) * 8 + lane / 8, p.M - 1 - m0) * (uint32_t)p.lda + 16 * tl.piece;
#pragma unroll
  for (int j = 0; j < T::LB; ++j)
    tl.boff[j] = (uint32_t)min((j * W + wave) * 8 + lane / 8, p.N - 1 - n0) * (uint32_t)p.ldb + 16 * tl.piece;
#pragma unroll
  for (int i = 0; i < T::LS; ++i) {
    const int f = i * T::kThreads + (int)threadIdx.x;   // row of the tile: tokens, then weights
    const int row = min(f, BM + BN - 1);
    if (row < BM) {
      tl.src[i] = p.sa + (size_t)(m0 + min(row, p.M - 1 - m0)) * p.ldsa;
      tl.dst[i] = 4 * ((row / (16 * TM) * 64 + row % 16) * TM + row / 16 % TM);
      tl.apart[i] = 64 * TM;
    } else {
      const int n = row - BM;
      tl.src[i] = p.sb + (size_t)(n0 + min(n, p.N - 1 - n0)) * p.ldsb;
      tl.dst[i] = 16 * BM + 4 * ((n / (16 * TN) * 64 + n % 16) * TN + n / 16 % TN);
      tl.apart[i] = 64 * TN;
    }
    if (f != row) tl.dst[i] = ~0u;
  }

  floatx4 acc[TM][TN];
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int q = 0; q < TN; ++q) acc[t][q] = floatx4{0.f, 0.f, 0.f, 0.f};

  tl.load_scales(0);
#pragma unroll
  for (int i = 0; i < S - 1; ++i)
    if (i < steps) tl.load(lds + i * T::kBytes, i, wave, lane);
  tl.store_scales(scales);
  wait_and_meet<0>();
  const uint8_t* my_a = scales + 4 * (wm * 64 + lane) * TM;
  const uint8_t* my_w = scales + 16 * BM + 4 * (wn * 64 + lane) * TN;
  int cur = 0, next = S - 1;
  const auto advance = [&] {
    cur = cur + 1 == S ? 0 : cur + 1;
    next = next + 1 == S ? 0 : next + 1;
  };
  for (int st = 0; st < steps; st += 2) {
    const int turn = st / 2 & 1;
    uint32_t sa[TM], sw[TN];
    read_words(my_a + turn * T::kScales, sa);
    read_words(my_w + turn * T::kScales, sw);
    if (st + 2 < steps) tl.load_scales(st / 2 + 1);
    if (st + S - 1 < steps) tl.load(lds + next * T::kBytes, st + S - 1, wave, lane);
    tl.template step<0>(lds + cur * T::kBytes, wave, lane, sa, sw, acc);
    advance();
    // the next stage has arrived (the S - 2 behind it may still be on their
    // way), this one is free
    if (st + S - 1 < steps) wait_and_meet<(S - 2) * T::kLoads>();
    else wait_and_meet<0>();
    if (st + 1 >= steps) break;
    if (st + S < steps) tl.load(lds + next * T::kBytes, st + S, wave, lane);
    tl.template step<1>(lds + cur * T::kBytes, wave, lane, sa, sw, acc);
    if (st + 2 < steps) tl.store_scales(scales + (turn ^ 1) * T::kScales);
    advance();
    if (st + S < steps) wait_and_meet<(S - 2) * T::kLoads>();
    else wait_and_meet<0>();
  }
  // the stages are free; each wave uses a part of its own
  static_assert(W * tile_store_bytes<TN, F32>() <= S * T::kBytes, "the stages hold the waves' tiles");
  store_tile<TM, TN, F32>(acc, lds + wave * tile_store_bytes<TN, F32>(), p.out, p.ldo, p.M, p.N,
                          m0 + wm * 16 * TM, n0 + wn * 16 * TN, lane);
}

template <int TM, int TN, int WM, int WN, int S>
hipError_t launch_tile(const MxGemm& p, hipStream_t s) {
  constexpr int BM = 16 * TM * WM, BN = 16 * TN * WN;
  const long long tm = ((long long)p.M + BM - 1) / BM, tn = ((long long)p.N + BN - 1) / BN;
  if (tm * tn > kMaxGemmBlocks) return hipErrorInvalidValue;
  const dim3 grid = grid_of((tm * tn + 7) / 8 * 8);
  if (p.out_f32)
    hipLaunchKernelGGL((mx_gemm_tile_kernel<TM, TN, WM, WN, S, true>), grid, dim3(WM * WN * kWave), 0, s,
                       p, (int)tm, (int)tn);
  else
    hipLaunchKernelGGL((mx_gemm_tile_kernel<TM, TN, WM, WN, S, false>), grid, dim3(WM * WN * kWave), 0, s,
                       p, (int)tm, (int)tn);
  return hipGetLastError();
}

template <int MT>
hipError_t launch_rows(const MxGemm& p, hipStream_t s) {
  const long long blocks = ((long long)p.M + 16 * MT - 1) / (16 * MT) * (((long long)p.N + 15) / 16);
  if (blocks > kMaxGemmBlocks) return hipErrorInvalidValue;
  const dim3 grid = grid_of(blocks);
#define MOE_ROWS(F, O) \
  hipLaunchKernelGGL((mx_gemm_rows_kernel<MT, F, O>), grid, dim3(8 * kWave), 0, s, p)
  const bool once = p.M <= 16 * MT;   // each weight is read by one block: past the caches
  if (p.out_f32) {
    if (once) MOE_ROWS(true, true);
    else MOE_ROWS(true, false);
  } else {
    if (once) MOE_ROWS(false, true);
    else MOE_ROWS(false, false);
  }
#undef MOE_ROWS
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemm& p, hipStream_t s) {
  if (p.M <= 16) return launch_rows<1>(p, s);
  if ((long long)p.M * p.N <= 256LL * 64 * 64) return launch_tile<2, 2, 2, 2, 3>(p, s);
  if ((long long)p.M * p.N <= 256LL * 128 * 128) return launch_tile<4, 2, 2, 4, 3>(p, s);
  return launch_tile<8, 4, 2, 4, 2>(p, s);
}

}  // namespace moe
