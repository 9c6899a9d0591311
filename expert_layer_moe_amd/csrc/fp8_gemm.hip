// Matrix product of fp8 (e4m3fn) codes with block scales:
//   out[m][n] = sum over K blocks b of sa[m][b] sb[n / 128][b]
//               (sum over k in b of a[m][k] b[n][k])
// ("AMD Instinct MI355X: ATOM ...": block-scale GEMM).  One fp8 MFMA covers a
// whole 128-wide K block, so each block's sum leaves the matrix cores on its
// own and joins the fp32 accumulator under its two scales: four FMAs a lane
// for every MFMA, which run beside the next MFMAs.
//
// The weights are the MFMA's A operand and the token rows its B operand: a
// lane's four sums are four columns of one token, under one product of
// scales.
//
// The fp8 MFMA cuts each product, before it adds it, to a multiple of 2^-13 of the
// largest power of two among the products of its eight k = 8 i .. 8 i + 7
// (measured, with a pair of opposite large products beside small ones).  So a block's sum is off by at most 7 x 2^-13 of
// the sum of the eights' largest products, 1.5e-5 for random codes, and a sum of
// like terms keeps well within the half step of its bf16 result; one that cancels
// need not.  For fp32 results the codes become bf16, exactly, and four bf16 MFMAs
// add up the block in fp32 (F32 below).
//
// Measured (bf16 results): 8192 x 4096 x 7168 207 to 227 us from card to card,
// 2.1 to 2.3 PFLOP/s, where the library product of the same size, with one scale
// for all, takes 169: the matrix cores are busy 49 % of the cycles.  Without the
// FMAs it would take a tenth less, without the loads a fifth, with zeros for
// operands 200 us.  (fp32 results: 430 us.)  1000 x 7168 x 2048 20.3 to 21.4 us;
// 1 x 4096 x 7168, 29 MB, 6.4 us (4.6 TB/s).
#include "moe_common.h"
#include "moe_kernels.h"

#include <algorithm>

namespace moe {
namespace {

typedef __attribute__((__vector_size__(8 * sizeof(int)))) int i32x8;
typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4;

constexpr int kBK = 128;   // K block

// 32 codes of one row: 16-byte pieces g and 4 + g of the row's K block for
// lane group g = lane / 16 (any order of K serves, as long as both operands
// have it).
struct Frag {
  u32x4 p[2];
};

template <bool F32>
struct Operand;
template <>
struct Operand<false> {
  i32x8 v;
  __device__ __forceinline__ void set(const i32x8& f) { v = f; }
  __device__ __forceinline__ void read(const uint8_t* row, int at0, int at1) {
    set(Frag{{ld16(row + at0), ld16(row + at1)}});
  }
  __device__ __forceinline__ void set(const Frag& f) {
    v = i32x8{(int)f.p[0][0], (int)f.p[0][1], (int)f.p[0][2], (int)f.p[0][3],
              (int)f.p[1][0], (int)f.p[1][1], (int)f.p[1][2], (int)f.p[1][3]};
  }
};
template <>
struct Operand<true> {
  __device__ __forceinline__ void set(const i32x8& f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fp8x8_to_bf16x8((uint32_t)f[2 * i], (uint32_t)f[2 * i + 1]);
  }
  bf16x8 v[4];
  __device__ __forceinline__ void read(const uint8_t* row, int at0, int at1) {
    set(Frag{{ld16(row + at0), ld16(row + at1)}});
  }
  __device__ __forceinline__ void set(const Frag& f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fp8x8_to_bf16x8(f.p[i / 2][2 * (i & 1)], f.p[i / 2][2 * (i & 1) + 1]);
  }
};

// D(16x16, fp32) = A(16x128) * B(128x16): lane l has row l % 16 of A, column
// l % 16 of B, and D[4 (l / 16) + i][l % 16] (i < 4).
__device__ __forceinline__ floatx4 mfma_block(const Operand<false>& a, const Operand<false>& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
      a.v, b.v, floatx4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ floatx4 mfma_block(const Operand<true>& a, const Operand<true>& b) {
  floatx4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) d = mfma16x16x32(a.v[i], b.v[i], d);
  return d;
}

// Columns n .. n + 3 of row m, as far as they exist.
template <bool F32>
__device__ __forceinline__ void store4(const Fp8Gemm& p, int m, int n, floatx4 v) {
  const size_t at = (size_t)m * p.ldo + n;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= p.N) break;
    if constexpr (F32) static_cast<float*>(p.out)[at + i] = v[i];
    else static_cast<uint16_t*>(p.out)[at + i] = f32_to_bf16_bits(v[i]);
  }
}

// A buffer from p on (unbounded: the kernels keep their offsets in range).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p, int bytes = -1) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}
// An offset behind the end of every buffer of less than 2 GB: loads give 0.
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t src, uint32_t lane_offset, uint32_t offset) {
  return __builtin_bit_cast(u32x4,
                            __builtin_amdgcn_raw_buffer_load_b128(src, lane_offset, offset, 0));
}

// Waits until at most N of this wave's loads are outstanding and its LDS
// accesses are done, then for the block; no memory access moves across.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | (N >> 4) << 14);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Loads straight to LDS: lane l's 4 or 16 bytes go to dst + 4 l or + 16 l.
// (As buffer loads: the compiler takes global ones for accesses that may
// complete out of order with LDS reads, and waits for all of either at each
// use.)  ONCE: data that no other block reads.
__device__ __forceinline__ void to_lds4(__amdgpu_buffer_rsrc_t src, uint32_t lane_offset,
                                          uint32_t offset, void* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)dst, 4,
                                           lane_offset, offset, 0, 0);
}
template <bool ONCE = false>
__device__ __forceinline__ void to_lds16(__amdgpu_buffer_rsrc_t src, uint32_t lane_offset,
                                         uint32_t offset, void* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)dst, 16,
                                           lane_offset, offset, 0, ONCE ? 2 : 0);
}
// Waits until at most N of the wave's loads are outstanding and its LDS reads
// are done; no memory access moves across.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | (N >> 4) << 14);
  asm volatile("" ::: "memory");
}

// The blocks of a call, at most kGridX of them along x (a multiple of the 8 XCDs;
// a dimension holds less than 2^32 threads): block block_index(), and behind the
// last one some without work.
constexpr unsigned kGridX = 1u << 22;
__device__ __forceinline__ unsigned block_index() { return blockIdx.y * gridDim.x + blockIdx.x; }
dim3 grid_of(long long blocks) {
  const long long y = (blocks + kGridX - 1) / kGridX;
  return dim3((unsigned)std::min<long long>(blocks, kGridX), (unsigned)y);
}

// ---- few rows --------------------------------------------------------------------
// One block per 16 columns and 16 MT rows; its 8 waves split the K blocks and
// meet in LDS.  Bound by reading the weights: they stream through rings in LDS,
// whole 128-byte lines of 8 rows a load, kAhead K blocks ahead, and with them
// the scales; the token rows, from L2, through registers as far ahead.  (Weights by way of
// registers, in half lines: 1 x 4096 x 7168 9.0 us, 6.4 so; 16 x 18432 x 7168 49
// and 34.  16 waves with half the blocks each: 7.9 and 53.)
//
// Rows and columns past the end read the last ones, unstored.  Pieces of K past
// the end: the tokens' lie outside the buffer and are 0, the weights' are those
// of the block's first piece (whose NaN the sum has anyway).
template <int MT, bool F32, bool ONCE>
struct Rows {
  static constexpr int W = 8, kSets = MT == 1 ? 4 : 3, kAhead = kSets - 1;
  // of a K block: 16 weight rows, token scales, weight scale (64 times)
  static constexpr int kAs = 16 * kBK, kWs = kAs + 256, kEntry = kWs + 256;
  static constexpr int kLoads = 4 + 2 * MT;
  int K;
  __amdgpu_buffer_rsrc_t wbuf, wsbuf, abuf, asbuf;
  uint32_t wrow[2], arow[MT], srow;   // this lane's rows
  int wpiece;                             // byte place of its weights in a row's block
  i32x8 a[kSets][MT];   // a Frag's pieces
  floatx4 acc[MT];

  __device__ __forceinline__ void issue(uint8_t* __restrict__ to, int kb, int lane, int set) {
    const int k0 = kb * kBK, g = lane / 16;
    const uint32_t at = k0 + wpiece < K ? wpiece : 0;
#pragma unroll
    for (int p = 0; p < 2; ++p) to_lds16<ONCE>(wbuf, wrow[p] + at, k0, to + 1024 * p);
    to_lds4(asbuf, srow, 4 * kb, to + kAs);
    to_lds4(wsbuf, 0, 4 * kb, to + kWs);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const u32x4 f0 = load16(abuf, k0 + 16 * g < K ? arow[t] : kNowhere, k0);
      const u32x4 f1 = load16(abuf, k0 + 64 + 16 * g < K ? arow[t] + 64 : kNowhere, k0);
      a[set][t] = __builtin_shufflevector(__builtin_bit_cast(i32x4, f0), __builtin_bit_cast(i32x4, f1),
                                          0, 1, 2, 3, 4, 5, 6, 7);
    }
  }

  // The K block in set i and `cur`; LOAD: block `ahead` goes to `to`.
  template <bool LOAD>
  __device__ __forceinline__ void step(const uint8_t* __restrict__ cur, uint8_t* __restrict__ to,
                                       int ahead, int lane, int i) {
    if constexpr (LOAD) {
      wait_loads<63>();   // the reads of the block that is loaded over
      issue(to, ahead, lane, (i + kAhead) % kSets);
      wait_loads<kAhead * kLoads>();
    }
    const int r = lane % 16, g = lane / 16;
    const float ws = *reinterpret_cast<const float*>(cur + kWs);
    Operand<F32> wo;
    wo.read(cur + r * kBK, 16 * (g ^ r % 8), 16 * ((g + 4) ^ r % 8));
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      Operand<F32> ao;
      ao.set(a[i][t]);
      const floatx4 d = mfma_block(wo, ao);
      const float sc = ws * reinterpret_cast<const float*>(cur + kAs)[16 * t + r];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[t][j] = fmaf(sc, d[j], acc[t][j]);
    }
  }
};

template <int MT, bool F32, bool ONCE>
__global__ __launch_bounds__(8 * kWave) __attribute__((amdgpu_waves_per_eu(4)))
void fp8_gemm_rows_kernel(Fp8Gemm p) {
  using RW = Rows<MT, F32, ONCE>;
  constexpr int W = RW::W;
  __shared__ __attribute__((aligned(16))) uint8_t ring[W][RW::kSets * RW::kEntry];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int r = lane % 16, g = lane / 16;
  const int blocks_n = (p.N + 15) / 16;
  const int n0 = (int)(block_index() % blocks_n) * 16, m0 = (int)(block_index() / blocks_n) * (16 * MT);
  if (m0 >= p.M) return;
  const int nb = (p.K + kBK - 1) / kBK;
  RW rw;
  rw.K = p.K;
  rw.wbuf = buffer_at(p.b + (size_t)n0 * p.ldb);
  rw.wsbuf = buffer_at(p.sb + (size_t)(n0 / kBK) * nb);
  // (of the block's rows: pieces behind them read as 0)
  rw.abuf = buffer_at(p.a + (size_t)m0 * p.lda, min(16 * MT, p.M - m0) * (int)p.lda);
  rw.asbuf = buffer_at(p.sa + (size_t)m0 * p.ldsa);
  rw.wpiece = 16 * (lane % 8 ^ lane / 8);
#pragma unroll
  for (int q = 0; q < 2; ++q)
    rw.wrow[q] = (uint32_t)min(8 * q + lane / 8, p.N - 1 - n0) * (uint32_t)p.ldb;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const uint32_t m = min(16 * t + r, p.M - 1 - m0);
    rw.arow[t] = m * (uint32_t)p.lda + 16 * g;
    rw.acc[t] = floatx4{0.f, 0.f, 0.f, 0.f};
  }
  rw.srow = 4u * (uint32_t)min(lane % (16 * MT), p.M - 1 - m0) * (uint32_t)p.ldsa;
  const int b0 = (int)((long long)nb * wave / W), n = (int)((long long)nb * (wave + 1) / W) - b0;
  uint8_t* mine = ring[wave];
  int j = 0;   // blocks done
  if (n >= RW::kSets) {
#pragma unroll
    for (int i = 0; i < RW::kAhead; ++i) {
      rw.issue(mine + i * RW::kEntry, b0 + i, lane, i);
      __builtin_amdgcn_sched_barrier(0);   // block after block, as the waits count
    }
    // whole rounds of the sets (behind the last block that one again, unused,
    // so that as many loads are on the way at every step), then the rest,
    // which is all loaded
#pragma unroll 1
    for (; j + RW::kSets <= n; j += RW::kSets)
#pragma unroll
      for (int i = 0; i < RW::kSets; ++i)
        rw.template step<true>(mine + i * RW::kEntry,
                               mine + (i + RW::kAhead) % RW::kSets * RW::kEntry,
                               b0 + min(j + i + RW::kAhead, n - 1), lane, i);
    wait_loads<0>();
#pragma unroll
    for (int i = 0; i < RW::kAhead; ++i)
      if (j + i < n) rw.template step<false>(mine + i * RW::kEntry, nullptr, 0, lane, i);
  } else {
#pragma unroll
    for (int i = 0; i < RW::kAhead; ++i)
      if (i < n) rw.issue(mine + i * RW::kEntry, b0 + i, lane, i);
    wait_loads<0>();
#pragma unroll
    for (int i = 0; i < RW::kAhead; ++i)
      if (i < n) rw.template step<false>(mine + i * RW::kEntry, nullptr, 0, lane, i);
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
    if (m < p.M) store4<F32>(p, m, n0 + 4 * g, s);
  }
}

// ---- tiles ---------------------------------------------------------------------------
// acc += s d, here: left to itself the compiler moves all FMAs of a K block
// behind its last MFMA (and the sums of all tiles into registers of their own).
__device__ __forceinline__ void add_scaled(floatx4& acc, const floatx4& d, float s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = fmaf(s, d[i], acc[i]);
    asm volatile("" : "+v"(a));
    acc[i] = a;
  }
}

// BM token rows x BN weight rows per block; wave (wm, wn) of WM x WN computes
// 16 TM rows x 16 TN columns.  The K blocks of both operands go from memory
// straight to LDS (16 bytes a lane, no registers) into S stages, S - 1 of
// them ahead of the one that is multiplied: rows of 128 bytes whose 16-byte
// piece c lies at place c ^ (row / 2 % 8), so that the 16 rows of an operand
// read fall on all banks once.  Rows past the end read the last one,
// unstored; pieces of K past the end are set to zero.  The token scales of 8 K
// blocks at a time lie in LDS, [block][row].
template <int TM, int TN, int WM, int WN, int S, int KB, bool F32>
struct Tile {
  static constexpr int W = WM * WN, BM = 16 * TM * WM, BN = 16 * TN * WN;
  static constexpr int LA = BM / 8 / W, LB = BN / 8 / W;   // loads of 8 rows per wave and stage
  static constexpr int SC = 8;                             // K blocks of a scale stage
  static constexpr int LS = BM * SC / kWave / W;           // its loads per wave
  static constexpr int kBlock = (BM + BN) * kBK;           // bytes of a K block
  static constexpr int kBytes = KB * kBlock;               // of a stage
  static constexpr int kLoads = KB * (LA + LB);            // a wave's loads of a stage
  static_assert(LA * 8 * W == BM && LB * 8 * W == BN, "whole loads");
  static_assert(kBK % (16 * TN) == 0, "one weight scale per wave and K block");
  static_assert(BM % kWave == 0 && LS * W * kWave == BM * SC, "whole scale loads");
  static_assert((S - 2) * KB <= SC - 2 && SC % KB == 0, "a scale stage arrives before its use");

  int K, nb;
  // from the tile's first row on: a, b, the scales of a, the scales of b
  __amdgpu_buffer_rsrc_t abuf, bbuf, sbuf, wbuf;
  uint32_t aoff[LA], boff[LB];               // this lane's rows and pieces
  uint32_t soff[LS], woff;                   // its rows of the scales
  int piece;                                 // byte place of its piece (the same in all its rows)

  // Loads a stage: K blocks kb .. kb + KB - 1 (past the end: the last one).
  __device__ __forceinline__ void load(uint8_t* __restrict__ stage, int kb, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int k0 = min(kb + i, nb - 1) * kBK;
      uint8_t* to = stage + i * kBlock + wave * 8 * kBK;
      const bool in = k0 + piece < K;
      if (k0 + kBK > K && !in) {
#pragma unroll
        for (int j = 0; j < LA + LB; ++j)
          *reinterpret_cast<u32x4*>(to + j * W * 8 * kBK + 16 * lane) = u32x4{0u, 0u, 0u, 0u};
      }
      if (in) {
#pragma unroll
        for (int j = 0; j < LA; ++j) to_lds16(abuf, aoff[j], k0, to + j * W * 8 * kBK);
#pragma unroll
        for (int j = 0; j < LB; ++j) to_lds16(bbuf, boff[j], k0, to + (LA + j) * W * 8 * kBK);
      }
    }
  }

  // Loads the scales of K blocks 8 chunk .. 8 chunk + 7 (past the end: of the
  // last block): the tokens', 64 rows of a block at a time, then the weights',
  // 8 lanes per block of columns (lanes past the tile's columns are not read).
  __device__ __forceinline__ void load_scales(float* __restrict__ to, int chunk, int wave,
                                              int lane) const {
#pragma unroll
    for (int i = 0; i < LS; ++i) {
      const int at = i * W + wave, j = at / (BM / kWave), first = at % (BM / kWave) * kWave;
      to_lds4(sbuf, soff[i], 4 * min(chunk * SC + j, nb - 1), to + j * BM + first);
    }
    if (wave == 0) to_lds4(wbuf, woff + 4 * min(chunk * SC + lane % SC, nb - 1), 0, to + SC * BM);
  }

  // The token scales of rows 16 t + r and the weight scale of K block kb.
  __device__ __forceinline__ float scales_of(const float* __restrict__ scale, int kb, int wave, int r,
                                             float (&sa)[TM]) const {
    const float* sp = scale + kb % SC * BM + (wave / WN * 16 + r) * TM;
    if constexpr (TM % 4 == 0) {
#pragma unroll
      for (int t = 0; t < TM; t += 4) {
        const floatx4 v = *reinterpret_cast<const floatx4*>(sp + t);
#pragma unroll
        for (int i = 0; i < 4; ++i) sa[t + i] = v[i];
      }
    } else {
#pragma unroll
      for (int t = 0; t < TM; ++t) sa[t] = sp[t];
    }
    return scale[SC * BM + wave % WN * 16 * TN / kBK * SC + kb % SC];
  }

  // One stage, K blocks kb .. kb + KB - 1: the stage S - 1 further on is
  // loaded into `next` while `cur` is multiplied.
  __device__ __forceinline__ void step(const uint8_t* __restrict__ cur, uint8_t* __restrict__ next,
                                       const float* __restrict__ scale, float* __restrict__ scale_next, int kb,
                                       int wave, int lane, floatx4 (&acc)[TM][TN]) {
    // the other stage of scales, last read in the K blocks before this stage's
    if (kb % SC == (KB > 2 ? 0 : 2)) load_scales(scale_next, kb / SC + 1, wave, lane);
    if (kb + (S - 1) * KB < nb) load(next, kb + (S - 1) * KB, wave, lane);
    const int r = lane % 16, g = lane / 16;
    const int sw0 = 16 * (g ^ (r / 2)), sw1 = sw0 ^ 64;   // places of pieces g, g + 4 of row r
    const uint8_t* at = cur + (wave / WN * 16 * TM + r) * kBK;
    const uint8_t* bt = cur + (BM + wave % WN * 16 * TN + r) * kBK;
    if constexpr (KB > 1) {
      // small tiles: every operand of the stage first (a stage's last K blocks
      // may lie past the end: they are the last one again, under scale 0)
      Operand<F32> wo[KB][TN], ao[KB][TM];
      float sc[KB][TM];
#pragma unroll
      for (int j = 0; j < KB; ++j) {
#pragma unroll
        for (int q = 0; q < TN; ++q) wo[j][q].read(bt + j * kBlock + q * 16 * kBK, sw0, sw1);
#pragma unroll
        for (int t = 0; t < TM; ++t) ao[j][t].read(at + j * kBlock + t * 16 * kBK, sw0, sw1);
        const float ws = scales_of(scale, kb + j, wave, r, sc[j]);
#pragma unroll
        for (int t = 0; t < TM; ++t) sc[j][t] = kb + j < nb ? ws * sc[j][t] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < KB; ++j)
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
          for (int q = 0; q < TN; ++q) {
            const floatx4 d = mfma_block(wo[j][q], ao[j][t]);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][q][i] = fmaf(sc[j][t], d[i], acc[t][q][i]);
          }
      return;
    }
    // token tile t's MFMAs run beside the FMAs of tile t - 1 and the operand
    // reads of tile t + 1
    Frag f;
    f.p[0] = ld16(at + sw0);
    f.p[1] = ld16(at + sw1);
    Operand<F32> wo[TN];
#pragma unroll
    for (int q = 0; q < TN; ++q) wo[q].read(bt + q * 16 * kBK, sw0, sw1);
    float sa[TM];
    const float ws = scales_of(scale, kb, wave, r, sa);
    floatx4 d_old[TN];
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      Operand<F32> ao;
      ao.set(f);
      if (t + 1 < TM) {
        f.p[0] = ld16(at + (t + 1) * 16 * kBK + sw0);
        f.p[1] = ld16(at + (t + 1) * 16 * kBK + sw1);
      }
      const float sc = ws * sa[t > 0 ? t - 1 : 0];
      floatx4 d[TN];
#pragma unroll
      for (int q = 0; q < TN; ++q) {
        d[q] = mfma_block(wo[q], ao);
        if (t > 0) add_scaled(acc[t - 1][q], d_old[q], sc);
      }
#pragma unroll
      for (int q = 0; q < TN; ++q) d_old[q] = d[q];
      if constexpr (!F32) {
        if (t == 0) {
          // the first MFMA needs four of the reads
          __builtin_amdgcn_sched_group_barrier(0x100, 2 + 2 * TN + 1 + (TM + 3) / 4, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
        if (t + 1 < TM) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);   // LDS reads
        if (t > 0)
#pragma unroll
          for (int q = 0; q < TN; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // an MFMA
            __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);   // four FMAs
          }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int q = 0; q < TN; ++q) add_scaled(acc[TM - 1][q], d_old[q], ws * sa[TM - 1]);
  }
};

template <int TM, int TN, int WM, int WN, int S, int KB, bool F32>
__global__ __launch_bounds__(WM * WN * kWave) __attribute__((amdgpu_waves_per_eu(TM * TN >= 64 ? 1 : 2)))
void fp8_gemm_tile_kernel(Fp8Gemm p, int tiles_m, int tiles_n) {
  using T = Tile<TM, TN, WM, WN, S, KB, F32>;
  constexpr int W = T::W, BM = T::BM, BN = T::BN, SC = T::SC;
  // One array for all: with several the compiler gives each an alias scope
  // of its own in place of those of step()'s arguments, and then waits for
  // every load to LDS ahead of any read.
  constexpr int kScales = SC * BM + kWave;   // token scales, weight scales
  __shared__ __attribute__((aligned(16))) uint8_t lds[S * T::kBytes + 2 * kScales * 4];
  float* scales = reinterpret_cast<float*>(lds + S * T::kBytes);
  static_assert(BN <= 8 * kBK && SC == 8, "a wave holds a stage's weight scales");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int wm = wave / WN, wn = wave % WN;
  const int r = lane % 16, g = lane / 16;
  // The hardware hands block b to XCD b % 8: give each XCD a contiguous range
  // of tiles, and walk them in groups of 8 rows of tiles, column by column,
  // so that its tiles share operands in its L2.
  const int total = tiles_m * tiles_n;
  const int xcd = block_index() % 8, at = block_index() / 8;
  const int tile = total / 8 * xcd + min(xcd, total % 8) + at;
  if (at >= total / 8 + (xcd < total % 8 ? 1 : 0)) return;
  constexpr int GM = 8;
  const int group = tile / (GM * tiles_n), in_group = tile - group * (GM * tiles_n);
  const int gm = min(GM, tiles_m - group * GM);
  const int tm = group * GM + in_group % gm, tn = in_group / gm;
  const int m0 = tm * BM, n0 = tn * BN;
  const int nb = (p.K + kBK - 1) / kBK;

  T tl;
  tl.K = p.K;
  tl.nb = nb;
  tl.wbuf = buffer_at(p.sb + (size_t)(n0 / kBK) * nb);
  tl.woff = 4u * ((uint32_t)min(lane / SC, (p.N - 1) / kBK - n0 / kBK) * (uint32_t)nb);
  tl.abuf = buffer_at(p.a + (size_t)m0 * p.lda);
  tl.bbuf = buffer_at(p.b + (size_t)n0 * p.ldb);
  tl.sbuf = buffer_at(p.sa + (size_t)m0 * p.ldsa);
  tl.piece = 16 * ((lane % 8) ^ ((wave * 4 + lane / 16) % 8));
#pragma unroll
  for (int j = 0; j < T::LA; ++j)
    tl.aoff[j] = (uint32_t)min((j * W + wave) * 8 + lane / 8, p.M - 1 - m0) * (uint32_t)p.lda + tl.piece;
#pragma unroll
  for (int j = 0; j < T::LB; ++j)
    tl.boff[j] = (uint32_t)min((j * W + wave) * 8 + lane / 8, p.N - 1 - n0) * (uint32_t)p.ldb + tl.piece;
#pragma unroll
  for (int i = 0; i < T::LS; ++i) {
    // a lane's rows of a wave's TM tiles lie side by side
    const int f = (i * W + wave) % (BM / kWave) * kWave + lane;
    const int row = f / (16 * TM) * (16 * TM) + f % TM * 16 + f / TM % 16;
    tl.soff[i] = 4u * ((uint32_t)min(row, p.M - 1 - m0) * (uint32_t)p.ldsa);
  }

  floatx4 acc[TM][TN];
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int q = 0; q < TN; ++q) acc[t][q] = floatx4{0.f, 0.f, 0.f, 0.f};

  tl.load_scales(scales, 0, wave, lane);
#pragma unroll
  for (int i = 0; i < S - 1; ++i)
    if (i * KB < nb) tl.load(lds + i * T::kBytes, i * KB, wave, lane);
  wait_and_meet<0>();
  int cur = 0, next = S - 1;
  for (int kb = 0; kb < nb; kb += KB) {
    tl.step(lds + cur * T::kBytes, lds + next * T::kBytes, scales + (kb / SC & 1) * kScales,
            scales + ((kb / SC & 1) ^ 1) * kScales, kb, wave, lane, acc);
    cur = cur + 1 == S ? 0 : cur + 1;
    next = next + 1 == S ? 0 : next + 1;
    // the next stage has arrived (the S - 2 behind it may still be on their
    // way), this one is free
    if (kb + (S - 1) * KB < nb) wait_and_meet<(S - 2) * T::kLoads>();
    else wait_and_meet<0>();
  }
  // Out through LDS, 16 rows at a time: as the MFMA leaves it, a lane has
  // four columns of one row, and a store would cover 16 rows x 32 bytes.  The
  // stages are free; each wave uses a part of its own.
  constexpr int kSize = F32 ? 4 : 2, kCols = 16 * TN;
  constexpr int kPitch = kCols * kSize + 16;
  static_assert(W * 16 * kPitch <= S * T::kBytes, "the stages hold the waves' tiles");
  uint8_t* mine = lds + wave * (16 * kPitch);
  const int nw = n0 + wn * kCols;
  constexpr int kVec = 16 / kSize, kLanes = kCols / kVec;   // values of a piece, pieces of a row
  const bool wide = ((size_t)p.ldo * kSize | (size_t)p.N * kSize | (size_t)p.out) % 16 == 0;
#pragma unroll
  for (int t = 0; t < TM; ++t) {
#pragma unroll
    for (int q = 0; q < TN; ++q) {
      uint8_t* to = mine + r * kPitch + (16 * q + 4 * g) * kSize;
      if constexpr (F32) *reinterpret_cast<floatx4*>(to) = acc[t][q];
      else
        *reinterpret_cast<u32x2*>(to) =
            u32x2{pack_bf16x2(acc[t][q][0], acc[t][q][1]), pack_bf16x2(acc[t][q][2], acc[t][q][3])};
    }
    const int mt = m0 + wm * 16 * TM + 16 * t;
    if (wide) {
#pragma unroll
      for (int i = lane; i < 16 * kLanes; i += kWave) {
        const int row = i / kLanes, c = i % kLanes * kVec;
        const u32x4 v = ld16(mine + row * kPitch + c * kSize);
        if (mt + row < p.M && nw + c < p.N)
          *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(p.out) +
                                    ((size_t)(mt + row) * p.ldo + nw + c) * kSize) = v;
      }
    } else {
      for (int i = lane; i < 16 * kCols; i += kWave) {
        const int row = i / kCols, c = i % kCols;
        if (mt + row >= p.M || nw + c >= p.N) continue;
        const size_t o = (size_t)(mt + row) * p.ldo + nw + c;
        const uint8_t* from = mine + row * kPitch + c * kSize;
        if constexpr (F32) static_cast<float*>(p.out)[o] = *reinterpret_cast<const float*>(from);
        else static_cast<uint16_t*>(p.out)[o] = *reinterpret_cast<const uint16_t*>(from);
      }
    }
  }
}

// TO_F32: also for fp32 results (the bf16 operands of a 256 x 256 tile do not fit
// the registers; a 64 x 128 one is never the fastest, two of 64 x 64 are).
template <int TM, int TN, int WM, int WN, int S, int KB = 1, bool TO_F32 = true>
hipError_t launch_tile(const Fp8Gemm& p, hipStream_t s) {
  constexpr int BM = 16 * TM * WM, BN = 16 * TN * WN;
  const long long tm = ((long long)p.M + BM - 1) / BM, tn = ((long long)p.N + BN - 1) / BN;
  if (tm * tn > kMaxGemmBlocks) return hipErrorInvalidValue;
  const dim3 grid = grid_of((tm * tn + 7) / 8 * 8);
  if (p.out_f32) {
    if constexpr (TO_F32)
      hipLaunchKernelGGL((fp8_gemm_tile_kernel<TM, TN, WM, WN, S, KB, true>), grid,
                         dim3(WM * WN * kWave), 0, s, p, (int)tm, (int)tn);
    else
      return hipErrorInvalidValue;
  } else {
    hipLaunchKernelGGL((fp8_gemm_tile_kernel<TM, TN, WM, WN, S, KB, false>), grid,
                       dim3(WM * WN * kWave), 0, s, p, (int)tm, (int)tn);
  }
  return hipGetLastError();
}

template <int MT>
hipError_t launch_rows(const Fp8Gemm& p, hipStream_t s) {
  const long long blocks = ((long long)p.M + 16 * MT - 1) / (16 * MT) * (((long long)p.N + 15) / 16);
  if (blocks > kMaxGemmBlocks) return hipErrorInvalidValue;
  const dim3 grid = grid_of(blocks);
#define MOE_ROWS(F, O) \
  hipLaunchKernelGGL((fp8_gemm_rows_kernel<MT, F, O>), grid, dim3(8 * kWave), 0, s, p)
  // each weight is read by one block: past the caches (where three blocks read
  // them, 37 x 1001 x 5136, that took 12.0 us in place of 8.0)
  const bool once = p.M <= 16 * MT;
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

// The kernels of different tiles and what they take: us per K block while
// each CU has at most one block, and with all blocks a CU holds (bf16 / fp32
// result; 1e9: not there).  Measured with K = 7168 (bf16) and 4096
// (fp32) on shapes whose tiles number 16 .. 256 and 512 .. 2048.
struct Shape {
  int bm, bn, per_cu;
  float one[2], full[2];
};
constexpr Shape kTiles[] = {
    {64, 32, 2, {.30f, .39f}, {.52f, .65f}},
    {64, 64, 2, {.42f, .55f}, {.65f, .71f}},
    {64, 128, 1, {.53f, 1e9f}, {.53f, 1e9f}},
    {128, 128, 1, {.70f, 1.1f}, {.70f, 1.1f}},
    {128, 256, 1, {1.05f, 1.7f}, {1.0f, 1.7f}},
    {256, 256, 1, {1.65f, 1e9f}, {1.75f, 1e9f}},
};

// The kernel with the least expected time: an index of kTiles, or kRows16 or
// kRows32.  Rows kernels: their waves split K, so a wave takes nb / 8 blocks, in
// 1.4 us a block with 16 rows, 1.8 with 32, while at most one block a CU runs, in
// proportion to the blocks beyond (24 x 4096 x 7168: 32-row blocks 12.3 us, the
// best tile 19.3; 64 x 4096 x 7168: 24.4 against 19.9).  Tiles: rounds of the
// blocks that the chip holds, 3 K blocks' worth of start and end.
constexpr int kRows16 = -2, kRows32 = -1;
int choose(int M, int N, int K, bool out_f32) {
  const int nb = (K + kBK - 1) / kBK;
  const auto ceil_div = [](long long a, long long b) { return (a + b - 1) / b; };
  const auto rows_us = [&](int rows, float us) {
    const float blocks = (float)(ceil_div(N, 16) * ceil_div(M, rows));
    return (float)ceil_div(nb, 8) * us * std::max(1.f, blocks / 256.f);
  };
  int best = kRows16;
  float least = rows_us(16, 1.4f);
  if (M > 16) {
    if (const float t = rows_us(32, 1.8f); t < least) least = t, best = kRows32;
    for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
      const Shape& k = kTiles[i];
      const long long blocks = ceil_div(M, k.bm) * ceil_div(N, k.bn);
      const float step = blocks <= 256 ? k.one[out_f32] : k.full[out_f32];
      const float t = (float)(nb + 3) * step * (float)ceil_div(blocks, 256 * k.per_cu);
      if (t < least) least = t, best = i;
    }
  }
  return best;
}

}  // namespace

const char* fp8_gemm_kernel_name(int M, int N, int K, bool out_f32) {
  static const char* const kNames[] = {"rows 16",       "rows 32",        "tile 64 x 32",
                                       "tile 64 x 64",  "tile 64 x 128",  "tile 128 x 128",
                                       "tile 128 x 256", "tile 256 x 256"};
  static_assert(sizeof(kNames) / sizeof(kNames[0]) == sizeof(kTiles) / sizeof(kTiles[0]) + 2, "names");
  return kNames[choose(M, N, K, out_f32) - kRows16];
}

hipError_t launch_fp8_gemm(const Fp8Gemm& p, hipStream_t s) {
  switch (choose(p.M, p.N, p.K, p.out_f32)) {
    case kRows16: return launch_rows<1>(p, s);
    case kRows32: return launch_rows<2>(p, s);
    case 0: return launch_tile<2, 1, 2, 2, 3, 2>(p, s);
    case 1: return launch_tile<2, 2, 2, 2, 4>(p, s);
    case 2: return launch_tile<2, 2, 2, 4, 4, 1, false>(p, s);
    case 3: return launch_tile<4, 2, 2, 4, 4>(p, s);
    case 4: return launch_tile<4, 4, 2, 4, 3>(p, s);
    default: return launch_tile<8, 4, 2, 4, 2, 1, false>(p, s);
  }
}

}  // namespace moe
