// The whole expert layer for a few token rows (at most 16) in two launches, or
// three.
//
// A decode step of one or a few sequences reads each chosen expert's weights
// once for one or two rows: k experts of 3 I H weights a token, tens of MB, so
// launches and dependences count as much as bytes.  few_logits_kernel computes
// the router logits (and clears what the next launch counts in).  In
// few_experts_kernel every block forms the top-k itself (T rows of E logits,
// cheaper than another launch), then takes work from a ticket counter:
//   h'(t, j)[c] = w(t, j) SiLU(W_gate x_t)[c] (W_up x_t)[c]
//   out[t][n]   = sum over experts and c of W2_e[n][c] h'(t, j)[c]
// The routing weight is applied to h', so one accumulator runs over all
// experts and no per-expert output rows exist.
//
// STAGED, the rows and h' fit in a block's LDS (one or two rows of 7168): both
// products in one launch, the down units waiting for the sums they read.
// Otherwise the gate/up units alone, and few_down_kernel after them: with many
// rows the waits cost more than a launch (16 rows of the 256-expert layer: 248
// us in two launches, 199 in three).
//
// Bound by HBM.  One row, bf16: 48 experts of I = 640 top-3 (83 MB) 28.0 us,
// 256 of I = 256 top-8 and a shared one (103 MB) 30.6 us, of which the weights
// take 16 and 20 at the rate of a large copy; the logits and their launch
// take 5, the top-k in every block 4, the handover of h' 3.  (The latter in fp8,
// 51 MB: 28.1 us, the same steps.)  16 rows, row-major (1.14 GB): 200 to 212 us,
// 5.4 to 5.7 TB/s.
#include "moe_common.h"
#include "moe_kernels.h"

#include <math.h>

#include <algorithm>
#include <type_traits>

namespace moe {
namespace {

constexpr int kRows = kFewRows;   // one MFMA tile of token rows
constexpr int kWaves = 8;
constexpr int kThreads = kWaves * kWave;
constexpr int kMaxTopk = 16;
constexpr int kMaxSeg = 257;      // 256 routed experts + 1 shared
constexpr int kDownCols = 32;      // output columns of a down unit

// h' is kept as two bf16, the value rounded and the rest rounded: 16 mantissa
// bits, so that h' adds nothing visible to the rounding of the output, at two
// MFMAs where the launch waits for HBM anyway.  In memory (not STAGED): the
// values [T (k + n_shared) + 1][I], then the rests, the last row of both zero;
// a 32-bit word holds two columns.

// STAGED, the gate and up sums themselves are in memory, and a word that no
// block has written yet is kUnset, a NaN that finished() never gives.
constexpr uint32_t kUnset = 0xffffffffu;
__device__ __forceinline__ uint32_t finished(float v) {
  return __float_as_uint(v) == kUnset ? 0x7fc00000u : __float_as_uint(v);
}

__device__ __forceinline__ void split_h(float v, uint32_t& hi, uint32_t& lo) {
  hi = f32_to_bf16_bits(v);
  lo = 0;
  if ((hi & 0x7f80u) != 0x7f80u) lo = f32_to_bf16_bits(v - bf16_bits_to_f32((uint16_t)hi));
  else if (hi & 0x7fu) hi = 0x7fc0u;   // NaN
}

// part[z][t][e] (rows few_logit_stride(E) apart): router logits over the z-th
// part of K (the 8 waves of a block split that part again and meet in LDS), 16
// experts per block; the second launch adds the parts up.  (8 parts, 128 blocks
// for 256 experts: with 4, one row took 36.7 us in all in place of 34.8.)  Rows
// with valid == 0 are not read.  Also sets the ticket counter and marks the
// sums unset (STAGED) or zeroes the zero rows of h' (rows of I).
__global__ __launch_bounds__(kThreads) void few_logits_kernel(
    const uint16_t* __restrict__ x, const uint8_t* __restrict__ valid,
    const uint16_t* __restrict__ R, float* __restrict__ part, uint32_t* __restrict__ hw,
    int rows, int I, bool staged, int32_t* __restrict__ ticket, int first_ticket, int T, int H, int E) {
  __shared__ floatx4 red[kWaves][kWave];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int m = lane % 16, g = lane / 16;
  const uint32_t gid = (blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
  const uint32_t n = gridDim.x * gridDim.y * kThreads;
  if (staged) {
    for (uint32_t i = gid; i < 2u * kFewParts * rows * I; i += n) hw[i] = kUnset;
  } else {
    const uint32_t used = (uint32_t)rows * (I / 2), half = I / 2;
    for (uint32_t i = gid; i < 2 * half; i += n) hw[used + i + (i < half ? 0 : used)] = 0u;
  }
  if (gid == 0) *ticket = first_ticket;
  const int e = blockIdx.x * 16 + m;
  const bool ev = e < E;
  const bool rv = m < T && (valid == nullptr || valid[m] != 0);
  const int steps = H / 32, parts = gridDim.y * kWaves, p = blockIdx.y * kWaves + wave;
  const int s0 = (int)((long long)steps * p / parts), s1 = (int)((long long)steps * (p + 1) / parts);
  const uint16_t* xp = x + (size_t)(rv ? m : 0) * H + 8 * g;
  const uint16_t* rp = R + (size_t)(ev ? e : 0) * H + 8 * g;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  constexpr int U = 4;   // steps loaded at once (a wave has 3 or 4 at H = 7168)
  for (int s = s0; s < s1; s += U) {
    u32x4 xa[U], rb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u >= s1) break;
      xa[u] = rv ? ld16(xp + 32 * (s + u)) : zero;
      rb[u] = ev ? ld16(rp + 32 * (s + u)) : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u >= s1) break;
      acc = mfma16x16x32(as_bf16x8(xa[u]), as_bf16x8(rb[u]), acc);
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave != 0 || !ev) return;
  for (int w = 1; w < kWaves; ++w)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += red[w][lane][i];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 4 * g + i;
    if (t < T) part[((size_t)blockIdx.y * T + t) * few_logit_stride(E) + e] = acc[i];
  }
}

// Weights by way of LDS, 16 bytes a lane at a time: chunks of kParts KB that
// hold a 16-row tile's next kSteps MFMA steps (packed and fp8 rows 1 KB, bf16
// one step, fp8 two).  WIDE, for bf16 rows: 2 KB, 128 bytes = a whole line of
// every row, the two halves of a line would be asked for twice (16 rows' gate/up
// launch 137 us in place of 168).
template <bool FP8, bool PW, bool WIDE = false>
struct WChunk {
  static_assert(!WIDE || !(FP8 || PW), "for bf16 rows");
  static constexpr int kSteps = FP8 || WIDE ? 2 : 1, kParts = WIDE ? 2 : 1;
  static constexpr int kBytes = PW ? 1024 : 64 * kParts;   // from one chunk of a tile to the next
  // K of the lane's first value of step u
  static __device__ __forceinline__ int k_of(int u, int g) {
    return FP8 && !PW ? 16 * g + 8 * u : 32 * u + 8 * g;
  }
  // The row whose share the lane loads (WIDE: of 8 rows), and the byte offset
  // of that share behind the row (packed: behind the tile).  WIDE: piece p of
  // row r takes the place of piece p ^ r % 8, so that the lanes of a step read
  // all banks.
  static __device__ __forceinline__ int load_row(int lane) { return WIDE ? lane / 8 : lane % 16; }
  static __device__ __forceinline__ uint32_t load_offset(int lane) {
    return WIDE ? 16 * (lane % 8 ^ lane / 8) : PW ? 16 * lane : 16 * (lane / 16);
  }
  static __device__ __forceinline__ bf16x8 get(const uint8_t* chunk, int u, int lane) {
    if constexpr (FP8) {
      const u32x2 v = ld8(chunk + (PW ? 512 * u + 8 * lane : 16 * lane + 8 * u));
      return fp8x8_to_bf16x8(v[0], v[1]);
    } else if constexpr (WIDE) {
      return as_bf16x8(ld16(chunk + 128 * (lane % 16) + 16 * ((4 * u + lane / 16) ^ lane % 8)));
    } else {
      return as_bf16x8(ld16(chunk + 16 * lane));
    }
  }
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p, int bytes = -1) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}
// An offset behind the end of every buffer of less than 2 GB: loads give 0.
constexpr uint32_t kNowhere = 0x80000000u;

// 16 bytes a lane from buffer + lane_offset + offset straight to dst + 16 lane;
// NT: data that no other block reads.
template <bool NT>
__device__ __forceinline__ void to_lds16(__amdgpu_buffer_rsrc_t src, uint32_t lane_offset,
                                         uint32_t offset, void* dst) {
  if constexpr (NT)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)dst, 16,
                                             lane_offset, offset, 0, 2);
  else
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)dst, 16,
                                             lane_offset, offset, 0, 0);
}

// A float at buffer + offset, the same for all lanes, by way of the vector
// cache: a scalar load would have to be waited for with the next LDS read.
__device__ __forceinline__ float load_float(__amdgpu_buffer_rsrc_t src, uint32_t offset) {
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(src, offset, 0, 0));
}
__device__ __forceinline__ void to_lds4(__amdgpu_buffer_rsrc_t src, uint32_t lane_offset, void* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)dst, 4,
                                           lane_offset, 0, 0, 0);
}

// Waits until at most N of the wave's loads are outstanding and its LDS reads
// are done; no memory access moves across.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | (N >> 4) << 14);
  asm volatile("" ::: "memory");
}

// For chunk set i, with AHEAD chunks of N loads behind it, and MORE in every odd
// set (the scales, of two chunks each); i a constant.
template <int AHEAD, int N, int MORE>
__device__ __forceinline__ void wait_chunk(int i) {
  static_assert(MORE == 0 || AHEAD % 2 == 1, "sets in pairs");
  if (i % 2 == 0) wait_loads<AHEAD * N + (AHEAD + 1) / 2 * MORE>();
  else wait_loads<AHEAD * N + AHEAD / 2 * MORE>();
}

struct FewTables {
  int16_t slot[kMaxSeg][kRows];   // assignment t (k + ns) + j of row t at this segment, or -1
  int16_t act[kMaxSeg];           // segments that some row chose, ascending
  uint32_t chosen[(kMaxSeg + 31) / 32];   // the same as bits
  float w[kRows][kMaxTopk + 1];   // routing weights; the shared slot holds 1
  int16_t pick[kRows * (kMaxTopk + 1)];   // an assignment's segment
  int16_t place[kMaxSeg];         // of a segment in act
  uint8_t bad[kRows];             // rows whose logits are NaN
  int n_act;
};

// A block's LDS, in one variable (with several the compiler gives each an
// alias scope of its own in place of those of the functions' arguments, and
// then waits for every load to LDS ahead of any read): the tables, the token
// rows (gate/up) or h' (down) of calls whose rows fit (STAGED), and a ring of
// weights per wave, which also holds its sums at the end of a unit.  STAGED:
// one block a CU, and room for the waves' sums of two segments of its range
// beside the ring, which stays full; otherwise two blocks a CU, one of which
// streams while the other adds up.
constexpr int kPad = kFewPad;   // bytes between staged rows: up to four rows on different banks
template <bool STAGED>
struct FewShared {
  static constexpr int kStage = STAGED ? kFewStage : 16, kRing = STAGED ? 10 * 1024 : 8 * 1024;
  static constexpr int kSums = STAGED ? 2 * kWaves * 2 * kWave : 1;
  // fp8: scales of the units of a range (kFewStage bounds them: at most 512
  // units of at most 127 blocks, 256 ranges), and of a down unit's experts
  static constexpr int kUnits = 3, kBlocks = 128, kDown = kFewStage / 4 / 128;
  FewTables tb;
  int tk;   // the block's next ticket
  __attribute__((aligned(16))) uint8_t stage[kStage];
  __attribute__((aligned(16))) uint8_t ring[kWaves][kRing];
  floatx4 sums[kSums];
  float up_scales[STAGED ? kUnits : 1][2][STAGED ? kBlocks : 1];
  float down_scales[STAGED ? kDown : 1];
};
static_assert(sizeof(FewShared<true>::sums) >= kFewStage, "gate sums of staged assignments");
static_assert(sizeof(FewShared<true>) <= 160 * 1024, "one block on a CU");
static_assert(sizeof(FewShared<false>) <= 80 * 1024, "two blocks on a CU");

// A logit as an unsigned number of the same order; 0 for NaN (and for experts
// already taken), below any logit.
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);   // -0 is 0
  return v != v ? 0u : u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// Largest key of the wave (DPP moves fused into the maxima).
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max_dpp<0x111>(v);   // row_shr 1
  v = max_dpp<0x112>(v);   // row_shr 2
  v = max_dpp<0x114>(v);   // row_shr 4
  v = max_dpp<0x118>(v);   // row_shr 8: lane 15 of each row has the row's
  v = max_dpp<0x142>(v);   // row_bcast 15
  v = max_dpp<0x143>(v);   // row_bcast 31: lane 63 has the wave's
  return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
}

// Row t's top-k by one wave, into the tables: lane l has experts 4 l .. + 3 and
// keeps the best of them that is left; k rounds of the best of all, the lowest
// expert among equal ones; weights = softmax over the picks.  A loop that
// stays a loop: run once per launch, unrolled rounds would be fetched from
// memory instruction by instruction (1 us each).
__device__ __forceinline__ void few_topk(const float* __restrict__ part, int t, int T, int E, int ns,
                                         int k, FewTables& tb) {
  const int lane = threadIdx.x % kWave, kk = k + ns, e0 = 4 * lane;
  floatx4 s = {0.f, 0.f, 0.f, 0.f};
  if (e0 < E) {
    floatx4 p[kFewLogitParts];
#pragma unroll
    for (int z = 0; z < kFewLogitParts; ++z)
      p[z] = *reinterpret_cast<const floatx4*>(part + ((size_t)z * T + t) * few_logit_stride(E) + e0);
#pragma unroll
    for (int z = 0; z < kFewLogitParts; ++z)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[c] += p[z][c];
  }
  uint32_t v[4], mine = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    v[c] = e0 + c < E ? logit_key(s[c]) : 0u;
    mine = max(mine, v[c]);
  }
  uint32_t top = 0, my_v = 0;
  int my_e = -1;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    const uint32_t best = wave_max(mine);
    const int my_best = v[0] == best ? e0 : v[1] == best ? e0 + 1 : v[2] == best ? e0 + 2 : e0 + 3;
    const int winner = __builtin_ctzll(__ballot(mine == best));
    int e = __builtin_amdgcn_readlane(my_best, winner);
    if (best == 0) e = -1;   // none left: the others are NaN
    if (j == 0) top = best;
    if (lane == j) {
      my_v = best;
      my_e = e;
    }
    mine = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (e == e0 + c) v[c] = 0;
      mine = max(mine, v[c]);
    }
  }
  // (equal infinities are an exact tie, not NaN)
  const float w = lane < k ? (my_v == top ? 1.f : expf(key_logit(my_v) - key_logit(top))) : 0.f;
  float sum = w;
#pragma unroll
  for (int d = 1; d < kMaxTopk; d <<= 1) sum += __shfl_xor(sum, d, kMaxTopk);
  const float my_w = w / sum;
  // NaN logits may leave fewer than k experts: the row's output is NaN
  if (!__all(lane >= k || (my_e >= 0 && my_w == my_w))) {
    if (lane == 0) tb.bad[t] = 1;
    return;
  }
  if (lane < kk) {
    const int e = lane < k ? my_e : E;
    tb.slot[e][t] = (int16_t)(t * kk + lane);
    tb.pick[t * kk + lane] = (int16_t)e;
    tb.w[t][lane] = lane < k ? my_w : 1.f;
    atomicOr(&tb.chosen[e / 32], 1u << (e % 32));
  }
}

struct FewArgs {
  const uint16_t* x;
  const uint8_t* valid;
  const void* w13;
  const void* w2;
  const float* s13;
  const float* s2;
  const float* part;
  uint32_t* hw;        // h'
  uint32_t plane;      // words from its values to their rests
  int32_t* ticket;
  FewTables* tables;   // not STAGED: block 0's, for the down launch
  uint16_t* out;
  int T, H, I, E, ns, k;
};

// By one thread.  (An address in vector registers: for a uniform one the
// compiler adds up the wave's tickets first and waits for the sum, and with it
// for all loads before it, on the spot.)
__device__ __forceinline__ int take_ticket(int32_t* ticket) {
  auto* p = (__attribute__((address_space(1))) int32_t*)ticket;
  asm volatile("" : "+v"(p));
  return __hip_atomic_fetch_add(p, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The tables the units work from and, STAGED, the token rows in LDS (a row of
// 2 H bytes every 2 H + kPad, 16 zero bytes behind the last): a row's top-k by
// a wave, the copy by the waves without one.  Called by every thread of the
// block.
template <bool STAGED>
__device__ __forceinline__ void few_route(const FewArgs& a, FewTables& tb, uint8_t* xs, int& s_tk) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int nseg = a.E + a.ns;
  uint32_t* slots = reinterpret_cast<uint32_t*>(&tb.slot[0][0]);
  for (int i = threadIdx.x; i < nseg * (kRows / 2); i += kThreads) slots[i] = 0xffffffffu;
  if (threadIdx.x < kRows) tb.bad[threadIdx.x] = 0;
  if (threadIdx.x < (kMaxSeg + 31) / 32) tb.chosen[threadIdx.x] = 0;
  __syncthreads();
  const int copy = a.T < kWaves ? a.T : 0;   // the first wave that copies
  if (STAGED && wave >= copy) {
    const int pieces = a.H / 8, threads = kThreads - copy * kWave;
    for (int i = threadIdx.x - copy * kWave; i < a.T * pieces; i += threads) {
      const int t = i / pieces, c = i - t * pieces;
      if (a.valid == nullptr || a.valid[t] != 0)
        *reinterpret_cast<u32x4*>(xs + t * (2 * a.H + kPad) + 16 * c) =
            ld16(a.x + (size_t)t * a.H + 8 * c);
    }
    if (threadIdx.x == kThreads - 1)
      *reinterpret_cast<u32x4*>(xs + a.T * (2 * a.H + kPad)) = u32x4{0u, 0u, 0u, 0u};
  }
  // The block's first ticket, behind this wave's loads.  Not STAGED, where no
  // unit waits for another, it is the block's index and the counter starts
  // behind those (one counter serves a ticket every 10 ns, so the last of 512
  // blocks would wait 5 us).
  if (threadIdx.x == kThreads - 1) s_tk = STAGED ? take_ticket(a.ticket) : blockIdx.x;
  for (int t = wave; t < a.T; t += kWaves)
    if (a.valid == nullptr || a.valid[t] != 0) few_topk(a.part, t, a.T, a.E, a.ns, a.k, tb);
  __syncthreads();
  if (threadIdx.x < nseg) {
    const int e = threadIdx.x;
    int n = 0;
    for (int i = 0; i < e / 32; ++i) n += __popc(tb.chosen[i]);
    const uint32_t word = tb.chosen[e / 32];
    n += __popc(word & ((1u << (e % 32)) - 1));
    const bool any = word >> (e % 32) & 1;
    if (any) tb.act[n] = (int16_t)e;
    tb.place[e] = (int16_t)n;
    if (e == nseg - 1) tb.n_act = n + any;
  }
  __syncthreads();
}

// h columns of a gate/up unit.
constexpr int few_cols(bool fp8) { return fp8 ? 16 : 8; }

// A gate/up unit's loads and sums of one wave: weights by way of LDS, token
// rows in LDS (STAGED) or registers, kAhead chunks ahead.
template <bool FP8, bool PW, bool STAGED>
struct GateUp {
  using WC = WChunk<FP8, PW, !FP8 && !PW>;
  static constexpr int NT = FP8 ? 2 : 1;
  static constexpr int kLoads = NT * WC::kParts, kEntry = 1024 * kLoads;   // of a chunk's weights
  static constexpr int kSets = FewShared<STAGED>::kRing / kEntry, kAhead = kSets - 1;
  static constexpr int kXSets = STAGED ? 1 : kSets;
  __amdgpu_buffer_rsrc_t wbuf[NT], xbuf, sbuf;
  uint32_t wl[WC::kParts], xl[WC::kSteps];
  uint32_t so[NT];   // byte offsets of the unit's scales in sbuf
  floatx4 acc[NT], part[NT];
  u32x4 x[kXSets][WC::kSteps];
  float sc[kXSets][NT];

  // Chunk c's weights to `to` and, not STAGED, the rest to set `set`.
  __device__ __forceinline__ void issue(uint8_t* __restrict__ to, int c, int set) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < WC::kParts; ++p)
        to_lds16<PW>(wbuf[n], wl[p], c * WC::kBytes, to + 1024 * (n * WC::kParts + p));
    if constexpr (!STAGED) {
#pragma unroll
      for (int u = 0; u < WC::kSteps; ++u)
        x[set][u] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(xbuf, xl[u], c * (64 * WC::kSteps), 0));
      if (FP8 && set % 2 == 1)
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[set][n] = load_float(sbuf, so[n] + c / 2 * 4);
    }
  }
  // The sums of the chunk in `cur`, x and scales in set `set`; fp8: scaled up
  // to here if `second`, the second half of a 128-wide block (STAGED: always,
  // blocks may be split between waves).
  __device__ __forceinline__ void multiply(const uint8_t* __restrict__ cur, int lane, int set, bool second) {
#pragma unroll
    for (int u = 0; u < WC::kSteps; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        floatx4& d = FP8 ? part[n] : acc[n];
        d = mfma16x16x32(WC::get(cur + 1024 * n, u, lane), as_bf16x8(x[set][u]), d);
      }
    if (FP8 && second)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[n][i] = fmaf(sc[set][n], part[n][i], acc[n][i]);
          part[n][i] = 0.f;
        }
  }
  // STAGED: chunk c out of `cur`.
  __device__ __forceinline__ void step_staged(const uint8_t* __restrict__ cur,
                                              const uint8_t* __restrict__ xs,
                                              const float* __restrict__ scales, int c, bool xv,
                                              int lane) {
    if constexpr (FP8)
#pragma unroll
      for (int n = 0; n < NT; ++n) sc[0][n] = scales[n * FewShared<true>::kBlocks + c / 2];
#pragma unroll
    for (int u = 0; u < WC::kSteps; ++u)
      x[0][u] = ld16(xs + (xv ? 2 * (c * 32 * WC::kSteps + WC::k_of(u, lane / 16)) : 0));
    multiply(cur, lane, 0, true);
  }
  // Not STAGED: set i's chunk in its place in the wave's ring; LOAD: chunk c
  // takes the place of the one before it.
  template <bool LOAD>
  __device__ __forceinline__ void step(const uint8_t* __restrict__ cur, uint8_t* __restrict__ to, int i,
                                       int c, int lane) {
    if constexpr (LOAD) {
      wait_loads<63>();   // the reads of the chunk that is loaded over
      issue(to, c, (i + kAhead) % kSets);
      wait_chunk<kAhead, kLoads + WC::kSteps, FP8 ? NT : 0>(i);
    }
    multiply(cur, lane, i, i % 2 == 1);
  }
};

// Where a gate/up unit's weights are, for the wave's loads: h' columns c0 ..
// c0 + few_cols - 1 of expert e.  bf16: the MFMA A operand holds 8 gate rows
// and the 8 up rows of the same columns; fp8: 16 gate rows, and 16 up rows in
// a second one (half a packed fp8 tile is half a line of memory).  The B
// operand holds the token rows (rows that did not choose e: zeros).
template <bool FP8, bool PW, bool STAGED>
__device__ __forceinline__ void at_unit(GateUp<FP8, PW, STAGED>& gu, const FewArgs& a, int lane, int e,
                                        int c0) {
  using GU = GateUp<FP8, PW, STAGED>;
  using WC = typename GU::WC;
  const int H = a.H, I = a.I;
  constexpr int kSize = FP8 ? 1 : 2;
#pragma unroll
  for (int n = 0; n < GU::NT; ++n)
    gu.wbuf[n] = buffer_at(static_cast<const uint8_t*>(a.w13) +
                           ((size_t)e * 2 * I + n * I + c0 / 16 * 16) * H * kSize);
  // bf16: the tile's rows 8 .. 15 are the up rows, I rows on
  const uint32_t up_rows = (uint32_t)I * H * kSize;
  const int lr = WC::load_row(lane);
#pragma unroll
  for (int p = 0; p < WC::kParts; ++p) {
    if constexpr (FP8) gu.wl[p] = WC::load_offset(lane) + (PW ? 0 : lr * H * kSize);
    else if constexpr (PW)   // lane (g, r)'s share lies at 256 g + 16 r
      gu.wl[p] = 256 * (lane / 16) + 16 * (c0 % 16 + lane % 8) + (lane % 16 >= 8 ? up_rows : 0u);
    else gu.wl[p] = WC::load_offset(lane) + (c0 % 16 + lr) * H * kSize + p * up_rows;
  }
}
// Index of the scales of those columns' gate (n = 0) or up (1) rows.
__device__ __forceinline__ uint32_t scales_at(const FewArgs& a, int e, int c0, int n) {
  return (e * (2 * a.I / 128) + (n * a.I + c0) / 128) * (a.H / 128);
}

// A unit by a block, the waves splitting K = H in 128-wide blocks and meeting
// in LDS: h' to memory.
template <bool FP8, bool PW>
__device__ __forceinline__ void gate_up_unit(const FewArgs& a, const FewTables* __restrict__ tb,
                                             uint8_t* __restrict__ ring, int e, int c0, int& next) {
  using GU = GateUp<FP8, PW, false>;
  using WC = typename GU::WC;
  constexpr int NT = GU::NT, kCols = few_cols(FP8), kRing = FewShared<false>::kRing;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int m = lane % 16, g = lane / 16;
  const int H = a.H, I = a.I;
  GU gu;
  at_unit(gu, a, lane, e, c0);
  gu.sbuf = buffer_at(a.s13);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    gu.so[n] = 4 * scales_at(a, e, c0, n);
    gu.acc[n] = gu.part[n] = floatx4{0.f, 0.f, 0.f, 0.f};
  }
  const bool xv = tb->slot[e][m] >= 0;
  // rows that did not choose e: zeros
  gu.xbuf = buffer_at(a.x, 2 * a.T * H);
#pragma unroll
  for (int u = 0; u < WC::kSteps; ++u) gu.xl[u] = xv ? 2 * (m * H + WC::k_of(u, g)) : kNowhere;
  // (rounded so that wave 0, which takes the tickets, has a block)
  const int nb = H / 128, cpb = 4 / WC::kSteps;
  const int s0 = (nb * wave + kWaves - 1) / kWaves * cpb, s1 = (nb * (wave + 1) + kWaves - 1) / kWaves * cpb;
  uint8_t* mine = ring + wave * kRing;
  if (s0 < s1) {
    // (behind the last chunk that one again, unused, so that as many loads are
    // on the way at every step)
#pragma unroll
    for (int i = 0; i < GU::kAhead; ++i) {
      gu.issue(mine + i * GU::kEntry, min(s0 + i, s1 - 1), i);
      __builtin_amdgcn_sched_barrier(0);   // chunk after chunk, as the waits count
    }
    if (threadIdx.x == 0) next = take_ticket(a.ticket);
    int c = s0;
#pragma unroll 1
    for (; c + GU::kSets <= s1; c += GU::kSets)
#pragma unroll
      for (int i = 0; i < GU::kSets; ++i)
        gu.template step<true>(mine + i * GU::kEntry,
                               mine + (i + GU::kAhead) % GU::kSets * GU::kEntry, i,
                               min(c + i + GU::kAhead, s1 - 1), lane);
    wait_loads<0>();
#pragma unroll
    for (int i = 0; i < GU::kAhead; ++i)
      if (c + i < s1) gu.template step<false>(mine + i * GU::kEntry, nullptr, i, 0, lane);
  }
  floatx4* red = reinterpret_cast<floatx4*>(mine);
#pragma unroll
  for (int n = 0; n < NT; ++n) red[n * kWave + lane] = gu.acc[n];
  __syncthreads();
  // thread -> (columns c, c + 1, row t)
  if (threadIdx.x < kCols / 2 * kRows) {
    const int c = threadIdx.x % (kCols / 2) * 2, t = threadIdx.x / (kCols / 2);
    const int slot = tb->slot[e][t];
    if (slot >= 0) {
      const int up = FP8 ? c : 8 + c;
      float gs[2] = {0.f, 0.f}, us[2] = {0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const floatx4* r = reinterpret_cast<const floatx4*>(ring + w * kRing);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          gs[i] += r[c / 4 * 16 + t][c % 4 + i];
          us[i] += r[(NT - 1) * kWave + up / 4 * 16 + t][up % 4 + i];
        }
      }
      const float wt = tb->w[t][slot - t * (a.k + a.ns)];
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) split_h(silu_mul(gs[i], us[i]) * wt, hi[i], lo[i]);
      // (read by the next launch)
      uint32_t* to = a.hw + ((size_t)slot * I + c0 + c) / 2;
      __hip_atomic_store(to, hi[0] | hi[1] << 16, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(to + a.plane, lo[0] | lo[1] << 16, __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    }
  }
}

// A range of the gate/up units' 128-wide blocks of K, unit after unit, STAGED:
// the calls' few units would not go evenly into the chip's CUs (288 into 256
// for one row of the 256-expert layer: 36.3 us, with equal shares 31.4), so each
// block takes an equal share of all their blocks instead, at most kFewParts of them
// sharing a unit.  Every wave takes its part of each unit's blocks in the range
// (a segment) as one stream: the ring runs on from segment to segment, only the
// sums stop, for the block to add the waves' up and send them to memory.
struct FewSplit {
  int nb, total, per, ranges;   // blocks of a unit, of all, of a range; ranges
  __device__ __forceinline__ FewSplit(int H, int n_gu) {
    nb = H / 128;
    total = n_gu * nb;
    per = max((total + 255) / 256, (nb + kFewParts - 2) / (kFewParts - 1));
    ranges = (total + per - 1) / per;
  }
  // the parts that share unit u: ranges first(u) .. last(u)
  __device__ __forceinline__ int first(int u) const { return u * nb / per; }
  __device__ __forceinline__ int last(int u) const { return (u * nb + nb - 1) / per; }
};

// A wave's place in its chunks of a range.
struct RangePlace {
  int u, end;   // unit, end of the range
  int c, c1;    // chunks of the segment to go
  // The wave's chunks of the segment of unit u in blocks [from, end).
  __device__ __forceinline__ void segment(int from, int nb, int cpb, int wave) {
    const int k0 = max(from - u * nb, 0), k1 = min(end - u * nb, nb), n = (k1 - k0) * cpb;
    c = k0 * cpb + n * wave / kWaves;
    c1 = k0 * cpb + n * (wave + 1) / kWaves;
  }
};

template <bool FP8, bool PW>
__device__ __forceinline__ void gate_up_range(const FewArgs& a, const FewTables* __restrict__ tb,
                                              const uint8_t* __restrict__ xs,
                                              uint8_t* __restrict__ ring, floatx4* __restrict__ sums,
                                              float* __restrict__ scales, const FewSplit& sp, int r,
                                              int& next) {
  using GU = GateUp<FP8, PW, true>;
  using WC = typename GU::WC;
  constexpr int NT = GU::NT, kCols = few_cols(FP8), kRing = FewShared<true>::kRing;
  constexpr int kValues = 16 * NT;   // of a row: gate columns, then up columns
  constexpr int cpb = 4 / WC::kSteps;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int m = lane % 16, n_cg = a.I / kCols, nb = sp.nb;
  const int r0 = r * sp.per, r1 = min(r0 + sp.per, sp.total);
  uint8_t* mine = ring + wave * kRing;
  GU gu;
  RangePlace ld, at;
  ld.u = at.u = r0 / nb;
  ld.end = at.end = r1;
  auto column = [&](int u) { return (u % n_cg) * kCols; };
  auto expert = [&](int u) { return __builtin_amdgcn_readfirstlane(tb->act[u / n_cg]); };
  // the next chunk to load: of the first segment from ld.u on that has one
  auto settle = [&]() {
    while (ld.c == ld.c1 && (ld.u + 1) * nb < r1) {
      ++ld.u;
      ld.segment(r0, nb, cpb, wave);
      at_unit(gu, a, lane, expert(ld.u), column(ld.u));
    }
  };
  constexpr int kUnits = FewShared<true>::kUnits, kBlocks = FewShared<true>::kBlocks;
  if constexpr (FP8) {
    // the scales of the range's units, gate or up of one by a wave
    const int u = min(ld.u + wave / 2, (r1 - 1) / nb);
    const uint32_t first = scales_at(a, expert(u), column(u), wave % 2);
    if (wave < 2 * kUnits)
      for (int i = 0; i < nb; i += kWave)
        to_lds4(buffer_at(a.s13), 4 * (first + min(i + lane, nb - 1)), scales + wave * kBlocks + i);
  }
  ld.segment(r0, nb, cpb, wave);
  at_unit(gu, a, lane, expert(ld.u), column(ld.u));
  settle();
  int ahead = 0;   // chunks on their way
#pragma unroll 1
  for (int i = 0; i < GU::kAhead && ld.c < ld.c1; ++i) {
    gu.issue(mine + i * GU::kEntry, ld.c++, 0);
    ++ahead;
    settle();
  }
  if constexpr (FP8) {
    // (what is behind a wave's scales: its ring)
    if (ahead == GU::kAhead) wait_loads<GU::kAhead * GU::kLoads>();
    else wait_loads<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
  if (threadIdx.x == 0) next = take_ticket(a.ticket);
  int from = 0, side = 0;
  const int u0 = at.u;
#pragma unroll 1
  for (; at.u * nb < r1; ++at.u) {
    const int e = expert(at.u);
    at.segment(r0, nb, cpb, wave);
#pragma unroll
    for (int n = 0; n < NT; ++n) gu.acc[n] = gu.part[n] = floatx4{0.f, 0.f, 0.f, 0.f};
    const bool xv = tb->slot[e][m] >= 0;
    // a lane without a row reads the 16 zero bytes behind them
    const uint8_t* xl = xs + (xv ? m * (2 * a.H + kPad) : a.T * (2 * a.H + kPad));
#pragma unroll 1
    for (int c = at.c; c < at.c1; ++c) {
      if (ahead == GU::kAhead) wait_loads<(GU::kAhead - 1) * GU::kLoads>();
      else wait_loads<0>();
      --ahead;
      if (ld.c < ld.c1) {
        gu.issue(mine + (from == 0 ? GU::kSets - 1 : from - 1) * GU::kEntry, ld.c++, 0);
        ++ahead;
        settle();
      }
      gu.step_staged(mine + from * GU::kEntry, xl, scales + (at.u - u0) * 2 * kBlocks, c, xv, lane);
      from = from + 1 == GU::kSets ? 0 : from + 1;
    }
    floatx4* red = sums + side * (kWaves * 2 * kWave);
#pragma unroll
    for (int n = 0; n < NT; ++n) red[(wave * 2 + n) * kWave + lane] = gu.acc[n];
    // (no __syncthreads: the loads may stay on their way.  A wave overwrites
    // this side after the next segment's barrier, when all have read it.)
    wait_loads<63>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const int v = threadIdx.x % kValues, t = threadIdx.x / kValues;
    const int slot = t < a.T ? tb->slot[e][t] : -1;
    if (slot >= 0) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        // (one read each: for pairs of them the compiler waits for all loads)
        int i = (w * 2 + v / 16) * kWave + v % 16 / 4 * 16 + t;
        asm volatile("" : "+v"(i));
        s += red[i][v % 4];
      }
      // readers wait for the words themselves to change, so nothing has to be
      // ordered around the stores
      const size_t at_part = ((size_t)slot * n_cg + at.u % n_cg) * kFewParts + r - sp.first(at.u);
      __hip_atomic_store(a.hw + at_part * kValues + v, finished(s), __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    }
    side ^= 1;
  }
}

__device__ __forceinline__ unsigned long long peek(const uint32_t* p) {
  return __hip_atomic_load(reinterpret_cast<const unsigned long long*>(p), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool unset(unsigned long long v) {
  return max((uint32_t)v, (uint32_t)(v >> 32)) == kUnset;
}

// All of h' to LDS, from the sums of its parts: row s (an assignment) every 4 I
// + kPad bytes, 8 columns' values (16 bytes), then their rests; 16 zero bytes
// behind the last row.  Waits for the sums that are unset: the ranges that
// write them have smaller tickets, which blocks take in order and only while
// they run, so each such range has ended or is running in a block that waits
// for nothing, and the wait ends.
//
// First the sums, four floats an item, three items and two parts of each at a
// time, as they come from beyond this XCD's L2: gate sums to `gates`, up sums
// to where their columns' h' goes; then h', two columns a lane.  Loops that
// stay loops: all this runs once, and is fetched from memory.
template <bool FP8>
__device__ __forceinline__ void stage_h(const FewArgs& a, const FewTables* __restrict__ tb,
                                        const FewSplit& sp, uint8_t* __restrict__ hs,
                                        float* __restrict__ gates) {
  constexpr int kCols = few_cols(FP8), kValues = 2 * kCols, kPer = kValues / 4, kItems = 3;
  const int I = a.I, kk = a.k + a.ns, n_cg = I / kCols, total = a.T * kk * n_cg * kPer;
  const int row_bytes = 4 * I + kPad;
#pragma unroll 1
  for (int j0 = threadIdx.x; j0 < total; j0 += kItems * kThreads) {
    const uint32_t* p[kItems];
    int parts[kItems];
    floatx4 sum[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int j = j0 + i * kThreads, s = j / kPer, slot = s / n_cg, t = slot / kk;
      parts[i] = 0;
      p[i] = a.hw + (size_t)s * kFewParts * kValues + j % kPer * 4;
      sum[i] = floatx4{0.f, 0.f, 0.f, 0.f};
      if (j < total && !tb->bad[t] && (a.valid == nullptr || a.valid[t] != 0)) {
        const int u = tb->place[tb->pick[slot]] * n_cg + s - slot * n_cg;
        parts[i] = sp.last(u) - sp.first(u) + 1;
      }
    }
#pragma unroll 1
    for (int q = 0; q < kFewParts; q += 2) {
      if (!__any(max(max(parts[0], parts[1]), parts[2]) > q)) break;
      static_assert(kItems == 3, "of parts");
      unsigned long long v[kItems][2][2];
      bool wait;
#pragma unroll 1
      do {
        wait = false;
#pragma unroll
        for (int i = 0; i < kItems; ++i)
          if (q < parts[i])
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t* from = p[i] + min(q + h, parts[i] - 1) * kValues;
              v[i][h][0] = peek(from);
              v[i][h][1] = peek(from + 2);
            }
#pragma unroll
        for (int i = 0; i < kItems; ++i)
          if (q < parts[i])
#pragma unroll
            for (int h = 0; h < 2; ++h) wait |= unset(v[i][h][0]) || unset(v[i][h][1]);
      } while (__any(wait));
#pragma unroll
      for (int i = 0; i < kItems; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (q + h < parts[i])
#pragma unroll
            for (int k = 0; k < 4; ++k)
              sum[i][k] += __uint_as_float((uint32_t)(v[i][h][k / 2] >> (k % 2 * 32)));
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int j = j0 + i * kThreads, s = j / kPer, slot = s / n_cg, c = j % kPer * 4;
      float* to = c < kCols ? gates + s * kCols + c
                            : reinterpret_cast<float*>(hs + slot * row_bytes) +
                                  (s - slot * n_cg) * kCols + c - kCols;
      if (parts[i] > 0) *reinterpret_cast<floatx4*>(to) = sum[i];
    }
  }
  if (threadIdx.x == 0)
    *reinterpret_cast<u32x4*>(hs + a.T * kk * row_bytes) = u32x4{0u, 0u, 0u, 0u};
  __syncthreads();
  // (the four lanes of 8 columns, of one wave, read before they write)
#pragma unroll 1
  for (int j = threadIdx.x; j < a.T * kk * (I / 2); j += kThreads) {
    const int slot = j / (I / 2), c = 2 * (j - slot * (I / 2)), t = slot / kk;
    uint8_t* row = hs + slot * row_bytes;
    const float* g = gates + slot * I + c;
    const float* u = reinterpret_cast<const float*>(row) + c;
    const float w = tb->w[t][slot - t * kk];
    uint32_t h0, l0, h1, l1;
    split_h(silu_mul(g[0], u[0]) * w, h0, l0);
    split_h(silu_mul(g[1], u[1]) * w, h1, l1);
    uint32_t* to = reinterpret_cast<uint32_t*>(row) + c / 8 * 8 + c % 8 / 2;
    to[0] = h0 | h1 << 16;
    to[4] = l0 | l1 << 16;
  }
}

// A down unit's loads and sums of one wave, W2 by way of LDS.
template <bool FP8, bool PW>
struct DownStaged {
  using WC = WChunk<FP8, PW>;
  static constexpr int kEntry = 2048, kLoads = 2;
  static constexpr int kEntries = FewShared<true>::kRing / kEntry, kAhead = kEntries - 1;
  const uint8_t* w2;   // row c0 of expert 0
  size_t expert;       // bytes of an expert
  uint32_t tile;       // of 16 rows
  uint32_t wl;
  int cpe;             // chunks of an expert
  int ai, q;           // the next chunk to load: chosen expert, chunk of it
  int row_bytes, zeros;
  floatx4 acc[2], part[2];

  __device__ __forceinline__ void issue(uint8_t* __restrict__ to, const FewTables* __restrict__ tb) {
    const int e = __builtin_amdgcn_readfirstlane(tb->act[ai]);
    const __amdgpu_buffer_rsrc_t buf = buffer_at(w2 + e * expert);
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) to_lds16<PW>(buf, wl, nt * tile + q * WC::kBytes, to + 1024 * nt);
    if (++q == cpe) q = 0, ++ai;
  }

  // Chunk q of expert e out of `cur`; the next one to load (if more) into `next`.
  __device__ __forceinline__ void step(const uint8_t* __restrict__ cur, uint8_t* __restrict__ to,
                                       const uint8_t* __restrict__ hs, const FewTables* __restrict__ tb,
                                       int e, int cq, bool more, int lane, const float* __restrict__ scale) {
    if (more) issue(to, tb);
    const int slot = tb->slot[e][lane % 16], g = lane / 16;
    float sc = 0.f;
    if constexpr (FP8) sc = *scale;
#pragma unroll
    for (int u = 0; u < WC::kSteps; ++u) {
      const uint8_t* hr = hs + (slot >= 0 ? slot * row_bytes + 4 * (cq * 32 * WC::kSteps + WC::k_of(u, g)) : zeros);
      const u32x4 hi = ld16(hr), lo = ld16(hr + (slot >= 0 ? 16 : 0));
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const bf16x8 w = WC::get(cur + 1024 * nt, u, lane);
        floatx4& d = FP8 ? part[nt] : acc[nt];
        d = mfma16x16x32(w, as_bf16x8(hi), d);
        d = mfma16x16x32(w, as_bf16x8(lo), d);
      }
    }
    if (FP8 && cq % 2 == 1)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[nt][i] = fmaf(sc, part[nt][i], acc[nt][i]);
          part[nt][i] = 0.f;
        }
  }
};

// out[t][n] of a row whose sum came out as NaN, from that row's experts alone.
// The MFMAs multiply every chosen expert's weights with all rows, by zeros for
// the rows without it, and by h' in two parts: a weight or scale that is not
// finite makes NaN of the rows without its expert (0 x inf) and of sums that are
// infinite (inf x a rest of 0 or of the other sign).  Only NaN can come of
// either, so every other sum stands.  hi(slot, c), lo(slot, c): 8 columns of h'.
template <bool FP8, bool PW, class HI, class LO>
__device__ __forceinline__ float row_alone(const FewArgs& a, const FewTables* __restrict__ tb, int t, int n,
                                           HI hi, LO lo) {
  if (a.valid != nullptr && a.valid[t] == 0) return 0.f;
  const int kk = a.k + a.ns, H = a.H, I = a.I;
  constexpr int kBlock = FP8 ? 128 : 32;   // columns under one scale (bf16: none)
  float sum = 0.f;
#pragma unroll 1
  for (int j = 0; j < kk; ++j) {
    const int slot = t * kk + j, e = tb->pick[slot];
#pragma unroll 1
    for (int c0 = 0; c0 < I; c0 += kBlock) {
      float part = FP8 ? 0.f : sum;
#pragma unroll 1
      for (int c = c0; c < c0 + kBlock; c += 8) {
        const size_t at = (size_t)e * H * I + (PW ? frag_index(n, c, I) : (size_t)n * I + c);
        bf16x8 w;
        if constexpr (FP8) {
          const u32x2 v = ld8(static_cast<const uint8_t*>(a.w2) + at);
          w = fp8x8_to_bf16x8(v[0], v[1]);
        } else {
          w = as_bf16x8(ld16(static_cast<const uint16_t*>(a.w2) + at));
        }
        const bf16x8 h = as_bf16x8(hi(slot, c)), l = as_bf16x8(lo(slot, c));
#pragma unroll
        for (int i = 0; i < 8; ++i) part = fmaf((float)w[i], (float)h[i] + (float)l[i], part);
      }
      if constexpr (FP8)
        sum = fmaf(a.s2[((size_t)e * (H / 128) + n / 128) * (I / 128) + c0 / 128], part, sum);
      else sum = part;
    }
    if (sum != sum) break;   // it stays NaN
  }
  return sum;
}

// The sums of the waves (each at the start of its part of the ring) to
// out[t][c0 .. c0 + 31].
template <bool FP8, bool PW>
__device__ __forceinline__ void store_out(const FewArgs& a, const FewTables* __restrict__ tb,
                                          const uint8_t* __restrict__ hs, uint8_t* __restrict__ ring,
                                          int c0, const floatx4 (&acc)[2]) {
  constexpr int kRing = FewShared<true>::kRing;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  floatx4* red = reinterpret_cast<floatx4*>(ring + wave * kRing);
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) red[nt * kWave + lane] = acc[nt];
  __syncthreads();
  const int c = threadIdx.x % kDownCols, t = threadIdx.x / kDownCols;
  if (t < a.T) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      s += reinterpret_cast<const floatx4*>(ring + w * kRing)[c / 16 * kWave + (c % 16) / 4 * 16 + t][c % 4];
    if (s != s && !tb->bad[t]) {
      const int row_bytes = 4 * a.I + kPad;
      const auto hi = [&](int slot, int i) { return ld16(hs + slot * row_bytes + 4 * i); };
      const auto lo = [&](int slot, int i) { return ld16(hs + slot * row_bytes + 4 * i + 16); };
      s = row_alone<FP8, PW>(a, tb, t, c0 + c, hi, lo);
    }
    a.out[(size_t)t * a.H + c0 + c] = tb->bad[t] ? 0x7fc0u : f32_to_bf16_bits(s);
  }
}

// out[t][c0 .. c0 + 31] for every row: W2 rows (two 16-column tiles) as the
// MFMA A operand, h' as B, K = all chosen experts' columns one after the
// other, split over the waves.  The first W2 loads are on their way while the
// block waits for h' (staged: it has it from its unit before).
template <bool FP8, bool PW>
__device__ __forceinline__ void down_unit_staged(const FewArgs& a, const FewTables* __restrict__ tb,
                                                 const FewSplit& sp, uint8_t* __restrict__ hs,
                                                 uint8_t* __restrict__ ring, floatx4* __restrict__ sums,
                                                 float* __restrict__ scales, bool staged, int c0,
                                                 int& next) {
  using DS = DownStaged<FP8, PW>;
  using WC = typename DS::WC;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int H = a.H, I = a.I;
  constexpr int kSize = FP8 ? 1 : 2, GC = FP8 ? 2 : 1;   // chunks under one scale
  DS d;
  d.w2 = static_cast<const uint8_t*>(a.w2) + (size_t)c0 * I * kSize;
  d.expert = (size_t)H * I * kSize;
  d.tile = 16 * I * kSize;
  d.wl = WC::load_offset(lane) + (PW ? 0 : WC::load_row(lane) * I * kSize);
  d.cpe = I / (32 * WC::kSteps);
  d.row_bytes = 4 * I + kPad;
  d.zeros = a.T * (a.k + a.ns) * d.row_bytes;
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) d.acc[nt] = d.part[nt] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int n = __builtin_amdgcn_readfirstlane(tb->n_act) * (d.cpe / GC);
  const int s0 = n * wave / kWaves * GC, s1 = n * (wave + 1) / kWaves * GC;
  int ai = s0 / d.cpe, q = s0 - ai * d.cpe;
  d.ai = ai;
  d.q = q;
  uint8_t* mine = ring + wave * FewShared<true>::kRing;
  // fp8: the scales of the columns' blocks, expert after expert
  const int n_scales = FP8 ? __builtin_amdgcn_readfirstlane(tb->n_act) * (I / 128) : 0;
  float sc = 0.f;
  if (FP8 && threadIdx.x < n_scales) {
    const int i = threadIdx.x / (I / 128);
    sc = a.s2[((size_t)tb->act[i] * (H / 128) + c0 / 128) * (I / 128) + threadIdx.x - i * (I / 128)];
  }
#pragma unroll
  for (int i = 0; i < DS::kAhead; ++i)
    if (s0 + i < s1) d.issue(mine + i * DS::kEntry, tb);
  if (threadIdx.x == 0) next = take_ticket(a.ticket);
  if (FP8 && threadIdx.x < n_scales) scales[threadIdx.x] = sc;
  if (!staged) stage_h<FP8>(a, tb, sp, hs, reinterpret_cast<float*>(sums));
  __syncthreads();
  int at = 0;
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    if (s + DS::kAhead <= s1) wait_loads<(DS::kAhead - 1) * DS::kLoads>();
    else wait_loads<0>();
    const int to = at == 0 ? DS::kEntries - 1 : at - 1;
    const int e = __builtin_amdgcn_readfirstlane(tb->act[ai]);
    d.step(mine + at * DS::kEntry, mine + to * DS::kEntry, hs, tb, e, q, s + DS::kAhead < s1, lane,
           scales + ai * (I / 128) + q / 2);
    if (++q == d.cpe) q = 0, ++ai;
    at = at + 1 == DS::kEntries ? 0 : at + 1;
  }
  store_out<FP8, PW>(a, tb, hs, ring, c0, d.acc);
}

// Calls whose rows and h' do not fit in LDS have their down product in a
// launch of its own, where h' is read like any other memory: 16 rows of the
// 256-expert layer, 378 MB of W2, 58 us packed (6.5 TB/s), 64 row-major.
//
// A wave's loads and sums: NT tiles of 16 columns, W2 by way of LDS, h' in
// registers, both kAhead chunks ahead.
template <bool FP8, bool PW, int NT, bool WIDE>
struct Down {
  using WC = WChunk<FP8, PW, WIDE>;
  static constexpr int kEntry = 1024 * NT * WC::kParts;
  static constexpr int kWaves = WIDE ? 12 : 16;   // of a block
  static constexpr int kSets = WIDE ? 5 - NT : FP8 ? 4 : 8 / NT, kAhead = kSets - 1;
  static constexpr int kLoads = NT * WC::kParts + 2 * WC::kSteps;   // of a chunk
  const uint8_t* w2;      // row c0 of expert 0
  __amdgpu_buffer_rsrc_t s2;
  const uint16_t* h;
  size_t expert, plane;   // bytes of an expert, values of a plane of h'
  uint32_t tile;          // bytes of 16 rows
  uint32_t wl;
  int I, H, c0, zero_row, cpe;   // cpe: chunks of an expert
  // the next chunk to load, and how many follow it
  int ai, q, left;
  int e;
  const uint16_t* hrow;   // this lane's
  floatx4 acc[NT], part[NT];
  u32x4 hi[kSets][WC::kSteps], lo[kSets][WC::kSteps];
  float sc[kSets];

  __device__ __forceinline__ void enter(const FewTables* __restrict__ tb, int lane) {
    e = __builtin_amdgcn_readfirstlane(tb->act[ai]);
    const int slot = tb->slot[e][lane % 16];
    hrow = h + (size_t)(slot >= 0 ? slot : zero_row) * I;
  }

  // The weights first: once a chunk's h' has arrived, so have they.  (Behind
  // the last chunk that one again, unused, so that as many loads are on the
  // way at every step.)
  __device__ __forceinline__ void issue(uint8_t* __restrict__ to, const FewTables* __restrict__ tb,
                                        int lane, int set) {
    const __amdgpu_buffer_rsrc_t buf = buffer_at(w2 + e * expert);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int p = 0; p < WC::kParts; ++p)
        to_lds16<PW>(buf, wl, nt * tile + p * (tile / 2) + q * WC::kBytes,
                     to + 1024 * (nt * WC::kParts + p));
#pragma unroll
    for (int u = 0; u < WC::kSteps; ++u) {
      const uint16_t* p = hrow + q * 32 * WC::kSteps + WC::k_of(u, lane / 16);
      hi[set][u] = ld16(p);
      lo[set][u] = ld16(p + plane);
    }
    if (FP8 && set % 2 == 1)
      sc[set] = load_float(s2, 4 * ((e * (H / 128) + c0 / 128) * (I / 128) + q / 2));
    if (left > 0) {
      --left;
      if (++q == cpe) {
        q = 0;
        ++ai;
        enter(tb, lane);
      }
    }
  }

  // The chunk in `cur`; LOAD: the next one to load goes to `to`.
  template <bool LOAD>
  __device__ __forceinline__ void step(const uint8_t* __restrict__ cur, uint8_t* __restrict__ to,
                                       const FewTables* __restrict__ tb, int lane, int set, bool second) {
    if constexpr (LOAD) {
      wait_loads<63>();   // the reads of the chunk that is loaded over
      issue(to, tb, lane, (set + kAhead) % kSets);
      wait_chunk<kAhead, kLoads, FP8 ? 1 : 0>(set);
    }
#pragma unroll
    for (int u = 0; u < WC::kSteps; ++u)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const bf16x8 w = WC::get(cur + 1024 * WC::kParts * nt, u, lane);
        floatx4& d = FP8 ? part[nt] : acc[nt];
        d = mfma16x16x32(w, as_bf16x8(hi[set][u]), d);
        d = mfma16x16x32(w, as_bf16x8(lo[set][u]), d);
      }
    if (FP8 && second)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[nt][i] = fmaf(sc[set], part[nt][i], acc[nt][i]);
          part[nt][i] = 0.f;
        }
  }
  // Set i's chunk, in its place in the wave's part of the ring.  (A wave's
  // chunks are whole pairs under a scale.)
  template <bool LOAD>
  __device__ __forceinline__ void run(uint8_t* ring, const FewTables* tb, int lane, int i) {
    step<LOAD>(ring + i * kEntry, ring + (i + kAhead) % kSets * kEntry, tb, lane, i, i % 2 == 1);
  }
};

template <class DN>
struct DownShared {
  FewTables tb;
  __attribute__((aligned(16))) uint8_t ring[DN::kWaves][DN::kSets * DN::kEntry];
};
static_assert(sizeof(FewTables) % 4 == 0 && sizeof(FewTables) <= kFewTableBytes, "copied by words");

// out[t][c0 .. c0 + 16 NT - 1] for every row: as down_unit_staged, by 16 waves.
template <bool FP8, bool PW, int NT, bool WIDE>
__global__ __launch_bounds__((Down<FP8, PW, NT, WIDE>::kWaves * kWave)) void few_down_kernel(FewArgs a) {
  using DN = Down<FP8, PW, NT, WIDE>;
  using WC = typename DN::WC;
  constexpr int kDownWaves = DN::kWaves;
  __shared__ DownShared<DN> sh;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int H = a.H, I = a.I, c0 = blockIdx.x * 16 * NT;
  constexpr int kSize = FP8 ? 1 : 2, GC = FP8 ? 2 : 1;   // GC: chunks under one scale
  for (int i = threadIdx.x; i < (int)(sizeof(FewTables) / 4); i += kDownWaves * kWave)
    reinterpret_cast<uint32_t*>(&sh.tb)[i] = reinterpret_cast<const uint32_t*>(a.tables)[i];
  __syncthreads();
  DN d;
  d.w2 = static_cast<const uint8_t*>(a.w2) + (size_t)c0 * I * kSize;
  d.s2 = buffer_at(a.s2);
  d.h = reinterpret_cast<const uint16_t*>(a.hw);
  d.expert = (size_t)H * I * kSize;
  d.plane = 2 * (size_t)a.plane;
  d.tile = 16 * I * kSize;
  d.wl = WC::load_offset(lane) + (PW ? 0 : WC::load_row(lane) * I * kSize);
  d.I = I;
  d.H = H;
  d.c0 = c0;
  d.zero_row = a.T * (a.k + a.ns);
  d.cpe = I / (32 * WC::kSteps);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) d.acc[nt] = d.part[nt] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int n = __builtin_amdgcn_readfirstlane(sh.tb.n_act) * (d.cpe / GC);
  const int s0 = n * wave / kDownWaves * GC, s1 = n * (wave + 1) / kDownWaves * GC;
  uint8_t* mine = sh.ring[wave];
  if (s0 < s1) {
    d.ai = s0 / d.cpe;
    d.q = s0 - d.ai * d.cpe;
    d.left = s1 - s0 - 1;
    d.enter(&sh.tb, lane);
#pragma unroll
    for (int i = 0; i < DN::kAhead; ++i) {
      d.issue(mine + i * DN::kEntry, &sh.tb, lane, i);
      __builtin_amdgcn_sched_barrier(0);   // chunk after chunk, as the waits count
    }
    // whole rounds of the sets, then the rest, which is all loaded
    int s = s0;
#pragma unroll 1
    for (; s + DN::kSets <= s1; s += DN::kSets)
#pragma unroll
      for (int i = 0; i < DN::kSets; ++i) d.template run<true>(mine, &sh.tb, lane, i);
    wait_loads<0>();
#pragma unroll
    for (int i = 0; i < DN::kAhead; ++i)
      if (s + i < s1) d.template run<false>(mine, &sh.tb, lane, i);
  }
  floatx4* red = reinterpret_cast<floatx4*>(mine);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) red[nt * kWave + lane] = d.acc[nt];
  __syncthreads();
  const int c = threadIdx.x % (16 * NT), t = threadIdx.x / (16 * NT);
  if (t < a.T) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kDownWaves; ++w)
      sum += reinterpret_cast<const floatx4*>(sh.ring[w])[c / 16 * kWave + (c % 16) / 4 * 16 + t][c % 4];
    if (sum != sum && !sh.tb.bad[t]) {
      const auto hi = [&](int slot, int i) { return ld16(d.h + (size_t)slot * I + i); };
      const auto lo = [&](int slot, int i) { return ld16(d.h + d.plane + (size_t)slot * I + i); };
      sum = row_alone<FP8, PW>(a, &sh.tb, t, c0 + c, hi, lo);
    }
    a.out[(size_t)t * H + c0 + c] = sh.tb.bad[t] ? 0x7fc0u : f32_to_bf16_bits(sum);
  }
}

template <bool FP8, bool PW, bool STAGED>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(STAGED ? 2 : 4)))
void few_experts_kernel(FewArgs a) {
  static_assert(kThreads >= kRows * kDownCols, "one output per thread");
  __shared__ FewShared<STAGED> sh;
  few_route<STAGED>(a, sh.tb, sh.stage, sh.tk);
  if (!STAGED && blockIdx.x == 0)
    for (int i = threadIdx.x; i < (int)(sizeof(FewTables) / 4); i += kThreads)
      reinterpret_cast<uint32_t*>(a.tables)[i] = reinterpret_cast<const uint32_t*>(&sh.tb)[i];
  constexpr int kCols = few_cols(FP8);
  const int n_cg = a.I / kCols, n_gu = __builtin_amdgcn_readfirstlane(sh.tb.n_act) * n_cg;
  const FewSplit sp(a.H, STAGED ? n_gu : 0);
  const int n_up = STAGED ? sp.ranges : n_gu, n_all = n_up + (STAGED ? a.H / kDownCols : 0);
  int tk = __builtin_amdgcn_readfirstlane(sh.tk);
  bool h_staged = false;   // the stage holds h' in place of the token rows (tickets grow)
  while (tk < n_all) {
    __syncthreads();   // tk, the ring and the stage are free
    int next = 0;   // the next ticket (thread 0), asked for behind the unit's first loads
    if constexpr (STAGED) {
      if (tk < n_up) {
        gate_up_range<FP8, PW>(a, &sh.tb, sh.stage, &sh.ring[0][0], sh.sums,
                               &sh.up_scales[0][0][0], sp, tk, next);
      } else {
        down_unit_staged<FP8, PW>(a, &sh.tb, sp, sh.stage, &sh.ring[0][0], sh.sums,
                                  sh.down_scales, h_staged,
                                  (tk - n_up) * kDownCols, next);
        h_staged = true;
      }
    } else {
      const int ai = tk / n_cg;
      gate_up_unit<FP8, PW>(a, &sh.tb, &sh.ring[0][0], __builtin_amdgcn_readfirstlane(sh.tb.act[ai]),
                            (tk - ai * n_cg) * kCols, next);
    }
    if (threadIdx.x == 0) sh.tk = next;
    __syncthreads();
    tk = __builtin_amdgcn_readfirstlane(sh.tk);
  }
}

}  // namespace

hipError_t launch_few(int wkind, bool packed, const void* x, const uint8_t* valid, const void* R,
                      const void* w13, const void* w2, const float* s13, const float* s2,
                      float* part, uint32_t* hw, int32_t* ticket, void* tables, void* out, int T,
                      int H, int I, int E, int n_shared, int k, hipStream_t s) {
  if (wkind == W_F32 || T < 1 || T > kFewRows || E + n_shared > kMaxSeg || k > kMaxTopk ||
      H % 128 != 0 || I % 32 != 0 || (long long)H * I >= kMaxFewArea || (wkind == W_FP8 && I % 128 != 0))
    return hipErrorInvalidValue;
  const int rows = T * (k + n_shared);
  const bool staged = few_staged(T, H, I, k + n_shared);
  // Blocks loop over the tickets.  STAGED: one a CU, or fewer if there are
  // fewer ranges and down units; otherwise a block for every gate/up unit, so
  // that they all run at once, from one to two a CU.
  const long long n_gu = (long long)(std::min(E, T * k) + n_shared) * (I / few_cols(wkind == W_FP8));
  const dim3 grid((unsigned)(staged ? std::min((kFewParts - 1) * n_gu + H / kDownCols, 256LL)
                                    : std::min(n_gu, 512LL)));
  hipLaunchKernelGGL(few_logits_kernel, dim3((E + 15) / 16, kFewLogitParts), dim3(kThreads), 0, s,
                     static_cast<const uint16_t*>(x), valid, static_cast<const uint16_t*>(R), part,
                     hw, rows, I, staged, ticket, staged ? 0 : (int)grid.x, T, H, E);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const FewArgs a{static_cast<const uint16_t*>(x), valid, w13, w2, s13, s2, part, hw,
                  (uint32_t)(rows + 1) * (I / 2), ticket, static_cast<FewTables*>(tables),
                  static_cast<uint16_t*>(out), T, H, I, E, n_shared, k};
  // The down launch: 32 columns a block, or 16 if that gives fewer rounds of
  // 256 blocks (one a CU) for its columns.
  const bool narrow = (H / 16 + 255) / 256 < (H / 32 + 255) / 256 * 2;
#define MOE_DOWN(F, P, N, W)                                                                  \
  hipLaunchKernelGGL((few_down_kernel<F, P, N, W>), dim3(H / (16 * N)),                       \
                     dim3(Down<F, P, N, W>::kWaves * kWave), 0, s, a)
#define MOE_FEW(F, P)                                                                         \
  if (staged) {                                                                               \
    hipLaunchKernelGGL((few_experts_kernel<F, P, true>), grid, dim3(kThreads), 0, s, a);      \
  } else {                                                                                    \
    hipLaunchKernelGGL((few_experts_kernel<F, P, false>), grid, dim3(kThreads), 0, s, a);     \
    if ((err = hipGetLastError()) != hipSuccess) return err;                                  \
    if (narrow) {                                                                             \
      if (F || P || I % 64 != 0) MOE_DOWN(F, P, 1, false);                                    \
      else MOE_DOWN(F, P, 1, (!F && !P));                                                     \
    } else {                                                                                  \
      if (F || P || I % 64 != 0) MOE_DOWN(F, P, 2, false);                                    \
      else MOE_DOWN(F, P, 2, (!F && !P));                                                     \
    }                                                                                         \
  }
  if (wkind == W_FP8) {
    if (packed) { MOE_FEW(true, true); } else { MOE_FEW(true, false); }
  } else {
    if (packed) { MOE_FEW(false, true); } else { MOE_FEW(false, false); }
  }
#undef MOE_DOWN
#undef MOE_FEW
  return hipGetLastError();
}

}  // namespace moe
