// The whole expert layer for a few token rows (at most 16) in two launches.
//
// A decode step of one or a few sequences reads each chosen expert's weights
// once for one or two rows: k experts of 3 I H weights a token, a few tens of
// MB, a few microseconds of HBM time, so launches and dependences count as
// much as bytes.  few_logits_kernel computes the router logits (and clears
// what the second launch counts in); few_experts_kernel does the rest: every
// block forms the top-k itself (T rows of E logits, cheaper than another
// launch), then takes units from a ticket counter, first the gate/up units
//   h'(t, j)[c] = w(t, j) SiLU(W_gate x_t)[c] (W_up x_t)[c]   (8 columns c)
// and then the down units
//   out[t][n] = sum over experts and c of W2_e[n][c] h'(t, j)[c]  (32 columns n).
// The routing weight is applied to h', so one accumulator runs over all
// experts and no per-expert output rows exist.
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
constexpr int kDnCols = 32;       // output columns of a down unit

// A word of h' that no gate/up unit has written yet: as a pair of bf16 it is
// a NaN pattern that pack_h never makes.
constexpr uint32_t kUnset = 0xffffffffu;

// h' as two bf16, the value rounded (low half) and the rest rounded (high
// half): 16 mantissa bits, so that h' adds nothing visible to the rounding of
// the output, at two MFMAs where the launch waits for HBM anyway.
__device__ __forceinline__ uint32_t pack_h(float v) {
  const uint32_t hi = f32_to_bf16_bits(v);
  if ((hi & 0x7f80u) == 0x7f80u) return (hi & 0x7fu) ? 0x7fc0u : hi;   // NaN, infinity
  return hi | (uint32_t)f32_to_bf16_bits(v - bf16_bits_to_f32((uint16_t)hi)) << 16;
}

// part[z][t][e]: router logits over the z-th part of K (the 8 waves of a
// block split that part again and meet in LDS), 16 experts per block; the
// second launch adds the parts up.  Rows with valid == 0 are not read.  Also
// marks every word of h' unset and zeroes the ticket counter.
__global__ __launch_bounds__(kThreads) void few_logits_kernel(
    const uint16_t* __restrict__ x, const uint8_t* __restrict__ valid,
    const uint16_t* __restrict__ R, float* __restrict__ part, uint32_t* __restrict__ hw,
    size_t n_hw, int32_t* __restrict__ ticket, int T, int H, int E) {
  __shared__ floatx4 red[kWaves][kWave];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int m = lane % 16, g = lane / 16;
  const size_t gid = ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
  for (size_t i = gid; i < n_hw; i += (size_t)gridDim.x * gridDim.y * kThreads) hw[i] = kUnset;
  if (gid == 0) *ticket = 0;
  const int e = blockIdx.x * 16 + m;
  const bool ev = e < E;
  const bool rv = m < T && (valid == nullptr || valid[m] != 0);
  const int steps = H / 32, parts = gridDim.y * kWaves, p = blockIdx.y * kWaves + wave;
  const int s0 = (int)((long long)steps * p / parts), s1 = (int)((long long)steps * (p + 1) / parts);
  const uint16_t* xp = x + (size_t)(rv ? m : 0) * H + 8 * g;
  const uint16_t* rp = R + (size_t)(ev ? e : 0) * H + 8 * g;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  constexpr int U = 8;   // steps loaded at once (a wave has 7 at H = 7168)
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
    if (t < T) part[((size_t)blockIdx.y * T + t) * E + e] = acc[i];
  }
}

// The weights of one lane in a 128-wide K block of its row: four MFMA steps of
// 8.  Row-major fp8 takes two steps with one load, 16 consecutive bytes, so
// the steps' K order is that of k_of.
template <bool FP8, bool PW>
struct WBlock {
  static constexpr bool kPair = FP8 && !PW;
  static constexpr int kLoads = kPair ? 2 : 4;
  typename std::conditional<FP8 && PW, u32x2, u32x4>::type v[kLoads];
  // K of the lane's first weight of step u
  static __device__ __forceinline__ int k_of(int u, int g) {
    return kPair ? 64 * (u / 2) + 16 * g + 8 * (u & 1) : 32 * u + 8 * g;
  }
  // Offset (elements) of lane group g's weights of row r behind those of row 0
  // of a 16-row tile, at K 0.
  static __device__ __forceinline__ uint32_t lane_offset(int r, int K, int g) {
    return PW ? (16 * g + r) * 8 : r * K + (kPair ? 16 : 8) * g;
  }
  // Loads one load's worth: `tile` points at a tile's first row, K 0; step i of
  // K block `block`.  The uniform part of the address stays in scalar registers.
  __device__ __forceinline__ void load1(const void* tile, uint32_t lane, int block, int i) {
    const uint32_t at = (uint32_t)block * (PW ? 2048 : 128) + i * (PW ? 512 : kPair ? 64 : 32);
    // packed: whole lines that no other block reads; row-major: a line's other
    // half is asked for next
    if constexpr (FP8) {
      const uint8_t* p = static_cast<const uint8_t*>(tile) + at;
      if constexpr (PW) v[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p + lane));
      else v[i] = ld16(p + lane);
    } else {
      const uint8_t* p = static_cast<const uint8_t*>(tile) + 2 * (size_t)at;
      if constexpr (PW) v[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + 2 * lane));
      else v[i] = ld16(p + 2 * lane);
    }
  }
  __device__ __forceinline__ void load(const void* tile, uint32_t lane, int block) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load1(tile, lane, block, i);
  }
  static __device__ __forceinline__ const void* tile_at(const void* base, size_t row, int K) {
    return static_cast<const uint8_t*>(base) + row * K * (FP8 ? 1 : 2);
  }
  __device__ __forceinline__ bf16x8 get(int u) const {
    if constexpr (kPair) return fp8x8_to_bf16x8(v[u / 2][2 * (u & 1)], v[u / 2][2 * (u & 1) + 1]);
    else if constexpr (FP8) return fp8x8_to_bf16x8(v[u][0], v[u][1]);
    else return as_bf16x8(v[u]);
  }
};

// Weights by way of LDS: chunks of 1 KB, 16 bytes a lane, that hold a 16-row
// tile's next kSteps MFMA steps (bf16 one, fp8 two).
template <bool FP8, bool PW>
struct WChunk {
  static constexpr int kSteps = FP8 ? 2 : 1;
  static constexpr int kBytes = PW ? 1024 : 64;   // from one chunk of a tile to the next
  // K of the lane's first value of step u
  static __device__ __forceinline__ int k_of(int u, int g) {
    return FP8 && !PW ? 16 * g + 8 * u : 32 * u + 8 * g;
  }
  // byte offset of lane (g, r)'s share behind the tile
  static __device__ __forceinline__ uint32_t lane_offset(int r, int K, int g) {
    return PW ? (FP8 ? 256 * g + 16 * r : (16 * g + r) * 16) : r * (K * (FP8 ? 1 : 2)) + 16 * g;
  }
  static __device__ __forceinline__ bf16x8 get(const uint8_t* chunk, int u, int lane) {
    if constexpr (FP8) {
      const u32x2 v = ld8(chunk + (PW ? 512 * u + 8 * lane : 16 * lane + 8 * u));
      return fp8x8_to_bf16x8(v[0], v[1]);
    } else {
      return as_bf16x8(ld16(chunk + 16 * lane));
    }
  }
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, -1, 0x00020000);
}

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

// Waits until at most N of the wave's loads are outstanding and its LDS reads
// are done; no memory access moves across.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | (N >> 4) << 14);
  asm volatile("" ::: "memory");
}

struct FewTables {
  int16_t slot[kMaxSeg][kRows];   // assignment t (k + ns) + j of row t at this segment, or -1
  int16_t act[kMaxSeg];           // segments that some row chose, ascending
  uint32_t chosen[(kMaxSeg + 31) / 32];   // the same as bits
  float w[kRows][kMaxTopk + 1];   // routing weights; the shared slot holds 1
  uint8_t bad[kRows];             // rows whose logits are NaN
  int n_act;
};

// A block's LDS, in one variable (with several the compiler gives each an
// alias scope of its own in place of those of the functions' arguments, and
// then waits for every load to LDS ahead of any read): the tables, the token
// rows (gate/up) or h' (down) of calls whose rows fit (STAGED), and a ring of
// weights per wave, which also holds its sums at the end of a unit.  Half a
// CU's LDS: two blocks on a CU.
constexpr int kPad = 64;   // bytes between staged rows: up to four rows on different banks
template <bool STAGED>
struct FewShared {
  static constexpr int kStage = STAGED ? 22 * 1024 : 16, kRing = STAGED ? 6 * 1024 : 8 * 1024;
  FewTables tb;
  int tk;   // the block's next ticket
  __attribute__((aligned(16))) uint8_t stage[kStage];
  __attribute__((aligned(16))) uint8_t ring[kWaves][kRing];
};
static_assert(sizeof(FewShared<true>) <= 80 * 1024 && sizeof(FewShared<false>) <= 80 * 1024,
              "two blocks on a CU");

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

// Row t's top-k by one wave (expert e in lane e % 64, register e / 64), into
// the tables: k rounds of the largest logit left, the lowest expert among
// equal ones, weights = softmax over the picks.  A loop that stays a loop: run
// once per launch, unrolled rounds are fetched from memory instruction by
// instruction (1 us each, against 0.2).
__device__ __forceinline__ void few_topk(const float* __restrict__ part, int ks, int t, int T, int E,
                                         int ns, int k, FewTables& tb) {
  const int lane = threadIdx.x % kWave, kk = k + ns;
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + kWave * i;
    v[i] = 0;
    if (e < E) {
      float p[kFewLogitParts];
#pragma unroll
      for (int z = 0; z < kFewLogitParts; ++z) p[z] = part[((size_t)z * T + t) * E + e];
      float s = 0.f;
#pragma unroll
      for (int z = 0; z < kFewLogitParts; ++z) s += p[z];
      v[i] = logit_key(s);
    }
  }
  uint32_t top = 0, my_v = 0;
  int my_e = -1;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    const uint32_t best = wave_max(max(max(v[0], v[1]), max(v[2], v[3])));
    unsigned long long at = __ballot(v[3] == best);
    int e = 3 * kWave;
#pragma unroll
    for (int i = 2; i >= 0; --i) {
      const unsigned long long b = __ballot(v[i] == best);
      if (b) at = b, e = kWave * i;
    }
    e = best != 0 ? e + __builtin_ctzll(at) : -1;
    if (j == 0) top = best;
    if (lane == j) {
      my_v = best;
      my_e = e;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e == lane + kWave * i) v[i] = 0;
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
  uint32_t* hw;        // h' [T (k + ns)][I], words of pack_h
  int32_t* ticket;
  uint16_t* out;
  int T, H, I, E, ns, k, ks;
};

__device__ __forceinline__ int take_ticket(int32_t* ticket) {
  return __hip_atomic_fetch_add(ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The tables the units work from and, STAGED, the token rows in LDS (a row of
// 2 H bytes every 2 H + kPad, 16 zero bytes behind the last): rows' top-k by
// the first waves, the copy by the others.  Called by every thread of the
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
  if (STAGED && wave >= a.T) {
    const int pieces = a.H / 8, threads = kThreads - a.T * kWave;
    for (int i = threadIdx.x - a.T * kWave; i < a.T * pieces; i += threads) {
      const int t = i / pieces, c = i - t * pieces;
      if (a.valid == nullptr || a.valid[t] != 0)
        *reinterpret_cast<u32x4*>(xs + t * (2 * a.H + kPad) + 16 * c) =
            ld16(a.x + (size_t)t * a.H + 8 * c);
    }
    if (threadIdx.x == kThreads - 1)
      *reinterpret_cast<u32x4*>(xs + a.T * (2 * a.H + kPad)) = u32x4{0u, 0u, 0u, 0u};
  }
  // the block's first ticket, behind this wave's loads (one counter serves a
  // ticket every 10 ns, so the last of 512 blocks waits 5 us)
  if (threadIdx.x == kThreads - 1) s_tk = take_ticket(a.ticket);
  for (int t = wave; t < a.T; t += kWaves)
    if (a.valid == nullptr || a.valid[t] != 0) few_topk(a.part, a.ks, t, a.T, a.E, a.ns, a.k, tb);
  __syncthreads();
  if (threadIdx.x < nseg) {
    const int e = threadIdx.x;
    int n = 0;
    for (int i = 0; i < e / 32; ++i) n += __popc(tb.chosen[i]);
    const uint32_t word = tb.chosen[e / 32];
    n += __popc(word & ((1u << (e % 32)) - 1));
    const bool any = word >> (e % 32) & 1;
    if (any) tb.act[n] = (int16_t)e;
    if (e == nseg - 1) tb.n_act = n + any;
  }
  __syncthreads();
}

// h columns of a gate/up unit.
constexpr int few_cols(bool fp8) { return fp8 ? 16 : 8; }

// A gate/up unit's loads and sums of one wave.
template <bool FP8, bool PW, bool STAGED>
struct GateUp {
  using WC = WChunk<FP8, PW>;
  static constexpr int NT = FP8 ? 2 : 1, XN = STAGED ? 0 : WC::kSteps;
  static constexpr int kLoads = NT + XN, kEntry = 1024 * kLoads;
  static constexpr int kEntries = FewShared<STAGED>::kRing / kEntry, kAhead = kEntries - 1;
  __amdgpu_buffer_rsrc_t wbuf[NT], xbuf;
  uint32_t wl, xl[2];
  floatx4 acc[NT], part[NT];

  __device__ __forceinline__ void issue(uint8_t* __restrict__ to, int c) const {
#pragma unroll
    for (int n = 0; n < NT; ++n) to_lds16<PW>(wbuf[n], wl, c * WC::kBytes, to + 1024 * n);
#pragma unroll
    for (int u = 0; u < XN; ++u)
      to_lds16<false>(xbuf, xl[u], c * (64 * WC::kSteps), to + 1024 * (NT + u));
  }

  // Chunk c out of `cur`, chunk c + kAhead (if there is one) into `next`.
  __device__ __forceinline__ void step(const uint8_t* __restrict__ cur, uint8_t* __restrict__ next,
                                       const uint8_t* __restrict__ xs, int c, int c1, bool xv, int lane,
                                       const float* __restrict__ const (&sp)[NT]) {
    if (c + kAhead < c1) issue(next, c + kAhead);
    const int g = lane / 16;
    float sc[NT];
    if constexpr (FP8)
#pragma unroll
      for (int n = 0; n < NT; ++n) sc[n] = sp[n][c / 2];
#pragma unroll
    for (int u = 0; u < WC::kSteps; ++u) {
      u32x4 x;
      if constexpr (STAGED) x = ld16(xs + (xv ? 2 * (c * 32 * WC::kSteps + WC::k_of(u, g)) : 0));
      else {
        x = ld16(cur + 1024 * (NT + u) + 16 * lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = xv ? x[i] : 0u;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        floatx4& d = FP8 ? part[n] : acc[n];
        d = mfma16x16x32(WC::get(cur + 1024 * n, u, lane), as_bf16x8(x), d);
      }
    }
    // fp8: the second half of a 128-wide block
    if (FP8 && c % 2 == 1)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[n][i] = fmaf(sc[n], part[n][i], acc[n][i]);
          part[n][i] = 0.f;
        }
  }
};

// h' columns c0 .. c0 + few_cols - 1 of expert e for every row that chose it.
// bf16: the MFMA A operand holds 8 gate rows and the 8 up rows of the same
// columns; fp8: 16 gate rows, and 16 up rows in a second one (half a packed
// fp8 tile is half a line of memory).  The B operand holds the token rows
// (rows that did not choose e: zeros).  The waves split K = H in 128-wide
// blocks and meet in LDS.
template <bool FP8, bool PW, bool STAGED>
__device__ __forceinline__ void gate_up_unit(const FewArgs& a, const FewTables* __restrict__ tb,
                                             const uint8_t* __restrict__ xs,
                                             uint8_t* __restrict__ ring, int e, int c0, int& next) {
  using GU = GateUp<FP8, PW, STAGED>;
  using WC = typename GU::WC;
  constexpr int NT = GU::NT, kCols = few_cols(FP8), kRing = FewShared<STAGED>::kRing;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int m = lane % 16, g = lane / 16;
  const int H = a.H, I = a.I;
  constexpr int kSize = FP8 ? 1 : 2;
  GU gu;
  const float* sp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    gu.wbuf[n] = buffer_at(static_cast<const uint8_t*>(a.w13) +
                           ((size_t)e * 2 * I + n * I + c0 / 16 * 16) * H * kSize);
    sp[n] = FP8 ? a.s13 + ((size_t)e * (2 * I / 128) + (n * I + c0) / 128) * (H / 128) : nullptr;
    gu.acc[n] = gu.part[n] = floatx4{0.f, 0.f, 0.f, 0.f};
  }
  // bf16: lanes 8 .. 15 of a group have the up rows, I rows on
  if constexpr (FP8) gu.wl = PW ? 16 * lane : WC::lane_offset(m, H, g);
  else gu.wl = WC::lane_offset(c0 % 16 + m % 8, H, g) + (m >= 8 ? (uint32_t)I * H * kSize : 0u);
  const bool xv = tb->slot[e][m] >= 0;
  // (rows past T: row 0 again, not used)
  gu.xbuf = buffer_at(a.x);
#pragma unroll
  for (int u = 0; u < 2; ++u) gu.xl[u] = 2 * ((xv ? m : 0) * H + WC::k_of(u, g));
  // staged rows: a lane without one reads the 16 zero bytes behind them
  const uint8_t* xl = xs + (xv ? m * (2 * H + kPad) : a.T * (2 * H + kPad));
  // (rounded so that wave 0, which takes the tickets, has a block)
  const int nb = H / 128, cpb = 4 / WC::kSteps;
  const int s0 = (nb * wave + kWaves - 1) / kWaves * cpb, s1 = (nb * (wave + 1) + kWaves - 1) / kWaves * cpb;
  uint8_t* mine = ring + wave * kRing;
#pragma unroll
  for (int i = 0; i < GU::kAhead; ++i)
    if (s0 + i < s1) gu.issue(mine + i * GU::kEntry, s0 + i);
  if (threadIdx.x == 0) next = take_ticket(a.ticket);
  int at = 0;
#pragma unroll 1
  for (int c = s0; c < s1; ++c) {
    if (c + GU::kAhead <= s1) wait_loads<(GU::kAhead - 1) * GU::kLoads>();
    else wait_loads<0>();
    const int to = at == 0 ? GU::kEntries - 1 : at - 1;
    gu.step(mine + at * GU::kEntry, mine + to * GU::kEntry, xl, c, s1, xv, lane, sp);
    at = at + 1 == GU::kEntries ? 0 : at + 1;
  }
  floatx4* red = reinterpret_cast<floatx4*>(mine);
#pragma unroll
  for (int n = 0; n < NT; ++n) red[n * kWave + lane] = gu.acc[n];
  __syncthreads();
  if (threadIdx.x < kCols * kRows) {
    const int c = threadIdx.x % kCols, t = threadIdx.x / kCols;
    const int slot = tb->slot[e][t];
    if (slot >= 0) {
      const int up = FP8 ? c : 8 + c;
      float gs = 0.f, us = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const floatx4* r = reinterpret_cast<const floatx4*>(ring + w * kRing);
        gs += r[c / 4 * 16 + t][c % 4];
        us += r[(NT - 1) * kWave + up / 4 * 16 + t][up % 4];
      }
      const float wt = tb->w[t][slot - t * (a.k + a.ns)];
      // readers wait for the word itself to change, so nothing has to be
      // ordered around the store
      __hip_atomic_store(a.hw + (size_t)slot * I + c0 + c, pack_h(silu_mul(gs, us) * wt),
                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
}

__device__ __forceinline__ unsigned long long peek(const uint32_t* p) {
  return __hip_atomic_load(reinterpret_cast<const unsigned long long*>(p), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool unset(unsigned long long v) {
  return (uint32_t)v == kUnset || (uint32_t)(v >> 32) == kUnset;
}

// Reads h' words (each lane N pairs from its p on, or none: zeros) until none
// of them is unset.  The units that write them have smaller tickets, which
// blocks take in order and only while they run, so each such unit has ended
// or is running in a block that waits for nothing: the wait ends.
template <int N>
__device__ __forceinline__ void read_h(const uint32_t* const (&p)[N], unsigned long long (&v)[N]) {
  for (;;) {
    bool again = false;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = p[i] == nullptr ? 0ull : peek(p[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) again |= unset(v[i]);
    if (!__any(again)) return;
    __builtin_amdgcn_s_sleep(1);
  }
}

// All of h' to LDS, its two parts apart: row s (an assignment) of 2 I bytes of
// high parts and 2 I of low parts every 4 I + kPad bytes, 16 zero bytes behind
// the last row.  By every thread of the block, 16 bytes a turn.
__device__ __forceinline__ void stage_h(const FewArgs& a, const FewTables* __restrict__ tb,
                                        uint8_t* __restrict__ hs) {
  const int I = a.I, quads = I / 4, total = a.T * (a.k + a.ns) * quads, row_bytes = 4 * I + kPad;
#pragma unroll 1
  for (int j0 = 0; j0 < total; j0 += 2 * kThreads) {
    unsigned long long v[4];
    int at[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = j0 + i * kThreads + (int)threadIdx.x;
      const int slot = j / quads, t = min(slot / (a.k + a.ns), a.T - 1);
      const bool in = j < total && !tb->bad[t] && (a.valid == nullptr || a.valid[t] != 0);
      at[i] = in ? slot * row_bytes + 8 * (j - slot * quads) : -1;
    }
    for (;;) {
      bool again = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t* p = a.hw + 4 * (uint32_t)(j0 + i * kThreads + (int)threadIdx.x);
        v[2 * i] = v[2 * i + 1] = 0;
        if (at[i] >= 0) {
          v[2 * i] = peek(p);
          v[2 * i + 1] = peek(p + 2);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) again |= unset(v[i]);
      if (!__any(again)) break;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (at[i] < 0) continue;
      const uint32_t w0 = (uint32_t)v[2 * i], w1 = (uint32_t)(v[2 * i] >> 32);
      const uint32_t w2 = (uint32_t)v[2 * i + 1], w3 = (uint32_t)(v[2 * i + 1] >> 32);
      *reinterpret_cast<u32x2*>(hs + at[i]) = u32x2{(w0 & 0xffffu) | w1 << 16, (w2 & 0xffffu) | w3 << 16};
      *reinterpret_cast<u32x2*>(hs + at[i] + 2 * I) =
          u32x2{w0 >> 16 | (w1 & 0xffff0000u), w2 >> 16 | (w3 & 0xffff0000u)};
    }
  }
  if (threadIdx.x == 0)
    *reinterpret_cast<u32x4*>(hs + a.T * (a.k + a.ns) * row_bytes) = u32x4{0u, 0u, 0u, 0u};
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
  int row_bytes, zeros, low;
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
      const uint8_t* hr = hs + (slot >= 0 ? slot * row_bytes + 2 * (cq * 32 * WC::kSteps + WC::k_of(u, g)) : zeros);
      const u32x4 hi = ld16(hr), lo = ld16(hr + (slot >= 0 ? low : 0));
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

// The sums of the waves (each at the start of its part of the ring) to
// out[t][c0 .. c0 + 31].
template <bool STAGED>
__device__ __forceinline__ void store_out(const FewArgs& a, const FewTables* __restrict__ tb,
                                          uint8_t* __restrict__ ring, int c0, const floatx4 (&acc)[2]) {
  constexpr int kRing = FewShared<STAGED>::kRing;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  floatx4* red = reinterpret_cast<floatx4*>(ring + wave * kRing);
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) red[nt * kWave + lane] = acc[nt];
  __syncthreads();
  const int c = threadIdx.x % kDnCols, t = threadIdx.x / kDnCols;
  if (t < a.T) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      s += reinterpret_cast<const floatx4*>(ring + w * kRing)[c / 16 * kWave + (c % 16) / 4 * 16 + t][c % 4];
    a.out[(size_t)t * a.H + c0 + c] = tb->bad[t] ? 0x7fc0u : f32_to_bf16_bits(s);
  }
}

// out[t][c0 .. c0 + 31] for every row: W2 rows (two 16-column tiles) as the
// MFMA A operand, h' as B, K = all chosen experts' columns one after the
// other, split over the waves.  The first W2 loads are on their way while the
// block waits for h' (staged: it has it from its unit before).
template <bool FP8, bool PW>
__device__ __forceinline__ void down_unit_staged(const FewArgs& a, const FewTables* __restrict__ tb,
                                                 uint8_t* __restrict__ hs, uint8_t* __restrict__ ring,
                                                 bool staged, int c0, int& next) {
  using DS = DownStaged<FP8, PW>;
  using WC = typename DS::WC;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int H = a.H, I = a.I;
  constexpr int kSize = FP8 ? 1 : 2, GC = FP8 ? 2 : 1;   // chunks under one scale
  DS d;
  d.w2 = static_cast<const uint8_t*>(a.w2) + (size_t)c0 * I * kSize;
  d.expert = (size_t)H * I * kSize;
  d.tile = 16 * I * kSize;
  d.wl = PW ? 16 * lane : WC::lane_offset(lane % 16, I, lane / 16);
  d.cpe = I / (32 * WC::kSteps);
  d.row_bytes = 4 * I + kPad;
  d.zeros = a.T * (a.k + a.ns) * d.row_bytes;
  d.low = 2 * I;
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) d.acc[nt] = d.part[nt] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int n = tb->n_act * (d.cpe / GC);
  const int s0 = n * wave / kWaves * GC, s1 = n * (wave + 1) / kWaves * GC;
  int ai = s0 / d.cpe, q = s0 - ai * d.cpe;
  d.ai = ai;
  d.q = q;
  uint8_t* mine = ring + wave * FewShared<true>::kRing;
#pragma unroll
  for (int i = 0; i < DS::kAhead; ++i)
    if (s0 + i < s1) d.issue(mine + i * DS::kEntry, tb);
  if (threadIdx.x == 0) next = take_ticket(a.ticket);
  if (!staged) stage_h(a, tb, hs);
  __syncthreads();
  int at = 0;
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    if (s + DS::kAhead <= s1) wait_loads<(DS::kAhead - 1) * DS::kLoads>();
    else wait_loads<0>();
    const int to = at == 0 ? DS::kEntries - 1 : at - 1;
    const int e = __builtin_amdgcn_readfirstlane(tb->act[ai]);
    d.step(mine + at * DS::kEntry, mine + to * DS::kEntry, hs, tb, e, q, s + DS::kAhead < s1, lane,
           a.s2 + ((size_t)e * (H / 128) + c0 / 128) * (I / 128) + q / 2);
    if (++q == d.cpe) q = 0, ++ai;
    at = at + 1 == DS::kEntries ? 0 : at + 1;
  }
  store_out<true>(a, tb, ring, c0, d.acc);
}

// The same with W2 and h' straight to registers, for calls whose h' does not
// fit in LDS.
template <bool FP8, bool PW>
__device__ __forceinline__ void down_unit(const FewArgs& a, const FewTables* __restrict__ tbp,
                                          uint8_t* __restrict__ ring, int c0, int& next) {
  const FewTables& tb = *tbp;
  using WB = WBlock<FP8, PW>;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int m = lane % 16, g = lane / 16;
  const int H = a.H, I = a.I;
  // a wave's work in groups of GS steps: fp8 a 128-wide block under one
  // scale, bf16 single steps (72 of them for 9 experts of 256 columns: 9 a
  // wave, where blocks of four would give three waves 12 and five 8)
  constexpr int GS = FP8 ? 4 : 1, kBatch = 4 / GS;   // groups loaded at once
  constexpr int kLoads = FP8 ? WB::kLoads : 1;
  const int gpe = I / (32 * GS);   // groups of an expert
  const int n = tb.n_act * gpe;
  const int s0 = n * wave / kWaves, s1 = n * (wave + 1) / kWaves;
  const uint32_t wl = WB::lane_offset(m, I, g);
  floatx4 acc[2];
  acc[0] = acc[1] = floatx4{0.f, 0.f, 0.f, 0.f};
  bool take = true;
  for (int s = s0; s < s1; s += kBatch) {
    typename std::conditional<FP8 && PW, u32x2, u32x4>::type wv[kBatch][2][kLoads];
    int ai = s / gpe, q = s - ai * gpe;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (s + i < s1) {
        const int e = __builtin_amdgcn_readfirstlane(tb.act[ai]);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const void* tile = WB::tile_at(a.w2, (size_t)e * H + c0 + 16 * nt, I);
          WB w;
          if constexpr (FP8) w.load(tile, wl, q);
          else w.load1(static_cast<const uint16_t*>(tile) + (size_t)q * (PW ? 512 : 32), wl, 0, 0);
#pragma unroll
          for (int l = 0; l < kLoads; ++l) wv[i][nt][l] = w.v[l];
        }
        if (++q == gpe) q = 0, ++ai;
      }
    }
    if (take && threadIdx.x == 0) next = take_ticket(a.ticket);
    take = false;
    ai = s / gpe, q = s - ai * gpe;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (s + i >= s1) continue;
      const int e = __builtin_amdgcn_readfirstlane(tb.act[ai]);
      const int slot = tb.slot[e][m];
      u32x4 hi[GS], lo[GS];
      {
        const uint32_t* p[4 * GS];
        unsigned long long v[4 * GS];
#pragma unroll
        for (int u = 0; u < GS; ++u) {
          const int k = GS == 4 ? 128 * q + WB::k_of(u, g) : 32 * q + 8 * g;
#pragma unroll
          for (int l = 0; l < 4; ++l)
            p[4 * u + l] = slot >= 0 ? a.hw + (size_t)slot * I + k + 2 * l : nullptr;
        }
        read_h<4 * GS>(p, v);
#pragma unroll
        for (int u = 0; u < GS; ++u)
#pragma unroll
          for (int l = 0; l < 4; ++l) {
            const uint32_t w0 = (uint32_t)v[4 * u + l], w1 = (uint32_t)(v[4 * u + l] >> 32);
            hi[u][l] = (w0 & 0xffffu) | (w1 << 16);
            lo[u][l] = (w0 >> 16) | (w1 & 0xffff0000u);
          }
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        if constexpr (FP8) {
          WB w;
#pragma unroll
          for (int l = 0; l < kLoads; ++l) w.v[l] = wv[i][nt][l];
          floatx4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int u = 0; u < GS; ++u) {
            p = mfma16x16x32(w.get(u), as_bf16x8(hi[u]), p);
            p = mfma16x16x32(w.get(u), as_bf16x8(lo[u]), p);
          }
          const float sc = a.s2[((size_t)e * (H / 128) + c0 / 128) * (I / 128) + q];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[nt][j] = fmaf(sc, p[j], acc[nt][j]);
        } else {
          acc[nt] = mfma16x16x32(as_bf16x8(wv[i][nt][0]), as_bf16x8(hi[0]), acc[nt]);
          acc[nt] = mfma16x16x32(as_bf16x8(wv[i][nt][0]), as_bf16x8(lo[0]), acc[nt]);
        }
      }
      if (++q == gpe) q = 0, ++ai;
    }
  }
  if (take && threadIdx.x == 0) next = take_ticket(a.ticket);
  store_out<false>(a, tbp, ring, c0, acc);
}

template <bool FP8, bool PW, bool STAGED>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(4)))
void few_experts_kernel(FewArgs a) {
  static_assert(kThreads == kRows * kDnCols, "one output per thread");
  __shared__ FewShared<STAGED> sh;
  few_route<STAGED>(a, sh.tb, sh.stage, sh.tk);
  constexpr int kCols = few_cols(FP8);
  const int n_cg = a.I / kCols, n_gu = sh.tb.n_act * n_cg, n_all = n_gu + a.H / kDnCols;
  int tk = __builtin_amdgcn_readfirstlane(sh.tk);
  bool h_staged = false;   // the stage holds h' in place of the token rows (tickets grow)
  while (tk < n_all) {
    __syncthreads();   // tk, the ring and the stage are free
    int next = 0;   // the next ticket (thread 0), asked for behind the unit's first loads
    if (tk < n_gu) {
      const int ai = tk / n_cg;
      gate_up_unit<FP8, PW, STAGED>(a, &sh.tb, sh.stage, &sh.ring[0][0],
                                    __builtin_amdgcn_readfirstlane(sh.tb.act[ai]),
                                    (tk - ai * n_cg) * kCols, next);
    } else {
      const int c0 = (tk - n_gu) * kDnCols;
      if constexpr (STAGED)
        down_unit_staged<FP8, PW>(a, &sh.tb, sh.stage, &sh.ring[0][0], h_staged, c0, next);
      else down_unit<FP8, PW>(a, &sh.tb, &sh.ring[0][0], c0, next);
      h_staged = true;
    }
    if (threadIdx.x == 0) sh.tk = next;
    __syncthreads();
    tk = __builtin_amdgcn_readfirstlane(sh.tk);
  }
}

}  // namespace

hipError_t launch_few(int wkind, bool packed, const void* x, const uint8_t* valid, const void* R,
                      const void* w13, const void* w2, const float* s13, const float* s2,
                      float* part, uint32_t* hw, int32_t* ticket, void* out, int T, int H, int I,
                      int E, int n_shared, int k, hipStream_t s) {
  if (wkind == W_F32 || T < 1 || T > kFewRows || E + n_shared > kMaxSeg || k > kMaxTopk ||
      H % 128 != 0 || I % 32 != 0 || (long long)H * I >= kMaxFewArea || (wkind == W_FP8 && I % 128 != 0))
    return hipErrorInvalidValue;
  const size_t n_hw = (size_t)T * (k + n_shared) * I;
  hipLaunchKernelGGL(few_logits_kernel, dim3((E + 15) / 16, kFewLogitParts), dim3(kThreads), 0, s,
                     static_cast<const uint16_t*>(x), valid, static_cast<const uint16_t*>(R), part,
                     hw, n_hw, ticket, T, H, E);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const FewArgs a{static_cast<const uint16_t*>(x), valid, w13, w2, s13, s2, part, hw, ticket,
                  static_cast<uint16_t*>(out), T, H, I, E, n_shared, k, kFewLogitParts};
  // A block for every gate/up unit, so that they all run at once, from one to
  // two a CU; blocks loop over the tickets.
  const long long n_gu = (long long)(std::min(E, T * k) + n_shared) * (I / few_cols(wkind == W_FP8));
  const long long units = n_gu + H / kDnCols;
  const dim3 grid((unsigned)std::min(units, std::max(256LL, std::min(n_gu, 512LL))));
  // rows and h' in LDS where they fit
  const bool staged = T < kWaves && (long long)T * (2 * H + kPad) + 16 <= FewShared<true>::kStage &&
                      (long long)T * (k + n_shared) * (4LL * I + kPad) + 16 <= FewShared<true>::kStage;
#define MOE_FEW(F, P)                                                                         \
  if (staged)                                                                                 \
    hipLaunchKernelGGL((few_experts_kernel<F, P, true>), grid, dim3(kThreads), 0, s, a);      \
  else                                                                                        \
    hipLaunchKernelGGL((few_experts_kernel<F, P, false>), grid, dim3(kThreads), 0, s, a)
  if (wkind == W_FP8) {
    if (packed) { MOE_FEW(true, true); } else { MOE_FEW(true, false); }
  } else {
    if (packed) { MOE_FEW(false, true); } else { MOE_FEW(false, false); }
  }
#undef MOE_FEW
  return hipGetLastError();
}

}  // namespace moe
