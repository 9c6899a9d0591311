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
#include "topk.h"

#include <algorithm>

namespace moe {
namespace {

constexpr int kRows = kFewRows;   // one MFMA tile of token rows
constexpr int kWaves = 8;
constexpr int kThreads = kWaves * kWave;
constexpr int kMaxSeg = 257;      // 256 routed experts + 1 shared
constexpr int kGuCols = 8;        // h columns of a gate/up unit
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
  for (int s = s0; s < s1; ++s) {
    const u32x4 a = rv ? ld16(xp + 32 * s) : zero;
    const u32x4 b = ev ? ld16(rp + 32 * s) : zero;
    acc = mfma16x16x32(as_bf16x8(a), as_bf16x8(b), acc);
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

// 8 weights of one lane and MFMA step.
template <bool FP8>
struct WFrag {
  typename std::conditional<FP8, u32x2, u32x4>::type v;
  __device__ __forceinline__ void load(const void* base, size_t off) {
    if constexpr (FP8) v = ld8(static_cast<const uint8_t*>(base) + off);
    else v = ld16(static_cast<const uint16_t*>(base) + off);
  }
  __device__ __forceinline__ bf16x8 get() const {
    if constexpr (FP8) return fp8x8_to_bf16x8(v[0], v[1]);
    else return as_bf16x8(v);
  }
};

struct FewTables {
  int16_t slot[kMaxSeg][kRows];   // assignment t (k + ns) + j of row t at this segment, or -1
  int16_t act[kMaxSeg];           // segments that some row chose, ascending
  float w[kRows][kMaxTopk + 1];   // routing weights; the shared slot holds 1
  uint8_t bad[kRows];             // rows whose logits are NaN
  int n_act;
};

// The top-k of every row (one wave per row, kWaves rows at a time) and the
// tables the units work from; called by every thread of the block.
__device__ __forceinline__ void few_route(const float* __restrict__ part, int ks,
                                          const uint8_t* __restrict__ valid, int T, int E, int ns,
                                          int k, FewTables& tb) {
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int nseg = E + ns, kk = k + ns;
  for (int i = threadIdx.x; i < nseg * kRows; i += kThreads) tb.slot[i / kRows][i % kRows] = -1;
  if (threadIdx.x < kRows) tb.bad[threadIdx.x] = 0;
  __syncthreads();
  for (int t = wave; t < T; t += kWaves) {
    if (valid != nullptr && valid[t] == 0) continue;
    float v[4];
    bool taken[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = lane + kWave * i;
      taken[i] = e >= E;
      float s = 0.f;
      if (e < E)
        for (int z = 0; z < ks; ++z) s += part[((size_t)z * T + t) * E + e];
      v[i] = s;
    }
    float my_w;
    int my_e;
    topk_row(v, taken, k, lane, my_e, my_w);
    // NaN logits pick no expert: the row's output is NaN
    const bool ok = lane >= k || ((unsigned)my_e < (unsigned)E && my_w == my_w);
    if (!__all(ok)) {
      if (lane == 0) tb.bad[t] = 1;
      continue;
    }
    if (lane < k) {
      tb.slot[my_e][t] = (int16_t)(t * kk + lane);
      tb.w[t][lane] = my_w;
    }
    if (ns && lane == 0) {
      tb.slot[E][t] = (int16_t)(t * kk + k);
      tb.w[t][k] = 1.f;
    }
  }
  __syncthreads();
  if (wave == 0) {
    int n = 0;
    for (int e0 = 0; e0 < nseg; e0 += kWave) {
      const int e = e0 + lane;
      bool any = false;
      if (e < nseg)
        for (int t = 0; t < T; ++t) any |= tb.slot[e][t] >= 0;
      const unsigned long long b = __ballot(any);
      if (any) tb.act[n + __popcll(b & ((1ull << lane) - 1))] = (int16_t)e;
      n += __popcll(b);
    }
    if (lane == 0) tb.n_act = n;
  }
  __syncthreads();
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

// K steps that a wave runs through at once (loads ahead of the MFMAs).
constexpr int kBatch = 4;

// h' columns c0 .. c0 + 7 of expert e for every row that chose it.  The MFMA
// A operand holds 8 gate rows and the 8 up rows of the same columns, the B
// operand the token rows (rows that did not choose e: zeros); the waves split
// K = H in 128-wide blocks and meet in LDS.
template <bool FP8, bool PW>
__device__ __forceinline__ void gate_up_unit(const FewArgs& a, const FewTables& tb, int e, int c0,
                                             floatx4 (&red)[kWaves][2][kWave]) {
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int m = lane % 16, g = lane / 16;
  const int H = a.H, I = a.I;
  const int row = m < 8 ? c0 + m : I + c0 + m - 8;
  const size_t wrow = (size_t)e * 2 * I + row;
  // row-major fp8: 16 bytes of a row hold a lane's share of two steps
  constexpr bool kPair = FP8 && !PW;
  const size_t woff = PW ? (wrow / 16) * (H / 32) * 512 + (size_t)(16 * g + row % 16) * 8
                         : wrow * H + (kPair ? 16 : 8) * g;
  const bool xv = tb.slot[e][m] >= 0;
  const uint16_t* xp = a.x + (size_t)(xv ? m : 0) * H + (kPair ? 16 : 8) * g;
  const float* sp = nullptr;
  if constexpr (FP8)
    sp = a.s13 + ((size_t)e * (2 * I / 128) + (g < 2 ? c0 : I + c0) / 128) * (H / 128);
  const int nb = H / 128;
  const int b0 = nb * wave / kWaves, b1 = nb * (wave + 1) / kWaves;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int b = b0; b < b1; ++b) {
    WFrag<FP8> w[kBatch];
    u32x4 xf[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int s = 4 * b + u;
      w[u].load(a.w13, woff + (PW ? (size_t)s * 512 : kPair ? (size_t)(s / 2) * 64 + 8 * (s & 1) : (size_t)s * 32));
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int s = 4 * b + u;
      xf[u] = xv ? ld16(xp + (kPair ? (s / 2) * 64 + 8 * (s & 1) : s * 32)) : zero;
    }
    if constexpr (FP8) {
      floatx4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < kBatch; ++u) p = mfma16x16x32(w[u].get(), as_bf16x8(xf[u]), p);
      const float sc = sp[b];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(sc, p[i], acc[i]);
    } else {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) acc = mfma16x16x32(w[u].get(), as_bf16x8(xf[u]), acc);
    }
  }
  red[wave][0][lane] = acc;
  __syncthreads();
  // thread -> (column c, row t): gate at MFMA row c, up at row 8 + c
  if (threadIdx.x < kGuCols * kRows) {
    const int c = threadIdx.x % kGuCols, t = threadIdx.x / kGuCols;
    const int slot = tb.slot[e][t];
    if (slot >= 0) {
      float gs = 0.f, us = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        gs += red[w][0][(c / 4) * 16 + t][c % 4];
        us += red[w][0][(2 + c / 4) * 16 + t][c % 4];
      }
      const float wt = tb.w[t][slot - t * (a.k + a.ns)];
      // readers wait for the word itself to change, so nothing has to be
      // ordered around the store
      __hip_atomic_store(a.hw + (size_t)slot * I + c0 + c, pack_h(silu_mul(gs, us) * wt),
                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
}

// out[t][c0 .. c0 + 31] for every row: W2 rows (two 16-column tiles) as the
// MFMA A operand, h' as B, K = all chosen experts' columns one after the
// other, split over the waves.  The h' words are read until none of them is
// unset: the units that write them have smaller tickets, which blocks take
// in order and only while they run, so each such unit has ended or is
// running in a block that waits for nothing, and the wait ends.
template <bool FP8, bool PW>
__device__ __forceinline__ void down_unit(const FewArgs& a, const FewTables& tb, int c0,
                                          floatx4 (&red)[kWaves][2][kWave]) {
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int m = lane % 16, g = lane / 16;
  const int H = a.H, I = a.I;
  constexpr int GS = FP8 ? kBatch : 1;   // K steps under one scale
  const int spe = I / 32;                // K steps of an expert
  const int n = tb.n_act * (spe / GS);
  const int s0 = n * wave / kWaves * GS, s1 = n * (wave + 1) / kWaves * GS;
  floatx4 acc[2];
  acc[0] = acc[1] = floatx4{0.f, 0.f, 0.f, 0.f};
  for (int s = s0; s < s1; s += kBatch) {
    WFrag<FP8> w[kBatch][2];
    const uint32_t* hp[kBatch];
    const float* sc = nullptr;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int su = min(s + u, s1 - 1);   // past the end: read again, not used
      const int ai = su / spe, q = su - ai * spe;
      const int e = tb.act[ai];
      const int slot = tb.slot[e][m];
      hp[u] = slot >= 0 && s + u < s1 ? a.hw + (size_t)slot * I + 32 * q + 8 * g : nullptr;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const size_t wrow = (size_t)e * H + c0 + 16 * nt;
        w[u][nt].load(a.w2, PW ? ((wrow / 16) * spe + q) * 512 + 8 * lane
                               : (wrow + m) * I + 32 * q + 8 * g);
      }
      if (FP8 && u == 0)
        sc = a.s2 + ((size_t)e * (H / 128) + c0 / 128) * (I / 128) + q / 4;
    }
    unsigned long long v[kBatch][4];
    for (;;) {
      bool unset = false;
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[u][i] = hp[u] == nullptr
                        ? 0ull
                        : __hip_atomic_load(reinterpret_cast<const unsigned long long*>(hp[u]) + i,
                                            __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          unset |= (uint32_t)v[u][i] == kUnset || (uint32_t)(v[u][i] >> 32) == kUnset;
      if (!__any(unset)) break;
      __builtin_amdgcn_s_sleep(2);
    }
    floatx4 p[2];
    p[0] = p[1] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      u32x4 hi, lo;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w0 = (uint32_t)v[u][i], w1 = (uint32_t)(v[u][i] >> 32);
        hi[i] = (w0 & 0xffffu) | (w1 << 16);
        lo[i] = (w0 >> 16) | (w1 & 0xffff0000u);
      }
      // (a step past the end has zeros for h')
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        floatx4& d = FP8 ? p[nt] : acc[nt];
        d = mfma16x16x32(w[u][nt].get(), as_bf16x8(hi), d);
        d = mfma16x16x32(w[u][nt].get(), as_bf16x8(lo), d);
      }
    }
    if constexpr (FP8) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] = fmaf(*sc, p[nt][i], acc[nt][i]);
    }
  }
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) red[wave][nt][lane] = acc[nt];
  __syncthreads();
  const int c = threadIdx.x % kDnCols, t = threadIdx.x / kDnCols;
  if (t < a.T) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) s += red[w][c / 16][(c % 16) / 4 * 16 + t][c % 4];
    a.out[(size_t)t * H + c0 + c] = tb.bad[t] ? 0x7fc0u : f32_to_bf16_bits(s);
  }
}

template <bool FP8, bool PW>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(4)))
void few_experts_kernel(FewArgs a) {
  static_assert(kThreads == kRows * kDnCols, "one output per thread");
  __shared__ FewTables tb;
  __shared__ floatx4 red[kWaves][2][kWave];
  __shared__ int s_tk;
  if (threadIdx.x == 0)
    s_tk = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  few_route(a.part, a.ks, a.valid, a.T, a.E, a.ns, a.k, tb);
  const int n_cg = a.I / kGuCols;
  const int n_gu = tb.n_act * n_cg, n_all = n_gu + a.H / kDnCols;
  int tk = __builtin_amdgcn_readfirstlane(s_tk);
  while (tk < n_all) {
    __syncthreads();   // s_tk and red are free
    if (threadIdx.x == 0)
      s_tk = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (tk < n_gu) {
      const int ai = tk / n_cg;
      gate_up_unit<FP8, PW>(a, tb, tb.act[ai], (tk - ai * n_cg) * kGuCols, red);
    } else {
      down_unit<FP8, PW>(a, tb, (tk - n_gu) * kDnCols, red);
    }
    __syncthreads();
    tk = __builtin_amdgcn_readfirstlane(s_tk);
  }
}

// Enough blocks for two on every CU; they loop over the tickets.
constexpr int kFewGrid = 512;

}  // namespace

hipError_t launch_few(int wkind, bool packed, const void* x, const uint8_t* valid, const void* R,
                      const void* w13, const void* w2, const float* s13, const float* s2,
                      float* part, uint32_t* hw, int32_t* ticket, void* out, int T, int H, int I,
                      int E, int n_shared, int k, hipStream_t s) {
  if (wkind == W_F32 || T < 1 || T > kFewRows || E + n_shared > kMaxSeg || k > kMaxTopk ||
      H % 128 != 0 || I % 32 != 0 || (wkind == W_FP8 && I % 128 != 0))
    return hipErrorInvalidValue;
  const size_t n_hw = (size_t)T * (k + n_shared) * I;
  hipLaunchKernelGGL(few_logits_kernel, dim3((E + 15) / 16, kFewLogitParts), dim3(kThreads), 0, s,
                     static_cast<const uint16_t*>(x), valid, static_cast<const uint16_t*>(R), part,
                     hw, n_hw, ticket, T, H, E);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const FewArgs a{static_cast<const uint16_t*>(x), valid, w13, w2, s13, s2, part, hw, ticket,
                  static_cast<uint16_t*>(out), T, H, I, E, n_shared, k, kFewLogitParts};
  const long long units = (long long)(std::min(E, T * k) + n_shared) * (I / kGuCols) + H / kDnCols;
  const dim3 grid((unsigned)std::min<long long>(units, kFewGrid));
#define MOE_FEW(F, P) \
  hipLaunchKernelGGL((few_experts_kernel<F, P>), grid, dim3(kThreads), 0, s, a)
  if (wkind == W_FP8) {
    if (packed) MOE_FEW(true, true);
    else MOE_FEW(true, false);
  } else {
    if (packed) MOE_FEW(false, true);
    else MOE_FEW(false, false);
  }
#undef MOE_FEW
  return hipGetLastError();
}

}  // namespace moe
