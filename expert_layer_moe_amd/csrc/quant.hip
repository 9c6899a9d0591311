// Token rows -> e4m3fn codes with one fp32 scale per 128 values ("Step3
// Inference Optimization on AMD Instinct MI308X", optimisation list: FP8
// blockscale), the a operand of the fp8 product; and the same of
// SiLU(gate) * up, between the two products of a dense layer.
//   scale = max(largest |v| of the block, 1e-12) / 448, code = e4m3(v / scale)
// with both divisions correctly rounded in fp32 and the code rounded to
// nearest even, so every code is determined by its input.
#include "moe_common.h"
#include "moe_kernels.h"

#include <algorithm>

namespace moe {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kTiny = 1e-12f;

// As the formula has it: expf to one unit in the last place, a correctly rounded
// division; 0 from v = -88.8 on, where exp(-v) overflows.  8192 x 2048 bf16 gates
// and ups are bound by it: 19.8 to 20.4 us.  (With exp2 and reciprocal instructions and a
// correction each they take 17.2, but scales are then off by up to 5.3 units of
// 2^-24 in place of 3.6.)
__device__ __forceinline__ float silu(float v) { return v / (1.f + expf(-v)); }

constexpr int kPer = 16;                    // values of a lane: 16 bytes of codes
constexpr int kLanes = 128 / kPer;          // lanes of a block of 128
constexpr int kGroups = 256 / kLanes;       // blocks a workgroup does at once

// kPer consecutive values at base + off.
template <bool BF16>
__device__ __forceinline__ void load(const void* base, size_t off, float (&v)[kPer]) {
  if constexpr (BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + off;
    u32x4 q[kPer / 8];
#pragma unroll
    for (int j = 0; j < kPer / 8; ++j) q[j] = ld16(p + 8 * j);
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
      v[2 * i] = __uint_as_float(q[i / 4][i % 4] << 16);
      v[2 * i + 1] = __uint_as_float(q[i / 4][i % 4] & 0xffff0000u);
    }
  } else {
    const float* p = static_cast<const float*>(base) + off;
#pragma unroll
    for (int j = 0; j < kPer / 4; ++j) {
      const floatx4 q = *reinterpret_cast<const floatx4*>(p + 4 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * j + i] = q[i];
    }
  }
}

// One pass: 8 lanes per block of 128 values, 16 values per lane, so that codes
// leave 16 bytes a lane.  Bound by memory (3 bytes a bf16 value), if the
// arithmetic stays small: one division per lane, r = 1 / scale; every v / scale
// is then q + (v - q scale) r with q = v r, which is the correctly rounded
// quotient for a correctly rounded r (Markstein; nothing here comes near
// overflow, and quotients too small for the remainder to be exact have code 0).
// 8192 x 7168 bf16: 32 us, 5.6 TB/s; with a division per value 43.
template <bool BF16, bool SILU>
__global__ __launch_bounds__(256) void quant_kernel(QuantRows p) {
  const uint32_t nb = (p.cols + 127u) / 128, total = (uint32_t)p.rows * nb;   // < 2^31
  const int part = threadIdx.x % kLanes;
  // every lane of a wave stays in the loop as long as any has a block (the
  // maximum is taken across lanes)
  for (uint32_t j0 = blockIdx.x * kGroups; j0 < total; j0 += gridDim.x * kGroups) {
    const uint32_t j = j0 + threadIdx.x / kLanes, row = j / nb, kb = j - row * nb;
    const int c = kb * 128 + kPer * part;
    const bool in = j < total && c < p.cols;
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = 0.f;
    if (in) {
      load<BF16>(p.in, (size_t)row * p.ld_in + c, v);
      if constexpr (SILU) {
        float u[kPer];
        load<BF16>(p.in, (size_t)row * p.ld_in + p.cols + c, u);
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = silu(v[i]) * u[i];
      }
    }
    float top = kTiny;
#pragma unroll
    for (int i = 0; i < kPer; ++i) top = fmaxf(top, fabsf(v[i]));
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float scale = top / kE4m3Max, r = 1.f / scale;
    // an infinite scale: no remainder, all finite values are 0
    const float back = scale < INFINITY ? scale : 0.f;
    if (!in) continue;
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = v[4 * i + k], y = x * r;
        f[k] = copysignf(fmaf(fmaf(-y, back, x), r, y), x);   // (-0 stays -0)
      }
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w, true);
      q[i] = (uint32_t)w;
    }
    *reinterpret_cast<u32x4*>(p.codes + (size_t)row * p.ld_codes + c) = q;
    if (part == 0) p.scales[(size_t)row * p.ld_scales + kb] = scale;
  }
}

}  // namespace

hipError_t launch_quant(const QuantRows& p, bool silu_mul, hipStream_t s) {
  const long long blocks = p.rows * ((p.cols + 127LL) / 128);
  if (blocks > kMaxQuantBlocks) return hipErrorInvalidValue;
  const dim3 grid((unsigned)std::min((blocks + kGroups - 1) / kGroups, 1LL << 20));
#define MOE_Q(B, S) hipLaunchKernelGGL((quant_kernel<B, S>), grid, dim3(256), 0, s, p)
  if (p.bf16) {
    if (silu_mul) MOE_Q(true, true);
    else MOE_Q(true, false);
  } else {
    if (silu_mul) MOE_Q(false, true);
    else MOE_Q(false, false);
  }
#undef MOE_Q
  return hipGetLastError();
}

}  // namespace moe
