// Token rows -> e4m3fn codes with one fp32 scale per 128 values ("Step3
// Inference Optimization on AMD Instinct MI308X", optimisation list: FP8
// blockscale), the a operand of the fp8 product; and the same of
// SiLU(gate) * up, between the two products of a dense layer.
//   scale = max(largest |v| of the block, 1e-12) / 448, code = e4m3(v / scale)
// with both divisions correctly rounded in fp32 and the code rounded to
// nearest even, so every code is determined by its input.
#include "moe_common.h"
#include "moe_kernels.h"

namespace moe {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kTiny = 1e-12f;

// 8 consecutive values at p.
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, size_t off, float (&v)[8]) {
  if constexpr (BF16) {
    const u32x4 q = ld16(static_cast<const uint16_t*>(base) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(q[i] << 16);
      v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
  } else {
    const float* p = static_cast<const float*>(base) + off;
    const floatx4 a = *reinterpret_cast<const floatx4*>(p);
    const floatx4 b = *reinterpret_cast<const floatx4*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
}

// 16 lanes per block of 128 values, 8 values per lane.
template <bool BF16, bool SILU>
__global__ __launch_bounds__(256) void quant_kernel(QuantRows p) {
  const int nb = (p.cols + 127) / 128;
  const long long total = (long long)p.rows * nb;
  const int lane16 = threadIdx.x % 16;
  const long long step = (long long)gridDim.x * 16;
  // every lane of a wave stays in the loop as long as any has a block (the
  // maximum is taken across lanes)
  const long long first = (long long)blockIdx.x * 16 + threadIdx.x / 16;
  for (long long j = first; j - threadIdx.x % kWave / 16 < total; j += step) {
    const long long row = j / nb;
    const int kb = (int)(j - row * nb);
    const int c = kb * 128 + 8 * lane16;
    const bool in = j < total && c < p.cols;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (in) {
      load8<BF16>(p.in, (size_t)row * p.ld_in + c, v);
      if constexpr (SILU) {
        float u[8];
        load8<BF16>(p.in, (size_t)row * p.ld_in + p.cols + c, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] / (1.f + expf(-v[i])) * u[i];
      }
    }
    float top = kTiny;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float scale = top / kE4m3Max;
    if (!in) continue;
    u32x2 q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] / scale, v[4 * i + 1] / scale, 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] / scale, v[4 * i + 3] / scale, w, true);
      q[i] = (uint32_t)w;
    }
    *reinterpret_cast<u32x2*>(p.codes + (size_t)row * p.ld_codes + c) = q;
    if (lane16 == 0) p.scales[(size_t)row * p.ld_scales + kb] = scale;
  }
}

}  // namespace

hipError_t launch_quant(const QuantRows& p, bool silu_mul, hipStream_t s) {
  const long long blocks = ((long long)p.rows * ((p.cols + 127) / 128) + 15) / 16;
  const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192));
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
