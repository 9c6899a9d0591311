// Matrix product of fp8 (e4m3fn) codes with block scales:
//   out[m][n] = sum over K blocks b of sa[m][b] sb[n / 128][b]
//               (sum over k in b of a[m][k] b[n][k])
// ("AMD Instinct MI355X: ATOM ...": block-scale GEMM).  One fp8 MFMA covers a
// whole 128-wide K block, so each block's sum leaves the matrix cores on its
// own and joins the fp32 accumulator under its two scales.
#include "moe_common.h"
#include "moe_kernels.h"

namespace moe {
namespace {

typedef __attribute__((__vector_size__(8 * sizeof(int)))) int i32x8;

// D(16x16, fp32) = A(16x128) * B(128x16), e4m3 inputs, 32 codes of a row per
// lane: lane l holds 16-byte pieces l / 16 and 4 + l / 16 of row l % 16 (any
// order of K serves, as long as A and B agree); D as mfma16x16x32.
__device__ __forceinline__ floatx4 mfma_block(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1) {
  const i32x8 a = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3],
                   (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
  const i32x8 b = {(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3],
                   (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, floatx4{0.f, 0.f, 0.f, 0.f}, 0, 0,
                                                          0, 0, 0, 0);
}

// 64 rows x 64 columns per block, 16 columns per wave, operands straight from
// memory.
__global__ __launch_bounds__(256) void fp8_gemm_kernel(Fp8Gemm p) {
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int r = lane % 16, g = lane / 16;
  const long long m0 = (long long)blockIdx.x * 64;
  const int n0 = blockIdx.y * 64 + wave * 16;
  if (n0 >= p.N) return;
  const int nb = (p.K + 127) / 128;
  const uint8_t* bp = p.b + (size_t)min(n0 + r, p.N - 1) * p.ldb;
  const float* sb = p.sb + (size_t)(n0 / 128) * nb;
  const uint8_t* ap[4];
  const float* sa[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const size_t m = (size_t)min(m0 + 16 * t + r, (long long)p.M - 1);
    ap[t] = p.a + m * p.lda;
    sa[t] = p.sa + m * p.ldsa;
  }
  const u32x4 zero = {0u, 0u, 0u, 0u};
  floatx4 acc[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) acc[t] = floatx4{0.f, 0.f, 0.f, 0.f};
  for (int kb = 0; kb < nb; ++kb) {
    const int k0 = kb * 128 + 16 * g, k1 = k0 + 64;
    const bool v0 = k0 < p.K, v1 = k1 < p.K;
    const u32x4 w0 = v0 ? ld16(bp + k0) : zero, w1 = v1 ? ld16(bp + k1) : zero;
    const float s = sb[kb];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const u32x4 a0 = v0 ? ld16(ap[t] + k0) : zero, a1 = v1 ? ld16(ap[t] + k1) : zero;
      const floatx4 d = mfma_block(w0, w1, a0, a1);
      const float sc = s * sa[t][kb];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(sc, d[i], acc[t][i]);
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const long long m = m0 + 16 * t + r;
    if (m >= p.M) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + 4 * g + i;
      if (n >= p.N) continue;
      if (p.out_f32) static_cast<float*>(p.out)[m * p.ldo + n] = acc[t][i];
      else static_cast<uint16_t*>(p.out)[m * p.ldo + n] = f32_to_bf16_bits(acc[t][i]);
    }
  }
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8Gemm& p, hipStream_t s) {
  const long long gx = ((long long)p.M + 63) / 64, gy = ((long long)p.N + 63) / 64;
  if (gx > 0x7fffffffLL || gy > 65535) return hipErrorInvalidValue;
  hipLaunchKernelGGL(fp8_gemm_kernel, dim3((unsigned)gx, (unsigned)gy), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace moe
