// Root-mean-square norm of token rows, with the addition of the residual ahead of
// it and, if asked for, e4m3fn codes of the result behind it:
//   r = x + residual, rounded to the type it is stored in
//   v = r / sqrt(mean(r^2) + eps) * weight, in fp32
// out = v rounded once; codes and scales are those that quant.hip makes of v.  The
// norm is that of the stored r, so that whoever reads r has the rows that v is of.
//
// One pass: a row stays in the registers of its block, 8 values a lane and piece.
#include "moe_common.h"
#include "moe_kernels.h"

#include <algorithm>

namespace moe {
namespace {

constexpr int kPer = 8;   // values of a lane's piece: 16 bytes of bf16

template <bool BF16>
struct Piece {
  u32x4 q[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* base, size_t at) {
    const uint8_t* p = static_cast<const uint8_t*>(base) + at * (BF16 ? 2 : 4);
    q[0] = ld16(p);
    if constexpr (!BF16) q[1] = ld16(p + 16);
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (BF16)
      return __uint_as_float(i & 1 ? q[0][i / 2] & 0xffff0000u : q[0][i / 2] << 16);
    else
      return __uint_as_float(q[i / 4][i % 4]);
  }
};

// v to base + at, rounded to bf16 or as it is; returns nothing, v as it was
template <bool BF16>
__device__ __forceinline__ void store(void* base, size_t at, const float (&v)[kPer]) {
  if constexpr (BF16) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + at) = q;
  } else {
    float* p = static_cast<float*>(base) + at;
    *reinterpret_cast<floatx4*>(p) = floatx4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<floatx4*>(p + 4) = floatx4{v[4], v[5], v[6], v[7]};
  }
}

// RES: 0 no residual, 1 fp32, 2 bf16.  P pieces a lane.
template <int P, bool XB, int RES, bool CODES>
__global__ __launch_bounds__(1024) void norm_kernel(NormRows p) {
  const int waves = blockDim.x / kWave, wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  __shared__ float part[2][16];
  int turn = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    float v[P][kPer];
    Piece<XB> x[P];
    Piece<RES == 2> res[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = (i * (int)blockDim.x + (int)threadIdx.x) * kPer;
      if (c >= p.cols) continue;
      x[i].load(p.x, (size_t)row * p.ld_x + c);
      if constexpr (RES != 0) res[i].load(p.res, (size_t)row * p.ld_res + c);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = (i * (int)blockDim.x + (int)threadIdx.x) * kPer;
      if (c >= p.cols) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[i][k] = 0.f;
        continue;
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        v[i][k] = x[i][k];
        if constexpr (RES != 0) v[i][k] += res[i][k];
        if constexpr (RES == 2) v[i][k] = bf16_bits_to_f32(f32_to_bf16_bits(v[i][k]));
      }
      if constexpr (RES != 0) store<RES == 2>(p.res_out, (size_t)row * p.ld_res_out + c, v[i]);
#pragma unroll
      for (int k = 0; k < kPer; ++k) sum = fmaf(v[i][k], v[i][k], sum);
    }
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) sum += __shfl_xor(sum, d);
    if (lane == 0) part[turn][wave] = sum;
    // (one barrier a row: a wave writes part[turn] again only behind the next
    // row's barrier, which all waves reach when they have read it)
    __syncthreads();
    sum = 0.f;
    for (int w = 0; w < waves; ++w) sum += part[turn][w];
    const float inv = 1.f / sqrtf(sum / (float)p.cols + p.eps);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = (i * (int)blockDim.x + (int)threadIdx.x) * kPer;
      const bool in = c < p.cols;
      if (in) {
        if (p.w_bf16) {
          Piece<true> w;
          w.load(p.w, c);
#pragma unroll
          for (int k = 0; k < kPer; ++k) v[i][k] = v[i][k] * inv * w[k];
        } else {
          Piece<false> w;
          w.load(p.w, c);
#pragma unroll
          for (int k = 0; k < kPer; ++k) v[i][k] = v[i][k] * inv * w[k];
        }
        if (!CODES || p.out != nullptr) {
          if (p.out_bf16) store<true>(p.out, (size_t)row * p.ld_out + c, v[i]);
          else store<false>(p.out, (size_t)row * p.ld_out + c, v[i]);
        }
      }
      if constexpr (CODES) {
        // 16 lanes hold a block of 128 (those behind the row hold zeros)
        float top = kFp8Tiny;
#pragma unroll
        for (int k = 0; k < kPer; ++k) top = fmaxf(top, fabsf(v[i][k]));
#pragma unroll
        for (int d = 1; d < 128 / kPer; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
        const Fp8Block b(top);
        if (in) {
          *reinterpret_cast<u32x2*>(p.codes + (size_t)row * p.ld_codes + c) =
              u32x2{b.codes(v[i]), b.codes(v[i] + 4)};
          if (c % 128 == 0) p.scales[(size_t)row * p.ld_scales + c / 128] = b.scale;
        }
      }
    }
  }
}

template <int P, bool XB, int RES>
void launch(const NormRows& p, dim3 grid, dim3 block, hipStream_t s) {
  if (p.codes) hipLaunchKernelGGL((norm_kernel<P, XB, RES, true>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((norm_kernel<P, XB, RES, false>), grid, block, 0, s, p);
}

template <int P>
void launch_typed(const NormRows& p, dim3 grid, dim3 block, hipStream_t s) {
  const int res = p.res == nullptr ? 0 : p.res_bf16 ? 2 : 1;
  if (p.x_bf16) {
    if (res == 0) launch<P, true, 0>(p, grid, block, s);
    else if (res == 1) launch<P, true, 1>(p, grid, block, s);
    else launch<P, true, 2>(p, grid, block, s);
  } else {
    if (res == 0) launch<P, false, 0>(p, grid, block, s);
    else if (res == 1) launch<P, false, 1>(p, grid, block, s);
    else launch<P, false, 2>(p, grid, block, s);
  }
}

}  // namespace

hipError_t launch_norm(const NormRows& p, hipStream_t s) {
  if (p.cols > kMaxNormCols) return hipErrorInvalidValue;
  // waves of 512 P values each
  const int pieces = (p.cols + kPer * kWave - 1) / (kPer * kWave);   // P = 1
  const int P = pieces <= 16 ? (pieces > 4 ? 2 : 1) : 4;
  const dim3 block(kWave * ((pieces + P - 1) / P)), grid((unsigned)std::min(p.rows, 1 << 20));
  if (P == 1) launch_typed<1>(p, grid, block, s);
  else if (P == 2) launch_typed<2>(p, grid, block, s);
  else launch_typed<4>(p, grid, block, s);
  return hipGetLastError();
}

}  // namespace moe
