// Root-mean-square norm of token rows, with the addition of the residual ahead of
// it and, if asked for, e4m3fn codes of the result behind it:
//   r = x + residual, rounded to the type it is stored in
//   v = r / sqrt(mean(r^2) + eps) * weight, in fp32: mean, root, quotient and product
//       rounded once each
// out = v rounded once; codes and scales are those that quant.hip makes of v.  The
// norm is that of the stored r, so that whoever reads r has the rows that v is of.
//
// One pass: a row stays in the registers of its block, 8 values a lane and piece, 2
// pieces a lane (1: 10 % slower where rows take more than 8 waves; 4, up to 10 %
// slower, for rows above 16384 alone, which 16 waves of 2 pieces do not hold).
// Bound by memory.  bf16 with a residual, 8192 x 7168 in us and TB/s: to bf16 82.0, 5.7;
// to codes 74.5, 5.5; of 512 to 16384 columns 5.4 to 5.9.  One row 3.4, the launch.
// fp32 with a residual 184.5, 5.1, to codes 148.5, 5.2; bf16 with an fp32 residual 129.5,
// 5.4, to codes 121.5, 5.3.
// Measured and not better: blocks that stay and load the next row ahead (79 to 92 us,
// 77 to 83 to codes), fewer blocks a CU.
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
  __device__ __forceinline__ void store(void* base, size_t at) const {
    u32x4* p = reinterpret_cast<u32x4*>(static_cast<uint8_t*>(base) + at * (BF16 ? 2 : 4));
    p[0] = q[0];
    if constexpr (!BF16) p[1] = q[1];
  }
  // v, rounded to bf16 or as it is
  __device__ __forceinline__ explicit Piece(const float (&v)[kPer]) {
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) q[0][i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) q[i / 4][i % 4] = __float_as_uint(v[i]);
    }
  }
  Piece() = default;
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (BF16)
      return __uint_as_float(i & 1 ? q[0][i / 2] & 0xffff0000u : q[0][i / 2] << 16);
    else
      return __uint_as_float(q[i / 4][i % 4]);
  }
};

// The value of the lane N places on among 16 (around), which hold one block of 128.
template <int N>
__device__ __forceinline__ float around(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0x120 + N, 0xf, 0xf, true));
}
__device__ __forceinline__ float max_of_16(float v) {
  v = fmaxf(v, around<1>(v));
  v = fmaxf(v, around<2>(v));
  v = fmaxf(v, around<4>(v));
  return fmaxf(v, around<8>(v));
}
__device__ __forceinline__ float sum_of_wave(float v) {
  v += around<1>(v);
  v += around<2>(v);
  v += around<4>(v);
  v += around<8>(v);
  const auto of = [&](int lane) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
  };
  return (of(0) + of(16)) + (of(32) + of(48));
}

// x / root for the values of a row: one division a row, inv = 1 / root, and q + (x - q
// root) inv with q = x inv, the quotient rounded once (Markstein; compared with the
// division for 600 roots and all mantissas of x).  Without the remainder a value has one
// rounding more, and some codes next to the middle of two become the other one.
struct Root {
  float root, inv, back;
  __device__ __forceinline__ explicit Root(float mean)
      // (an infinite root: no remainder, all finite values give 0)
      : root(sqrtf(mean)), inv(1.f / root), back(root < INFINITY ? root : 0.f) {}
  __device__ __forceinline__ float of(float x) const {
    const float q = x * inv;
    return fmaf(-fmaf(back, q, -x), inv, q);   // (so that -0 stays -0)
  }
};

// RES: 0 no residual, 1 fp32, 2 bf16.  P pieces a lane.
template <int P, bool XB, int RES, bool CODES>
__global__ __launch_bounds__(1024) void norm_kernel(NormRows p) {
  const int waves = blockDim.x / kWave, wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  __shared__ float part[2][16];
  int turn = 0;
  const auto col = [&](int i) { return (i * (int)blockDim.x + (int)threadIdx.x) * kPer; };
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    float v[P][kPer];
    Piece<XB> x[P];
    Piece<RES == 2> res[P];
    u32x4 w[P];   // (the first half of fp32 weights; the other one behind the barrier)
    // (lanes behind the row read its last piece: loads under a condition wait for
    // those ahead of them)
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = min(col(i), p.cols - kPer);
      x[i].load(p.x, (size_t)row * p.ld_x + c);
      if constexpr (RES != 0) res[i].load(p.res, (size_t)row * p.ld_res + c);
    }
    const auto load_w = [&](int i) {
      w[i] = ld16(static_cast<const uint8_t*>(p.w) + (p.w_bf16 ? 2 : 4) * min(col(i), p.cols - kPer));
    };
    if constexpr (P <= 2)
#pragma unroll
      for (int i = 0; i < P; ++i) load_w(i);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const bool in = col(i) < p.cols;
#pragma unroll
      for (int k = 0; k < kPer; ++k) v[i][k] = x[i][k];
      if constexpr (RES != 0) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[i][k] += res[i][k];
        const Piece<RES == 2> r(v[i]);
        if (in) r.store(p.res_out, (size_t)row * p.ld_res_out + col(i));
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[i][k] = r[k];
      }
      float of = 0.f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) of = fmaf(v[i][k], v[i][k], of);
      sum += in ? of : 0.f;
    }
    sum = sum_of_wave(sum);
    if (lane == 0) part[turn][wave] = sum;
    // (one barrier a row: a wave writes part[turn] again only behind the next
    // row's barrier, which all waves reach when they have read it)
    __syncthreads();
    sum = 0.f;
    for (int w = 0; w < waves; ++w) sum += part[turn][w];
    const Root root(sum / (float)p.cols + p.eps);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = col(i);
      const bool in = c < p.cols;
      if (in) {
        if constexpr (P > 2) load_w(i);
        if (p.w_bf16) {
          Piece<true> of;
          of.q[0] = w[i];
#pragma unroll
          for (int k = 0; k < kPer; ++k) v[i][k] = root.of(v[i][k]) * of[k];
        } else {
          Piece<false> of;
          of.q[0] = w[i];
          of.q[1] = ld16(static_cast<const float*>(p.w) + c + 4);
#pragma unroll
          for (int k = 0; k < kPer; ++k) v[i][k] = root.of(v[i][k]) * of[k];
        }
        if (!CODES || p.out != nullptr) {
          if (p.out_bf16) Piece<true>(v[i]).store(p.out, (size_t)row * p.ld_out + c);
          else Piece<false>(v[i]).store(p.out, (size_t)row * p.ld_out + c);
        }
      }
      if constexpr (CODES) {
        // 16 lanes hold a block of 128
        float top = kFp8Tiny;
#pragma unroll
        for (int k = 0; k < kPer; ++k) top = fmaxf(top, fabsf(v[i][k]));
        const Fp8Block b(max_of_16(in ? top : kFp8Tiny));
        if (in) {
          *reinterpret_cast<u32x2*>(p.codes + (size_t)row * p.ld_codes + c) =
              u32x2{b.codes(v[i]), b.codes(v[i] + 4)};
          if (c % 128 == 0) p.scales[(size_t)row * p.ld_scales + c / 128] = b.scale;
        }
      }
    }
  }
}

using Kernel = void (*)(NormRows);
template <int P, bool CODES>
Kernel kernel_of(const NormRows& p) {
  const int res = p.res == nullptr ? 0 : p.res_bf16 ? 2 : 1;
  if (p.x_bf16)
    return res == 0 ? norm_kernel<P, true, 0, CODES>
                    : res == 1 ? norm_kernel<P, true, 1, CODES> : norm_kernel<P, true, 2, CODES>;
  return res == 0 ? norm_kernel<P, false, 0, CODES>
                  : res == 1 ? norm_kernel<P, false, 1, CODES> : norm_kernel<P, false, 2, CODES>;
}

}  // namespace

hipError_t launch_norm(const NormRows& p, hipStream_t s) {
  if (p.cols > kMaxNormCols) return hipErrorInvalidValue;
  // waves of 512 P values each
  const int pieces = (p.cols + kPer * kWave - 1) / (kPer * kWave);
  const int P = pieces <= 32 ? 2 : 4;
  const dim3 block(kWave * ((pieces + P - 1) / P)), grid((unsigned)std::min(p.rows, 1 << 20));
  const Kernel kernel = P == 2 ? p.codes ? kernel_of<2, true>(p) : kernel_of<2, false>(p)
                               : p.codes ? kernel_of<4, true>(p) : kernel_of<4, false>(p);
  return enqueue(kernel, grid, block, s, p);
}

}  // namespace moe
