// 4-bit floats in blocks of 32 under a power of two ("MX" of the Open Compute
// Project's microscaling formats 1.0: elements e2m1, scales e8m0):
//   e = floor(log2(largest |v| of the block)) - 2, at least -127
//   code = e2m1(v / 2^e), to the nearest, ties to the even code, at most 6;
//   scale code = e + 127
// Token rows to codes, SiLU(gate) * up to codes, and codes to their values.
// Everything behind SiLU is exact but the rounding to a code, so each code is
// determined by its input.
#include "moe_common.h"
#include "moe_kernels.h"

#include <algorithm>

namespace moe {
namespace {

constexpr int kMx = 32;
constexpr int kPer = 8;             // values of a lane: 16 bytes of bf16, 4 of codes
constexpr int kLanes = kMx / kPer;  // lanes of a block
constexpr int kThreads = 256;

// n / d for n < 2^31 by a product (Granlund and Montgomery: m = floor(2^(31 + s) / d)
// + 1 with 2^s >= d).
struct Divider {
  uint32_t m, shift;
};
Divider divider(uint32_t d) {
  uint32_t s = 0;
  while ((1u << s) < d) ++s;
  return {(uint32_t)((1ull << (31 + s)) / d + 1), 31 + s};
}
__device__ __forceinline__ uint32_t operator/(uint32_t n, Divider d) {
  return (uint32_t)((uint64_t)n * d.m >> d.shift);
}

// The largest magnitude's bits of 8 values, as they are or packed; NaN and
// infinities come out on top.
struct Floats {
  float v[kPer];
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ uint32_t codes(float scale) const {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], scale, 3);
  }
};

template <bool BF16>
__device__ __forceinline__ Floats load(const void* base, size_t at) {
  Floats f;
  if constexpr (BF16) {
    const u32x4 q = ld16(static_cast<const uint16_t*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.v[2 * i] = __uint_as_float(q[i] << 16);
      f.v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
  } else {
    const float* p = static_cast<const float*>(base) + at;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const floatx4 q = *reinterpret_cast<const floatx4*>(p + 4 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) f.v[4 * j + i] = q[i];
    }
  }
  return f;
}

template <bool BF16, bool SILU>
__global__ __launch_bounds__(kThreads) void mx_quant_kernel(MxRows p, Divider per_row) {
  constexpr uint32_t kGroups = kThreads / kLanes;
  const uint32_t nb = p.cols / kMx, total = (uint32_t)p.rows * nb;   // < 2^31
  const int part = threadIdx.x % kLanes;
  for (uint32_t j0 = blockIdx.x * kGroups; j0 < total; j0 += gridDim.x * kGroups) {
    const uint32_t j = j0 + threadIdx.x / kLanes;
    if (j >= total) continue;   // (a block's lanes leave together)
    const uint32_t row = j / per_row, kb = j - row * nb;
    const size_t c = kb * (size_t)kMx + kPer * part;
    Floats f = load<BF16>(p.values, (size_t)row * p.ld_values + c);
    if constexpr (SILU) {
      const Floats u = load<BF16>(p.values, (size_t)row * p.ld_values + p.cols + c);
#pragma unroll
      for (int i = 0; i < kPer; ++i) f.v[i] = silu(f.v[i]) * u.v[i];
    }
    uint32_t top = f.top();
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    const uint32_t ex = top >> 23;   // of the largest, biased; 255: infinity or NaN
    const uint32_t code = ex == 255 ? 255 : ex > 2 ? ex - 2 : 0;
    // (2^-127 lies below the normal numbers)
    const float scale = __uint_as_float(code == 0 ? 0x00400000u : code << 23);
    const uint32_t q = code == 255 ? 0u : f.codes(scale);
    *reinterpret_cast<uint32_t*>(p.codes + (size_t)row * p.ld_codes + c / 2) = q;
    if (part == 0) p.scales[(size_t)row * p.ld_scales + kb] = (uint8_t)code;
  }
}

// e2m1 codes to fp32: the code's three low bits are an exponent and a mantissa
// bit, of which 0.5 (code 1) is the only one below the normal ones.
__device__ __forceinline__ float e2m1(uint32_t code) {
  const uint32_t m = code & 7;
  const float v = __uint_as_float((m << 22) + (126u << 23));   // (1 + low / 2) 2^(m / 2 - 1)
  const float size = m == 0 ? 0.f : m == 1 ? 0.5f : v;
  return code & 8 ? -size : size;
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void mx_dequant_kernel(MxRows p, Divider per_row) {
  constexpr uint32_t kGroups = kThreads / kLanes;
  const uint32_t nb = p.cols / kMx, total = (uint32_t)p.rows * nb;   // < 2^31
  const int part = threadIdx.x % kLanes;
  for (uint32_t j0 = blockIdx.x * kGroups; j0 < total; j0 += gridDim.x * kGroups) {
    const uint32_t j = j0 + threadIdx.x / kLanes;
    if (j >= total) continue;
    const uint32_t row = j / per_row, kb = j - row * nb;
    const size_t c = kb * (size_t)kMx + kPer * part;
    const uint32_t q = *reinterpret_cast<const uint32_t*>(p.codes + (size_t)row * p.ld_codes + c / 2);
    const uint32_t code = p.scales[(size_t)row * p.ld_scales + kb];
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      v[i] = code == 255 ? __uint_as_float(0x7fc00000u) : ldexpf(e2m1(q >> 4 * i), (int)code - 127);
    const size_t at = (size_t)row * p.ld_values + c;
    if constexpr (BF16) {
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = __float_as_uint(v[2 * i]) >> 16 | (__float_as_uint(v[2 * i + 1]) & 0xffff0000u);
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.values) + at) = o;
    } else {
      float* to = static_cast<float*>(p.values) + at;
      *reinterpret_cast<floatx4*>(to) = floatx4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<floatx4*>(to + 4) = floatx4{v[4], v[5], v[6], v[7]};
    }
  }
}

dim3 grid_for(const MxRows& p) {
  const long long blocks = (long long)p.rows * (p.cols / kMx), each = kThreads / kLanes;
  return dim3((unsigned)std::min((blocks + each - 1) / each, 1LL << 20));
}

}  // namespace

hipError_t launch_mx_quant(const MxRows& p, bool silu_mul, hipStream_t s) {
  if ((long long)p.rows * (p.cols / kMx) > kMaxMxBlocks) return hipErrorInvalidValue;
  const Divider d = divider(p.cols / kMx);
#define MOE_Q(B, S) hipLaunchKernelGGL((mx_quant_kernel<B, S>), grid_for(p), dim3(kThreads), 0, s, p, d)
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

hipError_t launch_mx_dequant(const MxRows& p, hipStream_t s) {
  if ((long long)p.rows * (p.cols / kMx) > kMaxMxBlocks) return hipErrorInvalidValue;
  const Divider d = divider(p.cols / kMx);
  if (p.bf16) hipLaunchKernelGGL((mx_dequant_kernel<true>), grid_for(p), dim3(kThreads), 0, s, p, d);
  else hipLaunchKernelGGL((mx_dequant_kernel<false>), grid_for(p), dim3(kThreads), 0, s, p, d);
  return hipGetLastError();
}

}  // namespace moe
