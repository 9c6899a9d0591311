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
#include <type_traits>

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

// The power of two of a scale code (2^-127 lies below the normal numbers).
__device__ __forceinline__ float scale_of(uint32_t code) {
  return __uint_as_float(code == 0 ? 0x00400000u : code << 23);
}

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

// silu() of 8 values, bit by bit (compared once for every fp32 value, and for 146 thousand
// gates whenever the tests run): v / d, d = 1 + exp(-v), as q + (v - q d) r with q = v r and
// r = 1 / d to half a step or nearly so, which rounds the quotient correctly (Markstein)
// while d and r are normal numbers.  Where they are not (v < -87 in any lane: rare), the
// division itself.
__device__ __forceinline__ void silu8(float (&v)[kPer]) {
  const float least = fminf(fminf(fminf(v[0], v[1]), fminf(v[2], v[3])),
                            fminf(fminf(v[4], v[5]), fminf(v[6], v[7])));
  if (__builtin_expect(least < -87.f, 0)) {
#pragma unroll 1
    for (int i = 0; i < kPer; ++i) {   // (around, so that they stay in registers)
      const float t = silu(v[0]);
#pragma unroll
      for (int j = 0; j + 1 < kPer; ++j) v[j] = v[j + 1];
      v[kPer - 1] = t;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float d = 1.f + expf(-v[i]), r0 = __builtin_amdgcn_rcpf(d), r = fmaf(fmaf(-d, r0, 1.f), r0, r0);
    const float q = v[i] * r;
    v[i] = fmaf(-fmaf(d, q, -v[i]), r, q);   // (so that -0 stays -0)
  }
}

// One pass, 8 values a lane, 4 lanes a block of 32.  Bound by memory: 8192 x 7168 bf16
// 28.0 us, 5.3 TB/s, fp32 46, 5.8; SiLU of 8192 x 2048 bf16 15.1, 5.0 TB/s (17.6 with a
// division a value), fp32 26, 5.5.  Two or four pieces a thread: within 1 % (SiLU: slower).
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
      silu8(f.v);
#pragma unroll
      for (int i = 0; i < kPer; ++i) f.v[i] *= u.v[i];
    }
    uint32_t top = f.top();
    // (of the four lanes: the neighbour's, then the other two's)
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xb1, 0xf, 0xf, true));
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4e, 0xf, 0xf, true));
    const uint32_t ex = top >> 23;   // of the largest, biased; 255: infinity or NaN
    const uint32_t code = ex == 255 ? 255 : ex > 2 ? ex - 2 : 0;
    const uint32_t q = code == 255 ? 0u : f.codes(scale_of(code));
    *reinterpret_cast<uint32_t*>(p.codes + (size_t)row * p.ld_codes + c / 2) = q;
    if (part == 0) p.scales[(size_t)row * p.ld_scales + kb] = (uint8_t)code;
  }
}

// 16 bytes a lane leave: 8 values of bf16, 4 of fp32 (whose halves of 32 bytes, stored
// one after the other, cost 10 us more), two pieces a thread, their loads ahead of
// their stores.  The matrix of 8192 x 7168: bf16 28.0 us, 5.3 TB/s (one piece 30.3),
// fp32 49.2, 5.4 TB/s (one piece 55.4, four 48.1).
template <bool BF16>
struct Dequant {
  static constexpr int kN = BF16 ? 8 : 4, kPieces = 2;
  static constexpr uint32_t kLanes = kMx / kN, kGroups = kThreads / kLanes, kEach = kGroups * kPieces;
  using Codes = std::conditional_t<BF16, uint32_t, uint16_t>;
};
template <bool BF16>
__global__ __launch_bounds__(kThreads) void mx_dequant_kernel(MxRows p, Divider per_row) {
  using D = Dequant<BF16>;
  const uint32_t nb = p.cols / kMx, total = (uint32_t)p.rows * nb;   // < 2^31
  const uint32_t part = threadIdx.x % D::kLanes;
  for (uint32_t j0 = blockIdx.x * D::kEach; j0 < total; j0 += gridDim.x * D::kEach) {
    uint32_t q[D::kPieces], code[D::kPieces], row[D::kPieces], kb[D::kPieces];
    const auto at = [&](int i) { return j0 + i * D::kGroups + threadIdx.x / D::kLanes; };
#pragma unroll
    for (int i = 0; i < D::kPieces; ++i) {
      const uint32_t j = min(at(i), total - 1);   // (behind the end: unstored)
      row[i] = j / per_row, kb[i] = j - row[i] * nb;
      q[i] = *reinterpret_cast<const typename D::Codes*>(p.codes + (size_t)row[i] * p.ld_codes +
                                                         kb[i] * (kMx / 2) + D::kN / 2 * part);
      code[i] = p.scales[(size_t)row[i] * p.ld_scales + kb[i]];
    }
#pragma unroll
    for (int i = 0; i < D::kPieces; ++i) {
      if (at(i) >= total) continue;
      const float scale = scale_of(code[i]);
      const size_t to = (size_t)row[i] * p.ld_values + (size_t)kb[i] * kMx + D::kN * part;
      u32x4 o;
      if constexpr (BF16) {
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], scale, 0));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], scale, 1));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], scale, 2));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], scale, 3));
        if (code[i] == 255) o = u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.values) + to) = o;
      } else {
        const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], scale, 0);
        const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], scale, 1);
        o = u32x4{__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(b[0]), __float_as_uint(b[1])};
        if (code[i] == 255) o = u32x4{0x7fc00000u, 0x7fc00000u, 0x7fc00000u, 0x7fc00000u};
        *reinterpret_cast<u32x4*>(static_cast<float*>(p.values) + to) = o;
      }
    }
  }
}

// blocks of the matrix, `each` of them a workgroup
dim3 grid_for(const MxRows& p, long long each) {
  const long long blocks = (long long)p.rows * (p.cols / kMx);
  return dim3((unsigned)std::min((blocks + each - 1) / each, 1LL << 20));
}

}  // namespace

hipError_t launch_mx_quant(const MxRows& p, bool silu_mul, hipStream_t s) {
  if ((long long)p.rows * (p.cols / kMx) > kMaxMxBlocks) return hipErrorInvalidValue;
  const Divider d = divider(p.cols / kMx);
  const auto kernel = p.bf16 ? silu_mul ? mx_quant_kernel<true, true> : mx_quant_kernel<true, false>
                             : silu_mul ? mx_quant_kernel<false, true> : mx_quant_kernel<false, false>;
  return enqueue(kernel, grid_for(p, kThreads / kLanes), dim3(kThreads), s, p, d);
}

hipError_t launch_mx_dequant(const MxRows& p, hipStream_t s) {
  if ((long long)p.rows * (p.cols / kMx) > kMaxMxBlocks) return hipErrorInvalidValue;
  const Divider d = divider(p.cols / kMx);
  if (p.bf16) return enqueue(mx_dequant_kernel<true>, grid_for(p, Dequant<true>::kEach), dim3(kThreads), s, p, d);
  return enqueue(mx_dequant_kernel<false>, grid_for(p, Dequant<false>::kEach), dim3(kThreads), s, p, d);
}

}  // namespace moe
