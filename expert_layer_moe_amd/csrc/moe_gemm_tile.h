// What the tiled products (fp8_gemm.hip, mxfp4_gemm.hip) share: loads straight
// to LDS and the waits for them, the order of a call's tiles, and a tile's way out.
#pragma once

#include <algorithm>

#include "moe_common.h"

namespace moe {

typedef __attribute__((__vector_size__(8 * sizeof(int)))) int i32x8;
typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4;

// A buffer from p on (unbounded: the kernels keep their offsets in range).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p, int bytes = -1) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}
// An offset behind the end of every buffer of at most 2^31 bytes (256 rows, 2^23 apart):
// loads give 0, also with the distance to a tile's later rows added, which stays below
// 2^31 as the rows do.
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t src, uint32_t lane_offset, uint32_t offset) {
  return __builtin_bit_cast(u32x4,
                            __builtin_amdgcn_raw_buffer_load_b128(src, lane_offset, offset, 0));
}

// Waits until at most N of this wave's loads are outstanding and its LDS
// accesses are done, then for the block; no memory access moves across.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | (N >> 4) << 14);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Loads straight to LDS: lane l's 4 or 16 bytes go to dst + 4 l or + 16 l.
// (As buffer loads: the compiler takes global ones for accesses that may
// complete out of order with LDS reads, and waits for all of either at each
// use.)  ONCE: data that no other block reads.
__device__ __forceinline__ void to_lds4(__amdgpu_buffer_rsrc_t src, uint32_t lane_offset,
                                          uint32_t offset, void* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)dst, 4,
                                           lane_offset, offset, 0, 0);
}
template <bool ONCE = false>
__device__ __forceinline__ void to_lds16(__amdgpu_buffer_rsrc_t src, uint32_t lane_offset,
                                         uint32_t offset, void* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)dst, 16,
                                           lane_offset, offset, 0, ONCE ? 2 : 0);
}
// Waits until at most N of the wave's loads are outstanding and its LDS reads
// are done; no memory access moves across.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | (N >> 4) << 14);
  asm volatile("" ::: "memory");
}

// The blocks of a call, at most kGridX of them along x (a multiple of the 8 XCDs;
// a dimension holds less than 2^32 threads): block block_index(), and behind the
// last one some without work.
constexpr unsigned kGridX = 1u << 22;
__device__ __forceinline__ unsigned block_index() { return blockIdx.y * gridDim.x + blockIdx.x; }
inline dim3 grid_of(long long blocks) {
  const long long y = (blocks + kGridX - 1) / kGridX;
  return dim3((unsigned)std::min<long long>(blocks, kGridX), (unsigned)y);
}

// Columns n .. n + 3 of row m, as far as they exist.
template <bool F32>
__device__ __forceinline__ void store4(void* out, long long ldo, int N, int m, int n, floatx4 v) {
  const size_t at = (size_t)m * ldo + n;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= N) break;
    if constexpr (F32) static_cast<float*>(out)[at + i] = v[i];
    else static_cast<uint16_t*>(out)[at + i] = f32_to_bf16_bits(v[i]);
  }
}

// A tile that block_index() takes, row tile and column tile; false: none.  The
// hardware hands block b to XCD b % 8: each XCD gets a contiguous range of tiles,
// and walks them in groups of 8 rows of tiles, column by column, so that its
// tiles share operands in its L2.
__device__ __forceinline__ bool tile_of_block(int tiles_m, int tiles_n, int& tm, int& tn) {
  const int total = tiles_m * tiles_n;
  const int xcd = block_index() % 8, at = block_index() / 8;
  const int tile = total / 8 * xcd + min(xcd, total % 8) + at;
  if (at >= total / 8 + (xcd < total % 8 ? 1 : 0)) return false;
  constexpr int GM = 8;
  const int group = tile / (GM * tiles_n), in_group = tile - group * (GM * tiles_n);
  const int gm = min(GM, tiles_m - group * GM);
  tm = group * GM + in_group % gm;
  tn = in_group / gm;
  return true;
}

// A wave's 16 TM rows x 16 TN columns, from row m0 and column n0 on, out through
// `mine`, its part of LDS (tile_store_bytes), 16 rows at a time: as the MFMA leaves
// it, lane (r, g) = (lane % 16, lane / 16) has four columns of one row, and a store
// would cover 16 rows x 32 bytes.
template <int TN, bool F32>
constexpr int tile_store_bytes() {
  return 16 * (16 * TN * (F32 ? 4 : 2) + 16);
}
template <int TM, int TN, bool F32>
__device__ __forceinline__ void store_tile(const floatx4 (&acc)[TM][TN], uint8_t* mine, void* out,
                                           long long ldo, int M, int N, int m0, int n0, int lane, int r, int g) {
  constexpr int kSize = F32 ? 4 : 2, kCols = 16 * TN;
  constexpr int kPitch = kCols * kSize + 16;
  constexpr int kVec = 16 / kSize, kLanes = kCols / kVec;   // values of a piece, pieces of a row
  const bool wide = ((size_t)ldo * kSize | (size_t)N * kSize | (size_t)out) % 16 == 0;
#pragma unroll
  for (int t = 0; t < TM; ++t) {
#pragma unroll
    for (int q = 0; q < TN; ++q) {
      uint8_t* to = mine + r * kPitch + (16 * q + 4 * g) * kSize;
      if constexpr (F32) *reinterpret_cast<floatx4*>(to) = acc[t][q];
      else
        *reinterpret_cast<u32x2*>(to) =
            u32x2{pack_bf16x2(acc[t][q][0], acc[t][q][1]), pack_bf16x2(acc[t][q][2], acc[t][q][3])};
    }
    const int mt = m0 + 16 * t;
    if (wide) {
#pragma unroll
      for (int i = lane; i < 16 * kLanes; i += kWave) {
        const int row = i / kLanes, c = i % kLanes * kVec;
        const u32x4 v = ld16(mine + row * kPitch + c * kSize);
        if (mt + row < M && n0 + c < N)
          *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(out) +
                                    ((size_t)(mt + row) * ldo + n0 + c) * kSize) = v;
      }
    } else {
      for (int i = lane; i < 16 * kCols; i += kWave) {
        const int row = i / kCols, c = i % kCols;
        if (mt + row >= M || n0 + c >= N) continue;
        const size_t o = (size_t)(mt + row) * ldo + n0 + c;
        const uint8_t* from = mine + row * kPitch + c * kSize;
        if constexpr (F32) static_cast<float*>(out)[o] = *reinterpret_cast<const float*>(from);
        else static_cast<uint16_t*>(out)[o] = *reinterpret_cast<const uint16_t*>(from);
      }
    }
  }
}

}  // namespace moe
