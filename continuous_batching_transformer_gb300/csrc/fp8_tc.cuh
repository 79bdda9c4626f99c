// fp8_tc.cuh -- e4m3 operands on the tensor cores: tiles of 64- and 128-byte rows in shared memory, the
// matrix instruction, and values as sums of several codes.
#pragma once
#include "paged_fp8.h"
#include "tc_common.cuh"

namespace tc {

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 inputs, 32 deep, fp32 accumulate, single CTA
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
// Instruction descriptor, kind::f8f6f4: e4m3 A and B (both K-major), fp32 D, M x N
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Instruction descriptor, kind::f16: fp16 A and B (both K-major), fp32 D, M x N
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// K-major tile of 64- or 128-byte rows in the swizzle of that size, groups of 8 rows next to each other
template <int ROW>
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t saddr) {
  static_assert(ROW == 64 || ROW == 128, "rows of 64 or 128 bytes");
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)1 << 16 | (uint64_t)(8 * ROW >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)(ROW == 64 ? 4 : 2) << 61;
}
// the same as two words: the high one is every tile's, the low one counts in 16-byte units and is moved by
// additions
template <int ROW>
__device__ __forceinline__ uint32_t rows_lo(const void* p) {
  return (uint32_t)sdesc_rows<ROW>(smem_u32(p));
}
template <int ROW>
__device__ __forceinline__ uint64_t rows_desc(uint32_t lo) {
  constexpr uint32_t hi = (uint32_t)((8 * ROW >> 4) | 1 << 14) | (ROW == 64 ? 4u : 2u) << 29;
  return (uint64_t)hi << 32 | lo;
}
// byte offset of (row, byte) in such a tile
template <int ROW>
__host__ __device__ __forceinline__ uint32_t swz(int row, int byte) {
  const int turn = ROW == 64 ? row >> 1 & 3 : row & 7;
  return (uint32_t)(row * ROW + (((byte >> 4) ^ turn) << 4) + (byte & 15));
}
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* m, uint64_t* bar, int at256,
                                              uint64_t policy) {
  tma_load_3d(dst, m, bar, 0, 0, at256, policy);
}

}  // namespace tc

// AND mask of 16 codes (one 16-byte unit) from their 16 visibility bits
CBT_D uint4 code_mask(uint32_t bits) {
  auto four = [](uint32_t b) { return ((b & 15u) * 0x00204081u & 0x01010101u) * 0xFFu; };
  return make_uint4(four(bits), four(bits >> 4), four(bits >> 8), four(bits >> 12));
}

// The power of two that brings magnitudes up to `top` (finite, >= 0) under 448, as an exponent to
// multiply by; within what fp32 holds, so that it and its reciprocal are normal numbers
CBT_D int fit_exponent(float top) {
  const uint32_t u = __float_as_uint(top);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u);
  return -min(max(e, -110), 120);
}

// K as rows of head_dim codes and V^T as rows of 64 positions: 64 positions a box
inline bool fp8_maps(const PagedKvFp8& kv, CUtensorMap* tk, CUtensorMap* tv) {
  return make_tmap_bytes(tk, kv.pool, kv.pool_bytes, kv.head_dim, kBlock) &&
         make_tmap_bytes(tv, kv.pool, kv.pool_bytes, kBlock, kv.head_dim);
}
