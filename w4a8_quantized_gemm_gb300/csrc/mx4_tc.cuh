// mx4_tc.cuh -- device code that the products of microscaled 4-bit operands share:
// the block-scaled instruction (tcgen05.mma kind::mxf4nvf4), its scales' way to
// Tensor Memory, and y's stores. G: the CTAs that one instruction spans (1 or 2).
#pragma once

#include "mx4_internal.h"

namespace egopq {

struct Mx4Params {
  const uint8_t* operand;
  const uint8_t* packed;
  const float* a_scale;
  const float* w_scale;
  const int32_t* offsets;
  void* y;
  int64_t M, N, K;
  int sets, nb, kb, type, split;
  uint64_t timeout_ns;
};

// 32 lanes x 16 bytes, to all four lane quarters: rows of 16 bytes, eight rows of
// 128 bytes a core matrix (stride 128), no swizzle
template <int G>
__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint32_t saddr) {
  const uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) |
                     static_cast<uint64_t>(128 >> 4) << 32 | static_cast<uint64_t>(1) << 46;
  if constexpr (G == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}
#define EGOPQ_MX4_MMA(GROUP, VEC)                                                              \
  asm volatile(                                                                                \
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                        \
      "tcgen05.mma.cta_group::" GROUP ".kind::mxf4nvf4.block_scale.scale_vec::" VEC             \
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                       \
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)                            \
      : "memory")
template <int FMT, int G>
__device__ __forceinline__ void tc_mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t sa, uint32_t sb, uint32_t accumulate) {
  if constexpr (G == 1 && FMT == EGOPQ_MX4_E8M0) EGOPQ_MX4_MMA("1", "2X");
  if constexpr (G == 1 && FMT == EGOPQ_MX4_E4M3) EGOPQ_MX4_MMA("1", "4X");
  if constexpr (G == 2 && FMT == EGOPQ_MX4_E8M0) EGOPQ_MX4_MMA("2", "2X");
  if constexpr (G == 2 && FMT == EGOPQ_MX4_E4M3) EGOPQ_MX4_MMA("2", "4X");
}
#undef EGOPQ_MX4_MMA
// e2m1 x e2m1, fp32 sums, K = 64, both K-major; id: which two of a word's four
// scales (0 or 2; with 4X all four).
template <int FMT>
__device__ __forceinline__ uint32_t idesc_mx4(int rows, int cols, int id) {
  return ((uint32_t)id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(cols >> 3) << 17) |
         ((FMT == EGOPQ_MX4_E8M0 ? 1u : 0u) << 23) | ((uint32_t)(rows >> 4) << 24) |
         ((uint32_t)id << 29);
}
// The instructions of one K block (its `steps` runs of 64 K) on operands at a_at and
// b_at in shared memory; scales at sa and sb, `sa_step` and `sb_step` columns a word
// of four.
template <int FMT, int G>
__device__ __forceinline__ void tc_block_mx4(uint32_t d, uint32_t a_at, uint32_t b_at, uint32_t sa,
                                             int sa_step, uint32_t sb, int sb_step, int rows,
                                             int cols, int steps, bool first) {
  for (int j = 0; j < steps; ++j) {
    const int at = FMT == EGOPQ_MX4_E4M3 ? j : j >> 1;
    const int id = FMT == EGOPQ_MX4_E4M3 ? 0 : (j & 1) * 2;
    tc_mma_mx4<FMT, G>(d, sdesc_kmajor_sw128(a_at + 32 * j), sdesc_kmajor_sw128(b_at + 32 * j),
                       idesc_mx4<FMT>(rows, cols, id), sa + sa_step * at, sb + sb_step * at,
                       !(first && j == 0));
  }
}
// Runs of 64 K in K block kb.
__device__ __forceinline__ int mx4_steps(int64_t K, int kb) {
  return (int)min((int64_t)4, (K - (int64_t)kb * 256 + 63) / 64);
}

__device__ __forceinline__ uint16_t mx4_bits16(int type, float v) {
  return type == kMx4Bf16 ? f32_to_bf16_bits(v) : __half_as_ushort(__float2half_rn(v));
}
__device__ __forceinline__ void store_y(void* y, int64_t at, int type, float v) {
  if (type == kMx4F32) static_cast<float*>(y)[at] = v;
  else static_cast<uint16_t*>(y)[at] = mx4_bits16(type, v);
}

}  // namespace egopq
