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

inline Mx4Params params_of(const Mx4GemmArgs& a) {
  Mx4Params p{};
  p.operand = a.operand;
  p.packed = a.packed;
  p.a_scale = a.a_scale;
  p.w_scale = a.w_scale;
  p.offsets = a.offsets;
  p.y = a.y;
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.sets = a.sets;
  p.nb = (int)((a.N + 127) / 128);
  p.kb = (int)mx4_kblocks(a.K);
  p.type = a.type;
  p.split = 1;
  p.timeout_ns = a.timeout_ns;
  return p;
}

// Descriptors hold addresses in 16-byte units in their lowest bits, and every
// address here is below 2^18: a place further on is an addition.
__device__ __forceinline__ uint64_t mx4_at(uint64_t desc, uint32_t bytes) {
  return desc + (bytes >> 4);
}
// Scales: 32 lanes x 16 bytes, to all four lane quarters: rows of 16 bytes, eight
// rows of 128 bytes a core matrix (stride 128), no swizzle.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(128 >> 4) << 32 |
         static_cast<uint64_t>(1) << 46;
}
template <int G>
__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (G == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                 : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                 : "memory");
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
// e2m1 x e2m1, fp32 sums, K = 64, both K-major. (Bits 4 and 29: which two of a
// word's four scales, 0 or 2; with 4X all four.)
template <int FMT>
__device__ __forceinline__ uint32_t idesc_mx4(int rows, int cols) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(cols >> 3) << 17) |
         ((FMT == EGOPQ_MX4_E8M0 ? 1u : 0u) << 23) | ((uint32_t)(rows >> 4) << 24);
}
// The instructions of one K block (its `steps` runs of 64 K) on the operands that a
// and b describe; scales at sa and sb, 4 and `sb_step` columns a word of four.
template <int FMT, int G>
__device__ __forceinline__ void tc_block_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t sa,
                                             uint32_t sb, int sb_step, uint32_t idesc, int steps,
                                             bool first) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int at = FMT == EGOPQ_MX4_E4M3 ? j : j >> 1;
    const uint32_t id = FMT == EGOPQ_MX4_E4M3 ? 0u : (uint32_t)(j & 1) * 2;
    if (j < steps)
      tc_mma_mx4<FMT, G>(d, mx4_at(a, 32 * j), mx4_at(b, 32 * j), idesc | id << 4 | id << 29,
                         sa + 4 * at, sb + sb_step * at, j > 0 || !first);
  }
}
// mbar_wait by threads that sleep in the hardware until the phase completes, or for a
// millisecond at a time: barriers and the tensor cores' instructions go through one
// queue, and threads that ask a barrier again and again slow both (a K block's
// instructions took 1800 cycles to issue beside ten warps that asked, for 510).
__device__ __forceinline__ bool mx4_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, 1000000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mx4_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                         uint64_t timeout_ns) {
  if (mx4_try(bar, parity)) return true;
  return mbar_wait(bar, parity, abort_flag, timeout_ns);
}
// A warp's wait, with the same answer in every lane.
__device__ __forceinline__ bool mx4_wait_warp(uint32_t bar, uint32_t parity,
                                              volatile int* abort_flag, uint64_t timeout_ns) {
  return __all_sync(0xffffffffu, mx4_wait(bar, parity, abort_flag, timeout_ns));
}

// A ring of `stages` buffers: the next item's, and the parity of its phase.
template <int STAGES>
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++s == STAGES) {
      s = 0;
      phase ^= 1;
    }
  }
};

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
