// mx4_quant.cuh -- a run of 256 values of a row to microscaled 4-bit codes, by one
// warp: what the quantization kernel does with memory, and the product of few rows
// with its own shared memory. The formats and the records: mx4_internal.h.
#pragma once

#include <cuda_fp8.h>

#include "mx4_internal.h"

namespace egopq {

constexpr int kE8M0 = EGOPQ_MX4_E8M0, kE4M3 = EGOPQ_MX4_E4M3;

// ---- conversions ----------------------------------------------------------------

// Eight fp32 values to e2m1 codes (to the nearest, ties to even, 6 at most), the
// first in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// The code of one real magnitude and sign, for values next to a border.
__device__ __forceinline__ uint32_t e2m1_double(double v) {
  const double a = fabs(v);
  const uint32_t m = (a > 0.25) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) +
                     (a >= 3.5) + (a > 5.0);
  return m | (v < 0.0 ? 8u : 0u);
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3);
  return __half2float(__half(h));
}
// 2^(byte - 127); 255 is NaN
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}

// Eight values of a row, as they lie in memory and as fp32.
template <int TYPE>
struct Eight {
  uint4 w[TYPE == kMx4F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) +
                                                    at * (TYPE == kMx4F32 ? 4 : 2));
    w[0] = __ldcs(q);
    if constexpr (TYPE == kMx4F32) w[1] = __ldcs(q + 1);
  }
  __device__ __forceinline__ void zero() {
    w[0] = make_uint4(0, 0, 0, 0);
    if constexpr (TYPE == kMx4F32) w[1] = w[0];
  }
  // The largest magnitude's pattern, of values stored as 16 bits (NaN above infinity
  // above all), and what it stands for.
  __device__ __forceinline__ uint32_t top16() const {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    const uint32_t m = __vmaxu2(__vimax3_u16x2(w[0].x & kAbs, w[0].y & kAbs, w[0].z & kAbs),
                                w[0].w & kAbs);
    return max(m & 0xffffu, m >> 16);
  }
  static __device__ __forceinline__ float of16(uint32_t pattern) {
    return TYPE == kMx4Bf16 ? __uint_as_float(pattern << 16)
                            : __half2float(__ushort_as_half((uint16_t)pattern));
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t a[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
    if constexpr (TYPE == kMx4F32) {
      const uint32_t b[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(a[i]);
        v[4 + i] = __uint_as_float(b[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (TYPE == kMx4Bf16) {
          v[2 * i] = __uint_as_float(a[i] << 16);
          v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a[i]));
          v[2 * i] = f.x;
          v[2 * i + 1] = f.y;
        }
      }
    }
  }
};

// Two fp32 at a time.
__device__ __forceinline__ void mul2(float& a0, float& a1, float b) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b));
}
__device__ __forceinline__ void mul2(float& a0, float& a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}
__device__ __forceinline__ void add2(float& a0, float& a1, float b) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b));
}
// a = b * c + a
__device__ __forceinline__ void fma2(float& a0, float& a1, float b0, float b1, float c) {
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "mov.b64 c, {%4, %4};\n\tfma.rn.f32x2 a, b, c, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1), "f"(c));
}

// 1 / v to a last place, for v that is no subnormal.
__device__ __forceinline__ float rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// ---- gated values -----------------------------------------------------------------
// h = silu(g) * u of two values in fp32, for -22 <= g. The exponent, below 32, is off by
// half a last place, 2^-20, and by 32 times log2(e)'s own 2^-26: the exponential by
// 0.96e-6. Its approximation adds 0.24e-6 (2^-22), the reciprocal's 0.12e-6, the sum,
// the products (r's, and for the codes that with 1/s, itself 0.12e-6 off) 0.06e-6 each:
// 1.74e-6 together, less than the 32 last places (1.9e-6 or more of a value) within
// which of a border 64 bits decide instead of fp32: the codes are those of the real h.
// That is a value in 30000 or so (which costs its warp about 2000 cycles, at 1/64 of
// the rate).
__device__ __forceinline__ void gated32(float& v0, float& v1, float g0, float g1, float u0,
                                        float u1) {
  v0 = g0, v1 = g1;
  mul2(v0, v1, -1.44269504f);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v0));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v1));
  add2(v0, v1, 1.f);
  v0 = rcp(v0), v1 = rcp(v1);
  mul2(v0, v1, g0, g1);
  mul2(v0, v1, u0, u1);
}
// Whether that does not hold, as g is below -22 or fp32 has run out of exponents on
// the way to v = h * r, before u (half a subnormal g loses a bit, but for the 16-bit
// types' g) or behind it (zeros are exact).
template <int TYPE>
__device__ __forceinline__ bool gated_weak(float g, float u, float v, float r) {
  return g != 0.f && u != 0.f &&
         (g < -22.f || (TYPE == kMx4F32 && fabsf(g) < 0x1p-100f) || fabsf(v) < 0x1p-100f ||
          fabsf(v) < 0x1p-100f * fabsf(r));
}
static __device__ __noinline__ double gated64(float g, float u, float r) {
  return (double)g / (1.0 + exp(-(double)g)) * (double)u * (double)r;
}
// How far above the number below it whose lowest mantissa bit is 2^-keep v lies, in
// last places and counted from kNear places below that number: every border
// between codes is such a number, and v is within kNear places of one where this is
// below 2 kNear. (The sign does not matter.)
constexpr uint32_t kNear = 32;
__device__ __forceinline__ uint32_t above_short(float v, int keep) {
  return (__float_as_uint(v) + kNear) & ((1u << (23 - keep)) - 1);
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min_abs3(float a, float b, float c) {
  float r;
  asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// max(|a|, |b|, |c|), NaN if one is
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// max(|a|, |b|), NaN if one is
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// v / 6, on the same side of the borders between e4m3 numbers (five bits; times six,
// seven) as the real quotient: a product with 1/6 and a step with its remainder, as
// for the codes below.
__device__ __forceinline__ float sixth(float v) {
  const float q = v * (1.f / 6.f);
  return fmaf(fmaf(-q, 6.f, v), 1.f / 6.f, q);
}

// Where a lane's results of a row's next runs go: its codes and its block's scale in
// their plain places and in the first run's record (null: not asked for).
struct RowOut {
  uint8_t *codes, *scales, *rec, *rec_scale;
};

// The i-th run of 256 values from where `out` points, all lanes of a warp.
template <int FMT, int TYPE, bool GATED>
__device__ __forceinline__ void quant_unit(const RowOut& out, int i_run, const Eight<TYPE>& g8,
                                           const Eight<TYPE>& u8, bool in, bool scaled, float r) {
  constexpr int kLanes = mx4_block(FMT) / 8;  // of one block
  const int lane = threadIdx.x & 31;
  float v[8], g[8], u[8];
  bool weak = false;
  float most;  // the block's largest magnitude (a NaN is)
  g8.values(g);
  if constexpr (!GATED && TYPE != kMx4F32) {
    // (of the stored patterns: the product with |r| keeps their order)
    uint32_t top = g8.top16();
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    most = Eight<TYPE>::of16(top);
    if (FMT == kE4M3 && scaled) most = fabsf(most * r);
  }
  if constexpr (GATED) {
    u8.values(u);
    float low = 1.f, gate = 0.f, tiny = 1.f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      gated32(v[i], v[i + 1], g[i], g[i + 1], u[i], u[i + 1]);
      low = min_abs3(low, v[i], v[i + 1]);
      if constexpr (TYPE == kMx4F32) tiny = min_abs3(tiny, g[i], g[i + 1]);
      gate = min3(gate, g[i], g[i + 1]);
      if constexpr (FMT == kE4M3) mul2(v[i], v[i + 1], r);
    }
    if (FMT == kE4M3) low = fminf(low, low * fabsf(r));
    if (low < 0x1p-100f || (TYPE == kMx4F32 && tiny < 0x1p-100f) || gate < -22.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) weak = weak || gated_weak<TYPE>(g[i], u[i], v[i], r);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = g[i];
    if (FMT == kE4M3 && scaled) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) mul2(v[i], v[i + 1], r);
    }
  }
  if constexpr (GATED || TYPE == kMx4F32) {
    most = max_abs(v[0], v[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) most = max_abs3(most, v[i], v[i + 1]);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1)
      most = max_abs(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  const uint32_t top = __float_as_uint(most);
  const bool bad = top >= 0x7f800000u;
  uint32_t byte;
  if constexpr (FMT == kE8M0)
    byte = bad ? 255u : (uint32_t)max((int)(top >> 23) - 2, 0);
  else
    byte = bad ? 0x7fu : __nv_cvt_float_to_fp8(sixth(most), __NV_SATFINITE, __NV_E4M3);
  if constexpr (GATED) {
    // next to a border between scales (a block of zeros is exact)
    const uint32_t over = FMT == kE8M0 ? above_short(most, 0) : above_short(sixth(most), 4);
    bool close = !bad && (weak || (top != 0 && over < 2 * kNear));
    if (__any_sync(0xffffffffu, close)) {
      // (a block's lanes go together; which of its values may be the largest is
      // certain from fp32 unless one is weak)
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) {
        const int other = __shfl_xor_sync(0xffffffffu, (close ? 1 : 0) | (weak ? 2 : 0), o);
        close = close || (other & 1);
        weak = weak || (other & 2);
      }
      double d = 0.0;
      if (close) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (weak || fabsf(v[i]) >= most * (1.f - 0x1p-16f))
            d = fmax(d, fabs(gated64(g[i], u[i], r)));
      }
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) d = fmax(d, __shfl_xor_sync(0xffffffffu, d, o));
      if (close) {
        if constexpr (FMT == kE8M0) {
          const int e = d > 0.0 ? ilogb(d) - 2 : -127;
          byte = (uint32_t)max(e + 127, 0);
        } else {
          byte = __nv_cvt_double_to_fp8(d / 6.0, __NV_SATFINITE, __NV_E4M3);
        }
      }
    }
  }
  float t[8];
  float inv, s = 0.f;
  if constexpr (FMT == kE8M0) {
    // 2^(127 - byte), byte at most 252: exact, as is the product where it matters
    inv = bad ? 0.f : __uint_as_float((254u - byte) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = v[i];
#pragma unroll
    for (int i = 0; i < 8; i += 2) mul2(t[i], t[i + 1], inv);
  } else {
    s = e4m3_value(byte);
    inv = s > 0.f ? rcp(s) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      t[i] = v[i], t[i + 1] = v[i + 1];
      mul2(t[i], t[i + 1], inv);
      // Borders m are numbers of three bits and s one of four, so m s has seven: v
      // is on it, or v / s at least .53 of m's last places away. t is off by four of
      // its last places; with the remainder, which is exact, it is off by 2^-20 of
      // one before it is rounded: on the border or on the right side of it. (An IEEE
      // quotient is too, but branches.)
      if constexpr (!GATED) {
        float r0 = v[i], r1 = v[i + 1];
        fma2(r0, r1, t[i], t[i + 1], -s);
        fma2(t[i], t[i + 1], r0, r1, inv);
      }
    }
  }
  uint32_t code = e2m1x8(t);
  if constexpr (GATED) {
    uint32_t over = kNear * 2;
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      over = __vimin3_u32(over, above_short(t[i], 2), above_short(t[i + 1], 2));
    if ((over < 2 * kNear || weak) && !bad) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (weak || (fabsf(t[i]) > 0.125f && above_short(t[i], 2) < 2 * kNear)) {
          double d = gated64(g[i], u[i], r);
          if constexpr (FMT == kE8M0) d = d * (double)inv;
          else d = s > 0.f ? d / (double)s : 0.0;
          code = (code & ~(15u << (4 * i))) | (e2m1_double(d) << (4 * i));
        }
      }
    }
  }
  if (bad) code = 0;
  if (out.codes && in) {
    *reinterpret_cast<uint32_t*>(out.codes + i_run * 128) = code;
    if (lane % kLanes == 0) out.scales[i_run * (256 / mx4_block(FMT))] = (uint8_t)byte;
  }
  if (out.rec) {
    *reinterpret_cast<uint32_t*>(out.rec + i_run * mx4_record_bytes(FMT)) = code;
    if (lane % kLanes == 0) out.rec_scale[i_run * mx4_record_bytes(FMT)] = (uint8_t)byte;
  }
}

}  // namespace egopq
