// mx4_quant.cu -- rows to microscaled 4-bit values and back, and weights in and
// out of their packed records. The formats and the records: mx4_internal.h.
#include <cuda_fp8.h>

#include "mx4_internal.h"

namespace egopq {

namespace {

constexpr int kE8M0 = EGOPQ_MX4_E8M0, kE4M3 = EGOPQ_MX4_E4M3;
constexpr int kQuantWarps = 4;

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

// Eight values of a row at p, as fp32.
template <int TYPE>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
  if constexpr (TYPE == kMx4F32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = __ldcs(q), b = __ldcs(q + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == kMx4Bf16) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
}

// ---- gated values -----------------------------------------------------------------
// h = silu(g) * u * r in fp32: the exponential is within 2 of its last places, the
// sum, the quotient and the products within half of one each, 2^-21 together. The
// codes are those of the real h: where fp32 lies within 2^-20 of a border (and
// where h is so small that fp32 has fewer bits), 64 bits decide.
// `weak`: a value for which that does not hold, as fp32 has run out of exponents
// on the way (zeros are exact).
__device__ __forceinline__ float gated32(float g, float u, float r, bool& weak) {
  const float h = __fdiv_rn(g, 1.f + expf(-g)) * u, v = h * r;
  weak = weak || (g != 0.f && u != 0.f &&
                  (g < -80.f || fabsf(h) < 0x1p-100f || fabsf(v) < 0x1p-100f));
  return v;
}
__device__ __forceinline__ double gated64(float g, float u, float r) {
  return (double)g / (1.0 + exp(-(double)g)) * (double)u * (double)r;
}
// Whether the positive number v lies within 8 of its last places of a number
// whose lowest mantissa bit is 2^-keep: every border between codes is one.
__device__ __forceinline__ bool near_short(float v, int keep) {
  const uint32_t low = (1u << (23 - keep)) - 1;
  return ((__float_as_uint(v) + 8u) & low) < 16u;
}

struct QuantParams {
  const void* x;
  const float* tensor_scale;
  const int32_t* offsets;
  const int32_t* index;
  uint8_t* codes;
  uint8_t* scales;
  uint8_t* operand;
  int64_t M, K, x_rows;
  int sets, kb;
};

// A warp takes 256 values of a row: eight a lane, so that a block of 32 (16) is
// four (two) neighbours and a row's 128 bytes of codes leave as one line. Bound
// by memory: 16 bytes a lane are on their way at a time, and the units of
// many rows keep enough warps on an SM to cover them.
template <int FMT, int TYPE, bool GATED>
__global__ void __launch_bounds__(kQuantWarps * 32) mx4_quant_kernel(const QuantParams p) {
  extern __shared__ int quant_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  int *first = nullptr, *block = nullptr;
  int64_t row0 = 0, rows = p.M;
  if (p.offsets) {
    first = quant_smem;
    block = first + p.sets + 1;
    if (warp == 0) mx4_scan_sets(p.offsets, p.sets, p.M, first, block);
    __syncthreads();
    row0 = first[0];
    rows = first[p.sets] - row0;
  }
  const float r = p.tensor_scale ? __fdiv_rn(1.f, __ldg(p.tensor_scale)) : 1.f;
  constexpr int kLanes = mx4_block(FMT) / 8;  // of one block
  const int64_t ld = GATED ? 2 * p.K : p.K;
  const int64_t units = rows * p.kb;
  for (int64_t w = (int64_t)blockIdx.x * kQuantWarps + warp; w < units;
       w += (int64_t)gridDim.x * kQuantWarps) {
    const int64_t row = row0 + w / p.kb;
    const int kb = (int)(w % p.kb);
    const int64_t k = (int64_t)kb * 256 + lane * 8;
    const bool in = k < p.K;
    int64_t src = row;
    if (p.index) src = __ldg(p.index + row);
    const bool have = in && src >= 0 && src < p.x_rows;
    float v[8], g[8], u[8];
    bool weak = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = g[i] = u[i] = 0.f;
    if (have) {
      if constexpr (GATED) {
        load8<TYPE>(p.x, src * ld + k, g);
        load8<TYPE>(p.x, src * ld + p.K + k, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = gated32(g[i], u[i], r, weak);
      } else {
        load8<TYPE>(p.x, src * ld + k, v);
        if (p.tensor_scale) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= r;
        }
      }
    }
    // the block's largest magnitude, as bits (NaN above infinity above all)
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool bad = top >= 0x7f800000u;
    // FMT's scale of a largest value, as its byte
    uint32_t byte;
    if constexpr (FMT == kE8M0) {
      byte = bad ? 255u : (uint32_t)max((int)(top >> 23) - 2, 0);
    } else {
      const float q = __fdiv_rn(__uint_as_float(top), 6.f);
      byte = bad ? 0x7fu : __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
    }
    if constexpr (GATED) {
      const float a = __uint_as_float(top);
      bool close = !bad && (weak || (FMT == kE8M0 ? near_short(a, 0)
                                                  : near_short(__fdiv_rn(a, 6.f), 4)));
      if (__any_sync(0xffffffffu, close)) {
        // every lane of a block comes along where one does: the shuffles are the
        // warp's, and what they bring to the other blocks is not used
        double d = 0.0;
        if (!bad && have) {
#pragma unroll 1
          for (int i = 0; i < 8; ++i) d = fmax(d, fabs(gated64(g[i], u[i], r)));
        }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) {
          d = fmax(d, __shfl_xor_sync(0xffffffffu, d, o));
          // (one mask for both: no lane leaves a shuffle out)
          const int other = __shfl_xor_sync(0xffffffffu, (close ? 1 : 0) | (weak ? 2 : 0), o);
          close = close || (other & 1);
          weak = weak || (other & 2);
        }
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
    float inv = 0.f, s = 0.f;
    if constexpr (FMT == kE8M0) {
      // 2^(127 - byte), byte at most 252: exact, as is the product where it matters
      inv = bad ? 0.f : __uint_as_float((254u - byte) << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = v[i] * inv;
    } else {
      // fp32's quotient is on the same side of a border (numbers of at most six
      // bits, times s) as the real one
      s = e4m3_value(byte);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = s > 0.f ? __fdiv_rn(v[i], s) : 0.f;
    }
    uint32_t code = e2m1x8(t);
    if constexpr (GATED) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = fabsf(t[i]);
        if (!bad && (weak || (a > 0.125f && near_short(a, 2)))) {
          double d = gated64(g[i], u[i], r);
          if constexpr (FMT == kE8M0) d = d * (double)inv;
          else d = s > 0.f ? d / (double)s : 0.0;
          code = (code & ~(15u << (4 * i))) | (e2m1_double(d) << (4 * i));
        }
      }
    }
    if (bad) code = 0;
    if (p.codes && in) {
      *reinterpret_cast<uint32_t*>(p.codes + row * (p.K / 2) + k / 2) = code;
      if (lane % kLanes == 0)
        p.scales[row * (p.K / mx4_block(FMT)) + k / mx4_block(FMT)] = (uint8_t)byte;
    }
    if (p.operand) {
      int64_t at = row;  // among the operand's rows
      if (p.offsets) {
        const int e = mx4_find_set(first, p.sets, (int)row);
        at = (int64_t)block[e] * 128 + (row - first[e]);
      }
      uint8_t* rec = p.operand + ((at >> 7) * p.kb + kb) * mx4_record_bytes(FMT);
      const int q = (int)(at & 127);
      *reinterpret_cast<uint32_t*>(rec + q * 128 + ((((lane >> 2) ^ q) & 7) << 4) + (lane & 3) * 4) =
          code;
      if (lane % kLanes == 0) {
        const int b = lane / kLanes;
        rec[kMx4Codes + (b >> 2) * 512 + (q & 31) * 16 + (q >> 5) * 4 + (b & 3)] = (uint8_t)byte;
      }
    }
  }
}

template <int FMT, int TYPE, bool GATED>
cudaError_t launch_quant(const Mx4QuantArgs& a, cudaStream_t st) {
  QuantParams p;
  p.x = a.x;
  p.tensor_scale = a.tensor_scale;
  p.offsets = a.offsets;
  p.index = a.index;
  p.codes = a.codes;
  p.scales = a.scales;
  p.operand = a.operand;
  p.M = a.M;
  p.K = a.K;
  p.x_rows = a.x_rows;
  p.sets = a.sets;
  p.kb = (int)mx4_kblocks(a.K);
  const int sms = device_sm_count();
  if (sms < 1) return cudaErrorInvalidConfiguration;
  const int64_t blocks = (a.M * p.kb + kQuantWarps - 1) / kQuantWarps;
  const int64_t most = (int64_t)sms * 16;
  const size_t smem = a.offsets ? 2 * (size_t)(a.sets + 1) * sizeof(int) : 0;
  PdlConfig c(dim3((unsigned)(blocks < most ? blocks : most), 1, 1), kQuantWarps * 32, smem, st);
  return cudaLaunchKernelEx(&c.cfg, mx4_quant_kernel<FMT, TYPE, GATED>, p);
}

template <int FMT>
cudaError_t launch_quant_type(const Mx4QuantArgs& a, cudaStream_t st) {
  switch (a.type) {
    case kMx4Bf16:
      return a.gated ? launch_quant<FMT, kMx4Bf16, true>(a, st)
                     : launch_quant<FMT, kMx4Bf16, false>(a, st);
    case kMx4F16:
      return a.gated ? launch_quant<FMT, kMx4F16, true>(a, st)
                     : launch_quant<FMT, kMx4F16, false>(a, st);
    default:
      return a.gated ? launch_quant<FMT, kMx4F32, true>(a, st)
                     : launch_quant<FMT, kMx4F32, false>(a, st);
  }
}

// ---- values back ------------------------------------------------------------------
// Eight values a thread; the code times its block's scale is exact in fp32.
template <int FMT, int TYPE>
__global__ void __launch_bounds__(256) mx4_dequant_kernel(const uint8_t* codes,
                                                          const uint8_t* scales, int64_t n,
                                                          const float* tensor_scale, void* y) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const float g = tensor_scale ? __ldg(tensor_scale) : 1.f;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x) {
    const uint32_t c = reinterpret_cast<const uint32_t*>(codes)[i];
    const uint32_t byte = scales[i / (mx4_block(FMT) / 8)];
    const float s = FMT == kE8M0 ? e8m0_value(byte) : e4m3_value(byte);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t h;
      asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
          "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
          : "=r"(h)
          : "r"(c >> (8 * j)));
      const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
      v[2 * j] = f.x * s;
      v[2 * j + 1] = f.y * s;
    }
    if (tensor_scale) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= g;
    }
    if constexpr (TYPE == kMx4F32) {
      float4* o = static_cast<float4*>(y) + 2 * i;
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (TYPE == kMx4Bf16) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
          w[j] = *reinterpret_cast<const uint32_t*>(&b);
        } else {
          const __half2 b = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
          w[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
      }
      static_cast<uint4*>(y)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <int FMT>
cudaError_t launch_dequant_type(const uint8_t* codes, const uint8_t* scales, int64_t n,
                                const float* ts, int type, void* y, cudaStream_t st) {
  const int sms = device_sm_count();
  if (sms < 1) return cudaErrorInvalidConfiguration;
  const int64_t blocks = (n + 255) / 256, most = (int64_t)sms * 8;
  PdlConfig c(dim3((unsigned)(blocks < most ? blocks : most), 1, 1), 256, 0, st);
  switch (type) {
    case kMx4Bf16:
      return cudaLaunchKernelEx(&c.cfg, mx4_dequant_kernel<FMT, kMx4Bf16>, codes, scales, n, ts, y);
    case kMx4F16:
      return cudaLaunchKernelEx(&c.cfg, mx4_dequant_kernel<FMT, kMx4F16>, codes, scales, n, ts, y);
    default:
      return cudaLaunchKernelEx(&c.cfg, mx4_dequant_kernel<FMT, kMx4F32>, codes, scales, n, ts, y);
  }
}

// ---- weights in and out of their records ---------------------------------------------
// A warp moves the 128 bytes of codes and the scales of one row and K block.
// Rows past N and values past K are zeros (in memory that the products read). No
// early launch here: a product may read a weight before its own wait.
template <int FMT, bool PACK>
__global__ void __launch_bounds__(256) mx4_pack_kernel(uint8_t* codes, uint8_t* scales, int64_t sets,
                                                       int64_t N, int64_t K, int64_t kb_n,
                                                       uint8_t* packed) {
  constexpr int kPer = 256 / mx4_block(FMT);  // scales of a row and K block
  const int lane = threadIdx.x & 31;
  const int64_t nb_n = (N + 127) / 128;
  const int64_t units = sets * nb_n * 128 * kb_n;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < units;
       w += (int64_t)gridDim.x * 8) {
    const int64_t kb = w % kb_n, rest = w / kb_n;
    const int q = (int)(rest & 127);
    const int64_t rb = rest >> 7;  // row block over all sets
    const int64_t set = rb / nb_n, n = (rb % nb_n) * 128 + q;
    uint8_t* rec = packed + (rb * kb_n + kb) * mx4_record_bytes(FMT);
    uint32_t* at = reinterpret_cast<uint32_t*>(rec + q * 128 + ((((lane >> 2) ^ q) & 7) << 4) +
                                               (lane & 3) * 4);
    const int64_t k = kb * 256 + lane * 8, row = set * N + n;
    uint32_t* plain = reinterpret_cast<uint32_t*>(codes + row * (K / 2) + k / 2);
    const bool in = n < N && k < K;
    if constexpr (PACK) *at = in ? *plain : 0u;
    else if (in) *plain = *at;
    if (lane < kPer) {
      uint8_t* sc = rec + kMx4Codes + (lane >> 2) * 512 + (q & 31) * 16 + (q >> 5) * 4 + (lane & 3);
      const int64_t b = kb * kPer + lane, blocks = K / mx4_block(FMT);
      const bool have = n < N && b < blocks;
      if constexpr (PACK) *sc = have ? scales[row * blocks + b] : (uint8_t)0;
      else if (have) scales[row * blocks + b] = *sc;
    }
  }
}

template <bool PACK>
cudaError_t launch_records(uint8_t* codes, uint8_t* scales, int64_t sets, int64_t N, int64_t K,
                           int format, uint8_t* packed, cudaStream_t st) {
  const int sms = device_sm_count();
  if (sms < 1) return cudaErrorInvalidConfiguration;
  const int64_t kb = mx4_kblocks(K), units = sets * ((N + 127) / 128) * 128 * kb;
  const int64_t blocks = (units + 7) / 8, most = (int64_t)sms * 8;
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  if (format == kE8M0)
    mx4_pack_kernel<kE8M0, PACK><<<grid, 256, 0, st>>>(codes, scales, sets, N, K, kb, packed);
  else
    mx4_pack_kernel<kE4M3, PACK><<<grid, 256, 0, st>>>(codes, scales, sets, N, K, kb, packed);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx4_quant(const Mx4QuantArgs& a, cudaStream_t st) {
  return a.format == kE8M0 ? launch_quant_type<kE8M0>(a, st) : launch_quant_type<kE4M3>(a, st);
}

cudaError_t launch_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K,
                               int format, const float* tensor_scale, int type, void* y,
                               cudaStream_t st) {
  const int64_t n = M * K / 8;
  return format == kE8M0 ? launch_dequant_type<kE8M0>(codes, scales, n, tensor_scale, type, y, st)
                         : launch_dequant_type<kE4M3>(codes, scales, n, tensor_scale, type, y, st);
}

cudaError_t launch_mx4_pack(const uint8_t* codes, const uint8_t* scales, int64_t sets, int64_t N,
                            int64_t K, int format, void* packed, cudaStream_t st) {
  return launch_records<true>(const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales), sets, N, K,
                              format, static_cast<uint8_t*>(packed), st);
}

cudaError_t launch_mx4_unpack(const void* packed, int64_t sets, int64_t N, int64_t K, int format,
                              uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  return launch_records<false>(codes, scales, sets, N, K, format,
                               static_cast<uint8_t*>(const_cast<void*>(packed)), st);
}

}  // namespace egopq
