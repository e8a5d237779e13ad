// mx4_quant.cu -- rows to microscaled 4-bit values and back, and weights in and
// out of their packed records. The formats and the records: mx4_internal.h.
#include "mx4_quant.cuh"

namespace egopq {

namespace {

constexpr int kQuantWarps = 4;

struct QuantParams {
  const void* x;
  const float* tensor_scale;
  const int32_t* offsets;
  const int32_t* index;
  uint8_t* codes;
  uint8_t* scales;
  uint8_t* operand;
  int64_t M, K, x_rows;
  int sets, kb, groups;  // K blocks of a row, and runs of U of them
};

// A warp takes U runs of 256 values of a row: eight values a lane, so that a block
// of 32 (16) is four (two) neighbours and a row's 128 bytes of codes leave as one
// line. All of a warp's loads are on their way before the first is used; few rows take
// U = 1, so that more warps share them. Measured: 4093 x 18944 bf16 to E8M0 36.5 us (5.4
// TB/s), to E4M3 44.7, gated 1021 x 18944 23.4 and 26.7. Nothing is full: captured on
// 4093 x 18944 fp16 and on the gated rows (E8M0 / E4M3 each), a scheduler issues in 69 and
// 67 % of its active cycles, memory runs at 53 / 41 and 36 / 34 % of its peak, the ALUs at
// 62 / 55 and 54 / 50. With seven warps a scheduler an instruction waits ten cycles, 1.5 to
// 2.7 of them for loads and two for the one before it.
// EARLY: the next kernel may begin at once; else not before every block's stores are
// performed (a variant of its own: the fence in the same one costs those without it 2 %).
template <int FMT, int TYPE, bool GATED, int U, bool EARLY>
__global__ void __launch_bounds__(kQuantWarps * 32, GATED ? 8 : 9) mx4_quant_kernel(const QuantParams p) {
  extern __shared__ int quant_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  if (EARLY && threadIdx.x == 0) griddep_launch_dependents();
  int *first = nullptr, *block = nullptr;
  int64_t row = 0, rows_end = p.M;
  if (p.offsets) {
    first = quant_smem;
    block = first + p.sets + 1;
    if (warp == 0) mx4_scan_sets(p.offsets, p.sets, p.M, 128, first, block, nullptr);
    __syncthreads();
    row = first[0];
    rows_end = first[p.sets];
  }
  const bool scaled = p.tensor_scale != nullptr;
  const float r = scaled ? __fdiv_rn(1.f, __ldg(p.tensor_scale)) : 1.f;
  const int64_t ld = GATED ? 2 * p.K : p.K;
  constexpr int kLanes = mx4_block(FMT) / 8;
  // this warp's runs: every `stride`-th, counted along the rows
  const int64_t at0 = (int64_t)blockIdx.x * kQuantWarps + warp;
  const int64_t stride = (int64_t)gridDim.x * kQuantWarps;
  const int64_t row_step = stride / p.groups;
  const int group_step = (int)(stride - row_step * p.groups);
  row += at0 / p.groups;
  int group = (int)(at0 % p.groups);
  while (row < rows_end) {
    int64_t src = row;
    if (p.index) src = __ldg(p.index + row);
    const bool have = src >= 0 && src < p.x_rows;
    Eight<TYPE> g8[U], u8[GATED ? U : 1];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t k = (int64_t)(group * U + i) * 256 + lane * 8;
      g8[i].zero();
      if constexpr (GATED) u8[i].zero();
      if (have && k < p.K) {
        g8[i].load(p.x, src * ld + k);
        if constexpr (GATED) u8[i].load(p.x, src * ld + p.K + k);
      }
    }
    RowOut out{};
    if (p.codes) {
      out.codes = p.codes + row * (p.K / 2) + group * U * 128 + lane * 4;
      out.scales = p.scales + row * (p.K / mx4_block(FMT)) +
                   group * U * (256 / mx4_block(FMT)) + lane / kLanes;
    }
    if (p.operand) {
      int64_t at = row;  // among the operand's rows
      if (p.offsets) {
        const int e = mx4_find_set(first, p.sets, (int)row);
        at = (int64_t)block[e] * 128 + (row - first[e]);
      }
      uint8_t* rec = p.operand + ((at >> 7) * p.kb + group * U) * mx4_record_bytes(FMT);
      const int q = (int)(at & 127), b = lane / kLanes;
      out.rec = rec + q * 128 + ((((lane >> 2) ^ q) & 7) << 4) + (lane & 3) * 4;
      out.rec_scale = rec + kMx4Codes + (b >> 2) * 512 + (q & 31) * 16 + (q >> 5) * 4 + (b & 3);
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (U == 1 || group * U + i < p.kb)
        quant_unit<FMT, TYPE, GATED>(out, i, g8[i], u8[GATED ? i : 0],
                                     (int64_t)(group * U + i) * 256 + lane * 8 < p.K, scaled, r);
    row += row_step;
    group += group_step;
    if (group >= p.groups) {
      group -= p.groups;
      ++row;
    }
  }
  if (!EARLY) __threadfence();  // (a block's end lets the next kernel begin)
}

template <int FMT, int TYPE, bool GATED, int U, bool EARLY>
cudaError_t launch_quant_u(const Mx4QuantArgs& a, int sms, cudaStream_t st) {
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
  p.groups = (p.kb + U - 1) / U;
  const int64_t blocks = (a.M * p.groups + kQuantWarps - 1) / kQuantWarps;
  // as many as are on the SMs at a time: a second round of blocks that takes as long
  // as the first would leave them half empty
  static std::atomic<int> held{0};
  int per_sm = held.load(std::memory_order_relaxed);
  if (per_sm < 1) {
    if (cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
            &per_sm, mx4_quant_kernel<FMT, TYPE, GATED, U, EARLY>, kQuantWarps * 32, 0);
        e != cudaSuccess)
      return e;
    held.store(per_sm < 1 ? 1 : per_sm, std::memory_order_relaxed);
    if (per_sm < 1) per_sm = 1;
  }
  const int64_t most = (int64_t)sms * per_sm;
  const size_t smem = a.offsets ? 2 * (size_t)(a.sets + 1) * sizeof(int) : 0;
  PdlConfig c(dim3((unsigned)(blocks < most ? blocks : most), 1, 1), kQuantWarps * 32, smem, st);
  return cudaLaunchKernelEx(&c.cfg, mx4_quant_kernel<FMT, TYPE, GATED, U, EARLY>, p);
}

template <int FMT, int TYPE, bool GATED>
cudaError_t launch_quant(const Mx4QuantArgs& a, cudaStream_t st) {
  constexpr int kMany = GATED || TYPE == kMx4F32 ? 2 : 4;
  const int sms = device_sm_count();
  if (sms < 1) return cudaErrorInvalidConfiguration;
  if (a.M * mx4_kblocks(a.K) <= (int64_t)sms * 96)
    return a.early ? launch_quant_u<FMT, TYPE, GATED, 1, true>(a, sms, st)
                   : launch_quant_u<FMT, TYPE, GATED, 1, false>(a, sms, st);
  return a.early ? launch_quant_u<FMT, TYPE, GATED, kMany, true>(a, sms, st)
                 : launch_quant_u<FMT, TYPE, GATED, kMany, false>(a, sms, st);
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

// ---- rows gathered in 4 bits ---------------------------------------------------------
// Ragged rows that are gathered from fewer: each was quantized once, and this moves
// codes and scales to their places among the records. A warp takes a row, sixteen K
// blocks at a time, 16 bytes a lane and four of them on their way; memory (L2, as to
// what is read) bounds it: 32768 rows of 3584 from 4096 take about 19 us.
template <int FMT>
__global__ void __launch_bounds__(256) mx4_gather_kernel(const QuantParams p) {
  extern __shared__ int quant_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  int *first = quant_smem, *block = first + p.sets + 1;
  if (warp == 0) mx4_scan_sets(p.offsets, p.sets, p.M, 128, first, block, nullptr);
  __syncthreads();
  constexpr int kPer = 256 / mx4_block(FMT), kWords = kPer / 4;  // scales of a K block
  constexpr int kRec = mx4_record_bytes(FMT);
  const int rows_end = first[p.sets], blocks = (int)(p.K / mx4_block(FMT));
  const int chunk = lane & 7, word = lane % kWords;
  for (int64_t row = first[0] + (int64_t)blockIdx.x * 8 + warp; row < rows_end;
       row += (int64_t)gridDim.x * 8) {
    const int64_t src = __ldg(p.index + row);
    const bool have = src >= 0 && src < p.x_rows;
    const int e = mx4_find_set(first, p.sets, (int)row);
    const int64_t at = (int64_t)block[e] * 128 + (row - first[e]);
    const int q = (int)(at & 127);
    uint8_t* rec = p.operand + (at >> 7) * p.kb * kRec;
    const uint8_t* codes = p.codes + src * (p.K / 2);
    const uint8_t* scales = p.scales + src * blocks;
    for (int kb0 = 0; kb0 < p.kb; kb0 += 16) {
      uint4 c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int kb = kb0 + 4 * j + (lane >> 3);
        c[j] = make_uint4(0, 0, 0, 0);
        if (have && (int64_t)kb * 256 + chunk * 32 < p.K)
          c[j] = *reinterpret_cast<const uint4*>(codes + kb * 128 + chunk * 16);
      }
      // a lane's words of four scales: of 32 / kWords K blocks at a time
      uint32_t w[kWords / 2];
#pragma unroll
      for (int j = 0; j < kWords / 2; ++j) {
        const int b = (kb0 + j * (32 / kWords) + lane / kWords) * kPer + word * 4;
        w[j] = 0;
        if (have) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (b + i < blocks) w[j] |= (uint32_t)scales[b + i] << (8 * i);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int kb = kb0 + 4 * j + (lane >> 3);
        if (kb < p.kb)
          *reinterpret_cast<uint4*>(rec + (int64_t)kb * kRec + q * 128 + ((chunk ^ q) & 7) * 16) =
              c[j];
      }
#pragma unroll
      for (int j = 0; j < kWords / 2; ++j) {
        const int kb = kb0 + j * (32 / kWords) + lane / kWords;
        if (kb < p.kb)
          *reinterpret_cast<uint32_t*>(rec + (int64_t)kb * kRec + kMx4Codes + word * 512 +
                                       (q & 31) * 16 + (q >> 5) * 4) = w[j];
      }
    }
  }
}

template <int FMT>
cudaError_t launch_gather(const Mx4QuantArgs& a, cudaStream_t st) {
  QuantParams p{};
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
  const int64_t blocks = (a.M + 7) / 8, most = (int64_t)sms * 8;
  PdlConfig c(dim3((unsigned)(blocks < most ? blocks : most), 1, 1), 256,
              2 * (size_t)(a.sets + 1) * sizeof(int), st);
  return cudaLaunchKernelEx(&c.cfg, mx4_gather_kernel<FMT>, p);
}

// ---- values back ------------------------------------------------------------------
// Eight values a thread and step, four steps' codes on their way at a time; the
// code times its block's scale is exact in fp32. Bound by memory: 4093 x 18944 to fp16
// takes 30 us, a copy's rate.
template <int FMT, int TYPE>
__device__ __forceinline__ void dequant8(uint32_t c, uint32_t byte, bool scaled, float g, void* y,
                                         int64_t i) {
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
  if (scaled) {
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

constexpr int kDequantSteps = 4;

template <int FMT, int TYPE>
__global__ void __launch_bounds__(256) mx4_dequant_kernel(const uint8_t* codes,
                                                          const uint8_t* scales, int64_t n,
                                                          const float* tensor_scale, void* y) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const bool scaled = tensor_scale != nullptr;
  const float g = scaled ? __ldg(tensor_scale) : 1.f;
  constexpr int kPer = mx4_block(FMT) / 8;
  for (int64_t i0 = (int64_t)blockIdx.x * 256 * kDequantSteps + threadIdx.x; i0 < n;
       i0 += (int64_t)gridDim.x * 256 * kDequantSteps) {
    uint32_t c[kDequantSteps], b[kDequantSteps];
#pragma unroll
    for (int q = 0; q < kDequantSteps; ++q) {
      const int64_t i = i0 + q * 256;
      c[q] = b[q] = 0;
      if (i < n) {
        c[q] = __ldcs(reinterpret_cast<const uint32_t*>(codes) + i);
        b[q] = __ldg(scales + i / kPer);
      }
    }
#pragma unroll
    for (int q = 0; q < kDequantSteps; ++q) {
      const int64_t i = i0 + q * 256;
      if (i < n) dequant8<FMT, TYPE>(c[q], b[q], scaled, g, y, i);
    }
  }
}

template <int FMT>
cudaError_t launch_dequant_type(const uint8_t* codes, const uint8_t* scales, int64_t n,
                                const float* ts, int type, void* y, cudaStream_t st) {
  const int sms = device_sm_count();
  if (sms < 1) return cudaErrorInvalidConfiguration;
  const int64_t per = 256 * kDequantSteps, blocks = (n + per - 1) / per, most = (int64_t)sms * 8;
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
// A warp moves the 128 bytes of codes and the scales of one row and K block (once a
// weight: 18944 x 3584 takes 72 us).
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
  __threadfence();  // (a block's end lets the next kernel begin)
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

cudaError_t launch_mx4_gather(const Mx4QuantArgs& a, cudaStream_t st) {
  return a.format == kE8M0 ? launch_gather<kE8M0>(a, st) : launch_gather<kE4M3>(a, st);
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
