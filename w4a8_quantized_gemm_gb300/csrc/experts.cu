// experts.cu -- the gated linears of a mixture of experts on packed int4
// weights, for few rows an expert, and the row moves around the products.
//
//   out[t] = sum_j w[t,j] * D_e( silu(G_e x_t) * (U_e x_t) ),  e = ids[t,j]
//
// G, U and D are packed int4 weights s * (q - z) (group 128); activations are
// bf16 (W4A16) or per-token int8 codes (W4A8, h quantized again as bf16). Rows
// are sorted by expert (RowPlan), so that the rows of one expert share each
// weight byte that is read.
#include "egopq_internal.h"

namespace egopq {

// ---- products for few rows an expert --------------------------------------------
// One CTA takes 32 packed weight rows of one expert (16 gate and the 16 up
// rows of the same outputs, or 32 rows of the down projection) times up to
// 8 * NT rows of that expert; its warps split K by groups of 128 and add their
// sums through shared memory in warp order.
//
// The products run on mma.m16n8k16 with the weights as the 16-row operand. A
// thread of the fragment (row r = lane / 4, columns by lane % 4) reads the
// 16-byte unit of row r, chunk lane % 4 of a packed record: its 32 codes are
// the thread's operand of all eight K steps of the group, once K is taken in
// the order (step, lane % 4) -> 32 * (lane % 4) + 4 * step, which the
// activations follow with 64 contiguous bytes a thread. So weights and
// activations go from memory straight into fragments: no shared memory, no
// shuffles, every load 16 bytes. The group's sum is scaled in fp32.
constexpr int kStreamWarps = 8;

template <int VARIANT>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (VARIANT == kW4A8) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

struct StreamParams {
  const void* act;         // bf16 or int8 codes [rows][K]
  const float* a_s;        // scales of those rows (W4A8)
  const uint8_t* packed;   // [E] packed weights of N rows
  uint16_t* y;             // bf16 [sorted rows][out columns]
  const int* head;
  const int4* tiles;
  const int32_t* order;    // sorted position -> slot, when the rows are gathered
  int k;                   // slots a token (row = slot / k); 0: rows are sorted positions
  int N, G;
};

// 16 int8 codes as fp16 pairs, in order: code + 128 as a byte under 0x64 is the
// fp16 number 1024 + code + 128 (every step exact).
__device__ __forceinline__ void codes_to_f16(const uint4& v, uint32_t* o) {
  const __half2 bias = __float2half2_rn(1152.f);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t u = w[q] ^ 0x80808080u;
    const uint32_t lo = prmt(u, 0x64646464u, 0x4140), hi = prmt(u, 0x64646464u, 0x4342);
    const __half2 l2 = __hsub2(*reinterpret_cast<const __half2*>(&lo), bias);
    const __half2 h2 = __hsub2(*reinterpret_cast<const __half2*>(&hi), bias);
    o[q * 2] = *reinterpret_cast<const uint32_t*>(&l2);
    o[q * 2 + 1] = *reinterpret_cast<const uint32_t*>(&h2);
  }
}

// 32 activations of one row at K offset 32 * (lane % 4) of a group, as the
// B-operand words of the group's eight K steps (words 2s and 2s + 1 of step s).
template <int VARIANT>
__device__ __forceinline__ void load_act(const void* act, int64_t at, bool live, uint32_t (&b)[16]) {
  if constexpr (VARIANT == kW4A8) {
    uint4 v[2] = {};
    if (live) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const int8_t*>(act) + at);
      v[0] = __ldg(src);
      v[1] = __ldg(src + 1);
    }
    codes_to_f16(v[0], b);
    codes_to_f16(v[1], b + 8);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 v = {};
      if (live)
        v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(act) + at) + i);
      b[i * 4] = v.x;
      b[i * 4 + 1] = v.y;
      b[i * 4 + 2] = v.z;
      b[i * 4 + 3] = v.w;
    }
  }
}

template <int VARIANT, bool GATE_UP, int NT>
__global__ void __launch_bounds__(32 * kStreamWarps, NT == 1 ? 2 : 1)
experts_stream_kernel(const StreamParams p) {
  constexpr int W = kStreamWarps;
  constexpr int LD = 8 * NT + 1;  // padded row of the partial sums
  __shared__ float red[W][32 * LD];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  if ((int)blockIdx.x >= p.head[1]) return;
  const int4 tile = __ldg(p.tiles + blockIdx.x);
  const int rows = tile.z;
  if (rows == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int G = p.G, K = G * 128;
  const uint8_t* rec =
      p.packed + (((int64_t)tile.x * (p.N >> 7) + (blockIdx.y >> 2)) * G) * 8512;
  const int r0 = (blockIdx.y & 3) * 32 + gid;  // this thread's first row of the record
  int64_t row_at[NT];
  bool live[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int j = nt * 8 + gid;
    live[nt] = j < rows;
    int64_t row = tile.y + j;
    if (GATE_UP && live[nt]) row = __ldg(p.order + row) / p.k;
    row_at[nt] = row * K + 32 * tig;
  }
  float sum[2][NT][4];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int q = 0; q < 4; ++q) sum[mt][nt][q] = 0.f;

  uint4 w[4];        // units of rows r0, r0 + 8, r0 + 16, r0 + 24
  uint16_t sc[4];
  uint8_t zb[4];
  auto load_w = [&](int g) {
    const uint8_t* rg = rec + (int64_t)g * 8512;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = r0 + 8 * q;
      w[q] = __ldg(reinterpret_cast<const uint4*>(rg + (tig * 128 + r) * 16));
      sc[q] = __ldg(reinterpret_cast<const uint16_t*>(rg + 8192 + 2 * r));
      zb[q] = __ldg(rg + 8448 + (r >> 1));
    }
  };
  if (warp < G) load_w(warp);
  for (int g = warp; g < G; g += W) {
    uint4 cw[4];
    float s[4];
    uint32_t z[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      cw[q] = w[q];
      s[q] = f16_bits_to_f32(sc[q]);
      z[q] = (r0 & 1) ? (zb[q] >> 4) : (zb[q] & 0xF);  // (rows r0 + 8q: one parity)
    }
    if (g + W < G) load_w(g + W);
    uint32_t b[NT][16];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      load_act<VARIANT>(p.act, row_at[nt] + (int64_t)g * 128, live[nt], b[nt]);
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t lo[16], hi[16];
      cvt_w4_unit<VARIANT>(cw[2 * mt], z[2 * mt], lo);
      cvt_w4_unit<VARIANT>(cw[2 * mt + 1], z[2 * mt + 1], hi);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int st = 0; st < 8; ++st)
          mma_16816<VARIANT>(acc, lo[2 * st], hi[2 * st], lo[2 * st + 1], hi[2 * st + 1],
                             b[nt][2 * st], b[nt][2 * st + 1]);
        sum[mt][nt][0] = fmaf(s[2 * mt], acc[0], sum[mt][nt][0]);
        sum[mt][nt][1] = fmaf(s[2 * mt], acc[1], sum[mt][nt][1]);
        sum[mt][nt][2] = fmaf(s[2 * mt + 1], acc[2], sum[mt][nt][2]);
        sum[mt][nt][3] = fmaf(s[2 * mt + 1], acc[3], sum[mt][nt][3]);
      }
    }
  }
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[warp][(mt * 16 + (q >> 1) * 8 + gid) * LD + nt * 8 + tig * 2 + (q & 1)] =
            sum[mt][nt][q];
  __syncthreads();
  // (idle warps past G wrote zeros)
  if constexpr (GATE_UP) {
    const int I = p.N >> 1;
    for (int i = threadIdx.x; i < 16 * 8 * NT; i += 32 * W) {
      const int c = i & 15, j = i >> 4;
      if (j >= rows) break;
      float gate = 0.f, up = 0.f;
#pragma unroll
      for (int q = 0; q < W; ++q) {
        gate += red[q][c * LD + j];
        up += red[q][(16 + c) * LD + j];
      }
      if constexpr (VARIANT == kW4A8) {
        const float as = __ldg(p.a_s + __ldg(p.order + tile.y + j) / p.k);
        gate *= as;
        up *= as;
      }
      p.y[(int64_t)(tile.y + j) * I + blockIdx.y * 16 + c] = f32_to_bf16_bits(gated(gate, up));
    }
  } else {
    for (int i = threadIdx.x; i < 32 * 8 * NT; i += 32 * W) {
      const int c = i & 31, j = i >> 5;
      if (j >= rows) break;
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < W; ++q) v += red[q][c * LD + j];
      if constexpr (VARIANT == kW4A8) v *= __ldg(p.a_s + tile.y + j);
      p.y[(int64_t)(tile.y + j) * p.N + blockIdx.y * 32 + c] = f32_to_bf16_bits(v);
    }
  }
}

// ---- the picks' outputs summed -----------------------------------------------------
// out[t] = sum_j w[t,j] * y[pos[t,j]] in fp32, j in order; a dropped pick adds
// nothing. A thread holds eight columns.
constexpr int kCombineThreads = 128;

__global__ void __launch_bounds__(kCombineThreads)
combine_kernel(const uint16_t* __restrict__ y, const float* __restrict__ weights,
               const int32_t* __restrict__ pos, int k, int64_t H, uint16_t* __restrict__ out) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const int64_t v = (int64_t)blockIdx.y * kCombineThreads + threadIdx.x;
  if (v * 8 >= H) return;
  float acc[8] = {};
  for (int j = 0; j < k; ++j) {
    const int at = __ldg(pos + t * k + j);
    if (at < 0) continue;
    const float w = __ldg(weights + t * k + j);
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(y + (int64_t)at * H) + v);
    const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[2 * i] = fmaf(w, __uint_as_float(q[i] << 16), acc[2 * i]);
      acc[2 * i + 1] = fmaf(w, __uint_as_float(q[i] & 0xFFFF0000u), acc[2 * i + 1]);
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = (uint32_t)f32_to_bf16_bits(acc[2 * i]) |
           ((uint32_t)f32_to_bf16_bits(acc[2 * i + 1]) << 16);
  reinterpret_cast<uint4*>(out + t * H)[v] = make_uint4(o[0], o[1], o[2], o[3]);
}

// ---- rows in sorted order -----------------------------------------------------------
// rows[p] = x[order[p] / k] for the p that have an expert: bf16 as they are, or
// int8 codes as fp16 (and their scales). One CTA a row.
constexpr int kGatherThreads = 128;

template <bool CODES>
__global__ void __launch_bounds__(kGatherThreads)
gather_rows_kernel(const void* __restrict__ x, const float* __restrict__ x_s,
                   const int32_t* __restrict__ order, const int* __restrict__ head, int k,
                   int64_t H, uint16_t* __restrict__ rows, float* __restrict__ rows_s) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int64_t p = blockIdx.x;
  if (p >= head[0]) return;
  const int64_t t = __ldg(order + p) / k;
  uint4* dst = reinterpret_cast<uint4*>(rows + p * H);
  if constexpr (CODES) {
    if (threadIdx.x == 0) rows_s[p] = __ldg(x_s + t);
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const int8_t*>(x) + t * H);
    for (int64_t v = threadIdx.x; v < H / 16; v += kGatherThreads) {
      const uint4 c = __ldg(src + v);
      uint32_t o[8];
      codes_to_f16(c, o);
      dst[2 * v] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[2 * v + 1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  } else {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + t * H);
    for (int64_t v = threadIdx.x; v < H / 8; v += kGatherThreads) dst[v] = __ldg(src + v);
  }
}

// ---- launches -----------------------------------------------------------------------
template <int VARIANT, bool GATE_UP>
static cudaError_t launch_stream(const StreamParams& p, int64_t tiles, int bt, cudaStream_t st) {
  PdlConfig c(dim3((unsigned)tiles, (unsigned)(p.N / 32), 1), 32 * kStreamWarps, 0, st);
  switch (bt) {
    case 8: return cudaLaunchKernelEx(&c.cfg, experts_stream_kernel<VARIANT, GATE_UP, 1>, p);
    case 16: return cudaLaunchKernelEx(&c.cfg, experts_stream_kernel<VARIANT, GATE_UP, 2>, p);
    default: return cudaLaunchKernelEx(&c.cfg, experts_stream_kernel<VARIANT, GATE_UP, 4>, p);
  }
}

static cudaError_t launch_combine(const ExpertsArgs& a, cudaStream_t st) {
  PdlConfig c(dim3((unsigned)a.T, (unsigned)((a.H / 8 + kCombineThreads - 1) / kCombineThreads), 1),
              kCombineThreads, 0, st);
  return cudaLaunchKernelEx(&c.cfg, combine_kernel, (const uint16_t*)a.y, a.weights,
                            (const int32_t*)a.plan.pos, a.k, a.H, a.out);
}

// Many rows an expert: the rows in sorted order, then the tcgen05 products.
template <int VARIANT>
static cudaError_t run_experts_tensor(const ExpertsArgs& a, cudaStream_t st) {
  constexpr bool kCodes = VARIANT == kW4A8;
  const int64_t n = a.T * a.k;
  cudaError_t e = launch_plan(a.ids, n, a.E, 192, a.plan, st);
  if (e != cudaSuccess) return e;
  if (kCodes) {
    e = launch_quant_act(a.x, a.T, a.H, a.x_q, a.x_s, a.x_gsum, nullptr, st);
    if (e != cudaSuccess) return e;
  }
  PdlConfig c(dim3((unsigned)n, 1, 1), kGatherThreads, 0, st);
  e = cudaLaunchKernelEx(&c.cfg, gather_rows_kernel<kCodes>,
                         kCodes ? (const void*)a.x_q : (const void*)a.x, (const float*)a.x_s,
                         (const int32_t*)a.plan.order, (const int*)a.plan.head, a.k, a.H, a.rows,
                         a.rows_s);
  if (e != cudaSuccess) return e;
  RaggedArgs r{};
  r.variant = VARIANT;
  r.gate_up = true;
  r.rows_max = n;
  r.N = 2 * a.I;
  r.K = a.H;
  r.E = a.E;
  r.act = a.rows;
  r.a_s = a.rows_s;
  r.packed = a.gate_up;
  r.y = a.h;
  r.plan = a.plan;
  r.timeout_ns = a.timeout_ns;
  if ((e = launch_ragged(r, st)) != cudaSuccess) return e;
  if (kCodes) {
    // (rows past the last one that has an expert are quantized too: nothing
    // reads them)
    e = launch_quant_act(a.h, experts_rows(n), a.I, nullptr, a.h_s, a.h_gsum, a.h_tc, st);
    if (e != cudaSuccess) return e;
  }
  r.gate_up = false;
  r.N = a.H;
  r.K = a.I;
  r.act = kCodes ? a.h_tc : (const void*)a.h;
  r.a_s = a.h_s;
  r.packed = a.down;
  r.y = a.y;
  if ((e = launch_ragged(r, st)) != cudaSuccess) return e;
  return launch_combine(a, st);
}

template <int VARIANT>
static cudaError_t run_experts(const ExpertsArgs& a, cudaStream_t st) {
  if (a.tensor) return run_experts_tensor<VARIANT>(a, st);
  constexpr bool kCodes = VARIANT == kW4A8;
  const int64_t n = a.T * a.k;
  // rows of a tile: a token picks an expert once as a rule, so hardly an expert
  // has more than T (one that has takes several tiles)
  const int bt = a.T <= 8 ? 8 : (a.T <= 16 ? 16 : 32);
  const int64_t tiles = plan_max_tiles(n, a.E, bt);
  cudaError_t e = launch_plan(a.ids, n, a.E, bt, a.plan, st);
  if (e != cudaSuccess) return e;
  if (kCodes) {
    e = launch_quant_act(a.x, a.T, a.H, a.x_q, a.x_s, a.x_gsum, nullptr, st);
    if (e != cudaSuccess) return e;
  }
  StreamParams p;
  p.act = kCodes ? (const void*)a.x_q : (const void*)a.x;
  p.a_s = a.x_s;
  p.packed = a.gate_up;
  p.y = a.h;
  p.head = a.plan.head;
  p.tiles = a.plan.tiles;
  p.order = a.plan.order;
  p.k = a.k;
  p.N = (int)(2 * a.I);
  p.G = (int)(a.H / 128);
  if ((e = launch_stream<VARIANT, true>(p, tiles, bt, st)) != cudaSuccess) return e;
  if (kCodes) {
    // (rows past the last one that has an expert are quantized too: nothing
    // reads them)
    e = launch_quant_act(a.h, n, a.I, a.h_q, a.h_s, a.h_gsum, nullptr, st);
    if (e != cudaSuccess) return e;
  }
  p.act = kCodes ? (const void*)a.h_q : (const void*)a.h;
  p.a_s = a.h_s;
  p.packed = a.down;
  p.y = a.y;
  p.k = 0;
  p.N = (int)a.H;
  p.G = (int)(a.I / 128);
  if ((e = launch_stream<VARIANT, false>(p, tiles, bt, st)) != cudaSuccess) return e;
  return launch_combine(a, st);
}

cudaError_t launch_experts(const ExpertsArgs& a, cudaStream_t st) {
  return a.variant == kW4A8 ? run_experts<kW4A8>(a, st) : run_experts<kW4A16>(a, st);
}

}  // namespace egopq
