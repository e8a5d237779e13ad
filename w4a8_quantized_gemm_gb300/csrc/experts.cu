// experts.cu -- the gated linears of a mixture of experts on packed int4
// weights: the products for few rows an expert, and the row moves and sums
// around the products.
//
//   out[t] = sum_j w[t,j] * D_e( silu(G_e x_t) * (U_e x_t) ),  e = ids[t,j]
//
// G, U and D are packed int4 weights s * (q - z) (group 128); activations are
// bf16 (W4A16) or per-token int8 codes (W4A8, h quantized again as bf16).
//
// Three ways, by the number of rows an expert has (experts_way):
//   few     up to 8 tokens: the matrix instruction's 8 columns are the tokens
//           themselves, every CTA finds the picked experts in the ids alone,
//           and the down product sums over the experts in registers: no plan,
//           no per-pick output
//   stream  rows sorted by expert (RowPlan), tiles of up to 32 rows of one
//   tensor  the tcgen05 products of tc_experts.cu over sorted rows
#include "egopq_internal.h"

namespace egopq {

// ---- products for few rows an expert --------------------------------------------
// A warp takes 32 packed weight rows of one expert (16 gate and the 16 up rows
// of the same outputs, or 32 rows of the down projection) times up to 8 * NT
// rows, over every W-th group of K; the CTA's W warps add their sums through
// shared memory in warp order.
//
// The products run on mma.m16n8k16 with the weights as the 16-row operand. A
// thread of the fragment (row r = lane / 4, columns by lane % 4) reads the
// 16-byte unit of row r, chunk lane % 4 of a packed record: its 32 codes are
// the thread's operand of all eight K steps of the group, once K is taken in
// the order (step, lane % 4) -> 32 * (lane % 4) + 4 * step, which the
// activations follow with 32 contiguous values a thread. So no shuffle and no
// transposition stands between memory and the matrix instruction.
//
// The weights stream from HBM once: each warp keeps kStages - 1 groups of its
// rows in flight (2.1 KB each) with cp.async into a ring of its own, which no
// other warp waits for. Bound by HBM where the rows are few; the conversion of
// the codes (about 2.5 instructions a pair) is next.
constexpr int kStages = 4;
constexpr int kStageBytes = 2176;  // 4 x 512 codes, 64 scales, 16 zero points, padding
constexpr int kWarps = 4;          // K parts of a CTA
constexpr int kFewWarps = 16;      // the few-token down product's
constexpr int kFewTokens = 8;
constexpr int kFewSlots = 128;     // picks of a few-token batch

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
  uint16_t* h;             // gate and up products: bf16 [sorted row or slot][N / 2]
  float* y;                // down product: fp32 [sorted row][N]
  uint16_t* out;           // few tokens, down product: bf16 [T][N]
  const int* head;         // plan
  const int4* tiles;
  const int32_t* order;
  const int32_t* ids;      // few tokens
  const float* weights;
  int T, k, E, N, G;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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

// 32 activations of one row as they lie in memory (two 16-byte vectors of
// codes, four of bf16), and as the B-operand words of a group's eight K steps.
template <int VARIANT>
struct ActRaw {
  static constexpr int kVec = VARIANT == kW4A8 ? 2 : 4;
  uint4 v[kVec];
  __device__ __forceinline__ void load(const void* act, int64_t at, bool live) {
    const uint8_t* src = static_cast<const uint8_t*>(act) + at * (VARIANT == kW4A8 ? 1 : 2);
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      v[i] = live ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void words(uint32_t (&b)[16]) const {
    if constexpr (VARIANT == kW4A8) {
      codes_to_f16(v[0], b);
      codes_to_f16(v[1], b + 8);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        b[4 * i] = v[i].x;
        b[4 * i + 1] = v[i].y;
        b[4 * i + 2] = v[i].z;
        b[4 * i + 3] = v[i].w;
      }
    }
  }
};

// sum += the products of this warp's n_units (record, activations) units with
// the 32 weight rows from rbase. rec_of(i): unit i's record; load_x(i, nt,
// raw): its activations for column tile nt; after(i): called once unit i is
// in `sum`.
template <int VARIANT, int NT, typename Rec, typename LoadX, typename After>
__device__ __forceinline__ void stream_units(uint8_t* ring, int n_units, int rbase, Rec rec_of,
                                             LoadX load_x, After after, float (&sum)[2][NT][4]) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const uint32_t ring_at = smem_u32(ring);
  auto issue = [&](int i) {
    if (i < n_units) {
      const uint8_t* rec = rec_of(i);
      const uint32_t st = ring_at + (uint32_t)(i % kStages) * kStageBytes;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        cp_async16(st + (q * 32 + lane) * 16, rec + (tig * 128 + rbase + gid + 8 * q) * 16);
      if (lane < 16) cp_async4(st + 2048 + lane * 4, rec + 8192 + 2 * rbase + lane * 4);
      else if (lane < 20) cp_async4(st + 2048 + lane * 4, rec + 8448 + rbase / 2 + (lane - 16) * 4);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);
  ActRaw<VARIANT> raw[NT];
  if (n_units > 0) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) load_x(0, nt, raw[nt]);
  }
  for (int i = 0; i < n_units; ++i) {
    cp_async_wait<kStages - 2>();
    __syncwarp();  // unit i has landed, and every lane has read unit i - 1
    issue(i + kStages - 1);
    const uint8_t* st = ring + (i % kStages) * kStageBytes;
    uint32_t b[NT][16];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      raw[nt].words(b[nt]);
      if (i + 1 < n_units) load_x(i + 1, nt, raw[nt]);
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t a[2][16];
      float s[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int row = gid + 8 * (2 * mt + q);
        const uint4 v = *reinterpret_cast<const uint4*>(st + ((2 * mt + q) * 32 + lane) * 16);
        s[q] = f16_bits_to_f32(*reinterpret_cast<const uint16_t*>(st + 2048 + 2 * row));
        const uint32_t zb = st[2112 + (row >> 1)];
        cvt_w4_unit<VARIANT>(v, (row & 1) ? (zb >> 4) : (zb & 0xF), a[q]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          mma_16816<VARIANT>(acc, a[0][2 * j], a[1][2 * j], a[0][2 * j + 1], a[1][2 * j + 1],
                             b[nt][2 * j], b[nt][2 * j + 1]);
        sum[mt][nt][0] = fmaf(s[0], acc[0], sum[mt][nt][0]);
        sum[mt][nt][1] = fmaf(s[0], acc[1], sum[mt][nt][1]);
        sum[mt][nt][2] = fmaf(s[1], acc[2], sum[mt][nt][2]);
        sum[mt][nt][3] = fmaf(s[1], acc[3], sum[mt][nt][3]);
      }
    }
    after(i);
  }
}

// The warp's 32 x 8 NT sums into its rows of `red` ([32][LD] a warp).
template <int NT, int LD>
__device__ __forceinline__ void put_sums(float* red, const float (&sum)[2][NT][4]) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[(mt * 16 + (q >> 1) * 8 + gid) * LD + nt * 8 + tig * 2 + (q & 1)] = sum[mt][nt][q];
}

template <int NT>
__device__ __forceinline__ void zero_sums(float (&sum)[2][NT][4]) {
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int q = 0; q < 4; ++q) sum[mt][nt][q] = 0.f;
}

// ---- few tokens: the picked experts, from the ids alone -----------------------------
// Every CTA reads the (at most 128) ids and marks the picked experts in a bit
// set; expert number b is the b-th set bit.
struct FewPicks {
  uint32_t seen[kMaxSets / 32];
  int ids[kFewSlots];
};

// Fills `f` (all threads; ends with a barrier); returns the number of experts.
__device__ __forceinline__ int few_picks(FewPicks& f, const StreamParams& p) {
  const int n = p.T * p.k, words = (p.E + 31) / 32;
  for (int i = threadIdx.x; i < words; i += blockDim.x) f.seen[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int v = __ldg(p.ids + i);
    f.ids[i] = v;
    if (v >= 0 && v < p.E) atomicOr(&f.seen[v >> 5], 1u << (v & 31));
  }
  __syncthreads();
  int count = 0;
  for (int w = 0; w < words; ++w) count += __popc(f.seen[w]);
  return count;
}

// The b-th picked expert (b below the count).
__device__ __forceinline__ int few_expert(const FewPicks& f, int b) {
  int w = 0;
  for (int c = __popc(f.seen[0]); b >= c; c = __popc(f.seen[w])) {
    b -= c;
    ++w;
  }
  uint32_t m = f.seen[w];
  for (; b > 0; --b) m &= m - 1;
  return w * 32 + __ffs(m) - 1;
}

// Token t's first slot with expert e, or -1.
__device__ __forceinline__ int few_slot(const FewPicks& f, const StreamParams& p, int t, int e) {
  for (int j = 0; j < p.k; ++j)
    if (f.ids[t * p.k + j] == e) return t * p.k + j;
  return -1;
}

// ---- h = silu(G x) * (U x) -----------------------------------------------------------
template <int VARIANT, int NT, bool FEW>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 ? 5 : (NT == 2 ? 3 : 2))
experts_gate_up_kernel(const StreamParams p) {
  constexpr int LD = 8 * NT + 1;  // padded row of the partial sums
  static_assert(kWarps * kStages * kStageBytes >= kWarps * 32 * LD * 4, "sums reuse the ring");
  __shared__ __align__(128) uint8_t ring[kWarps][kStages * kStageBytes];
  __shared__ FewPicks few;
  __shared__ int few_slots[kFewTokens];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int G = p.G, K = G * 128;
  int set, rows, first = 0;  // the expert, its rows here, the first one's sorted position
  if constexpr (FEW) {
    if ((int)blockIdx.x >= few_picks(few, p)) return;
    set = few_expert(few, blockIdx.x);
    if (threadIdx.x < kFewTokens)
      few_slots[threadIdx.x] =
          (int)threadIdx.x < p.T ? few_slot(few, p, threadIdx.x, set) : -1;
    __syncthreads();
    rows = p.T;
  } else {
    if ((int)blockIdx.x >= p.head[1]) return;
    const int4 tile = __ldg(p.tiles + blockIdx.x);
    set = tile.x;
    first = tile.y;
    rows = tile.z;
    if (rows == 0) return;
  }
  const uint8_t* rec =
      p.packed + (((int64_t)set * (p.N >> 7) + (blockIdx.y >> 2)) * G) * 8512;
  int64_t at[NT];
  bool live[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int j = nt * 8 + gid;
    live[nt] = FEW ? few_slots[gid] >= 0 : j < rows;
    const int64_t row = FEW ? gid : (live[nt] ? __ldg(p.order + first + j) / p.k : 0);
    at[nt] = row * K + 32 * tig;
  }
  float sum[2][NT][4];
  zero_sums<NT>(sum);
  const int n_units = warp < G ? (G - warp + kWarps - 1) / kWarps : 0;
  stream_units<VARIANT, NT>(
      ring[warp], n_units, (blockIdx.y & 3) * 32,
      [&](int i) { return rec + (int64_t)(warp + i * kWarps) * 8512; },
      [&](int i, int nt, ActRaw<VARIANT>& raw) {
        raw.load(p.act, at[nt] + (int64_t)(warp + i * kWarps) * 128, live[nt]);
      },
      [](int) {}, sum);
  __syncthreads();  // every warp is done with its ring
  float* red = reinterpret_cast<float*>(ring[0]);
  put_sums<NT, LD>(red + warp * 32 * LD, sum);
  __syncthreads();
  const int I = p.N >> 1;
  for (int i = threadIdx.x; i < 16 * 8 * NT; i += 32 * kWarps) {
    const int c = i & 15, j = i >> 4;
    if (j >= rows) break;
    const int64_t to = FEW ? few_slots[j] : first + j;
    if (to < 0) continue;
    float gate = 0.f, up = 0.f;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) {
      gate += red[(q * 32 + c) * LD + j];
      up += red[(q * 32 + 16 + c) * LD + j];
    }
    if constexpr (VARIANT == kW4A8) {
      const float as = __ldg(p.a_s + (FEW ? j : __ldg(p.order + first + j) / p.k));
      gate *= as;
      up *= as;
    }
    p.h[to * I + blockIdx.y * 16 + c] = f32_to_bf16_bits(gated(gate, up));
  }
}

// ---- y = D h, a sorted row at a time ----------------------------------------------------
template <int VARIANT, int NT>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 ? 5 : (NT == 2 ? 3 : 2))
experts_down_kernel(const StreamParams p) {
  constexpr int LD = 8 * NT + 1;
  __shared__ __align__(128) uint8_t ring[kWarps][kStages * kStageBytes];
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
  float sum[2][NT][4];
  zero_sums<NT>(sum);
  const int n_units = warp < G ? (G - warp + kWarps - 1) / kWarps : 0;
  stream_units<VARIANT, NT>(
      ring[warp], n_units, (blockIdx.y & 3) * 32,
      [&](int i) { return rec + (int64_t)(warp + i * kWarps) * 8512; },
      [&](int i, int nt, ActRaw<VARIANT>& raw) {
        raw.load(p.act,
                 (int64_t)(tile.y + nt * 8 + gid) * K + (warp + i * kWarps) * 128 + 32 * tig,
                 nt * 8 + gid < rows);
      },
      [](int) {}, sum);
  __syncthreads();
  float* red = reinterpret_cast<float*>(ring[0]);
  put_sums<NT, LD>(red + warp * 32 * LD, sum);
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * 8 * NT; i += 32 * kWarps) {
    const int c = i & 31, j = i >> 5;
    if (j >= rows) break;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) v += red[(q * 32 + c) * LD + j];
    if constexpr (VARIANT == kW4A8) v *= __ldg(p.a_s + tile.y + j);
    p.y[(int64_t)(tile.y + j) * p.N + blockIdx.y * 32 + c] = v;
  }
}

// ---- few tokens: out = sum over the experts of w * D h ----------------------------------
// One CTA a block of 32 output columns; its warps share the (expert, group)
// units of all picked experts, and since column t is token t for every expert,
// the weighted sums over the experts stay in registers.
template <int VARIANT>
__global__ void __launch_bounds__(32 * kFewWarps, 1)
experts_few_down_kernel(const StreamParams p) {
  constexpr int LD = kFewTokens + 1;
  extern __shared__ __align__(128) uint8_t few_ring[];  // [kFewWarps][kStages * kStageBytes]
  __shared__ FewPicks few;
  __shared__ int expert[kFewSlots];
  __shared__ int slot[kFewSlots][kFewTokens];      // token's row of h, -1: not picked
  __shared__ float weight[kFewSlots][kFewTokens];  // its weight (and the row's scale)
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int G = p.G, K = G * 128;
  const int count = few_picks(few, p);
  for (int i = threadIdx.x; i < count * kFewTokens; i += 32 * kFewWarps) {
    const int b = i / kFewTokens, t = i % kFewTokens;
    const int e = few_expert(few, b);
    if (t == 0) expert[b] = e;
    int s = -1;
    float w = 0.f;
    if (t < p.T) {
      s = few_slot(few, p, t, e);
      // (a token that lists an expert twice: h is in the first slot, the
      // weights add up)
      for (int j = s; j >= 0 && j < (t + 1) * p.k; ++j)
        if (few.ids[j] == e) w += __ldg(p.weights + j);
      if (VARIANT == kW4A8 && s >= 0) w *= __ldg(p.a_s + s);
    }
    slot[b][t] = s;
    weight[b][t] = w;
  }
  __syncthreads();
  const int units = count * G;
  const int n_units = warp < units ? (units - warp + kFewWarps - 1) / kFewWarps : 0;
  float sum[2][1][4], total[2][1][4];
  zero_sums<1>(sum);
  zero_sums<1>(total);
  stream_units<VARIANT, 1>(
      few_ring + warp * kStages * kStageBytes, n_units, (blockIdx.x & 3) * 32,
      [&](int i) {
        const int u = warp + i * kFewWarps, b = u / G;
        return p.packed + (((int64_t)expert[b] * (p.N >> 7) + (blockIdx.x >> 2)) * G + (u - b * G)) *
                              8512;
      },
      [&](int i, int, ActRaw<VARIANT>& raw) {
        const int u = warp + i * kFewWarps, b = u / G;
        const int s = slot[b][gid];
        raw.load(p.act, (int64_t)s * K + (u - b * G) * 128 + 32 * tig, s >= 0);
      },
      [&](int i) {
        const int u = warp + i * kFewWarps, b = u / G;
        if (i + 1 < n_units && (u + kFewWarps) / G == b) return;
        const float w0 = weight[b][2 * tig], w1 = weight[b][2 * tig + 1];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            // (a token without this expert adds nothing, whatever its column holds)
            total[mt][0][q] = fmaf((q & 1) ? w1 : w0, sum[mt][0][q], total[mt][0][q]);
            sum[mt][0][q] = 0.f;
          }
      },
      sum);
  __syncthreads();
  float* red = reinterpret_cast<float*>(few_ring);
  put_sums<1, LD>(red + warp * 32 * LD, total);
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * kFewTokens; i += 32 * kFewWarps) {
    const int c = i & 31, t = i >> 5;
    if (t >= p.T) break;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kFewWarps; ++q) v += red[(q * 32 + c) * LD + t];
    p.out[(int64_t)t * p.N + blockIdx.x * 32 + c] = f32_to_bf16_bits(v);
  }
}

// ---- the picks' outputs summed -----------------------------------------------------
// out[t] = sum_j w[t,j] * y[pos[t,j]] in fp32, j in order; a dropped pick adds
// nothing. A thread holds eight columns.
constexpr int kCombineThreads = 128;

template <typename Y>  // float or uint16_t (bf16)
__global__ void __launch_bounds__(kCombineThreads)
combine_kernel(const Y* __restrict__ y, const float* __restrict__ weights,
               const int32_t* __restrict__ pos, int k, int64_t H, uint16_t* __restrict__ out) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const int64_t v = (int64_t)blockIdx.y * kCombineThreads + threadIdx.x;
  if (v * 8 >= H) return;
  float acc[8] = {};
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int at = __ldg(pos + t * k + j);
    if (at < 0) continue;
    const float w = __ldg(weights + t * k + j);
    if constexpr (sizeof(Y) == 4) {
      const float4* src = reinterpret_cast<const float4*>(y + (int64_t)at * H) + 2 * v;
      const float4 a = __ldg(src), b = __ldg(src + 1);
      const float q[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, q[i], acc[i]);
    } else {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(y + (int64_t)at * H) + v);
      const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] = fmaf(w, __uint_as_float(q[i] << 16), acc[2 * i]);
        acc[2 * i + 1] = fmaf(w, __uint_as_float(q[i] & 0xFFFF0000u), acc[2 * i + 1]);
      }
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = (uint32_t)f32_to_bf16_bits(acc[2 * i]) |
           ((uint32_t)f32_to_bf16_bits(acc[2 * i + 1]) << 16);
  reinterpret_cast<uint4*>(out + t * H)[v] = make_uint4(o[0], o[1], o[2], o[3]);
}

// ---- rows quantized, and rows in sorted order -----------------------------------------
// Codes of a bf16 row as egopq_quant_act_i8 defines them (fp32 scale
// absmax / 127, fp32 quotient rounded half to even): int8, or the same
// integers as fp16 for the tensor cores. R threads a row.
__device__ __forceinline__ float absmax8(const uint4& v, float m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m = fmaxf(m, fabsf(__uint_as_float(w[j] << 16)));
    m = fmaxf(m, fabsf(__uint_as_float(w[j] & 0xFFFF0000u)));
  }
  return m;
}
__device__ __forceinline__ void codes8(const uint4& v, float s, float inv, bool zero, float (&q)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    q[2 * j] = zero ? 0.f : quant_code(__uint_as_float(w[j] << 16), s, inv);
    q[2 * j + 1] = zero ? 0.f : quant_code(__uint_as_float(w[j] & 0xFFFF0000u), s, inv);
  }
}
__device__ __forceinline__ uint4 codes_f16(const float (&q)[8]) {
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 h = __floats2half2_rn(q[2 * j], q[2 * j + 1]);
    o[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint2 codes_i8(const float (&q)[8]) {
  uint32_t o[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j >> 2] |= ((uint32_t)(int)q[j] & 0xFFu) << (8 * (j & 3));
  return make_uint2(o[0], o[1]);
}

// Maximum over the R threads of a row (R = 32, or the whole block).
template <int R>
__device__ __forceinline__ float row_max(float m, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if constexpr (R > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = part[0];
#pragma unroll
    for (int i = 1; i < R / 32; ++i) m = fmaxf(m, part[i]);
  }
  return m;
}

constexpr int kRowThreads = 128;
constexpr int kRowVecs = 8;  // 16-byte vectors a thread keeps of its row

// Rows [0, rows) (or those below head[0], where head is given) of x [.][K].
template <int R, bool F16>
__global__ void __launch_bounds__(kRowThreads)
quant_rows_kernel(const uint16_t* __restrict__ x, const int* __restrict__ head, int64_t rows,
                  int64_t K, void* __restrict__ codes, float* __restrict__ scales) {
  __shared__ float part[kRowThreads / 32];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int64_t m = (int64_t)blockIdx.x * (kRowThreads / R) + threadIdx.x / R;
  if (head) rows = head[0];
  if (m >= rows) return;  // (a whole warp, or the whole block)
  const int t = threadIdx.x % R;
  const uint4* src = reinterpret_cast<const uint4*>(x + m * K);
  const int64_t nvec = K / 8;
  uint4 v[kRowVecs];
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < kRowVecs; ++i)
    if (t + i * R < nvec) v[i] = __ldg(src + t + i * R);
#pragma unroll
  for (int i = 0; i < kRowVecs; ++i)
    if (t + i * R < nvec) a = absmax8(v[i], a);
  for (int64_t i = t + kRowVecs * R; i < nvec; i += R) a = absmax8(__ldg(src + i), a);
  a = row_max<R>(a, part);
  const float s = __fdiv_rn(a, 127.0f), inv = quant_recip(s);
  if (t == 0) scales[m] = s;
  auto put = [&](const uint4& u, int64_t i) {
    float q[8];
    codes8(u, s, inv, a == 0.f, q);
    if constexpr (F16) reinterpret_cast<uint4*>(static_cast<uint16_t*>(codes) + m * K)[i] = codes_f16(q);
    else reinterpret_cast<uint2*>(static_cast<int8_t*>(codes) + m * K)[i] = codes_i8(q);
  };
#pragma unroll
  for (int i = 0; i < kRowVecs; ++i)
    if (t + i * R < nvec) put(v[i], t + i * R);
  for (int64_t i = t + kRowVecs * R; i < nvec; i += R) put(__ldg(src + i), i);
}

// rows[pos[t, j]] = token t's activations, for each of its picks that has an
// expert: bf16 as they are, or (CODES) their fp16 codes, and rows_s their
// scales. One CTA a token: x is read once, each copy written once.
template <bool CODES>
__global__ void __launch_bounds__(kRowThreads)
scatter_rows_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ pos, int k,
                    int64_t K, uint16_t* __restrict__ rows, float* __restrict__ rows_s) {
  __shared__ float part[kRowThreads / 32];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int64_t m = blockIdx.x;
  const uint4* src = reinterpret_cast<const uint4*>(x + m * K);
  const int64_t nvec = K / 8;
  float s = 0.f, inv = 0.f, a = 0.f;
  if constexpr (CODES) {
    for (int64_t i = threadIdx.x; i < nvec; i += kRowThreads) a = absmax8(__ldg(src + i), a);
    a = row_max<kRowThreads>(a, part);
    s = __fdiv_rn(a, 127.0f);
    inv = quant_recip(s);
    for (int j = threadIdx.x; j < k; j += kRowThreads) {
      const int at = __ldg(pos + m * k + j);
      if (at >= 0) rows_s[at] = s;
    }
  }
  for (int64_t i = threadIdx.x; i < nvec; i += kRowThreads) {
    uint4 v = __ldg(src + i);
    if constexpr (CODES) {
      float q[8];
      codes8(v, s, inv, a == 0.f, q);
      v = codes_f16(q);
    }
    for (int j = 0; j < k; ++j) {
      const int at = __ldg(pos + m * k + j);
      if (at >= 0) reinterpret_cast<uint4*>(rows + (int64_t)at * K)[i] = v;
    }
  }
}

// ---- launches -----------------------------------------------------------------------
template <bool F16>
static cudaError_t launch_quant_rows(const uint16_t* x, const int* head, int64_t rows, int64_t K,
                                     void* codes, float* scales, cudaStream_t st) {
  // a warp a row where there are rows for every warp of the GPU (32768 x 1280:
  // a block a row leaves most of its threads without work), else a block
  if (rows >= 4096 && K <= 32 * kRowVecs * 8) {
    PdlConfig c(dim3((unsigned)((rows + 3) / 4), 1, 1), kRowThreads, 0, st);
    return cudaLaunchKernelEx(&c.cfg, quant_rows_kernel<32, F16>, x, head, rows, K, codes, scales);
  }
  PdlConfig c(dim3((unsigned)rows, 1, 1), kRowThreads, 0, st);
  return cudaLaunchKernelEx(&c.cfg, quant_rows_kernel<kRowThreads, F16>, x, head, rows, K, codes,
                            scales);
}

template <typename Y>
static cudaError_t launch_combine(const ExpertsArgs& a, const Y* y, cudaStream_t st) {
  PdlConfig c(dim3((unsigned)a.T, (unsigned)((a.H / 8 + kCombineThreads - 1) / kCombineThreads), 1),
              kCombineThreads, 0, st);
  return cudaLaunchKernelEx(&c.cfg, combine_kernel<Y>, y, a.weights, (const int32_t*)a.plan.pos,
                            a.k, a.H, a.out);
}

// Many rows an expert: the rows in sorted order, then the tcgen05 products.
template <int VARIANT>
static cudaError_t run_tensor(const ExpertsArgs& a, cudaStream_t st) {
  constexpr bool kCodes = VARIANT == kW4A8;
  const int64_t n = a.T * a.k;
  cudaError_t e = launch_plan(a.ids, n, a.E, 0, a.plan, st);
  if (e != cudaSuccess) return e;
  PdlConfig c(dim3((unsigned)a.T, 1, 1), kRowThreads, 0, st);
  e = cudaLaunchKernelEx(&c.cfg, scatter_rows_kernel<kCodes>, a.x, (const int32_t*)a.plan.pos, a.k,
                         a.H, a.rows, a.rows_s);
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
    e = launch_quant_rows<true>(a.h, a.plan.head, n, a.I, a.h_q, a.h_s, st);
    if (e != cudaSuccess) return e;
  }
  r.gate_up = false;
  r.N = a.H;
  r.K = a.I;
  r.act = kCodes ? a.h_q : (const void*)a.h;
  r.a_s = a.h_s;
  r.packed = a.down;
  r.y = static_cast<uint16_t*>(a.y);
  if ((e = launch_ragged(r, st)) != cudaSuccess) return e;
  return launch_combine(a, (const uint16_t*)a.y, st);
}

template <int VARIANT>
static cudaError_t run_few(const ExpertsArgs& a, StreamParams p, cudaStream_t st) {
  const int64_t n = a.T * a.k;
  const int64_t most = n < a.E ? n : a.E;
  PdlConfig c(dim3((unsigned)most, (unsigned)(a.I / 16), 1), 32 * kWarps, 0, st);
  cudaError_t e = cudaLaunchKernelEx(&c.cfg, experts_gate_up_kernel<VARIANT, 1, true>, p);
  if (e != cudaSuccess) return e;
  if (VARIANT == kW4A8) {
    // (a slot without an expert holds no row: its codes are never read)
    e = launch_quant_rows<false>(a.h, nullptr, n, a.I, a.h_q, a.h_s, st);
    if (e != cudaSuccess) return e;
  }
  p.act = VARIANT == kW4A8 ? a.h_q : (const void*)a.h;
  p.a_s = a.h_s;
  p.packed = a.down;
  p.N = (int)a.H;
  p.G = (int)(a.I / 128);
  constexpr size_t kSmem = (size_t)kFewWarps * kStages * kStageBytes;
  static SmemOptIn opt_in;
  if ((e = opt_in.ensure(experts_few_down_kernel<VARIANT>, kSmem)) != cudaSuccess) return e;
  PdlConfig d(dim3((unsigned)(a.H / 32), 1, 1), 32 * kFewWarps, kSmem, st);
  return cudaLaunchKernelEx(&d.cfg, experts_few_down_kernel<VARIANT>, p);
}

template <int VARIANT, int NT>
static cudaError_t run_stream(const ExpertsArgs& a, StreamParams p, cudaStream_t st) {
  const int64_t n = a.T * a.k;
  const int64_t tiles = plan_max_tiles(n, a.E, 8 * NT);
  PdlConfig c(dim3((unsigned)tiles, (unsigned)(a.I / 16), 1), 32 * kWarps, 0, st);
  cudaError_t e = cudaLaunchKernelEx(&c.cfg, experts_gate_up_kernel<VARIANT, NT, false>, p);
  if (e != cudaSuccess) return e;
  if (VARIANT == kW4A8) {
    e = launch_quant_rows<false>(a.h, a.plan.head, n, a.I, a.h_q, a.h_s, st);
    if (e != cudaSuccess) return e;
  }
  p.act = VARIANT == kW4A8 ? a.h_q : (const void*)a.h;
  p.a_s = a.h_s;
  p.packed = a.down;
  p.N = (int)a.H;
  p.G = (int)(a.I / 128);
  PdlConfig d(dim3((unsigned)tiles, (unsigned)(a.H / 32), 1), 32 * kWarps, 0, st);
  e = cudaLaunchKernelEx(&d.cfg, experts_down_kernel<VARIANT, NT>, p);
  if (e != cudaSuccess) return e;
  return launch_combine(a, (const float*)a.y, st);
}

template <int VARIANT>
static cudaError_t run_experts(const ExpertsArgs& a, cudaStream_t st) {
  if (a.way == kExpertsTensor) return run_tensor<VARIANT>(a, st);
  const int64_t n = a.T * a.k;
  StreamParams p{};
  p.act = VARIANT == kW4A8 ? (const void*)a.x_q : (const void*)a.x;
  p.a_s = a.x_s;
  p.packed = a.gate_up;
  p.h = a.h;
  p.y = static_cast<float*>(a.y);
  p.out = a.out;
  p.head = a.plan.head;
  p.tiles = a.plan.tiles;
  p.order = a.plan.order;
  p.ids = a.ids;
  p.weights = a.weights;
  p.T = (int)a.T;
  p.k = a.k;
  p.E = a.E;
  p.N = (int)(2 * a.I);
  p.G = (int)(a.H / 128);
  // rows of a tile: the average expert's in one tile as a rule (an expert with
  // more takes several, whose weights then come from L2)
  const int nt = n <= (int64_t)6 * a.E ? 1 : (n <= (int64_t)12 * a.E ? 2 : 4);
  cudaError_t e = cudaSuccess;
  if (a.way == kExpertsStream) e = launch_plan(a.ids, n, a.E, 8 * nt, a.plan, st);
  if (e == cudaSuccess && VARIANT == kW4A8)
    e = launch_quant_rows<false>(a.x, nullptr, a.T, a.H, a.x_q, a.x_s, st);
  if (e != cudaSuccess) return e;
  if (a.way == kExpertsFew) return run_few<VARIANT>(a, p, st);
  return nt == 1   ? run_stream<VARIANT, 1>(a, p, st)
         : nt == 2 ? run_stream<VARIANT, 2>(a, p, st)
                   : run_stream<VARIANT, 4>(a, p, st);
}

cudaError_t launch_experts(const ExpertsArgs& a, cudaStream_t st) {
  return a.variant == kW4A8 ? run_experts<kW4A8>(a, st) : run_experts<kW4A16>(a, st);
}

ExpertsWay experts_way(int64_t T, int k, int E, int path) {
  if (path == EGOPQ_PATH_TC) return kExpertsTensor;
  const int64_t n = T * k;
  if (path == EGOPQ_PATH_AUTO && n > kStreamRows * E) return kExpertsTensor;
  return T <= kFewTokens && n <= kFewSlots ? kExpertsFew : kExpertsStream;
}

}  // namespace egopq
