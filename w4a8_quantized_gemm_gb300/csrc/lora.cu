// lora.cu -- low-rank adapters of many requests at once, beside a shared
// projection:
//
//   y[m] = bf16( y0[m] + scale_a * B_a (A_a x[m]) ),  a = ids[m]
//
// A [L][r][K], B [L][N][r] bf16; adapter a uses its first ranks[a] rows of A
// (columns of B). A row with ids outside [0, L) keeps y0. Rows are sorted by
// adapter (RowPlan), so that the rows of one adapter share its weights.
//
// Two kernels: A x into fp32 sums [splits][M][r] (K split over warps and, for
// few rows, over CTAs: the sums of the parts are added in order by the second
// kernel, so the result does not depend on timing), then the product with B
// and the addition to y0. Both run on mma.m16n8k16 with fragments loaded
// straight from memory: the order of K inside a fragment is free as long as
// both operands share it, so each thread reads 16 contiguous bytes of its row.
#include "egopq_internal.h"

namespace egopq {

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kLoraWarps = 8;
constexpr int kLoraTile = 16;      // rows of a tile
constexpr int kLoraMaxRank = 128;

struct LoraParams {
  const uint16_t* y_in;
  const uint16_t* x;
  const uint16_t* A;
  const uint16_t* B;
  const float* scale;
  const int32_t* ranks;
  uint16_t* y_out;
  float* h;
  const int* head;
  const int4* tiles;
  const int32_t* order;
  int64_t M, N, K;
  int r, splits;
};

// ranks[a] as a number in [0, r]
__device__ __forceinline__ int adapter_rank(const LoraParams& p, int a) {
  return p.ranks ? max(0, min(p.r, __ldg(p.ranks + a))) : p.r;
}

// h[split][sorted row][0, rank) = the split's part of A_a x. One CTA a tile of
// 16 rows and a part of K, whose warps take 32-wide steps of it in turn; NR
// n8-tiles of ranks at a time.
template <int NR>
__global__ void __launch_bounds__(32 * kLoraWarps)
lora_shrink_kernel(const LoraParams p) {
  __shared__ float red[kLoraWarps][16][8 * NR + 1];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  if ((int)blockIdx.x >= p.head[1]) return;
  const int4 tile = __ldg(p.tiles + blockIdx.x);
  if (tile.z == 0) return;
  const int rank = adapter_rank(p, tile.x);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  // K in steps of 32: this CTA's are [s0, s1)
  const int steps = (int)(p.K / 32);
  const int s0 = (int)((int64_t)blockIdx.y * steps / p.splits);
  const int s1 = (int)((int64_t)(blockIdx.y + 1) * steps / p.splits);
  const bool live0 = gid < tile.z, live1 = gid + 8 < tile.z;
  const uint16_t* x0 = p.x + (live0 ? (int64_t)__ldg(p.order + tile.y + gid) * p.K : 0) + 8 * tig;
  const uint16_t* x1 =
      p.x + (live1 ? (int64_t)__ldg(p.order + tile.y + gid + 8) * p.K : 0) + 8 * tig;
  const uint16_t* Ab = p.A + (int64_t)tile.x * p.r * p.K + 8 * tig;
  for (int c0 = 0; c0 < rank; c0 += 8 * NR) {
    float acc[NR][4];
#pragma unroll
    for (int t = 0; t < NR; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[t][q] = 0.f;
#pragma unroll 2
    for (int s = s0 + warp; s < s1; s += kLoraWarps) {
      uint4 a0 = {}, a1 = {};
      if (live0) a0 = __ldg(reinterpret_cast<const uint4*>(x0 + s * 32));
      if (live1) a1 = __ldg(reinterpret_cast<const uint4*>(x1 + s * 32));
#pragma unroll
      for (int t = 0; t < NR; ++t) {
        const int j = c0 + t * 8 + gid;
        uint4 b = {};
        if (j < rank) b = __ldg(reinterpret_cast<const uint4*>(Ab + (int64_t)j * p.K + s * 32));
        mma_bf16(acc[t], a0.x, a1.x, a0.y, a1.y, b.x, b.y);
        mma_bf16(acc[t], a0.z, a1.z, a0.w, a1.w, b.z, b.w);
      }
    }
#pragma unroll
    for (int t = 0; t < NR; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[warp][(q >> 1) * 8 + gid][t * 8 + tig * 2 + (q & 1)] = acc[t][q];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * 8 * NR; i += 32 * kLoraWarps) {
      const int j = i % (8 * NR), row = i / (8 * NR);
      if (row < tile.z && c0 + j < rank) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kLoraWarps; ++w) v += red[w][row][j];
        p.h[((int64_t)blockIdx.y * p.M + tile.y + row) * p.r + c0 + j] = v;
      }
    }
    __syncthreads();
  }
}

// y = bf16(y0 + scale * B_a h). One CTA a tile of 16 rows and 32 * kLoraWarps
// columns, 32 a warp. The tile's h -- the splits added in order, scaled in
// fp32, and rounded to bf16 once, as the product's operand: relative 2^-8 of
// the update, below the rounding of y itself where the update is no larger
// than y -- lies in shared memory. Column c of the warp's n8-tile t is column
// (c / 2) * 8 + 2t + c % 2 of its 32, so that a thread's sums over the four
// tiles are eight neighbouring columns: one 16-byte load and store a row.
__global__ void __launch_bounds__(32 * kLoraWarps)
lora_expand_kernel(const LoraParams p) {
  constexpr int LD = kLoraMaxRank + 8;
  __shared__ __align__(16) uint16_t hs[16][LD];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int n_tiles = p.head[1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int64_t n0 = ((int64_t)blockIdx.y * kLoraWarps + warp) * 32;
  int4 tile;
  int rank = 0;
  if ((int)blockIdx.x < n_tiles) {
    tile = __ldg(p.tiles + blockIdx.x);
    if (tile.z == 0) return;
    rank = adapter_rank(p, tile.x);
    const float sc = __ldg(p.scale + tile.x);
    const int kr = (rank + 15) & ~15;
    for (int i = threadIdx.x; i < 16 * kr; i += 32 * kLoraWarps) {
      const int row = i / kr, j = i - row * kr;
      float v = 0.f;
      if (row < tile.z && j < rank)
        for (int s = 0; s < p.splits; ++s)
          v += p.h[((int64_t)s * p.M + tile.y + row) * p.r + j];
      hs[row][j] = f32_to_bf16_bits(sc * v);
    }
  } else {
    // tiles past the table copy the rows without an adapter, which the plan
    // lists last (nothing to do where y is updated in place)
    const int first = p.head[0] + ((int)blockIdx.x - n_tiles) * 16;
    tile = make_int4(0, first, min(16, (int)p.M - first), 0);
    if (tile.z <= 0 || p.y_in == p.y_out) return;
  }
  __syncthreads();
  if (n0 >= p.N) return;
  float acc[4][4];
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[t][q] = 0.f;
  const uint16_t* Bb = p.B + ((int64_t)tile.x * p.N + n0) * p.r;
  for (int j0 = 0; j0 < rank; j0 += 16) {
    // 16 ranks: thread column tig holds ranks 4 tig .. 4 tig + 3 of them
    const int j = j0 + 4 * tig;
    const uint2 a0 = *reinterpret_cast<const uint2*>(&hs[gid][j]);
    const uint2 a1 = *reinterpret_cast<const uint2*>(&hs[gid + 8][j]);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int col = (gid >> 1) * 8 + 2 * t + (gid & 1);
      uint2 b = {};
      if (j < p.r) b = __ldg(reinterpret_cast<const uint2*>(Bb + (int64_t)col * p.r + j));
      // columns of B past the adapter's rank meet zeros of h, but may hold
      // anything: leave them out
      if (j + 3 >= rank) {
        if (j >= rank) b = make_uint2(0u, 0u);
        else if (j + 1 >= rank) b = make_uint2(b.x & 0xFFFFu, 0u);
        else if (j + 2 >= rank) b.y = 0u;
        else b.y &= 0xFFFFu;
      }
      mma_bf16(acc[t], a0.x, a1.x, a0.y, a1.y, b.x, b.y);
    }
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int row = gid + 8 * half;
    if (row >= tile.z) continue;
    const int64_t at = (int64_t)__ldg(p.order + tile.y + row) * p.N + n0 + 8 * tig;
    const uint4 v = *reinterpret_cast<const uint4*>(p.y_in + at);
    const uint32_t q[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
      o[t] = (uint32_t)f32_to_bf16_bits(__uint_as_float(q[t] << 16) + acc[t][2 * half]) |
             ((uint32_t)f32_to_bf16_bits(__uint_as_float(q[t] & 0xFFFF0000u) +
                                         acc[t][2 * half + 1])
              << 16);
    *reinterpret_cast<uint4*>(p.y_out + at) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

int lora_tile(int64_t) { return kLoraTile; }

int lora_splits(int64_t M, int64_t K) {
  // parts of K so that about a CTA an SM runs, none of fewer steps than warps
  const int64_t tiles = (M + kLoraTile - 1) / kLoraTile;
  int64_t s = 128 / (tiles > 0 ? tiles : 1);
  const int64_t most = K / (32 * kLoraWarps);
  if (s > most) s = most;
  if (s > 8) s = 8;
  return s < 1 ? 1 : (int)s;
}

cudaError_t launch_lora(const LoraArgs& a, cudaStream_t st) {
  LoraParams p;
  p.y_in = a.y_in;
  p.x = a.x;
  p.A = a.A;
  p.B = a.B;
  p.scale = a.scale;
  p.ranks = a.ranks;
  p.y_out = a.y_out;
  p.h = a.h;
  p.head = a.plan.head;
  p.tiles = a.plan.tiles;
  p.order = a.plan.order;
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.r = a.r;
  p.splits = lora_splits(a.M, a.K);
  cudaError_t e = launch_plan(a.ids, a.M, a.L, kLoraTile, a.plan, st);
  if (e != cudaSuccess) return e;
  const int64_t tiles = plan_max_tiles(a.M, a.L, kLoraTile);
  {
    PdlConfig c(dim3((unsigned)tiles, (unsigned)p.splits, 1), 32 * kLoraWarps, 0, st);
    e = a.r <= 16 ? cudaLaunchKernelEx(&c.cfg, lora_shrink_kernel<2>, p)
        : a.r <= 32 ? cudaLaunchKernelEx(&c.cfg, lora_shrink_kernel<4>, p)
                    : cudaLaunchKernelEx(&c.cfg, lora_shrink_kernel<8>, p);
    if (e != cudaSuccess) return e;
  }
  // (the rows without an adapter make at most ceil(M / 16) tiles more)
  const int64_t grid = tiles + (a.M + 15) / 16;
  PdlConfig c(dim3((unsigned)grid,
                   (unsigned)((a.N + 32 * kLoraWarps - 1) / (32 * kLoraWarps)), 1),
              32 * kLoraWarps, 0, st);
  return cudaLaunchKernelEx(&c.cfg, lora_expand_kernel, p);
}

}  // namespace egopq
