// lora.cu -- low-rank adapters of many requests at once, beside a shared
// projection:
//
//   y[m] = bf16( y0[m] + scale_a * B_a (A_a x[m]) ),  a = ids[m]
//
// A [L][r][K], B [L][N][r] bf16; adapter a uses its first ranks[a] rows of A
// (columns of B). A row with ids outside [0, L) keeps y0.
//
// One kernel where its tiles run at once: a cluster of CTAs takes up to 32 rows
// of one adapter, splits K for A x, adds the parts through distributed shared
// memory in rank order and splits the columns for the product with B. Up to 128
// rows (decode) the cluster finds its rows in the ids alone; more rows are
// sorted by adapter first (RowPlan), and many tiles of narrow rows take two
// kernels (lora_many). Results do not depend on timing.
//
// All products run on mma.m16n8k16 with fragments loaded straight from memory:
// the order of K inside a fragment is free as long as both operands share it,
// so each thread reads 16 (A, x) or 8 (B) contiguous bytes of its row.
#include "egopq_internal.h"

#include <algorithm>

namespace egopq {

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

constexpr int kLoraWarps = 8;
constexpr int kLoraThreads = 32 * kLoraWarps;
constexpr int kLoraMaxRank = 128;
constexpr int kLoraFewRows = 128;  // rows of a batch without a plan
constexpr int kManyTile = 128;  // rows of a tile of the two kernels (lora_many)
constexpr int kManyCtas = 304;  // CTAs that their first is split for, two an SM
constexpr int kLoraCluster = 8;
constexpr int kHsLd = kLoraMaxRank + 8;  // padded row of the bf16 A x in shared memory (16-byte rows)

struct LoraParams {
  const uint16_t* y_in;
  const uint16_t* x;
  const uint16_t* A;
  const uint16_t* B;
  const float* scale;
  const int32_t* ranks;
  const int32_t* ids;
  uint16_t* y_out;
  const int* head;
  const int4* tiles;
  const int32_t* order;
  float* h;  // [splits][M][r] partial sums of A x, sorted rows (two kernels)
  int64_t M, N, K;
  int L, r, max_slabs, clusters, splits;
  bool beside;  // early: y_in alone comes from the kernel in front (launch_plan)
};

// ranks[a] as a number in [0, r]
__device__ __forceinline__ int adapter_rank(const LoraParams& p, int a) {
  return p.ranks ? max(0, min(p.r, __ldcg(p.ranks + a))) : p.r;
}

// acc[mt][t] += x rows (two a thread and row tile: xr[2 mt], xr[2 mt + 1], null
// where there is none) times ranks [c0, c0 + 8 NR) of A over the 32-wide K
// steps s0, s0 + step, ... below s1. Pointers include the thread's 8 * tig. A
// step's loads are all issued before its products (missing rows and ranks read
// the first and are replaced by zeros: no branch between the loads; past L1, as
// the kernel may be early).
template <int MT, int NR>
__device__ __forceinline__ void shrink_steps(float (&acc)[MT][NR][4], const uint16_t* const* xr,
                                             const uint16_t* Ab, int64_t K, int c0, int rank,
                                             int s0, int s1, int step) {
  const int gid = (threadIdx.x & 31) >> 2;
  auto keep = [](uint4 v, bool in) {
    return make_uint4(in ? v.x : 0u, in ? v.y : 0u, in ? v.z : 0u, in ? v.w : 0u);
  };
  const uint16_t* Aj[NR];
#pragma unroll
  for (int t = 0; t < NR; ++t) {
    const int j = c0 + t * 8 + gid;
    Aj[t] = Ab + (int64_t)(j < rank ? j : 0) * K;
  }
  for (int s = s0; s < s1; s += step) {
    uint4 a[2 * MT], b[NR];
#pragma unroll
    for (int q = 0; q < 2 * MT; ++q)
      a[q] = __ldcg(reinterpret_cast<const uint4*>((xr[q] ? xr[q] : Ab) + (int64_t)s * 32));
#pragma unroll
    for (int t = 0; t < NR; ++t) b[t] = __ldcg(reinterpret_cast<const uint4*>(Aj[t] + s * 32));
#pragma unroll
    for (int q = 0; q < 2 * MT; ++q) a[q] = keep(a[q], xr[q] != nullptr);
#pragma unroll
    for (int t = 0; t < NR; ++t) {
      const uint4 v = keep(b[t], c0 + t * 8 + gid < rank);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mma_bf16(acc[mt][t], a[2 * mt].x, a[2 * mt + 1].x, a[2 * mt].y, a[2 * mt + 1].y, v.x, v.y);
        mma_bf16(acc[mt][t], a[2 * mt].z, a[2 * mt + 1].z, a[2 * mt].w, a[2 * mt + 1].w, v.z, v.w);
      }
    }
  }
}

// Eight neighbouring columns of y plus their updates, rounded.
__device__ __forceinline__ uint4 add_row(const uint4& v, const float (&acc)[4][4], int half) {
  const uint32_t q[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const __nv_bfloat162 r =
        __floats2bfloat162_rn(__uint_as_float(q[t] << 16) + acc[t][2 * half],
                              __uint_as_float(q[t] & 0xFFFF0000u) + acc[t][2 * half + 1]);
    o[t] = *reinterpret_cast<const uint32_t*>(&r);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Eight ranks of B (a thread's: j .. j + 7) without those past the adapter's
// rank, which meet zeros of h but may hold anything.
__device__ __forceinline__ uint4 keep_ranks(uint4 v, int j, int rank) {
  uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = j + 2 * i + 1 < rank ? q[i] : (j + 2 * i < rank ? q[i] & 0xFFFFu : 0u);
  return make_uint4(q[0], q[1], q[2], q[3]);
}

// y_out = bf16(y_in + hs B^T) for a tile's rows (16 MT of them; `rows` live,
// row_of(i) names row i of y) over 32-column chunks first, first + step, ...
// below `last`; JS = ceil(r / 32). Column c of a chunk's n8-tile t is column
// (c / 2) * 8 + 2t + c % 2 of it, so that a thread's sums over the four tiles
// are eight neighbouring columns of y: one 16-byte access a row. A thread holds
// eight ranks a step of 32, as hs has them. y and B come through a ring in
// shared memory, a warp's own, in which a lane reads back what it copied (no
// barrier). begin() puts the first kSlots chunks on their way, before hs is
// known; a slot is filled again once its chunk is done.
template <int MT, int JS>
struct Expand {
  static constexpr int kSlotBytes = (4 * JS + 2 * MT) * 512;
  // CTAs of an SM that the ring and the registers leave room for
  static constexpr int kCtas = MT * JS == 1 ? 3 : 2;
  static constexpr int kSlots = (kCtas == 3 ? 8192 : 12288) / kSlotBytes;
  static_assert(kSlots >= 1, "a ring holds one chunk at least");
  const uint16_t* y_in;
  uint16_t* y_out;
  const uint16_t* Bt;
  int64_t at[2 * MT];  // this thread's place in its rows of y, -1: no row
  int r, rank, rows;
  uint32_t ring;  // this lane's first 16 bytes

  template <typename RowOf>
  __device__ __forceinline__ Expand(const LoraParams& p, const uint16_t* Bset, int rank_, int rows_,
                                    uint32_t ring_, RowOf row_of)
      : y_in(p.y_in), y_out(p.y_out), r(p.r), rank(rank_), rows(rows_) {
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    ring = ring_ + lane * 16;
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i)
      at[i] = i * 8 + gid < rows ? (int64_t)row_of(i * 8 + gid) * p.N + 8 * tig : -1;
    Bt = Bset + (int64_t)((gid >> 1) * 8 + (gid & 1)) * r + 8 * tig;
  }
  // chunk c's ranks 32 js and up of B, and with the last of them its y
  __device__ __forceinline__ void fetch(int64_t c, int64_t last, int slot, int js) {
    if (c < last) {
      const uint32_t to = ring + slot * kSlotBytes;
      if (js * 32 < rank) {
        const uint16_t* src = Bt + c * 32 * r + js * 32;
        // (ranks past the adapter's are dropped: zeros)
        const bool in = js * 32 + 8 * (int)(threadIdx.x & 3) < rank;  // r is a multiple of 8
#pragma unroll
        for (int t = 0; t < 4; ++t)
          cp_async16_zfill(to + (js * 4 + t) * 512, in ? src + 2 * t * r : Bt, in ? 16u : 0u);
      }
      if (js == JS - 1) {
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i)
          if (at[i] >= 0) cp_async16_zfill(to + (4 * JS + i) * 512, y_in + at[i] + c * 32, 16u);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ static uint4 piece(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
  }
  __device__ __forceinline__ void begin(int64_t first, int64_t last, int64_t step) {
#pragma unroll
    for (int d = 0; d < kSlots; ++d)
#pragma unroll
      for (int js = 0; js < JS; ++js) fetch(first + d * step, last, d, js);
  }
  __device__ __forceinline__ void run(const uint16_t (*hs)[kHsLd], int64_t first, int64_t last,
                                      int64_t step) {
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    int slot = 0;
    for (int64_t c = first; c < last; c += step) {
      const uint32_t from = ring + slot * kSlotBytes;
      float acc[MT][4][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[m][t][q] = 0.f;
#pragma unroll
      for (int js = 0; js < JS; ++js) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kSlots * JS - 1) : "memory");
        if (js * 32 < rank) {
          const int j = js * 32 + 8 * tig;
          uint4 b[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            b[t] = piece(from + (js * 4 + t) * 512);
            if (rank & 7) b[t] = keep_ranks(b[t], j, rank);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            if (m * 16 >= rows) break;
            const uint4 a0 = *reinterpret_cast<const uint4*>(&hs[m * 16 + gid][j]);
            const uint4 a1 = *reinterpret_cast<const uint4*>(&hs[m * 16 + gid + 8][j]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              mma_bf16(acc[m][t], a0.x, a1.x, a0.y, a1.y, b[t].x, b[t].y);
              mma_bf16(acc[m][t], a0.z, a1.z, a0.w, a1.w, b[t].z, b[t].w);
            }
          }
        }
        // (the lane's own copies only: what it has read it may overwrite)
        if (js < JS - 1) fetch(c + kSlots * step, last, slot, js);
      }
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i)
        if (at[i] >= 0)
          *reinterpret_cast<uint4*>(y_out + at[i] + c * 32) =
              add_row(piece(from + (4 * JS + i) * 512), acc[i >> 1], i & 1);
      fetch(c + kSlots * step, last, slot, JS - 1);
      slot = slot + 1 == kSlots ? 0 : slot + 1;
    }
  }
};

template <int MT, int NT>
__device__ __forceinline__ void zero_acc(float (&acc)[MT][NT][4]) {
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[m][t][q] = 0.f;
}

// ---- the kernel ------------------------------------------------------------------------
__device__ __forceinline__ void st_dsmem_u16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}

// Cluster (tile, slab): 8 CTAs. CTA c sums A x over its eighth of K for up to
// 16 MT rows of one adapter, takes an eighth of the (row, rank) sums from all
// parts through distributed shared memory, scales them, rounds them once to
// bf16 (the operand of the product with B: relative 2^-8 of the update at most,
// below the rounding of y itself where the update is no larger than y) and
// gives them to all eight; then every CTA updates its columns, the first of
// which are on their way since its part of A x was done. A slab is a range of
// columns; each slab sums A x again. The slabs are as many as fill the device
// with the tiles that the ids make, which only the device knows.
// Bound by its chain of waits: ids, A and x, two cluster barriers, B and y (67
// rows, 64 adapters of rank 32, 3584 x 18944: 17 us, of which about 2 for the
// rows, 5 for A x, 2 for the exchange, 6 for 48 MB of B and y). Asking B into L2
// ahead was slower (19 us: A queues behind it), as were B and y by way of
// registers, 25 us. Beside a linear (p.beside) all up to y runs while the linear
// does: 256 rows of 3584 x 3584 at rank 16 take 35.5 us together, 39.5 one after
// the other.
template <int NR, int MT, int JS, bool PLAN>
__global__ void __launch_bounds__(kLoraThreads, Expand<MT, JS>::kCtas)
lora_kernel(const LoraParams p) {
  constexpr int kRows = 16 * MT, kRed = 8 * NR + 1;
  // the warps' rings; before they are filled, red [kLoraWarps][kRows][kRed]
  extern __shared__ __align__(128) uint8_t rings[];
  constexpr int kRing = Expand<MT, JS>::kSlots * Expand<MT, JS>::kSlotBytes;
  float* red = reinterpret_cast<float*>(rings);
  __shared__ float part[kRows][JS * 32];
  __shared__ __align__(16) uint16_t hs[kRows][kHsLd];
  __shared__ uint32_t seen[PLAN ? 1 : kMaxSets / 32];
  __shared__ int rows_of[PLAN ? kRows : kLoraFewRows];
  __shared__ int sets[PLAN ? 1 : kLoraFewRows];  // a row's adapter, -1: none
  __shared__ int n_rows_s;
  auto wait = [] {
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
  };
  if (!p.beside) wait();
  auto leave = [&] {  // (a grid's end follows that of the one before)
    if (p.beside) griddep_wait();
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int rank_c = (int)cluster_ctarank();
  const int number = (int)(blockIdx.x / kLoraCluster);
  // this cluster's tile (or adapter, by its number in the batch) and slab of
  // columns: the tiles that there are share the grid's clusters
  int slabs = 1, slab = 0, b = 0;
  auto share = [&](int tiles) {
    slabs = max(1, min(p.max_slabs, p.clusters / tiles));
    slab = number % slabs;
    b = number / slabs;
  };
  // the adapter (-1: rows without one, which are copied) and its rows, in order
  int set = -1, n_rows = 0;
  if constexpr (PLAN) {
    int4 tile;
    const int n_tiles = __ldcg(p.head + 1), n_sorted = __ldcg(p.head);
    share(n_tiles + (int)((p.M - n_sorted + kRows - 1) / kRows));
    if (b < n_tiles) {
      tile = __ldcg(p.tiles + b);
      set = tile.x;
    } else {
      const int64_t first = n_sorted + (int64_t)(b - n_tiles) * kRows;
      tile = make_int4(-1, (int)first, (int)max((int64_t)0, min((int64_t)kRows, p.M - first)), 0);
    }
    n_rows = tile.z;
    if (n_rows == 0 || (set < 0 && p.y_in == p.y_out)) return leave();  // (the whole cluster)
    if ((int)threadIdx.x < n_rows) rows_of[threadIdx.x] = __ldcg(p.order + tile.y + threadIdx.x);
  } else {
    const int M = (int)p.M, words = (p.L + 31) / 32;
    int v = -1;
    if ((int)threadIdx.x < M) v = __ldcg(p.ids + threadIdx.x);
    for (int i = threadIdx.x; i < words; i += kLoraThreads) seen[i] = 0;
    __syncthreads();
    if ((int)threadIdx.x < M) {
      if (v >= 0 && v < p.L) atomicOr(&seen[v >> 5], 1u << (v & 31));
      else v = -1;
      sets[threadIdx.x] = v;
    }
    __syncthreads();
    // the b-th adapter of the batch (its bit, counted from below); one past the
    // last: the rows without an adapter
    int w = 0, n_sets = 0;
    for (int i = 0; i < words; ++i) n_sets += __popc(seen[i]);
    share(n_sets + 1);
    while (w < words && b >= __popc(seen[w])) b -= __popc(seen[w++]);
    if (w == words) {
      if (b > 0 || p.y_in == p.y_out) return leave();  // (the whole cluster)
    } else {
      uint32_t m = seen[w];
      for (; b > 0; --b) m &= m - 1;
      set = w * 32 + __ffs(m) - 1;
    }
    if (warp == 0) {
      int n = 0;
      for (int i0 = 0; i0 < M; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t hit = __ballot_sync(0xffffffffu, i < M && sets[i] == set);
        if ((hit >> lane) & 1) rows_of[n + __popc(hit & ((1u << lane) - 1))] = i;
        n += __popc(hit);
      }
      if (lane == 0) n_rows_s = n;
    }
  }
  __syncthreads();
  if constexpr (!PLAN) n_rows = n_rows_s;
  // this CTA's columns, 32 at a time
  const int64_t chunks = p.N / 32, parts = (int64_t)slabs * kLoraCluster;
  const int64_t me = (int64_t)slab * kLoraCluster + rank_c;
  const int64_t c_lo = me * chunks / parts, c_hi = (me + 1) * chunks / parts;
  if (set < 0) {
    if (p.beside) wait();
    // (all rows' vectors at once: row by row a tile of 32 took 10 us)
    const int nv = (int)(c_hi - c_lo) * 4;  // 16-byte vectors of a row
#pragma unroll 4
    for (int i = threadIdx.x; i < n_rows * nv; i += kLoraThreads) {
      const int row = i / nv;
      const int64_t at = (int64_t)rows_of[row] * p.N + (c_lo * 4 + i - row * nv) * 8;
      *reinterpret_cast<uint4*>(p.y_out + at) =
          __ldcg(reinterpret_cast<const uint4*>(p.y_in + at));
    }
    return;
  }
  const int rank = adapter_rank(p, set);
  const float sc = __ldcg(p.scale + set);
  const uint16_t* Bset = p.B + (int64_t)set * p.N * p.r;
  const int steps = (int)(p.K / 32);
  const int s0 = rank_c * steps / kLoraCluster, s1 = (rank_c + 1) * steps / kLoraCluster;
  const uint16_t* Ab = p.A + (int64_t)set * p.r * p.K + 8 * tig;
  for (int t0 = 0; t0 < n_rows; t0 += kRows) {
    const int rows = min(kRows, n_rows - t0);
    Expand<MT, JS> ex(p, Bset, rank, rows, smem_u32(rings) + warp * kRing,
                      [&](int i) { return rows_of[t0 + i]; });
    {
      const uint16_t* xr[2 * MT];
#pragma unroll
      for (int q = 0; q < 2 * MT; ++q)
        xr[q] = gid + 8 * q < rows ? p.x + (int64_t)rows_of[t0 + gid + 8 * q] * p.K + 8 * tig
                                   : nullptr;
      for (int c0 = 0; c0 < rank; c0 += 8 * NR) {
        float acc[MT][NR][4];
        zero_acc<MT, NR>(acc);
        shrink_steps<MT, NR>(acc, xr, Ab, p.K, c0, rank, s0 + warp, s1, kLoraWarps);
        float* mine = red + warp * kRows * kRed;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int t = 0; t < NR; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              mine[(m * 16 + (q >> 1) * 8 + gid) * kRed + t * 8 + tig * 2 + (q & 1)] =
                  acc[m][t][q];
        __syncthreads();
        for (int i = threadIdx.x; i < rows * 8 * NR; i += kLoraThreads) {
          const int j = i % (8 * NR), row = i / (8 * NR);
          float v = 0.f;
#pragma unroll
          for (int k = 0; k < kLoraWarps; ++k) v += red[(k * kRows + row) * kRed + j];
          if (c0 + j < JS * 32) part[row][c0 + j] = v;
        }
        __syncthreads();
      }
    }
    if (p.beside && t0 == 0) wait();
    ex.begin(c_lo + warp, c_hi, kLoraWarps);  // (red has been read)
    cluster_sync_all();  // every CTA's part is in its shared memory, and hs is free
    // an eighth of the rows' sums, in fours of ranks to a thread's row
    const int kr = (rank + 31) & ~31;
    const uint32_t part_at = smem_u32(part), hs_at = smem_u32(hs);
    for (int i = rank_c * kLoraThreads + threadIdx.x; i < kRows * kr;
         i += kLoraCluster * kLoraThreads) {
      const int row = i / kr, j = i - row * kr;
      float v = 0.f;
      const bool in = row < rows && j < rank;
      if (in) {
        const uint32_t at = part_at + (uint32_t)(row * JS * 32 + j) * 4;
        float q[kLoraCluster];
#pragma unroll
        for (int c = 0; c < kLoraCluster; ++c) q[c] = ld_dsmem_f32(map_to_rank(at, c));
#pragma unroll
        for (int c = 0; c < kLoraCluster; ++c) v += q[c];
      }
      // (ranks past the adapter's are zeros, whatever its scale is)
      const uint16_t h = in ? f32_to_bf16_bits(sc * v) : 0;
      const uint32_t to = hs_at + (uint32_t)(row * kHsLd + j) * 2;
#pragma unroll
      for (int c = 0; c < kLoraCluster; ++c) st_dsmem_u16(map_to_rank(to, c), h);
    }
    cluster_sync_all();  // (also the block's barrier) hs is whole; nothing remote follows
    ex.run(hs, c_lo + warp, c_hi, kLoraWarps);
    if (t0 + kRows < n_rows) __syncthreads();  // (the rings are red's again)
  }
}

// ---- very many rows: two kernels with A x between them in memory ------------------------
// h[split][sorted row][0, rank) = the split's part of A_a x. One CTA a tile of
// 32 rows and a part of K, which its warps share in 32-wide steps; each warp
// keeps kShrinkStages - 1 steps of its rows and of A in flight into a ring of
// its own (a lane reads back what it wrote: no barrier), and the warps add
// their sums to shared memory in turn. x is read once; A_a comes from L2, once
// a tile. Bound by the latency of its few steps: 4093 rows of 3584 at rank 64
// read 28 MB in 13 us (2.2 TB/s).
constexpr int kShrinkWarps = 4;
constexpr int kShrinkStages = 3;

template <int NR>
__global__ void __launch_bounds__(32 * kShrinkWarps)
lora_shrink_kernel(const LoraParams p) {
  constexpr int kStep = (4 + NR) * 512;  // bytes of a step: 4 row pairs' parts of x, NR of A
  extern __shared__ __align__(128) uint8_t ring[];  // [kShrinkWarps][kShrinkStages][kStep]
  __shared__ float red[kLoraTile][8 * NR + 1];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  constexpr int kSub = kManyTile / kLoraTile;
  const int number = (int)(blockIdx.x / kSub);
  if (number >= p.head[1]) return;
  int4 tile = __ldg(p.tiles + number);
  const int skip = (int)(blockIdx.x % kSub) * kLoraTile;
  tile.y += skip;
  tile.z = min(kLoraTile, tile.z - skip);
  if (tile.z <= 0) return;
  const int rank = adapter_rank(p, tile.x);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int steps = (int)(p.K / 32);
  const int s0 = (int)((int64_t)blockIdx.y * steps / p.splits) + warp;
  const int s1 = (int)((int64_t)(blockIdx.y + 1) * steps / p.splits);
  const uint16_t* xr[4];
  uint32_t x_bytes[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int row = q * 8 + gid;
    x_bytes[q] = row < tile.z ? 16u : 0u;
    xr[q] = p.x + (row < tile.z ? (int64_t)__ldg(p.order + tile.y + row) * p.K : 0) + 8 * tig;
  }
  uint8_t* mine = ring + warp * kShrinkStages * kStep;
  const uint32_t mine_at = smem_u32(mine) + lane * 16;
  // (a row without a rank or a token is read from row 0 and its bytes dropped)
  const uint16_t* Ab = p.A + (int64_t)tile.x * p.r * p.K + 8 * tig;
  for (int c0 = 0; c0 < rank; c0 += 8 * NR) {
    const uint16_t* ar[NR];
    uint32_t a_bytes[NR];
#pragma unroll
    for (int t = 0; t < NR; ++t) {
      const int j = c0 + t * 8 + gid;
      a_bytes[t] = j < rank ? 16u : 0u;
      ar[t] = Ab + (int64_t)(j < rank ? j : 0) * p.K;
    }
    auto issue = [&](int s, int stage) {
      if (s < s1) {
        const uint32_t st = mine_at + stage * kStep;
        const uint32_t off = (uint32_t)s * 32;
#pragma unroll
        for (int q = 0; q < 4; ++q) cp_async16_zfill(st + q * 512, xr[q] + off, x_bytes[q]);
#pragma unroll
        for (int t = 0; t < NR; ++t) cp_async16_zfill(st + (4 + t) * 512, ar[t] + off, a_bytes[t]);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    float acc[2][NR][4];
    zero_acc<2, NR>(acc);
#pragma unroll
    for (int i = 0; i < kShrinkStages - 1; ++i) issue(s0 + i * kShrinkWarps, i);
    int get = 0;
    for (int s = s0; s < s1; s += kShrinkWarps) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kShrinkStages - 2) : "memory");
      const uint8_t* st = mine + get * kStep + lane * 16;
      uint4 a[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) a[q] = *reinterpret_cast<const uint4*>(st + q * 512);
#pragma unroll
      for (int t = 0; t < NR; ++t) {
        const uint4 b = *reinterpret_cast<const uint4*>(st + (4 + t) * 512);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          mma_bf16(acc[mt][t], a[2 * mt].x, a[2 * mt + 1].x, a[2 * mt].y, a[2 * mt + 1].y, b.x, b.y);
          mma_bf16(acc[mt][t], a[2 * mt].z, a[2 * mt + 1].z, a[2 * mt].w, a[2 * mt + 1].w, b.z, b.w);
        }
      }
      // (the lane's own copies only: what it has read it may overwrite)
      issue(s + (kShrinkStages - 1) * kShrinkWarps, get == 0 ? kShrinkStages - 1 : get - 1);
      get = get + 1 == kShrinkStages ? 0 : get + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    for (int k = 0; k < kShrinkWarps; ++k) {
      if (warp == k) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int t = 0; t < NR; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float& v = red[mt * 16 + (q >> 1) * 8 + gid][t * 8 + tig * 2 + (q & 1)];
              v = k == 0 ? acc[mt][t][q] : v + acc[mt][t][q];
            }
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < tile.z * 8 * NR; i += 32 * kShrinkWarps) {
      const int j = i % (8 * NR), row = i / (8 * NR);
      if (c0 + j < rank)
        p.h[((int64_t)blockIdx.y * p.M + tile.y + row) * p.r + c0 + j] = red[row][j];
    }
    __syncthreads();
  }
}

// y = bf16(y0 + scale * B_a h). One CTA a tile of 128 rows and 256 columns, 32 a
// warp, whose part of B stays in registers (32 JS ranks at a time) while the
// rows go by, sixteen at a time, kAhead sixteens of y on their way; the tile's h
// (the splits added in order, scaled, rounded to bf16 once: see lora_kernel)
// lies in shared memory. Bound by y0 and y and by a CTA's start (plan, B, h, then
// y): 2 x 29 MB at 4093 x 3584 take about 23 us, where a copy of them alone takes
// 16 to 19.
template <int JS>
__global__ void __launch_bounds__(kLoraThreads, 2)
lora_expand_kernel(const LoraParams p) {
  // sixteens of rows whose y is on its way: what B leaves room for (4093 rows of
  // 3584, four / three / two of them: rank 64 41.5 / 43.7 / 42.9 us, rank 128
  // 72.5 / 67.9 / 63.8)
  constexpr int kAhead = JS < 4 ? 4 : 2;
  constexpr int LD = JS * 32 + 8;  // padded row of h: 16-byte rows, no bank conflicts
  __shared__ __align__(16) uint16_t hs[kManyTile][LD];
  // Every block of the first kernel waited for the plan before it let this one
  // start, so the plan, y and the weights are there and are asked for before
  // the wait (past L1: another kernel wrote them while this SM was busy).
  const int n_tiles = __ldcg(p.head + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  int4 tile;
  int rank = 0;
  if ((int)blockIdx.x < n_tiles) {
    tile = __ldcg(p.tiles + blockIdx.x);
    if (tile.z == 0) return griddep_wait();  // (a grid's end follows that of the one before)
    rank = adapter_rank(p, tile.x);
  } else {
    // tiles past the table copy the rows without an adapter, which the plan
    // lists last (nothing to do where y is updated in place)
    const int64_t first = __ldcg(p.head) + (int64_t)((int)blockIdx.x - n_tiles) * kManyTile;
    if (first >= p.M || p.y_in == p.y_out) return griddep_wait();
    tile = make_int4(0, (int)first, (int)min((int64_t)kManyTile, p.M - first), 0);
  }
  const int64_t c = (int64_t)blockIdx.y * kLoraWarps + warp;  // this warp's 32 columns
  const bool in = c * 32 < p.N;
  // B: column n of n8-tile t is column (n / 2) * 8 + 2t + n % 2 of the warp's,
  // so that a thread's sums over the four tiles are eight neighbouring columns
  // of y; eight ranks a thread and step of 32, as hs has them
  uint4 b[JS][4];
  {
    const uint16_t* src = p.B + ((int64_t)tile.x * p.N + c * 32 + (gid >> 1) * 8 + (gid & 1)) * p.r;
#pragma unroll
    for (int js = 0; js < JS; ++js) {
      const int j = js * 32 + 8 * tig;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        b[js][t] = make_uint4(0, 0, 0, 0);
        if (in && j < rank) b[js][t] = __ldcg(reinterpret_cast<const uint4*>(src + 2 * t * p.r + j));
      }
    }
    if (rank & 7) {
#pragma unroll
      for (int js = 0; js < JS; ++js)
#pragma unroll
        for (int t = 0; t < 4; ++t) b[js][t] = keep_ranks(b[js][t], js * 32 + 8 * tig, rank);
    }
  }
  // y of sixteen rows: this thread's two, a negative place where there is none
  int64_t at[kAhead][2];
  uint4 y[kAhead][2];
  auto fetch = [&](int m, int slot) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = m * 16 + half * 8 + gid;
      at[slot][half] = in && row < tile.z
                           ? (int64_t)__ldcg(p.order + tile.y + row) * p.N + c * 32 + 8 * tig
                           : -1;
    }
#pragma unroll
    for (int half = 0; half < 2; ++half)
      if (at[slot][half] >= 0)
        y[slot][half] = __ldcg(reinterpret_cast<const uint4*>(p.y_in + at[slot][half]));
  };
#pragma unroll
  for (int m = 0; m < kAhead; ++m) fetch(m, m);
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  if (rank > 0) {
    // a thread takes four ranks of a row (r is a multiple of 8)
    const float sc = __ldg(p.scale + tile.x);
    constexpr int kVec = JS * 8;  // fours of ranks in a row of hs
    constexpr int kEach = kManyTile * kVec / kLoraThreads;
    constexpr int kBatch = kEach < 4 ? kEach : 4;  // loads on their way at once
    for (int e0 = 0; e0 < kEach; e0 += kBatch) {
      float4 v[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s = 0; s < p.splits; ++s) {
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const int i = threadIdx.x + (e0 + e) * kLoraThreads, row = i / kVec, j = i % kVec * 4;
          if (row < tile.z && j < rank) {
            const float4 q = *reinterpret_cast<const float4*>(
                p.h + ((int64_t)s * p.M + tile.y + row) * p.r + j);
            v[e].x += q.x;
            v[e].y += q.y;
            v[e].z += q.z;
            v[e].w += q.w;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int i = threadIdx.x + (e0 + e) * kLoraThreads, row = i / kVec, j = i % kVec * 4;
        // (ranks past the adapter's were never written: leave them out)
        const __nv_bfloat162 lo = __floats2bfloat162_rn(j < rank ? sc * v[e].x : 0.f,
                                                        j + 1 < rank ? sc * v[e].y : 0.f);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(j + 2 < rank ? sc * v[e].z : 0.f,
                                                        j + 3 < rank ? sc * v[e].w : 0.f);
        *reinterpret_cast<uint2*>(&hs[row][j]) = make_uint2(
            *reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
    }
  }
  __syncthreads();
  const int m_end = (tile.z + 15) / 16;
  for (int m0 = 0; m0 < m_end; m0 += kAhead) {
#pragma unroll
    for (int slot = 0; slot < kAhead; ++slot) {
      const int m = m0 + slot;
      if (m >= m_end) break;
      float acc[4][4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[t][q] = 0.f;
#pragma unroll
      for (int js = 0; js < JS; ++js) {
        if (js * 32 >= rank) break;
        const uint4 a0 = *reinterpret_cast<const uint4*>(&hs[m * 16 + gid][js * 32 + 8 * tig]);
        const uint4 a1 = *reinterpret_cast<const uint4*>(&hs[m * 16 + gid + 8][js * 32 + 8 * tig]);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          mma_bf16(acc[t], a0.x, a1.x, a0.y, a1.y, b[js][t].x, b[js][t].y);
          mma_bf16(acc[t], a0.z, a1.z, a0.w, a1.w, b[js][t].z, b[js][t].w);
        }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half)
        if (at[slot][half] >= 0)
          *reinterpret_cast<uint4*>(p.y_out + at[slot][half]) = add_row(y[slot][half], acc, half);
      if (m + kAhead < m_end) fetch(m + kAhead, slot);
    }
  }
}

bool lora_few(int64_t M) { return M <= kLoraFewRows; }

// Whether a batch with a plan takes the two kernels. The cluster kernel holds 38
// tiles of 32 rows at once (a little more at high ranks, where its second round
// costs less than the two kernels' way of B) and repeats its chain of waits for
// the next ones; rows end a tile in the middle once an adapter, 3 / 8 of a tile
// on the measured mean. The two kernels read B once for every 128 rows of an
// adapter, which with few rows each and wide y costs more than those rounds, and
// start a CTA a 256 columns, where the cluster kernel goes through wide rows
// without a stop. Two kernels / cluster kernel, us, K = 3584, every row with an
// adapter:
//   N = 3584   2 adapters of rank 16, 1100 rows 18.4 / 16.0, 1200 rows 18.9 /
//              21.9; 8 of rank 64, 1000 rows 31.5 / 23.4, 1200 rows 33.5 / 34.7;
//              8 of rank 128, 1300 rows 55.1 / 52.8, 1400 rows 44.8 / 53.5; 32 of
//              rank 16, 800 rows 18.4 / 17.6, 900 rows 18.4 / 21.6; 128 of rank
//              16, 1000 rows 39.9 / 39.2
//   N = 7168   64 of rank 32, 1000 rows 43.4 / 33.7, 2100 rows 48.8 / 50.0; 128
//              of rank 16, 2100 rows 56.3 / 53.6; 8 of rank 64, 2500 rows 47.2 /
//              61.2
//   N = 9472   8 of rank 64, 1000 rows 45.8 / 30.8, 2500 rows 55.6 / 67.4
//   N = 12288  32 of rank 16, 1200 rows 37.3 / 36.2, 1400 rows 36.9 / 38.0, of
//              rank 64, 1700 rows 64.5 / 57.2, 2100 rows 71.4 / 73.5; 64 of rank
//              32, 2100 rows 72.3 / 59.2
//   N = 18944  8 of rank 16, 1000 rows 40.0 / 27.5, 4093 rows 101 / 92; 32 of
//              rank 32, 4093 rows 133 / 106, 16384 rows 444 / 358; 2 of rank 64,
//              2500 rows 84 / 91, 16384 rows 444 / 447
// A batch of more rows than one that takes them takes them too. (N below 16384
// also keeps the second kernel's column blocks within what a grid has in y.)
static bool lora_many(int64_t M, int64_t N, int L, int r) {
  const int64_t sets = std::min<int64_t>(L, M);
  return N < 16384 && 8 * M + 3 * kLoraTile * sets > 8 * kLoraTile * (r > 64 ? 44 : 38) &&
         160 * M >= sets * (N - 2048);
}

// Parts of K of the first kernel: about two CTAs an SM, each of two steps a warp
// or more.
static int lora_splits(int64_t M, int64_t K) {
  int64_t s = kManyCtas / (M / kLoraTile + 1);
  const int64_t most = K / (64 * kShrinkWarps);
  if (s > most) s = most;
  return s < 1 ? 1 : (int)s;
}

int64_t lora_h_rows(int64_t M) { return std::max<int64_t>(M, kManyCtas * kLoraTile); }

template <int NR>
static cudaError_t launch_shrink(const LoraParams& p, int64_t tiles, cudaStream_t st) {
  constexpr size_t kSmem = (size_t)kShrinkWarps * kShrinkStages * (4 + NR) * 512;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.ensure(lora_shrink_kernel<NR>, kSmem);
  if (e != cudaSuccess) return e;
  PdlConfig c(dim3((unsigned)tiles, (unsigned)p.splits, 1), 32 * kShrinkWarps, kSmem, st);
  return cudaLaunchKernelEx(&c.cfg, lora_shrink_kernel<NR>, p);
}

template <int NR, int MT, int JS, bool PLAN>
static cudaError_t launch_lora_kernel(LoraParams p, int64_t most, cudaStream_t st) {
  using Ex = Expand<MT, JS>;
  constexpr int kRing = Ex::kSlots * Ex::kSlotBytes, kRed = 16 * MT * (8 * NR + 1) * 4;
  constexpr size_t kSmem = (size_t)kLoraWarps * (kRing > kRed ? kRing : kRed);
  auto kern = lora_kernel<NR, MT, JS, PLAN>;
  static SmemOptIn opt_in;
  if (cudaError_t e = opt_in.ensure(kern, kSmem); e != cudaSuccess) return e;
  // clusters for every tile there could be, or for all SMs, which the tiles that
  // there are share
  p.clusters = device_sm_count() * Ex::kCtas / kLoraCluster;
  const int64_t clusters = std::max(most, std::min<int64_t>(most * p.max_slabs, p.clusters));
  if (clusters * kLoraCluster >= (1LL << 31)) return cudaErrorNotSupported;
  PdlConfig c(dim3((unsigned)(clusters * kLoraCluster), 1, 1), kLoraThreads, kSmem, st);
  cudaLaunchAttribute attr[2];
  attr[0] = c.attr[0];
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kLoraCluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  c.cfg.attrs = attr;
  c.cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&c.cfg, kern, p);
}

template <int MT, bool PLAN>
static cudaError_t launch_lora_rank(const LoraParams& p, int64_t most, cudaStream_t st) {
  return p.r <= 16   ? launch_lora_kernel<2, MT, 1, PLAN>(p, most, st)
         : p.r <= 32 ? launch_lora_kernel<4, MT, 1, PLAN>(p, most, st)
         : p.r <= 64 ? launch_lora_kernel<8, MT, 2, PLAN>(p, most, st)
                     : launch_lora_kernel<8, MT, 4, PLAN>(p, most, st);
}

cudaError_t launch_lora_plan(const LoraArgs& a, cudaStream_t st) {
  if (lora_few(a.M)) return cudaSuccess;
  return launch_plan(a.ids, a.M, a.L, lora_many(a.M, a.N, a.L, a.r) ? kManyTile : kLoraTile, a.plan, st,
                     true);
}

cudaError_t launch_lora(const LoraArgs& a, cudaStream_t st, bool beside) {
  LoraParams p;
  p.y_in = a.y_in;
  p.x = a.x;
  p.A = a.A;
  p.B = a.B;
  p.scale = a.scale;
  p.ranks = a.ranks;
  p.ids = a.ids;
  p.y_out = a.y_out;
  p.head = a.plan.head;
  p.tiles = a.plan.tiles;
  p.order = a.plan.order;
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.L = a.L;
  p.r = a.r;
  p.beside = beside;
  const bool few = lora_few(a.M);
  // (the rows without an adapter make at most ceil(M / tile) tiles more)
  const int64_t sets = a.L < a.M ? a.L : a.M;
  const bool many = lora_many(a.M, a.N, a.L, a.r);
  const int bt = many ? kManyTile : kLoraTile;
  const int64_t most = few ? sets + 1 : plan_max_tiles(a.M, a.L, bt) + (a.M + bt - 1) / bt;
  // slabs of 2048 columns at least
  p.max_slabs = (int)((a.N + 2047) / 2048);
  if (few) return launch_lora_rank<1, false>(p, most, st);
  cudaError_t e = cudaSuccess;
  if (!beside && (e = launch_plan(a.ids, a.M, a.L, bt, a.plan, st)) != cudaSuccess) return e;
  if (!many) return launch_lora_rank<2, true>(p, most, st);
  p.splits = lora_splits(a.M, a.K);
  p.h = a.h;
  const int64_t tiles = plan_max_tiles(a.M, a.L, bt) * (kManyTile / kLoraTile);
  e = a.r <= 16   ? launch_shrink<2>(p, tiles, st)
      : a.r <= 32 ? launch_shrink<4>(p, tiles, st)
                  : launch_shrink<8>(p, tiles, st);
  if (e != cudaSuccess) return e;
  PdlConfig c(dim3((unsigned)most, (unsigned)((a.N + 255) / 256), 1), kLoraThreads, 0, st);
  return a.r <= 32   ? cudaLaunchKernelEx(&c.cfg, lora_expand_kernel<1>, p)
         : a.r <= 64 ? cudaLaunchKernelEx(&c.cfg, lora_expand_kernel<2>, p)
                     : cudaLaunchKernelEx(&c.cfg, lora_expand_kernel<4>, p);
}

}  // namespace egopq
