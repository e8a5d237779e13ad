// mx4_pair.cu -- products of microscaled 4-bit operands with many rows: two CTAs, a
// cluster, share one instruction (cta_group::2) of 256 weight rows by up to 256 rows.
// Each holds 128 of the weight rows and half of the rows in shared memory, and
// 128 x 256 sums in its Tensor Memory.
//
// At four bits an operand byte feeds so many products that shared memory and L2 bind
// before the tensor cores do: a 128 x 128 tile needs 128 bytes of operands a cycle
// and CTA at the instructions' full rate, this one 64.
//
// Tensor Memory has 512 columns and two accumulators of 256 and two sets of scales
// need more, so the accumulators overlap: columns [kAcc1, 256) belong to both. A
// tile's instructions wait until the epilogue has read those of the tile before;
// the rest is read while they run.
#include "mx4_tc.cuh"

namespace egopq {

namespace {

constexpr int kBT = 256;      // rows of a tile at most
constexpr int kEpiWarps = 8;  // two for each 32 lanes of Tensor Memory
constexpr int kThreads = (kEpiWarps + 2) * 32;

template <int FMT>
struct Cfg {
  static constexpr int kRec = mx4_record_bytes(FMT);
  static constexpr int kScale = kRec - kMx4Codes;
  static constexpr int kAtoms = kScale / 512;
  // a stage: a weight record, half of the tile's rows, the scales of all of them
  static constexpr int kRowsAt = kRec;
  static constexpr int kRowScaleAt = kRec + 16384;
  static constexpr int kStage = kRowScaleAt + 2 * kScale;
  static constexpr int kStages = FMT == EGOPQ_MX4_E8M0 ? 6 : 5;
  static constexpr int kMiscAt = kStages * kStage;
  static constexpr int kMisc = 256;
  // scales: 128 weight rows' and 256 rows' words, in two sets
  static constexpr int kSetCols = 12 * kAtoms;
  static constexpr int kScaleAt = 512 - 2 * kSetCols;
  static constexpr int kAcc1 = kScaleAt - kBT;
  static constexpr int kShared = kBT - kAcc1;  // columns of both accumulators
  static_assert(kAcc1 >= 0 && kShared % 16 == 0 && kShared <= 96, "Tensor Memory");
  static_assert(kRec % 1024 == 0 && kStage % 1024 == 0, "swizzle atoms");
};

// ---- barriers of a pair -----------------------------------------------------------
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// mbar_wait for a barrier that the other CTA arrives on.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                             uint64_t timeout_ns) {
  if (try_wait_cluster(bar, parity)) return true;
  if (!mbar_wait(bar, parity, abort_flag, timeout_ns)) return false;
  return try_wait_cluster(bar, parity);  // (done: for its scope)
}
// Arrives on the barrier at this place in both CTAs when every instruction so far
// has completed.
__device__ __forceinline__ void commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void commit_own(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}

struct Unit {
  const uint8_t* w;     // this CTA's first weight record
  const uint8_t* rows;  // the tile's first row record
  int64_t row0;         // first row of y
  int count, cols;      // rows; the instruction's columns
  int n0;               // this CTA's first column of y
  int set;
};

// Sixteen columns (rows of y) of one lane's weight row. Two-byte results of an even
// N leave in pairs: lanes exchange, the even one taking one row of y, the odd one
// the next.
__device__ __forceinline__ void store16(const Mx4Params& p, const Unit& un, int c, int64_t n,
                                        const uint32_t (&v)[16], float g) {
  const int left = un.count - c;
  const bool odd = threadIdx.x & 1;
  if (p.type != kMx4F32 && (p.N & 1) == 0) {
    uint16_t* y = static_cast<uint16_t*>(p.y) + (un.row0 + c + (odd ? 1 : 0)) * p.N + (n & ~1);
    const bool in = n < p.N;
#pragma unroll
    for (int q = 0; q < 16; q += 2) {
      const float v0 = __uint_as_float(v[q]) * g, v1 = __uint_as_float(v[q + 1]) * g;
      const float other = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
      const float lo = odd ? other : v0, hi = odd ? v1 : other;
      uint32_t w;
      if (p.type == kMx4Bf16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        w = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        const __half2 b = __floats2half2_rn(lo, hi);
        w = *reinterpret_cast<const uint32_t*>(&b);
      }
      if (in && q + (odd ? 1 : 0) < left) *reinterpret_cast<uint32_t*>(y) = w;
      y += 2 * p.N;
    }
    return;
  }
  if (n >= p.N) return;
  int64_t at = (un.row0 + c) * p.N + n;
#pragma unroll
  for (int q = 0; q < 16; ++q, at += p.N)
    if (q < left) store_y(p.y, at, p.type, __uint_as_float(v[q]) * g);
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1) mx4_pair_kernel(const Mx4Params p) {
  using C = Cfg<FMT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const uint32_t bars = base + C::kMiscAt;
  auto full = [&](int s) { return bars + 8u * s; };
  auto peer_full = [&](int s) { return bars + 8u * (C::kStages + s); };
  auto empty = [&](int s) { return bars + 8u * (2 * C::kStages + s); };
  auto done = [&](int b) { return bars + 8u * (3 * C::kStages + b); };
  auto early = [&] { return bars + 8u * (3 * C::kStages + 2); };
  auto fin = [&] { return bars + 8u * (3 * C::kStages + 3); };
  uint8_t* misc = smem + C::kMiscAt + 8 * (3 * C::kStages + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 4);
  int* first = reinterpret_cast<int*>(smem + C::kMiscAt + C::kMisc);
  int* block = first + p.sets + 1;
  int* tile = block + p.sets + 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(peer_full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) mbar_init(done(b), 1);
    mbar_init(early(), 2 * kEpiWarps);
    mbar_init(fin(), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kEpiWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == 0) {
    // (the offsets were there before this kernel could begin: see mx4_few_kernel)
    if (p.offsets) mx4_scan_sets(p.offsets, p.sets, p.M, kBT, first, block, tile);
    else if (lane < 2) {
      first[lane] = lane ? (int)p.M : 0;
      block[lane] = 0;
      tile[lane] = lane ? (int)((p.M + kBT - 1) / kBT) : 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // (both CTAs' barriers are there before either arrives on one)
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint64_t tmo = p.timeout_ns;
  const int nbp = (p.nb + 1) / 2;
  const int team = (int)blockIdx.x / 2, teams = (int)gridDim.x / 2;
  const int total = tile[p.sets] * nbp;
  const int n_units = team < total ? (total - team + teams - 1) / teams : 0;
  const int n_items = n_units * p.kb;
  auto unit_at = [&](int i) {
    const int u = team + i * teams;
    const int e = mx4_find_set(tile, p.sets, u / nbp);
    const int tiles = tile[e + 1] - tile[e];
    const int local = u - tile[e] * nbp;
    const int n = local / tiles, t = local - n * tiles;
    Unit r;
    r.set = e;
    // (of an odd number of blocks the last pair's second is the last again: its
    // columns of y do not exist)
    r.w = p.packed + ((int64_t)e * p.nb + min(2 * n + rank, p.nb - 1)) * p.kb * C::kRec;
    r.rows = p.operand + (int64_t)(block[e] + 2 * t) * p.kb * C::kRec;
    r.row0 = (int64_t)first[e] + (int64_t)t * kBT;
    r.count = min(kBT, first[e + 1] - (int)r.row0);
    r.cols = (r.count + 15) & ~15;
    r.n0 = (2 * n + rank) * 128;
    return r;
  };

  if (warp == kEpiWarps) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      int issued = 0;
      Unit un{};
      const int ahead = min(C::kStages, n_items);
      auto load_w = [&](const Unit& x, int kb, int s) {
        const uint32_t bytes =
            C::kRec + x.cols / 2 * 128 + (x.cols > 128 ? 2 : 1) * C::kScale;
        mbar_arrive_expect_tx(full(s), bytes);
        bulk_load(base + s * C::kStage, x.w + (int64_t)kb * C::kRec, C::kRec, full(s));
      };
      // this CTA's half of the rows: of the first record, the second, or both
      auto load_rows = [&](const Unit& x, int kb, int s) {
        const uint8_t* rec = x.rows + (int64_t)kb * C::kRec;
        const uint8_t* next = rec + (int64_t)p.kb * C::kRec;
        const uint32_t to = base + s * C::kStage;
        const int half = x.cols / 2, from = rank * half;
        const int here = max(0, min(half, 128 - from));  // rows in the first record
        if (here) bulk_load(to + C::kRowsAt, rec + from * 128, here * 128, full(s));
        if (here < half)
          bulk_load(to + C::kRowsAt + here * 128, next + (from + here - 128) * 128,
                    (half - here) * 128, full(s));
        bulk_load(to + C::kRowScaleAt, rec + kMx4Codes, C::kScale, full(s));
        if (x.cols > 128)
          bulk_load(to + C::kRowScaleAt + C::kScale, next + kMx4Codes, C::kScale, full(s));
      };
      // (weights before this kernel's own wait: see mx4_few_kernel)
      for (int i = 0; i < ahead; ++i) {
        if (i % p.kb == 0) un = unit_at(i / p.kb);
        load_w(un, i % p.kb, i);
      }
      griddep_wait();
      griddep_launch_dependents();
      for (int i = 0; i < ahead; ++i) {
        if (i % p.kb == 0) un = unit_at(i / p.kb);
        load_rows(un, i % p.kb, i);
        ++issued;
      }
      int unit = (ahead - 1) / p.kb, kb = (ahead - 1) % p.kb;
      for (int i = ahead; i < n_items; ++i) {
        const int s = i % C::kStages;
        if (!mbar_wait(empty(s), ((i / C::kStages) & 1) ^ 1, abort_flag, tmo)) break;
        if (++kb == p.kb) {
          kb = 0;
          un = unit_at(++unit);
        }
        load_w(un, kb, s);
        load_rows(un, kb, s);
        ++issued;
      }
      for (int i = (issued > C::kStages ? issued - C::kStages : 0); i < issued; ++i) {
        volatile int no_abort = 0;
        mbar_wait(full(i % C::kStages), (i / C::kStages) & 1, &no_abort, tmo);
      }
      // the leader's arrivals on this CTA's barriers are there before it leaves
      for (int i = (issued > C::kStages ? issued - C::kStages : 0); i < issued; ++i)
        if (!mbar_wait(empty(i % C::kStages), (i / C::kStages) & 1, abort_flag, tmo)) break;
    }
  } else if (warp == kEpiWarps + 1) {
    if (lane == 0 && rank == 1) {
      // ------------------------------------------------- this CTA's part is there
      for (int i = 0; i < n_items; ++i) {
        const int s = i % C::kStages;
        if (!mbar_wait(full(s), (i / C::kStages) & 1, abort_flag, tmo)) break;
        arrive_cluster(map_to_rank(peer_full(s), 0));
      }
    } else if (lane == 0) {
      // -------------------------------------------------------------- issuer
      bool ok = true;
      int i = 0;
      for (int k = 0; k < n_units && ok; ++k) {
        const int cols = unit_at(k).cols;
        const uint32_t d = tmem + (k & 1) * C::kAcc1;
        // the shared columns have been read of the tile before, and so all of the
        // one before that
        if (k >= 1) ok = wait_cluster(early(), (k - 1) & 1, abort_flag, tmo);
        for (int kb = 0; kb < p.kb && ok; ++kb, ++i) {
          const int s = i % C::kStages;
          ok = mbar_wait(full(s), (i / C::kStages) & 1, abort_flag, tmo) &&
               wait_cluster(peer_full(s), (i / C::kStages) & 1, abort_flag, tmo);
          // the scales' set is free once the instructions of two K blocks before
          // have completed
          if (ok && i >= 2)
            ok = mbar_wait(empty((i - 2) % C::kStages), ((i - 2) / C::kStages) & 1, abort_flag, tmo);
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = base + s * C::kStage;
          const uint32_t sa = tmem + C::kScaleAt + (i & 1) * C::kSetCols, sb = sa + 4 * C::kAtoms;
#pragma unroll
          for (int j = 0; j < C::kAtoms; ++j) {
            tc_cp_scales<2>(sa + 4 * j, at + kMx4Codes + j * 512);
            tc_cp_scales<2>(sb + 8 * j, at + C::kRowScaleAt + j * 512);
            if (cols > 128)
              tc_cp_scales<2>(sb + 8 * j + 4, at + C::kRowScaleAt + C::kScale + j * 512);
          }
          tc_block_mx4<FMT, 2>(d, at, at + C::kRowsAt, sa, 4, sb, 8, 256, cols,
                               mx4_steps(p.K, kb), kb == 0);
          commit_both(empty(s));
        }
        if (ok) commit_both(done(k & 1));
      }
      if (i > 0) {  // what was issued ends before either CTA does
        commit_own(fin());
        volatile int no_abort = 0;
        mbar_wait(fin(), 0, &no_abort, tmo);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    griddep_wait();
    const uint32_t early_at = map_to_rank(early(), 0);
    const int mine = warp >> 2;  // of the pieces of 16 columns: the even or the odd ones
    bool ok = true;
    for (int k = 0; k < n_units; ++k) {
      const Unit un = unit_at(k);
      const int b = k & 1;
      float g = p.a_scale ? __ldg(p.a_scale) : 1.f;
      if (p.w_scale) g *= __ldg(p.w_scale + un.set);
      ok = mbar_wait(done(b), (k >> 1) & 1, abort_flag, tmo);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + b * C::kAcc1 + ((uint32_t)((warp & 3) * 32) << 16);
      const int64_t n = un.n0 + (warp & 3) * 32 + lane;
      // the shared columns first: accumulator 0's last, accumulator 1's first
      constexpr int kFirst = (C::kShared / 16 + 1) / 2;
      const int c0 = b ? 0 : C::kAcc1;
      uint32_t v[kFirst][16];
#pragma unroll
      for (int j = 0; j < kFirst; ++j) {
        const int c = (2 * j + mine) * 16;
        if (c < C::kShared && c0 + c < un.cols) tmem_ld16(d + c0 + c, v[j]);
      }
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(early_at);
#pragma unroll
      for (int j = 0; j < kFirst; ++j) {
        const int c = (2 * j + mine) * 16;
        if (c < C::kShared && c0 + c < un.cols) store16(p, un, c0 + c, n, v[j], g);
      }
      // (read before the next tile's are, and so before the instructions that
      // wait for those)
      const int from = b ? C::kShared : 0, to = min(un.cols, b ? kBT : C::kAcc1);
      for (int c = from + mine * 16; c < to; c += 32) {
        uint32_t u[16];
        tmem_ld16(d + c, u);
        tmem_wait_ld();
        store16(p, un, c, n, u, g);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // (neither leaves while the other's instructions or arrivals may reach it)
  if (warp == kEpiWarps + 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <int FMT>
cudaError_t launch_pair(const Mx4GemmArgs& a, cudaStream_t st) {
  using C = Cfg<FMT>;
  Mx4Params p;
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
  const int64_t tiles = a.offsets ? mx4_tiles(a.M, a.sets, kBT) : (a.M + kBT - 1) / kBT;
  const int64_t most = tiles * ((p.nb + 1) / 2);
  const int pairs = device_sm_count() / 2;
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  if (most >= (1LL << 31) || (most / pairs + 1) * p.kb >= (1LL << 31))
    return cudaErrorNotSupported;
  const size_t smem = C::kMiscAt + C::kMisc + 3 * (size_t)(a.sets + 1) * sizeof(int);
  auto kern = mx4_pair_kernel<FMT>;
  static SmemOptIn opt_in;
  if (cudaError_t e = opt_in.ensure(kern, smem); e != cudaSuccess) return e;
  PdlConfig c(dim3((unsigned)(2 * (most < pairs ? most : pairs)), 1, 1), kThreads, smem, st);
  cudaLaunchAttribute attr[2] = {c.attr[0], {}};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  c.cfg.attrs = attr;
  c.cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&c.cfg, kern, p);
}

}  // namespace

cudaError_t launch_mx4_pair(const Mx4GemmArgs& a, cudaStream_t st) {
  return a.format == EGOPQ_MX4_E8M0 ? launch_pair<EGOPQ_MX4_E8M0>(a, st)
                                    : launch_pair<EGOPQ_MX4_E4M3>(a, st);
}

cudaError_t take_error_word_mx4_pair(unsigned* out) { return take_local_error_word(out); }

}  // namespace egopq
