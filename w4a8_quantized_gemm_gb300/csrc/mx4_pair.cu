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
// the rest, 0.63 of a tile's columns (E4M3, whose scales take more, 0.44), is read while
// they run.
//
// Measured: 4096 x 18944 x 3584 87 us (6.4 PFLOP/s; E4M3, with twice the scales to
// copy, 96), 8192 x 8192 x 8192 149 us (7.4), the tensor pipe busy for 68 % of the first
// (E4M3 63). A K block takes some 540 cycles, of which its instructions are 512, and a
// change of tiles 2000, in which they stand still: with few K blocks (K = 1408 has six)
// that is over a third of a tile.
#include "mx4_tc.cuh"
#include "tc_kernel.cuh"  // (encode_fn)

namespace egopq {

namespace {

constexpr int kBT = 256;      // rows of a tile at most
constexpr int kEpiWarps = 8;  // two for each 32 lanes of Tensor Memory
// then: the instructions' issuer, the scales' (of the weight rows and of each 128
// rows), and two producers
constexpr int kMmaWarp = kEpiWarps, kCopyWarp = kMmaWarp + 1, kCopies = 3,
              kWeightWarp = kCopyWarp + kCopies, kRowWarp = kWeightWarp + 1;
constexpr int kThreads = (kRowWarp + 1) * 32;

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
  // scales: 128 weight rows' and 256 rows' words, in sets
  static constexpr int kSetCols = 12 * kAtoms;
  static constexpr int kSets = FMT == EGOPQ_MX4_E8M0 ? 4 : 3;
  static constexpr int kScaleAt = 512 - kSets * kSetCols;
  static constexpr int kAcc1 = kScaleAt - kBT;
  static constexpr int kShared = kBT - kAcc1;  // columns of both accumulators
  static_assert(kAcc1 >= 0 && kShared % 16 == 0 && kShared <= 144, "Tensor Memory");
  static_assert(kRec % 1024 == 0 && kStage % 1024 == 0, "swizzle atoms");
};

// ---- barriers of a pair -----------------------------------------------------------
// Arrives on another CTA's barrier, for Tensor Memory that has been read (its fence is
// beside the call), so it orders no memory of this thread's beyond the CTA: a
// release to the cluster waits 0.7 us for that.
__device__ __forceinline__ void arrive_remote(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// Rows of 128 bytes from row y on, to this CTA's shared memory; `bar` may be the
// other CTA's.
__device__ __forceinline__ void load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(y)
      : "memory");
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

// The operands as tensors of 128-byte rows, a record kRec / 128 of them (a bulk copy
// without a tensor map could not tell the other CTA's barrier of its arrival).
struct Maps {
  CUtensorMap weight;  // a record
  CUtensorMap rows;    // 128 rows
  CUtensorMap part;    // 32 rows
  CUtensorMap scale;   // a record's scales
};

struct Unit {
  int w;                // this CTA's first weight record
  int rows;             // the tile's first row record
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
    const uint32_t take = odd ? 0x3276u : 0x5410u;  // (of this lane's two values and the other's)
#pragma unroll
    for (int q = 0; q < 16; q += 2) {
      const float v0 = __uint_as_float(v[q]) * g, v1 = __uint_as_float(v[q + 1]) * g;
      uint32_t w;
      if (p.type == kMx4Bf16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v0, v1);
        w = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        const __half2 b = __floats2half2_rn(v0, v1);
        w = *reinterpret_cast<const uint32_t*>(&b);
      }
      w = __byte_perm(w, __shfl_xor_sync(0xffffffffu, w, 1), take);
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
__global__ void __launch_bounds__(kThreads, 1) mx4_pair_kernel(const __grid_constant__ Maps maps,
                                                                const Mx4Params p) {
  using C = Cfg<FMT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const uint32_t bars = base + C::kMiscAt;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (C::kStages + s); };
  auto done = [&](int b) { return bars + 8u * (2 * C::kStages + b); };
  auto early = [&] { return bars + 8u * (2 * C::kStages + 2); };
  auto fin = [&] { return bars + 8u * (2 * C::kStages + 3); };
  auto brought = [&](int q) { return bars + 8u * (2 * C::kStages + 4 + q); };
  uint8_t* misc = smem + C::kMiscAt + 8 * (2 * C::kStages + 4 + C::kSets);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 4);
  int* first = reinterpret_cast<int*>(smem + C::kMiscAt + C::kMisc);
  int* block = first + p.sets + 1;
  int* tile = block + p.sets + 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 2);  // (the leader's two producers; both CTAs' bytes)
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) mbar_init(done(b), 1);
    mbar_init(early(), 2 * kEpiWarps);
    mbar_init(fin(), 1 + kCopies);
    for (int q = 0; q < C::kSets; ++q) mbar_init(brought(q), kCopies);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
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
    r.w = (e * p.nb + min(2 * n + rank, p.nb - 1)) * p.kb;
    r.rows = (block[e] + 2 * t) * p.kb;
    r.row0 = (int64_t)first[e] + (int64_t)t * kBT;
    r.count = min(kBT, first[e + 1] - (int)r.row0);
    // (above 128 all 256, garbage among them: one copy then brings a half, where one of
    // 32 rows at a time takes longer than the instructions: 900 x 18944 x 3584 32.2 /
    // 29.5 us, 700 x 8192 x 8192 31.1 / 29.6)
    r.cols = r.count <= 128 ? (r.count + 15) & ~15 : kBT;
    r.n0 = (2 * n + rank) * 128;
    return r;
  };

  // Producers, a thread for weights and one for rows and their scales, in each CTA.
  // The leader's tell its barrier what both bring.
  auto produce = [&](auto&& bytes_of, auto&& load) {
    Ring<C::kStages> r;
    int i = 0;
    bool ok = true;
    for (int k = 0; k < n_units && ok; ++k) {
      const Unit un = unit_at(k);
      const uint32_t bytes = 2 * bytes_of(un);
      for (int kb = 0; kb < p.kb; ++kb, ++i, r.next()) {
        if (i >= C::kStages && !mx4_wait(empty(r.s), r.phase ^ 1, abort_flag, tmo)) {
          ok = false;
          break;
        }
        if (rank == 0) mbar_arrive_expect_tx(full(r.s), bytes);
        load(un, kb, base + r.s * C::kStage, map_to_rank(full(r.s), 0));
      }
    }
    // What is on its way has landed, and the leader's arrivals are there, before this
    // CTA leaves: an item's copies have been waited for by its instructions.
    for (int j = max(0, i - C::kStages); j < i; ++j) {
      volatile int no_abort = 0;
      if (rank == 0) mx4_wait(full(j % C::kStages), (j / C::kStages) & 1, &no_abort, tmo);
      if (!mx4_wait(empty(j % C::kStages), (j / C::kStages) & 1, &no_abort, tmo)) break;
    }
  };
  constexpr int kRecRows = C::kRec / 128;
  if (warp == kWeightWarp) {
    // Weights need no wait: nothing that may still run in front of this kernel
    // writes them (what makes weights lets no kernel begin before it has ended).
    if (lane == 0)
      produce([&](const Unit&) { return (uint32_t)C::kRec; },
              [&](const Unit& x, int kb, uint32_t to, uint32_t bar) {
                int rec = x.w + kb;
                if (!dbg_record_ok((uint64_t)rec * C::kRec, C::kRec,
                                   (uint64_t)p.sets * p.nb * p.kb * C::kRec))
                  rec = 0;
                load_pair(to, &maps.weight, bar, rec * kRecRows);
              });
  } else if (warp == kRowWarp) {
    if (lane == 0) {
      griddep_wait();
      griddep_launch_dependents();
      produce(
          [&](const Unit& x) {
            return x.cols == kBT ? 16384u + 2 * C::kScale
                                 : (uint32_t)(x.cols + 63) / 64 * 32 * 128 + C::kScale;
          },
          [&](const Unit& x, int kb, uint32_t to, uint32_t bar) {
            const int rec = (x.rows + kb) * kRecRows, next = rec + p.kb * kRecRows;
            if (x.cols == kBT) {
              load_pair(to + C::kRowsAt, &maps.rows, bar, rank ? next : rec);
            } else {
              // this CTA's half, 32 rows at a time
              for (int c = 0; c < x.cols / 2; c += 32)
                load_pair(to + C::kRowsAt + c * 128, &maps.part, bar,
                          rec + rank * x.cols / 2 + c);
            }
            load_pair(to + C::kRowScaleAt, &maps.scale, bar, rec + 128);
            if (x.cols == kBT)
              load_pair(to + C::kRowScaleAt + C::kScale, &maps.scale, bar, next + 128);
          });
    }
  } else if (warp >= kCopyWarp && warp < kCopyWarp + kCopies) {
    // ------------------------------------------------------------------- scales
    // An instruction takes its warp 50 cycles and more to issue, those of a K block
    // 512 to run: beside the products' issuer, the weight rows' and each 128 rows'
    // scales have a warp of their own (E4M3's twelve copies in one took 940 cycles).
    // The warps run whole, so that what an instruction reads is formed in uniform
    // registers, and one lane issues (a branch of one lane around all of it took
    // twice the time).
    if (rank == 0) {
      const int part = warp - kCopyWarp;
      const uint64_t scales = sdesc_scales(
          base + (part == 0 ? (uint32_t)kMx4Codes : C::kRowScaleAt + (part - 1) * C::kScale));
      const uint32_t to = tmem + C::kScaleAt + (part == 0 ? 0 : 4 * C::kAtoms + 4 * (part - 1));
      const int step = part == 0 ? 4 : 8;
      bool ok = true;
      int i = 0;
      Ring<C::kStages> r, before;  // item i, item i - kSets
      Ring<C::kSets> set;
      for (int k = 0; k < n_units && ok; ++k) {
        const bool have = part < 2 || unit_at(k).cols == kBT;
        for (int kb = 0; kb < p.kb; ++kb, ++i, r.next(), set.next()) {
          // its parts are there, and the instructions that read the set last have
          // completed
          ok = mx4_wait_warp(full(r.s), r.phase, abort_flag, tmo);
          if (ok && i >= C::kSets) {
            ok = mx4_wait_warp(empty(before.s), before.phase, abort_flag, tmo);
            before.next();
          }
          if (!ok) break;
          tc_fence_after();
          const uint64_t from = mx4_at(scales, r.s * C::kStage);
          const uint32_t at = to + set.s * C::kSetCols;
          if (lane == 0) {
            if (have) {
#pragma unroll
              for (int q = 0; q < C::kAtoms; ++q)
                tc_cp_scales<2>(at + step * q, mx4_at(from, q * 512));
            }
            commit_own(brought(set.s));
          }
          __syncwarp();
        }
      }
      if (lane == 0) commit_own(fin());  // what was issued ends before either CTA does
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------- issuer
    if (rank == 0) {
      const uint64_t operand = sdesc_kmajor_sw128(base);
      const int last_steps = mx4_steps(p.K, p.kb - 1);
      bool ok = true;
      Ring<C::kStages> r;
      Ring<C::kSets> set;
      for (int k = 0; k < n_units && ok; ++k) {
        const uint32_t idesc = idesc_mx4<FMT>(256, unit_at(k).cols);
        const uint32_t d = tmem + (k & 1) * C::kAcc1;
        // the shared columns have been read of the tile before, and so all of the
        // one before that
        if (k >= 1) ok = mx4_wait_warp(early(), (k - 1) & 1, abort_flag, tmo);
        for (int kb = 0; kb < p.kb && ok; ++kb, r.next(), set.next()) {
          // (with the scales the operands that they came with)
          ok = mx4_wait_warp(brought(set.s), set.phase, abort_flag, tmo);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sa = tmem + C::kScaleAt + set.s * C::kSetCols;
          const uint64_t a = mx4_at(operand, r.s * C::kStage), b = mx4_at(a, C::kRowsAt);
          const bool last = kb + 1 == p.kb;
          const int steps = last ? last_steps : 4;
          if (lane == 0) {
            tc_block_mx4<FMT, 2>(d, a, b, sa, sa + 4 * C::kAtoms, 8, idesc, steps, kb == 0);
            commit_both(empty(r.s));
            if (last) commit_both(done(k & 1));
          }
          __syncwarp();
        }
      }
      if (lane == 0) commit_own(fin());
      __syncwarp();
      volatile int no_abort = 0;
      mx4_wait_warp(fin(), 0, &no_abort, tmo);
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
      ok = mx4_wait_warp(done(b), (k >> 1) & 1, abort_flag, tmo);
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
        if (c < C::kShared && c0 + c < un.count) tmem_ld16(d + c0 + c, v[j]);
      }
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_remote(early_at);
#pragma unroll
      for (int j = 0; j < kFirst; ++j) {
        const int c = (2 * j + mine) * 16;
        if (c < C::kShared && c0 + c < un.count) store16(p, un, c0 + c, n, v[j], g);
      }
      // (read before the next tile's are, and so before the instructions that
      // wait for those)
      const int from = b ? C::kShared : 0, to = min(un.count, b ? kBT : C::kAcc1);
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
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// A buffer as a tensor of 128-byte rows, read `box` rows at a time.
bool make_map(CUtensorMap* map, const void* ptr, int64_t rows, int box) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {128, (cuuint64_t)rows};
  cuuint64_t strides[1] = {128};
  cuuint32_t boxes[2] = {128, (cuuint32_t)box};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, boxes,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT>
cudaError_t launch_pair(const Mx4GemmArgs& a, cudaStream_t st) {
  using C = Cfg<FMT>;
  const Mx4Params p = params_of(a);
  const int64_t tiles = a.offsets ? mx4_tiles(a.M, a.sets, kBT) : (a.M + kBT - 1) / kBT;
  const int64_t most = tiles * ((p.nb + 1) / 2);
  const int pairs = device_sm_count() / 2;
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  if (most >= (1LL << 31) || (most / pairs + 1) * p.kb >= (1LL << 31))
    return cudaErrorNotSupported;
  // the operands' rows of 128 bytes
  const int64_t rec_rows = C::kRec / 128;
  const int64_t blocks = a.offsets ? mx4_row_blocks(a.M, a.sets) : (a.M + 127) / 128;
  const int64_t w_rows = (int64_t)a.sets * p.nb * p.kb * rec_rows;
  const int64_t x_rows = blocks * p.kb * rec_rows;
  if (w_rows >= (1LL << 31) || x_rows >= (1LL << 31)) return cudaErrorNotSupported;
  Maps maps;
  if (!make_map(&maps.weight, a.packed, w_rows, (int)rec_rows) ||
      !make_map(&maps.rows, a.operand, x_rows, 128) ||
      !make_map(&maps.part, a.operand, x_rows, 32) ||
      !make_map(&maps.scale, a.operand, x_rows, C::kScale / 128))
    return cudaErrorInvalidValue;
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
  return cudaLaunchKernelEx(&c.cfg, kern, maps, p);
}

}  // namespace

cudaError_t launch_mx4_pair(const Mx4GemmArgs& a, cudaStream_t st) {
  return a.format == EGOPQ_MX4_E8M0 ? launch_pair<EGOPQ_MX4_E8M0>(a, st)
                                    : launch_pair<EGOPQ_MX4_E4M3>(a, st);
}

cudaError_t take_error_word_mx4_pair(unsigned* out) { return take_local_error_word(out); }
cudaError_t set_record_limit_mx4_pair(unsigned long long bytes) {
  return set_local_record_limit(bytes);
}

}  // namespace egopq
