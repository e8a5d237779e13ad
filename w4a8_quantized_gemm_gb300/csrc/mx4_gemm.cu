// mx4_gemm.cu -- products of microscaled 4-bit rows and weights on the tensor
// cores' block-scaled instructions (tcgen05.mma kind::mxf4nvf4).
//
//   y[m][n] = g_a g_w sum_b s_a[m][b] s_w[n][b] sum_{k in b} c_a[m][k] c_w[n][k]
//
// The instruction multiplies codes, applies both blocks' scales and adds up in
// fp32, so a tile is: one bulk copy a K block and operand (records,
// mx4_internal.h), the scales copied from shared to Tensor Memory, four
// instructions of 64 K each, and an epilogue that applies the tensors' scales and
// rounds once. Weights are the instruction's 128 rows and a tile of one set's rows
// its columns, as many as there are (a multiple of 16): few rows, or a ragged
// set's last ones, cost what they are.
#include "mx4_internal.h"

namespace egopq {

namespace {

constexpr int kBT = 128;      // rows of a tile at most
constexpr int kEpiWarps = 4;  // one for each 32 lanes of Tensor Memory
constexpr int kThreads = (kEpiWarps + 2) * 32;

template <int FMT>
struct Cfg {
  static constexpr int kRec = mx4_record_bytes(FMT);
  static constexpr int kScale = kRec - kMx4Codes;
  static constexpr int kAtoms = kScale / 512;  // of a K block and 128 rows
  static constexpr int kStage = 2 * kRec;      // a weight record and a row record
  static constexpr int kStages = 6;
  static constexpr int kMiscAt = kStages * kStage;
  static constexpr int kMisc = 256;
  // Tensor Memory: two accumulators, then each stage's scales
  static constexpr int kScaleCols = 8 * kAtoms;
  static_assert(2 * kBT + kStages * kScaleCols <= 512, "Tensor Memory");
  static_assert(kRec % 1024 == 0, "swizzle atoms");
};

struct GemmParams {
  const uint8_t* operand;
  const uint8_t* packed;
  const float* a_scale;
  const float* w_scale;
  const int32_t* offsets;
  void* y;
  int64_t M, N, K;
  int sets, nb, kb, type;
  uint64_t timeout_ns;
};

__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint32_t saddr) {
  // 32 lanes x 16 bytes, to all four lane quarters: rows of 16 bytes, eight rows
  // of 128 bytes a core matrix (stride 128), no swizzle
  const uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) |
                     static_cast<uint64_t>(128 >> 4) << 32 | static_cast<uint64_t>(1) << 46;
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}
template <int FMT>
__device__ __forceinline__ void tc_mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t sa, uint32_t sb, uint32_t accumulate) {
  if constexpr (FMT == EGOPQ_MX4_E8M0)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
// e2m1 x e2m1, fp32 sums, K = 64, both K-major; id: which two of a word's four
// scales (0 or 2; with 4X all four).
template <int FMT>
__device__ __forceinline__ uint32_t idesc_mx4(int rows, int cols, int id) {
  return ((uint32_t)id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(cols >> 3) << 17) |
         ((FMT == EGOPQ_MX4_E8M0 ? 1u : 0u) << 23) | ((uint32_t)(rows >> 4) << 24) |
         ((uint32_t)id << 29);
}

__device__ __forceinline__ void store_y(void* y, int64_t at, int type, float v) {
  if (type == kMx4F32) static_cast<float*>(y)[at] = v;
  else
    static_cast<uint16_t*>(y)[at] = type == kMx4Bf16
                                        ? f32_to_bf16_bits(v)
                                        : __half_as_ushort(__float2half_rn(v));
}

// A unit of work: a block of weight rows times a tile of one set's rows.
struct Unit {
  const uint8_t* w;     // its first weight record
  const uint8_t* rows;  // its first row record
  int64_t row0;         // first row of y
  int count;            // rows
  int n0;               // first column of y
  int set;
};

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1) mx4_gemm_kernel(const GemmParams p) {
  using C = Cfg<FMT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = base + C::kMiscAt;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (C::kStages + s); };
  auto done = [&](int b) { return bars + 8u * (2 * C::kStages + b); };
  auto free_acc = [&](int b) { return bars + 8u * (2 * C::kStages + 2 + b); };
  auto fin = [&] { return bars + 8u * (2 * C::kStages + 4); };
  uint8_t* misc = smem + C::kMiscAt + 8 * (2 * C::kStages + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 4);
  int* first = reinterpret_cast<int*>(smem + C::kMiscAt + C::kMisc);
  int* block = first + p.sets + 1;  // (a tile is a block of 128 rows)

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(done(b), 1);
      mbar_init(free_acc(b), kEpiWarps);
    }
    mbar_init(fin(), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kEpiWarps + 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == 0) {
    // (the offsets were there before this kernel could begin: the quantization in
    // front of a ragged product waits for them itself, every block of it)
    if (p.offsets) mx4_scan_sets(p.offsets, p.sets, p.M, first, block);
    else if (lane < 2) {
      first[lane] = lane ? (int)p.M : 0;
      block[lane] = lane ? (int)((p.M + kBT - 1) / kBT) : 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint64_t tmo = p.timeout_ns;
  const int total = block[p.sets] * p.nb;
  const int n_units = (int)blockIdx.x < total
                          ? (total - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x
                          : 0;
  // Neighbouring blocks take one weight block and a set's tiles one after the
  // other, so that a weight is read from memory once.
  auto unit_at = [&](int i) {
    const int u = (int)blockIdx.x + i * (int)gridDim.x;
    const int e = mx4_find_set(block, p.sets, u / p.nb);
    const int tiles = block[e + 1] - block[e];
    const int local = u - block[e] * p.nb;
    const int n = local / tiles, t = local - n * tiles;
    Unit r;
    r.set = e;
    r.w = p.packed + ((int64_t)e * p.nb + n) * p.kb * C::kRec;
    r.rows = p.operand + (int64_t)(block[e] + t) * p.kb * C::kRec;
    r.row0 = (int64_t)first[e] + (int64_t)t * kBT;
    r.count = min(kBT, first[e + 1] - (int)r.row0);
    r.n0 = n * 128;
    return r;
  };

  if (warp == kEpiWarps) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      const int n_items = n_units * p.kb;
      int issued = 0;
      Unit un{};
      // the first weights are on their way before this kernel's own wait: nothing
      // that may still run in front of it writes weights
      const int ahead = min(C::kStages, n_items);
      auto bytes_of = [&](const Unit& x) {
        return (uint32_t)(C::kRec + ((x.count + 7) & ~7) * 128 + C::kScale);
      };
      auto load_w = [&](const Unit& x, int kb, int s) {
        mbar_arrive_expect_tx(full(s), bytes_of(x));
        bulk_load(base + s * C::kStage, x.w + (int64_t)kb * C::kRec, C::kRec, full(s));
      };
      auto load_rows = [&](const Unit& x, int kb, int s) {
        const uint8_t* rec = x.rows + (int64_t)kb * C::kRec;
        const uint32_t to = base + s * C::kStage + C::kRec;
        bulk_load(to, rec, (uint32_t)((x.count + 7) & ~7) * 128, full(s));
        bulk_load(to + kMx4Codes, rec + kMx4Codes, C::kScale, full(s));
      };
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
      for (int i = ahead; i < n_items; ++i) {
        const int s = i % C::kStages;
        if (!mbar_wait(empty(s), ((i / C::kStages) & 1) ^ 1, abort_flag, tmo)) break;
        if (i % p.kb == 0) un = unit_at(i / p.kb);
        load_w(un, i % p.kb, s);
        load_rows(un, i % p.kb, s);
        ++issued;
      }
      for (int i = (issued > C::kStages ? issued - C::kStages : 0); i < issued; ++i) {
        volatile int no_abort = 0;
        mbar_wait(full(i % C::kStages), (i / C::kStages) & 1, &no_abort, tmo);
      }
    }
  } else if (warp == kEpiWarps + 1) {
    // ---------------------------------------------------------------- issuer
    if (lane == 0) {
      bool ok = true;
      int i = 0;
      for (int k = 0; k < n_units && ok; ++k) {
        const int cols = (unit_at(k).count + 15) & ~15;
        const int b = k & 1;
        if (k >= 2) ok = mbar_wait(free_acc(b), ((k >> 1) & 1) ^ 1, abort_flag, tmo);
        const uint32_t d = tmem + b * kBT;
        for (int kb = 0; kb < p.kb && ok; ++kb, ++i) {
          const int s = i % C::kStages;
          ok = mbar_wait(full(s), (i / C::kStages) & 1, abort_flag, tmo);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a_at = base + s * C::kStage, b_at = a_at + C::kRec;
          // a stage's scales have columns of their own: they are free once the
          // stage is
          const uint32_t sa = tmem + 2 * kBT + s * C::kScaleCols, sb = sa + 4 * C::kAtoms;
#pragma unroll
          for (int j = 0; j < C::kAtoms; ++j) {
            tc_cp_scales(sa + 4 * j, a_at + kMx4Codes + j * 512);
            tc_cp_scales(sb + 4 * j, b_at + kMx4Codes + j * 512);
          }
          const int steps = (int)min((int64_t)4, (p.K - (int64_t)kb * 256 + 63) / 64);
          for (int j = 0; j < steps; ++j) {
            const int at = C::kAtoms == 4 ? j : j >> 1, id = C::kAtoms == 4 ? 0 : (j & 1) * 2;
            tc_mma_mx4<FMT>(d, sdesc_kmajor_sw128(a_at + 32 * j), sdesc_kmajor_sw128(b_at + 32 * j),
                            idesc_mx4<FMT>(128, cols, id), sa + 4 * at, sb + 4 * at,
                            (kb | j) != 0);
          }
          tc_commit(empty(s));
        }
        if (ok) tc_commit(done(b));
      }
      if (i > 0) {  // what was issued ends before the block does
        tc_commit(fin());
        volatile int no_abort = 0;
        mbar_wait(fin(), 0, &no_abort, tmo);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    griddep_wait();
    bool ok = true;
    for (int k = 0; k < n_units && ok; ++k) {
      const Unit un = unit_at(k);
      const int b = k & 1;
      float g = p.a_scale ? __ldg(p.a_scale) : 1.f;
      if (p.w_scale) g *= __ldg(p.w_scale + un.set);
      ok = mbar_wait(done(b), (k >> 1) & 1, abort_flag, tmo);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + b * kBT + ((uint32_t)(warp * 32) << 16);
      const int64_t n = un.n0 + warp * 32 + lane;
      const bool in = n < p.N;
      for (int c = 0; c < un.count; c += 16) {
        uint32_t v[16];
        tmem_ld16(d + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 16; ++q)
          if (in && c + q < un.count)
            store_y(p.y, (un.row0 + c + q) * p.N + n, p.type, __uint_as_float(v[q]) * g);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(free_acc(b));
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kEpiWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int FMT>
cudaError_t launch_fmt(const Mx4GemmArgs& a, cudaStream_t st) {
  using C = Cfg<FMT>;
  GemmParams p;
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
  p.timeout_ns = a.timeout_ns;
  const int64_t tiles =
      a.offsets ? mx4_row_blocks(a.M, a.sets) : (a.M + kBT - 1) / kBT;
  const int64_t most = tiles * p.nb;
  const int sms = device_sm_count();
  if (sms < 1) return cudaErrorInvalidConfiguration;
  if (most >= (1LL << 31) || (most / sms + 1) * p.kb >= (1LL << 31)) return cudaErrorNotSupported;
  const size_t smem = C::kMiscAt + C::kMisc + 2 * (size_t)(a.sets + 1) * sizeof(int);
  auto kern = mx4_gemm_kernel<FMT>;
  static SmemOptIn opt_in;
  if (cudaError_t e = opt_in.ensure(kern, smem); e != cudaSuccess) return e;
  PdlConfig c(dim3((unsigned)(most < sms ? most : sms), 1, 1), kThreads, smem, st);
  return cudaLaunchKernelEx(&c.cfg, kern, p);
}

}  // namespace

cudaError_t launch_mx4_gemm(const Mx4GemmArgs& a, cudaStream_t st) {
  return a.format == EGOPQ_MX4_E8M0 ? launch_fmt<EGOPQ_MX4_E8M0>(a, st)
                                    : launch_fmt<EGOPQ_MX4_E4M3>(a, st);
}

cudaError_t take_error_word_mx4_gemm(unsigned* out) { return take_local_error_word(out); }

}  // namespace egopq
