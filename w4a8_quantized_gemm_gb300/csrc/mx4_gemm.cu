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
#include "mx4_quant.cuh"
#include "mx4_tc.cuh"

namespace egopq {

namespace {

constexpr int kBT = 64;       // rows of a tile at most
constexpr int kEpiWarps = 4;  // one for each 32 lanes of Tensor Memory
constexpr int kMmaWarp = kEpiWarps, kWeightWarp = kMmaWarp + 1, kRowWarp = kMmaWarp + 2;
constexpr int kExtraWarps = 4;  // beside the epilogue's, where rows are quantized here
constexpr int kMaxSplit = 8;  // CTAs that share a unit's K, a cluster

// Rows that the kernel quantizes itself (XT their type; kNone: they come as records):
// a handful, of one linear, once a CTA and for the K blocks that are its own. They
// then lie in shared memory behind the ring, and a stage holds weights alone. That
// leaves out a kernel and the wait for its results.
constexpr int kNone = -1;
constexpr int kOwnRows = 16;             // at most
// Runs of 256 values a CTA, at most. Calls that quantize so / apart, us, behind one
// another in a graph (outside of one, where the host's time counts, a launch less is 2
// us less):
//   18944 x 3584   1 row (7 runs) 8.9 / 11.3   8 (56) 11.3 / 12.2   12 (84) 12.8 / 12.5
//     gated        1 (7) 9.2 / 11.3   4 (28) 10.9 / 11.7   6 (42) 12.1 / 12.0
//   3584 x 18944   1 (10) 9.6 / 11.7   6 (60) 11.7 / 11.8   8 (80) 12.2 / 11.8
//     gated        1 (10) 10.4 / 11.7   2 (20) 11.0 / 11.7   4 (40) 12.8 / 12.3
//   3584 x 3584    1 (2) 5.3 / 6.5   8 (16) 5.6 / 6.7   16 (32) 6.5 / 7.4
constexpr int kOwnRuns = 64, kOwnGatedRuns = 32;
constexpr int kOwnBytes = 40960;         // codes and scales, at most

// Two CTAs share an SM, so that one's loads cover the other's ends.
template <int FMT, int XT>
struct Cfg {
  static constexpr bool kOwn = XT != kNone;
  static constexpr int kQuantWarps = kEpiWarps + kExtraWarps;
  static constexpr int kThreads = (kRowWarp + 1 + (kOwn ? kExtraWarps : 0)) * 32;
  static constexpr int kRec = mx4_record_bytes(FMT);
  static constexpr int kScale = kRec - kMx4Codes;
  static constexpr int kAtoms = kScale / 512;  // of a K block and 128 rows
  static constexpr int kRowsAt = kRec;         // a stage: a weight record, rows' codes, scales
  static constexpr int kRowScaleAt = kRec + kBT * 128;
  static constexpr int kStage = kOwn ? kRec : kRowScaleAt + kScale;
  static constexpr int kStages = kOwn || FMT == EGOPQ_MX4_E8M0 ? 4 : 3;
  static constexpr int kMiscAt = kStages * kStage;
  static constexpr int kMisc = 256;
  // Tensor Memory: two accumulators, then each stage's scales
  static constexpr int kScaleCols = 8 * kAtoms;
  static constexpr int kCols = 256;
  static_assert(2 * kBT + kStages * kScaleCols <= kCols, "Tensor Memory");
  static_assert(kRec % 1024 == 0 && kStage % 1024 == 0, "swizzle atoms");
  static_assert(kStages * kStage >= kBT * 512, "partial sums");
};

// A unit of work: a block of weight rows times a tile of one set's rows.
struct Unit {
  const uint8_t* w;     // its first weight record
  const uint8_t* rows;  // its first row record
  int64_t row0;         // first row of y
  int count;            // rows
  int half;             // first row in its records
  int n0;               // first column of y
  int set;
};

// x: the rows, where the kernel quantizes them (GATED: [gate | up]); p.operand else.
template <int FMT, int XT, bool GATED>
__global__ void __launch_bounds__(Cfg<FMT, XT>::kThreads, 2)
    mx4_few_kernel(const Mx4Params p, const void* x) {
  using C = Cfg<FMT, XT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t bars = base + C::kMiscAt;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (C::kStages + s); };
  auto done = [&](int b) { return bars + 8u * (2 * C::kStages + b); };
  auto free_acc = [&](int b) { return bars + 8u * (2 * C::kStages + 2 + b); };
  auto fin = [&] { return bars + 8u * (2 * C::kStages + 4); };
  auto own = [&] { return bars + 8u * (2 * C::kStages + 5); };
  uint8_t* misc = smem + C::kMiscAt + 8 * (2 * C::kStages + 6);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 4);
  int* first = reinterpret_cast<int*>(smem + C::kMiscAt + C::kMisc);
  int* block = first + p.sets + 1;
  int* tile = block + p.sets + 1;
  // own rows: behind the sets, 1024-byte aligned: [K block][codes of 16 rows], then
  // [K block][scales]
  constexpr int kOwnAt = C::kMiscAt + 1024;
  static_assert(C::kMisc + 6 * sizeof(int) <= 1024, "one set's words");

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), C::kOwn ? 1 : 2);  // (producers)
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(done(b), 1);
      mbar_init(free_acc(b), kEpiWarps);
    }
    mbar_init(fin(), 1);
    mbar_init(own(), C::kQuantWarps);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), C::kCols);
    tmem_relinquish();
  }
  if (warp == 0) {
    // (the offsets were there before this kernel could begin: the quantization in
    // front of a ragged product waits for them itself, every block of it)
    if (p.offsets) mx4_scan_sets(p.offsets, p.sets, p.M, kBT, first, block, tile);
    else if (lane < 2) {
      first[lane] = lane ? (int)p.M : 0;
      block[lane] = 0;
      tile[lane] = lane ? (int)((p.M + kBT - 1) / kBT) : 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint64_t tmo = p.timeout_ns;
  // A cluster of `split` CTAs takes a unit, each an equal run of its K blocks.
  const int split = p.split, rank = split > 1 ? (int)cluster_ctarank() : 0;
  const int team = (int)blockIdx.x / split, teams = (int)gridDim.x / split;
  const int total = tile[p.sets] * p.nb;
  const int n_units = team < total ? (total - team + teams - 1) / teams : 0;
  const int kb0 = p.kb * rank / split, kb_n = p.kb * (rank + 1) / split - kb0;
  // Neighbouring CTAs take one weight block and a set's tiles one after the
  // other, so that a weight is read from memory once.
  auto unit_at = [&](int i) {
    const int u = team + i * teams;
    const int e = mx4_find_set(tile, p.sets, u / p.nb);
    const int tiles = tile[e + 1] - tile[e];
    const int local = u - tile[e] * p.nb;
    const int n = local / tiles, t = local - n * tiles;
    Unit r;
    r.set = e;
    r.w = p.packed + (((int64_t)e * p.nb + n) * p.kb + kb0) * C::kRec;
    r.row0 = (int64_t)first[e] + (int64_t)t * kBT;
    r.count = min(kBT, first[e + 1] - (int)r.row0);
    // (a tile begins at row 0 or 64 of a record: its scales two columns in)
    r.rows = p.operand + ((int64_t)(block[e] + t * kBT / 128) * p.kb + kb0) * C::kRec;
    r.half = t * kBT % 128;
    r.n0 = n * 128;
    return r;
  };

  // Producers, a thread each for weights and rows: issuing a copy takes some 60
  // cycles, and a stage's barriers more. Each tells the stage's barrier what it
  // brings.
  auto produce = [&](auto&& bytes_of, auto&& load) {
    Ring<C::kStages> r;
    int i = 0;
    bool ok = true;
    for (int k = 0; k < n_units && ok; ++k) {
      const Unit un = unit_at(k);
      const uint32_t bytes = bytes_of(un);
      for (int kb = 0; kb < kb_n; ++kb, ++i, r.next()) {
        if (i >= C::kStages && !mx4_wait(empty(r.s), r.phase ^ 1, abort_flag, tmo)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(full(r.s), bytes);
        load(un, kb, base + r.s * C::kStage, full(r.s));
      }
    }
    for (int j = max(0, i - C::kStages); j < i; ++j) {  // what is on its way lands
      volatile int no_abort = 0;
      mx4_wait(full(j % C::kStages), (j / C::kStages) & 1, &no_abort, tmo);
    }
  };
  if constexpr (C::kOwn) {
    // (the epilogue's warps and those behind the last role)
    const int qw = warp < kEpiWarps ? warp : warp > kRowWarp ? warp - (kRowWarp + 1) + kEpiWarps : -1;
    if (qw >= 0) {
      griddep_wait();
      if (threadIdx.x == 0) griddep_launch_dependents();
      if (n_units > 0) {
        // Runs of 256 values, two of a warp's on their way at a time.
        constexpr int kAhead = 2, kLanes = mx4_block(FMT) / 8, kStep = C::kQuantWarps;
        const bool scaled = p.a_scale != nullptr;
        const float rg = scaled ? __fdiv_rn(1.f, __ldg(p.a_scale)) : 1.f;
        const int64_t ld = GATED ? 2 * p.K : p.K;
        const int runs = (int)p.M * kb_n;
        for (int u0 = qw; u0 < runs; u0 += kStep * kAhead) {
          Eight<XT> g8[kAhead], u8[kAhead];
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            const int u = u0 + j * kStep, row = u / kb_n, kb = u - row * kb_n;
            const int64_t k = (int64_t)(kb0 + kb) * 256 + lane * 8;
            g8[j].zero();
            u8[j].zero();
            if (u < runs && k < p.K) {
              g8[j].load(x, row * ld + k);
              if constexpr (GATED) u8[j].load(x, row * ld + p.K + k);
            }
          }
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            const int u = u0 + j * kStep, row = u / kb_n, kb = u - row * kb_n;
            if (u >= runs) break;
            const int b = lane / kLanes;
            RowOut out{};
            out.rec = smem + kOwnAt + kb * 2048 + row * 128 + ((((lane >> 2) ^ row) & 7) << 4) +
                      (lane & 3) * 4;
            out.rec_scale = smem + kOwnAt + kb_n * 2048 + kb * C::kScale + (b >> 2) * 512 +
                            row * 16 + (b & 3);
            quant_unit<FMT, XT, GATED>(out, 0, g8[j], u8[j], true, scaled, rg);
          }
        }
        fence_proxy_async_smem();  // (the tensor cores read what these threads wrote)
        __syncwarp();
        if (lane == 0) mbar_arrive(own());
      }
    }
  }
  if (warp == kWeightWarp) {
    // Weights need no wait: nothing that may still run in front of this kernel
    // writes them (what makes weights lets no kernel begin before it has ended).
    if (lane == 0)
      produce([&](const Unit&) { return (uint32_t)C::kRec; },
              [&](const Unit& x, int kb, uint32_t to, uint32_t bar) {
                const uint8_t* rec = x.w + (int64_t)kb * C::kRec;
                if (!dbg_record_ok((uint64_t)(rec - p.packed), C::kRec,
                                   (uint64_t)p.sets * p.nb * p.kb * C::kRec))
                  rec = p.packed;
                bulk_load(to, rec, C::kRec, bar);
              });
  } else if (warp == kRowWarp) {
    if (!C::kOwn && lane == 0) {
      griddep_wait();
      griddep_launch_dependents();
      produce([&](const Unit& x) { return (uint32_t)((x.count + 7) & ~7) * 128 + C::kScale; },
              [&](const Unit& x, int kb, uint32_t to, uint32_t bar) {
                const uint8_t* rec = x.rows + (int64_t)kb * C::kRec;
                bulk_load(to + C::kRowsAt, rec + x.half * 128, (uint32_t)((x.count + 7) & ~7) * 128,
                          bar);
                bulk_load(to + C::kRowScaleAt, rec + kMx4Codes, C::kScale, bar);
              });
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- issuer
    // (The warp runs whole, so that what an instruction reads is formed in uniform
    // registers, and one lane issues.)
    const uint64_t operand = sdesc_kmajor_sw128(base), scales = sdesc_scales(base);
    const int last_steps = mx4_steps(p.K, p.kb - 1);
    bool ok = true, any = false;
    if (C::kOwn && n_units > 0) ok = mx4_wait_warp(own(), 0, abort_flag, tmo);
    Ring<C::kStages> r;
    for (int k = 0; k < n_units && ok; ++k) {
      const Unit un = unit_at(k);
      const uint32_t idesc = idesc_mx4<FMT>(128, (un.count + 15) & ~15);
      const int b = k & 1;
      if (k >= 2) ok = mx4_wait_warp(free_acc(b), ((k >> 1) & 1) ^ 1, abort_flag, tmo);
      const uint32_t d = tmem + b * kBT;
      for (int kb = 0; kb < kb_n && ok; ++kb, r.next()) {
        ok = mx4_wait_warp(full(r.s), r.phase, abort_flag, tmo);
        if (!ok) break;
        tc_fence_after();
        any = true;
        // a stage's scales have columns of their own: they are free once the
        // stage is
        const uint32_t sa = tmem + 2 * kBT + r.s * C::kScaleCols, sb = sa + 4 * C::kAtoms;
        const uint64_t from = mx4_at(scales, r.s * C::kStage);
        const uint64_t from_r = C::kOwn ? mx4_at(scales, kOwnAt + kb_n * 2048 + kb * C::kScale)
                                        : mx4_at(from, C::kRowScaleAt);
        const uint64_t at_w = mx4_at(operand, r.s * C::kStage);
        const uint64_t at_r = C::kOwn ? mx4_at(operand, kOwnAt + kb * 2048)
                                      : mx4_at(at_w, C::kRowsAt);
        const int steps = kb0 + kb + 1 == p.kb ? last_steps : 4;
        if (lane == 0) {
#pragma unroll
          for (int j = 0; j < C::kAtoms; ++j) {
            tc_cp_scales<1>(sa + 4 * j, mx4_at(from, kMx4Codes + j * 512));
            tc_cp_scales<1>(sb + 4 * j, mx4_at(from_r, j * 512));
          }
          tc_block_mx4<FMT, 1>(d, at_w, at_r, sa, sb + un.half / 32, 4, idesc, steps, kb == 0);
          tc_commit(empty(r.s));
          if (kb + 1 == kb_n) tc_commit(done(b));
        }
        __syncwarp();
      }
    }
    if (any) {  // what was issued ends before the block does
      if (lane == 0) tc_commit(fin());
      __syncwarp();
      volatile int no_abort = 0;
      mx4_wait_warp(fin(), 0, &no_abort, tmo);
    }
  } else if (warp < kEpiWarps) {
    // ---------------------------------------------------------------- epilogue
    griddep_wait();
    bool ok = true;
    for (int k = 0; k < n_units && ok; ++k) {
      const Unit un = unit_at(k);
      const int b = k & 1;
      float g = p.a_scale ? __ldg(p.a_scale) : 1.f;
      if (p.w_scale) g *= __ldg(p.w_scale + un.set);
      ok = mx4_wait_warp(done(b), (k >> 1) & 1, abort_flag, tmo);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + b * kBT + ((uint32_t)(warp * 32) << 16);
      const int64_t n = un.n0 + warp * 32 + lane;
      const bool in = n < p.N;
      // (of a split unit: the sums as they are, [column][128], over the stages,
      // which all instructions have read)
      float* part = reinterpret_cast<float*>(smem) + warp * 32 + lane;
      for (int c = 0; c < un.count; c += 16) {
        uint32_t v[16];
        tmem_ld16(d + c, v);
        tmem_wait_ld();
        if (split > 1) {
#pragma unroll
          for (int q = 0; q < 16; ++q) part[(c + q) * 128] = __uint_as_float(v[q]);
          continue;
        }
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
  if (split > 1) {
    // One unit a cluster. CTA r adds up columns r, r + split, ..: the parts in
    // their order, whoever came first.
    cluster_sync_all();
    if (warp < kEpiWarps && n_units > 0) {
      const Unit un = unit_at(0);
      float g = p.a_scale ? __ldg(p.a_scale) : 1.f;
      if (p.w_scale) g *= __ldg(p.w_scale + un.set);
      const int64_t n = un.n0 + warp * 32 + lane;
      if (n < p.N)
        for (int c = rank; c < un.count; c += split) {
          const uint32_t at = base + (uint32_t)(c * 128 + warp * 32 + lane) * 4;
          float sum = 0.f;
#pragma unroll
          for (int r = 0; r < kMaxSplit; ++r)
            if (r < split) sum += ld_dsmem_f32(map_to_rank(at, r));
          store_y(p.y, (un.row0 + c) * p.N + n, p.type, sum * g);
        }
    }
    cluster_sync_all();  // (no CTA leaves while another reads its parts)
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

int64_t few_units(const Mx4GemmArgs& a) {
  return (a.offsets ? mx4_tiles(a.M, a.sets, kBT) : (a.M + kBT - 1) / kBT) * ((a.N + 127) / 128);
}

// Fewer units than the SMs hold CTAs: K is split.
int few_split(int64_t units, int64_t kb, int sms) {
  int64_t s = 2 * (int64_t)sms / units;
  if (s > kMaxSplit) s = kMaxSplit;
  if (s > kb) s = kb;
  return s < 1 ? 1 : (int)s;
}

template <int FMT, int XT, bool GATED>
cudaError_t launch_few(const Mx4GemmArgs& a, const void* x, cudaStream_t st) {
  using C = Cfg<FMT, XT>;
  Mx4Params p = params_of(a);
  const int64_t most = few_units(a);
  const int sms = device_sm_count();
  if (sms < 1) return cudaErrorInvalidConfiguration;
  if (most >= (1LL << 31) || (most / sms + 1) * p.kb >= (1LL << 31)) return cudaErrorNotSupported;
  p.split = few_split(most, p.kb, sms);
  const int64_t slots = 2 * sms;
  const int kb_most = (p.kb + p.split - 1) / p.split;
  size_t smem = C::kMiscAt + (C::kOwn ? 1024 + kb_most * (2048 + C::kScale)
                                      : C::kMisc + 3 * (size_t)(a.sets + 1) * sizeof(int));
  // Never three CTAs an SM, which Tensor Memory holds two of: the third's wait for it
  // and a cluster's for its other CTAs could wait for one another.
  if (smem < 80 * 1024) smem = 80 * 1024;
  auto kern = mx4_few_kernel<FMT, XT, GATED>;
  static SmemOptIn opt_in;
  if (cudaError_t e = opt_in.ensure(kern, smem); e != cudaSuccess) return e;
  PdlConfig c(dim3((unsigned)(p.split > 1 ? most * p.split : most < slots ? most : slots), 1, 1),
              C::kThreads, smem, st);
  cudaLaunchAttribute attr[2] = {c.attr[0], {}};
  if (p.split > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    c.cfg.attrs = attr;
    c.cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&c.cfg, kern, p, x);
}

template <int FMT>
cudaError_t launch_own(const Mx4GemmArgs& a, const Mx4QuantArgs& q, cudaStream_t st) {
  if (q.type == kMx4Bf16)
    return q.gated ? launch_few<FMT, kMx4Bf16, true>(a, q.x, st)
                   : launch_few<FMT, kMx4Bf16, false>(a, q.x, st);
  return q.gated ? launch_few<FMT, kMx4F16, true>(a, q.x, st)
                 : launch_few<FMT, kMx4F16, false>(a, q.x, st);
}

// Whether a linear's rows are few enough for the kernel to quantize, `runs` a CTA.
bool own_fits(const Mx4GemmArgs& a, int sms, int runs) {
  if (a.offsets || a.M > kOwnRows) return false;
  const int64_t kb = mx4_kblocks(a.K), split = few_split(few_units(a), kb, sms);
  const int64_t kb_most = (kb + split - 1) / split;
  return a.M * kb_most <= runs &&
         kb_most * (2048 + mx4_record_bytes(a.format) - kMx4Codes) <= kOwnBytes;
}

// Which kernel a product takes. One linear: by a rough model of what each would take, in
// us: a start, K blocks one after the other (with the columns of a tile), and a split
// unit's sums. Measured, E8M0, products alone:
//   N x K          rows   this kernel / pairs
//   3584 x 3584    64: 7.0 / 7.0   128: 8.2 / 7.5   192: 10.1 / 8.0
//   18944 x 3584   17: 10.6 / 9.1  64: 14.3 / 9.3
//   3584 x 18944   17: 9.9 / 23.6  192: 18.3 / 25.7  256: 24.1 / 26.1  384: 35.0 / 25.9
//   50257 x 2048   17: 11.5 / 12.1  64: 13.4 / 12.6  128: 16.6 / 13.9
//   512 x 3584     17: 4.0 / 6.7   512: 6.9 / 8.0
// The model is up to a third off (a split K's blocks cost less than it says, pairs of few
// units start sooner) and picks the slower side in three of these places, each next to
// where the two cross: 128 rows of 3584 x 3584 (this kernel, 0.7 us), 256 of 3584 x 18944
// (pairs, 2.0) and 17 of 50257 x 2048 (pairs, 0.6).
// Ragged rows, whose sets only the device knows: by their mean over all sets, 64 sets of
// 2560 x 3584, mean 32: 64.0 / 64.4, 64: 72.1 / 70.8, 96: 86.9 / 78.3; of 2048 x 1408,
// mean 32: 28.9 / 30.8, 64: 33.6 / 33.1, 96: 43.6 / 37.5. Empty sets count, so rows that
// lie in few of the sets may go this way where pairs are faster: 4096 rows in 16 of the 64
// 50.6 / 35.2 and 27.3 / 19.7, in 8 50.1 / 33.3 and 26.9 / 19.8.
// Rows that a linear may quantize itself, over a split K, take the same kernel behind a
// quantization of their own, so that both add up alike (K in one piece is the same sum
// in either kernel); where pairs would be faster it costs some 1.2 us: 16 rows of 16384 x
// 2048 8.0 / 6.6, 12 of 19456 x 2304 8.3 / 7.4, 14 of 9856 x 1024 5.6 / 4.5.
bool takes_few(const Mx4GemmArgs& a, int sms) {
  if (a.offsets) return a.M <= 64 * (int64_t)a.sets;
  const int64_t kb = mx4_kblocks(a.K), units = few_units(a);
  const int split = few_split(units, kb, sms);
  if (split > 1 && own_fits(a, sms, kOwnRuns)) return true;
  const int64_t rounds = split > 1 ? 1 : (units + 2 * sms - 1) / (2 * sms);
  const double rows = a.M < kBT ? (double)a.M : kBT;
  const double few = 4.0 + (double)(rounds * ((kb + split - 1) / split)) * (0.45 + 0.002 * rows) +
                     (split > 1 ? 0.15 * rows / split : 0.0);
  const int64_t pair_units = (a.M + 255) / 256 * (((a.N + 127) / 128 + 1) / 2);
  const int64_t pairs = sms / 2 > 0 ? sms / 2 : 1;
  const double pair = 4.5 + 0.28 * (double)((pair_units + pairs - 1) / pairs * kb);
  return few <= pair;
}

}  // namespace

bool mx4_own_rows(const Mx4GemmArgs& a, const Mx4QuantArgs& q) {
  const int sms = device_sm_count();
  return sms >= 1 && q.type != kMx4F32 && own_fits(a, sms, q.gated ? kOwnGatedRuns : kOwnRuns);
}

cudaError_t launch_mx4_own(const Mx4GemmArgs& a, const Mx4QuantArgs& q, cudaStream_t st) {
  return a.format == EGOPQ_MX4_E8M0 ? launch_own<EGOPQ_MX4_E8M0>(a, q, st)
                                    : launch_own<EGOPQ_MX4_E4M3>(a, q, st);
}

cudaError_t launch_mx4_gemm(const Mx4GemmArgs& a, cudaStream_t st) {
  const int sms = device_sm_count();
  if (sms < 1) return cudaErrorInvalidConfiguration;
  if (!takes_few(a, sms)) return launch_mx4_pair(a, st);
  return a.format == EGOPQ_MX4_E8M0 ? launch_few<EGOPQ_MX4_E8M0, kNone, false>(a, nullptr, st)
                                    : launch_few<EGOPQ_MX4_E4M3, kNone, false>(a, nullptr, st);
}

cudaError_t take_error_word_mx4_gemm(unsigned* out) { return take_local_error_word(out); }
cudaError_t set_record_limit_mx4_gemm(unsigned long long bytes) {
  return set_local_record_limit(bytes);
}

}  // namespace egopq
