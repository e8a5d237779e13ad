// tc_gemm.cu -- host side of the tcgen05 tensor-core GEMM (tc_kernel.cuh) for
// the linears: token tiles, grids, tensor maps, launches.
#include "tc_kernel.cuh"

namespace egopq {

// ---- bounded-wait self test -----------------------------------------------------
__global__ void selftest_timeout_kernel(uint64_t timeout_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // nothing ever arrives on `bar`: the wait must give up and flag a timeout
  if (threadIdx.x == 0) mbar_wait(smem_u32(&bar), 0, &abort_flag, timeout_ns);
  __syncthreads();
}

cudaError_t launch_selftest_timeout(uint64_t timeout_ns, cudaStream_t st) {
  selftest_timeout_kernel<<<1, 32, 0, st>>>(timeout_ns);
  return cudaGetLastError();
}
static int tc_sm_count() {
  const int n = device_sm_count();
  return n > 0 ? n : 148;
}

// Split of the work over the GPU. With enough tiles, a persistent grid (one
// CTA per SM) strides over them with all of K; otherwise each tile's K groups
// are split over a cluster of ks CTAs. ks minimises rounds * groups-per-unit.
static void choose_split(int64_t tiles, int G, int sms, double split_cost, bool one_wave,
                         int* ks_out, int* persistent_out) {
  // enough tiles to fill the GPU: persistent, all of K per tile
  if (tiles >= sms) {
    *ks_out = 1;
    *persistent_out = 1;
    return;
  }
  // otherwise split K over a cluster, one round, as many SMs busy as possible
  // (a split costs `split_cost` groups of prologue and reduction per CTA)
  double best = 1e30;
  int best_ks = 1;
  for (int ks = 1; ks <= 8 && ks <= G; ++ks) {
    const int64_t units = tiles * ks;
    if (one_wave && ks > 1 && units > sms) break;
    const int64_t rounds = (units + sms - 1) / sms;
    const double cost = (double)rounds * ((G + ks - 1) / ks + (ks > 1 ? split_cost : 0.0));
    if (cost < best - 1e-9) {
      best = cost;
      best_ks = ks;
    }
  }
  *ks_out = best_ks;
  *persistent_out = 0;
}

// Grid plan of one GEMM: a persistent grid over the first `units` tiles of the
// banded order and, for wide tiles whose last round would leave most SMs idle,
// a second launch splitting the remaining `tail` tiles' K over clusters of
// `tail_ks` CTAs; or, with too few tiles to fill the GPU, one split-K grid
// over all tiles (persistent = 0, split ks).
struct GridPlan {
  int persistent = 0;
  int ks = 1;
  int64_t units = 0, tail = 0;
  int tail_ks = 1;
  double cost = 0.0;  // CTA time in groups of one unit of this width
};

// the second launch of a split tail, in groups of a full-grid CTA: its launch
// behind the first, pipeline fill, cluster reduction and stores (measured on
// GB300: ~14 us beside the split groups' own time, ~26 groups of 192 tokens;
// so the 3584 x 18944 linear at 4096 tokens takes a tail, 386 -> 334 us,
// and the 3584 x 3584 one, 28 groups a tile, does not)
constexpr double kTailLaunchCost = 24.0;

static GridPlan plan_grid(int64_t tiles, int G, int sms, bool wide) {
  GridPlan g;
  const double split_cost = wide ? 2.0 : 1.0;
  choose_split(tiles, G, sms, split_cost, wide, &g.ks, &g.persistent);
  if (!g.persistent) {
    const int64_t units = tiles * g.ks;
    g.cost = (double)((units + sms - 1) / sms) *
             ((G + g.ks - 1) / g.ks + (g.ks > 1 ? split_cost : 0.0));
    return g;
  }
  const int64_t rounds = (tiles + sms - 1) / sms;
  g.units = tiles;
  g.cost = (double)rounds * G;
  if (!wide || rounds < 2) return g;
  const int64_t tail = tiles - (rounds - 1) * sms;
  int ks = 1;
  for (int k = 2; k <= 8 && k <= G && tail * k <= sms; ++k) ks = k;
  if (ks < 2) return g;
  const double split = (double)(rounds - 1) * G + (G + ks - 1) / ks + split_cost + kTailLaunchCost;
  if (split < g.cost) {
    g.units = (rounds - 1) * sms;
    g.tail = tail;
    g.tail_ks = ks;
    g.cost = split;
  }
  return g;
}

// Band height (in m-tiles) for the persistent tile order, which walks bands of
// `band` m-tiles with m fastest inside a band: each weight tile is read from
// DRAM once per band, each activation tile once if the band's activations stay
// in L2. So DRAM traffic is lowest when one operand stays L2-resident while
// the other streams once: all m-tiles in one band when the whole activation
// matrix fits the L2 budget (weights stream once), one m-tile a band (n
// fastest) when the whole weight matrix fits (activations stream once),
// otherwise the tallest band whose activation tiles fit.
static int choose_band(int64_t m_tiles, int64_t n_tiles, double act_tile, double w_tile) {
  constexpr double kL2Budget = 48e6;  // bytes of one operand kept resident (129 MB L2)
  if (m_tiles * act_tile <= kL2Budget) return (int)m_tiles;
  if (n_tiles * w_tile <= kL2Budget) return 1;
  int band = (int)(kL2Budget / act_tile);
  if (band < 1) band = 1;
  if (band > m_tiles) band = (int)m_tiles;
  return band;
}

template <int VARIANT, int BT, bool PARTIALS>
static cudaError_t launch_tc(const GemmArgs& a, cudaStream_t st) {
  using C = TcCfg<VARIANT, BT>;
  CUtensorMap act_map, w8_map;
  memset(&w8_map, 0, sizeof(w8_map));
  constexpr bool kCodes = (VARIANT == kW4A8 || VARIANT == kW8A8);  // quantized activations
  const void* act_ptr = kCodes ? (const void*)a.a_tc : (const void*)a.x;
  const CUtensorMapDataType adt =
      kCodes ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  int act3d = 0;
  if constexpr (C::kFp8) {
    if (!make_act_map_planes(&act_map, act_ptr, a.M, a.K, BT)) return cudaErrorInvalidValue;
  } else {
    act3d = make_act_map_3d(&act_map, adt, act_ptr, a.M, a.K, BT) ? 1 : 0;
    if (!act3d && !make_map(&act_map, adt, 2, act_ptr, a.M, a.K, 64, BT))
      return cudaErrorInvalidValue;
  }
  if constexpr (C::kW16) {
    if (!make_map(&w8_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.w16, a.N, a.K, 64, 128))
      return cudaErrorInvalidValue;
  } else if constexpr (C::kW8) {
    if (!make_map(&w8_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.w8, a.N, a.K, 128, 128))
      return cudaErrorInvalidValue;
  }
  const int G = (int)(a.K / 128);
  const int64_t m_tiles = (a.M + BT - 1) / BT;
  const int64_t n_tiles = a.N / 128;
  const int64_t tiles = m_tiles * n_tiles;
  if (m_tiles > 65535 || n_tiles > 65535 || tiles >= (1LL << 31)) return cudaErrorInvalidValue;
  const int sms = tc_sm_count() * C::kCtasPerSm;  // CTA slots of one wave
  // (wide tiles reduce 128 x BT partial sums through DSMEM, about two groups'
  // worth, and split only while every CTA of the split fits one wave: a
  // second wave of split clusters measured slower than no split, e.g. the
  // 3584 x 3584 linear at 512 tokens 53 us split four ways against 23 us)
  const GridPlan plan = plan_grid(tiles, G, sms, C::kWide);
  const int ks = plan.ks, persistent = plan.persistent;
  TcParams p{};
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.G = G;
  p.ks = ks;
  p.m_tiles = (int)m_tiles;
  p.n_tiles = (int)n_tiles;
  p.persistent = persistent;
  p.units = (int)plan.units;
  p.tail_base = (int)plan.units;
  p.act3d = act3d;
  p.band = persistent ? choose_band(m_tiles, n_tiles, (double)BT * a.K * 2.0,
                                    (double)128 * a.K * (C::kW16 ? 2.0 : (C::kW8 ? 1.0 : 0.5)))
                      : 1;
  p.a_s = a.a_s;
  p.a_gsum = a.a_gsum;
  p.s8 = a.s8;
  p.partials = a.partials;
  p.seg = seg_table(a);
  p.timeout_ns = a.timeout_ns;
  YMaps ymaps;
  memset(&ymaps, 0, sizeof(ymaps));
  if constexpr (C::kTmaEpi && !PARTIALS) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return cudaErrorInvalidValue;
    for (int j = 0; j < p.seg.count; ++j) {
      cuuint64_t dims[2] = {(cuuint64_t)p.seg.N[j], (cuuint64_t)a.M};
      cuuint64_t strides[1] = {(cuuint64_t)(p.seg.N[j] * 2)};
      cuuint32_t box[2] = {128, (cuuint32_t)C::kDrainCols};
      cuuint32_t estr[2] = {1, 1};
      if (fn(&ymaps.map[j], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.seg.y[j], dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    }
  }
  auto kern = tc_gemm_kernel<VARIANT, BT, PARTIALS>;
  // opt-in to the large shared-memory carve-out, once per device
  static SmemOptIn opt_in;
  if (cudaError_t e = opt_in.ensure(kern, C::kSmemBytes); e != cudaSuccess) return e;
  if constexpr (C::kRegSplit) {
    // the warpgroups' register budgets must fit in what the block is launched
    // with, or a setmaxnreg increase would wait for ever (checked once: the
    // register count is a property of the compiled kernel)
    static std::atomic<int> regs_ok{0};  // 0 unchecked, 1 fits, 2 does not
    if (regs_ok.load(std::memory_order_relaxed) == 0) {
      cudaFuncAttributes fa;
      cudaError_t e = cudaFuncGetAttributes(&fa, kern);
      if (e != cudaSuccess) return e;
      regs_ok.store(C::kDrainWGs * C::kRegDrain + C::kConvSets * C::kRegConv + C::kRegOther <=
                            (C::kWarps / 4) * fa.numRegs
                        ? 1
                        : 2,
                    std::memory_order_relaxed);
    }
    if (regs_ok.load(std::memory_order_relaxed) != 1) return cudaErrorInvalidConfiguration;
  }
  cudaLaunchConfig_t cfg = {};
  if (persistent)
    cfg.gridDim = dim3((unsigned)(plan.units < sms ? plan.units : sms), 1, 1);
  else
    cfg.gridDim = dim3((unsigned)ks, (unsigned)m_tiles, (unsigned)n_tiles);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = persistent ? 1u : (unsigned)ks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, act_map, w8_map, p, ymaps);
  if (e != cudaSuccess || plan.tail == 0) return e;
  // the split tail: the last tiles of the banded order, K over clusters
  p.persistent = 2;
  p.ks = plan.tail_ks;
  cfg.gridDim = dim3((unsigned)plan.tail_ks, (unsigned)plan.tail, 1);
  attr[0].val.clusterDim.x = (unsigned)plan.tail_ks;
  return cudaLaunchKernelEx(&cfg, kern, act_map, w8_map, p, ymaps);
}

// Time of a grid of `bt`-token wide tiles in units of one group of one
// 128-token tile: the cost of the grid plan_grid makes, times the relative
// cost of a group at that width.
static double wide_grid_cost(int64_t M, int64_t n_tiles, int G, int sms, int bt,
                             bool wide = true) {
  // one 192-token group against one 128-token group, CTA time in a full grid
  // (measured on GB300 over the 7B prefill shapes: 1.0-1.14 as the 192-token
  // kernel improved; every value in that range makes the same choices there)
  constexpr double kFullGroupCost = 1.12;
  const int64_t tiles = ((M + bt - 1) / bt) * n_tiles;
  return plan_grid(tiles, G, sms, wide).cost * (bt == kFullBT ? kFullGroupCost : 1.0);
}

int tc_token_tile(int variant, int64_t M, int64_t N, int64_t K) {
  if (M <= 16) return 16;
  if (M <= 32) return 32;
  if (M <= 64) return 64;
  // above 64 tokens every variant takes 192 tokens unless that grid costs
  // more (the int8-weight variants without the per-group tiles' split tails
  // and one-wave splits)
  if (variant == kW4A8 || variant == kW4A16 || variant == kW16A16 || variant == kW8A16 ||
      variant == kW8A8) {
    const int sms = tc_sm_count();
    const int G = (int)(K / 128);
    const int64_t n_tiles = N / 128;
    const bool wide = variant != kW8A16 && variant != kW8A8;  // (split tails, one-wave splits)
    return wide_grid_cost(M, n_tiles, G, sms, kFullBT, wide) <
                   wide_grid_cost(M, n_tiles, G, sms, kWideBT, wide)
               ? kFullBT
               : kWideBT;
  }
  return 128;
}

int tc_launches(int variant, int64_t M, int64_t N, int64_t K) {
  const int bt = tc_token_tile(variant, M, N, K);
  const bool per_group = (variant == kW4A8 || variant == kW4A16 || variant == kW16A16);
  if (bt <= 64 || !per_group) return 1;  // (only wide per-group tiles split a tail)
  const int64_t tiles = ((M + bt - 1) / bt) * (N / 128);
  return plan_grid(tiles, (int)(K / 128), tc_sm_count(), true).tail > 0 ? 2 : 1;
}

template <int VARIANT, bool PARTIALS>
static cudaError_t launch_tc_bt(const GemmArgs& a, cudaStream_t st) {
  constexpr bool kPerGroup = (VARIANT == kW4A8 || VARIANT == kW4A16 || VARIANT == kW16A16);
  switch (tc_token_tile(VARIANT, a.M, a.N, a.K)) {
    case 16:
      return launch_tc<VARIANT, 16, PARTIALS>(a, st);
    case 32:
      return launch_tc<VARIANT, 32, PARTIALS>(a, st);
    case 64:
      return launch_tc<VARIANT, 64, PARTIALS>(a, st);
    case kFullBT:
      if constexpr (kPerGroup || VARIANT == kW8A16 || VARIANT == kW8A8)
        return launch_tc<VARIANT, kFullBT, PARTIALS>(a, st);
      break;
    default:
      return launch_tc<VARIANT, 128, PARTIALS>(a, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_tc_gemm(const GemmArgs& a, cudaStream_t st) {
  if (a.M == 0) return cudaSuccess;
  switch (a.variant) {
    case kW4A8:
      return a.partials ? launch_tc_bt<kW4A8, true>(a, st) : launch_tc_bt<kW4A8, false>(a, st);
    case kW4A16:
      return launch_tc_bt<kW4A16, false>(a, st);
    case kW8A16:
      return launch_tc_bt<kW8A16, false>(a, st);
    case kW16A16:
      return launch_tc_bt<kW16A16, false>(a, st);
    case kW8A8:
      // the fp16 activation-code form exists for M > kTcFp8MaxM only (the
      // e4m3 planes below it are specific to 4-bit weights); smaller M run
      // on the GEMV
      if (a.M <= kTcFp8MaxM) return cudaErrorNotSupported;
      if (tc_token_tile(kW8A8, a.M, a.N, a.K) == kFullBT)
        return launch_tc<kW8A8, kFullBT, false>(a, st);
      return launch_tc<kW8A8, 128, false>(a, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t take_error_word_tc_gemm(unsigned* out) { return take_local_error_word(out); }
cudaError_t set_record_limit_tc_gemm(unsigned long long bytes) {
  return set_local_record_limit(bytes);
}

}  // namespace egopq
