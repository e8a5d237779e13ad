// tc_experts.cu -- the experts' products on the tensor cores: the 192-token
// tiles of tc_kernel.cuh over sorted rows, each expert's range with its own
// packed weights. A persistent grid walks the (expert, weight block, row tile)
// units, whose number only the device knows.
#include "tc_kernel.cuh"

namespace egopq {

template <int VARIANT, int MODE>
static cudaError_t launch_ragged_mode(const RaggedArgs& a, cudaStream_t st) {
  using C = TcCfg<VARIANT, kFullBT>;
  constexpr size_t kSmem = C::kSmemBytes + (kTcMaxSets + 4) * sizeof(int);
  static_assert(kSmem <= kMaxSmem, "shared memory of the ragged products");
  CUtensorMap act_map, none;
  memset(&none, 0, sizeof(none));
  YMaps ymaps;
  memset(&ymaps, 0, sizeof(ymaps));
  if (!make_act_map_3d(&act_map,
                       VARIANT == kW4A8 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                       a.act, a.rows_max, a.K, kFullBT))
    return cudaErrorInvalidValue;
  TcParams p{};
  p.M = a.rows_max;
  p.N = a.N;
  p.K = a.K;
  p.G = (int)(a.K / 128);
  p.ks = 1;
  p.n_tiles = (int)(a.N / 128);
  p.persistent = 1;
  p.act3d = 1;
  p.a_s = a.a_s;
  p.timeout_ns = a.timeout_ns;
  p.seg.count = 1;
  p.seg.packed[0] = a.packed;
  p.seg.y[0] = a.y;
  p.seg.N[0] = a.N;
  p.set_offset = a.plan.offset;
  p.sets = a.E;
  // units at most (the device counts them): as many CTAs as SMs, or fewer
  const int64_t most = plan_max_tiles(a.rows_max, a.E, kFullBT) * p.n_tiles;
  const int sms = device_sm_count();
  if (sms < 1) return cudaErrorInvalidConfiguration;
  if (most >= (1LL << 31) || (most / sms + 1) * p.G >= (1LL << 31)) return cudaErrorNotSupported;
  auto kern = tc_gemm_kernel<VARIANT, kFullBT, false, MODE>;
  static SmemOptIn opt_in;
  if (cudaError_t e = opt_in.ensure(kern, kSmem); e != cudaSuccess) return e;
  // (the register split must fit what the block is launched with: see launch_tc)
  static std::atomic<int> regs_ok{0};
  if (regs_ok.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    if (cudaError_t e = cudaFuncGetAttributes(&fa, kern); e != cudaSuccess) return e;
    regs_ok.store(C::kDrainWGs * C::kRegDrain + C::kConvSets * C::kRegConv + C::kRegOther <=
                          (C::kWarps / 4) * fa.numRegs
                      ? 1
                      : 2,
                  std::memory_order_relaxed);
  }
  if (regs_ok.load(std::memory_order_relaxed) != 1) return cudaErrorInvalidConfiguration;
  PdlConfig c(dim3((unsigned)(most < sms ? most : sms), 1, 1), C::kThreads, kSmem, st);
  return cudaLaunchKernelEx(&c.cfg, kern, act_map, none, p, ymaps);
}

cudaError_t launch_ragged(const RaggedArgs& a, cudaStream_t st) {
  if (a.variant == kW4A8)
    return a.gate_up ? launch_ragged_mode<kW4A8, kTcGateUp>(a, st)
                     : launch_ragged_mode<kW4A8, kTcDown>(a, st);
  return a.gate_up ? launch_ragged_mode<kW4A16, kTcGateUp>(a, st)
                   : launch_ragged_mode<kW4A16, kTcDown>(a, st);
}

cudaError_t take_error_word_tc_experts(unsigned* out) { return take_local_error_word(out); }
cudaError_t set_record_limit_tc_experts(unsigned long long bytes) {
  return set_local_record_limit(bytes);
}

}  // namespace egopq
