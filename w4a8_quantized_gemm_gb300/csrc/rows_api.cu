// rows_api.cu -- C ABI of the operators whose weights each row picks: the
// router, the experts' gated linears, the low-rank adapters. Argument checks
// and workspace layout only; nothing is allocated here.
#include <cmath>

#include "egopq_internal.h"

using namespace egopq;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s per bounded wait

// Parts of a workspace, each 256-byte aligned; with a null base only the size
// is added up.
struct Carver {
  uint8_t* base;
  size_t used = 0;
  explicit Carver(void* p) : base(static_cast<uint8_t*>(p)) {}
  template <typename T>
  T* take(int64_t count) {
    T* at = base ? reinterpret_cast<T*>(base + used) : nullptr;
    used += ((size_t)count * sizeof(T) + 255) / 256 * 256;
    return at;
  }
};

void carve_plan(Carver& c, RowPlan& plan, int64_t n, int S, int64_t tiles, bool pos) {
  plan.head = c.take<int>(2);
  plan.offset = c.take<int32_t>(S + 1);
  plan.order = c.take<int32_t>(n);
  plan.pos = pos ? c.take<int32_t>(n) : nullptr;
  plan.tiles = c.take<int4>(tiles);
}

size_t carve_experts(void* ws, ExpertsArgs& a) {
  Carver c(ws);
  const int64_t n = a.T * a.k;
  const bool codes = a.variant == kW4A8, tensor = a.way == kExpertsTensor;
  if (a.way != kExpertsFew)
    carve_plan(c, a.plan, n, a.E, tensor ? 0 : plan_max_tiles(n, a.E, 8), true);
  if (!tensor && (codes || a.way == kExpertsStream)) a.x_q = c.take<uint16_t>(a.T * a.H);
  if (!tensor && codes) a.x_s = c.take<float>(a.T);
  if (tensor) a.rows_s = c.take<float>(n);
  if (tensor || codes) {
    a.h_q = c.take<uint16_t>(n * a.I);
    a.h_s = c.take<float>(n);
  }
  a.h = c.take<uint16_t>(n * a.I * (tensor && !codes ? 2 : 1));
  if (tensor) {
    // the sorted activations are dead once the gate and up products have run
    a.rows = c.take<uint16_t>(n * a.H);
    a.y = a.rows;
  } else if (a.way == kExpertsStream) {
    a.y = c.take<float>(n * a.H);
  }
  return c.used;
}

int lora_result(cudaError_t e, int64_t M) {
  if (e == cudaErrorNotSupported)
    return fail(EGOPQ_ERR_UNSUPPORTED_SHAPE, "too many rows for one call (M=%lld)", (long long)M);
  return e == cudaSuccess ? EGOPQ_OK : cuda_fail(e, "adapters launch");
}

size_t carve_lora(void* ws, LoraArgs& a) {
  Carver c(ws);
  if (lora_few(a.M)) {
    c.take<int>(1);  // (needs none; a size of zero would say "refused")
    return c.used;
  }
  // (for either way of a planned batch, so that a batch of fewer rows fits too)
  carve_plan(c, a.plan, a.M, a.L, plan_max_tiles(a.M, a.L, kLoraTile), false);
  a.h = c.take<float>(lora_h_rows(a.M) * a.r);
  return c.used;
}

int check_experts_shape(int64_t T, int k, int E, int64_t H, int64_t I, int group, int variant) {
  if (T < 0 || k <= 0 || E <= 0 || H <= 0 || I <= 0)
    return fail(EGOPQ_ERR_INVALID_ARG, "bad sizes T=%lld k=%d E=%d H=%lld I=%lld", (long long)T, k,
                E, (long long)H, (long long)I);
  if (variant != EGOPQ_VARIANT_W4A8 && variant != EGOPQ_VARIANT_W4A16)
    return fail(EGOPQ_ERR_INVALID_ARG, "experts run W4A8 or W4A16 (got variant %d)", variant);
  if (E > kMaxSets)
    return fail(EGOPQ_ERR_UNSUPPORTED_SHAPE, "at most %d experts (got %d)", kMaxSets, E);
  if (T >= kMaxDim || H >= kMaxDim || I >= kMaxDim || T > (kMaxDim - 1) / k)
    return fail(EGOPQ_ERR_UNSUPPORTED_SHAPE, "sizes T=%lld k=%d H=%lld I=%lld exceed 2^31 - 1",
                (long long)T, k, (long long)H, (long long)I);
  if (int rc = check_w4_shape(0, H, I, group)) return rc;
  // (so that E weights of 2I or H rows stay below 2^31 rows)
  if (H >= (1 << 20) || I >= (1 << 20))
    return fail(EGOPQ_ERR_UNSUPPORTED_SHAPE, "H (%lld) and I (%lld) must be below 2^20",
                (long long)H, (long long)I);
  return EGOPQ_OK;
}

int check_lora_shape(int64_t M, int64_t N, int64_t K, int L, int r) {
  if (M < 0 || N <= 0 || K <= 0 || L <= 0 || r <= 0)
    return fail(EGOPQ_ERR_INVALID_ARG, "bad sizes M=%lld N=%lld K=%lld L=%d r=%d", (long long)M,
                (long long)N, (long long)K, L, r);
  if (M >= kMaxDim || N >= (1 << 24) || K >= kMaxDim)
    return fail(EGOPQ_ERR_UNSUPPORTED_SHAPE, "sizes M=%lld N=%lld K=%lld are too large",
                (long long)M, (long long)N, (long long)K);
  if (L > kMaxSets)
    return fail(EGOPQ_ERR_UNSUPPORTED_SHAPE, "at most %d adapters (got %d)", kMaxSets, L);
  if (r > 128 || r % 8)
    return fail(EGOPQ_ERR_UNSUPPORTED_SHAPE, "rank must be a multiple of 8, at most 128 (got %d)", r);
  if (K % 128 || N % 128)
    return fail(EGOPQ_ERR_UNSUPPORTED_SHAPE, "K (%lld) and N (%lld) must be multiples of 128",
                (long long)K, (long long)N);
  return EGOPQ_OK;
}

int check_aligned(const void* p, uintptr_t to, const char* name) {
  if (reinterpret_cast<uintptr_t>(p) & (to - 1))
    return fail(EGOPQ_ERR_MISALIGNED, "%s is not %d-byte aligned", name, (int)to);
  return EGOPQ_OK;
}

bool overlap(const uint16_t* a, int64_t na, const uint16_t* b, int64_t nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + 2 * (uintptr_t)nb && pb < pa + 2 * (uintptr_t)na;
}

// The adapters' update writes rows of y while other rows (and other columns of
// the same rows) are still formed from x: y may be updated in place, row for
// row, but not lie on x.
int check_lora_overlap(const LoraArgs& a) {
  if (overlap(a.x, a.M * a.K, a.y_out, a.M * a.N))
    return fail(EGOPQ_ERR_INVALID_ARG, "the output overlaps x");
  if (a.y_in != a.y_out && overlap(a.y_in, a.M * a.N, a.y_out, a.M * a.N))
    return fail(EGOPQ_ERR_INVALID_ARG, "y_out overlaps y_in and is not y_in");
  return EGOPQ_OK;
}

// A row's own picks and weights, which are read (or written) one by one: a batch
// may be a slice of a larger one, at any row.
int check_picks(const void* p, const char* name) {
  return p ? check_aligned(p, 4, name) : fail(EGOPQ_ERR_INVALID_ARG, "%s is NULL", name);
}

}  // namespace

extern "C" {

int egopq_moe_route(const void* logits, int logits_bf16, const float* bias, int64_t T, int E, int k,
                    int score, int n_group, int topk_group, int group_score, int renorm,
                    float scale, float* weights, int32_t* ids, egopq_stream_t stream) {
  if (T < 0 || E <= 0 || k <= 0 || n_group <= 0 || topk_group <= 0)
    return fail(EGOPQ_ERR_INVALID_ARG, "bad sizes T=%lld E=%d k=%d n_group=%d topk_group=%d",
                (long long)T, E, k, n_group, topk_group);
  if (score != EGOPQ_SCORE_SOFTMAX && score != EGOPQ_SCORE_SIGMOID)
    return fail(EGOPQ_ERR_INVALID_ARG, "unknown score %d", score);
  if (group_score != EGOPQ_GROUP_MAX && group_score != EGOPQ_GROUP_TOP2)
    return fail(EGOPQ_ERR_INVALID_ARG, "unknown group score %d", group_score);
  if (E % n_group || topk_group > n_group)
    return fail(EGOPQ_ERR_INVALID_ARG, "%d experts in %d groups, %d of them kept", E, n_group,
                topk_group);
  if (k > topk_group * (E / n_group))
    return fail(EGOPQ_ERR_INVALID_ARG, "k = %d of the %d experts of the kept groups", k,
                topk_group * (E / n_group));
  if (!std::isfinite(scale)) return fail(EGOPQ_ERR_INVALID_ARG, "scale is not finite");
  if (E > 512 || k > 32 || n_group > 32 || T >= kMaxDim)
    return fail(EGOPQ_ERR_UNSUPPORTED_SHAPE,
                "at most 512 experts, 32 picks and 32 groups (got E=%d k=%d n_group=%d T=%lld)", E,
                k, n_group, (long long)T);
  if (T == 0) return EGOPQ_OK;
  int rc = check_ptrs(1, "logits", logits);
  if (rc) return rc;
  if ((rc = check_picks(weights, "weights")) || (rc = check_picks(ids, "ids"))) return rc;
  if ((rc = check_aligned(bias, 16, "bias"))) return rc;
  if ((rc = check_arch())) return rc;
  RouteArgs a;
  a.logits = logits;
  a.bias = bias;
  a.weights = weights;
  a.ids = ids;
  a.T = T;
  a.E = E;
  a.k = k;
  a.n_group = n_group;
  a.topk_group = topk_group;
  a.bf16 = logits_bf16 != 0;
  a.sigmoid = score == EGOPQ_SCORE_SIGMOID;
  a.top2 = group_score == EGOPQ_GROUP_TOP2 && topk_group < n_group;
  a.renorm = renorm != 0;
  a.scale = scale;
  cudaError_t e = launch_route(a, (cudaStream_t)stream);
  return e == cudaSuccess ? EGOPQ_OK : cuda_fail(e, "moe_route launch");
}

int egopq_moe_pack_gate_up(const uint8_t* w_q, const uint16_t* scale_f16, const uint8_t* zero,
                           int64_t E, int64_t I, int64_t K, int group, void* packed,
                           egopq_stream_t stream) {
  if (E <= 0 || I <= 0 || K <= 0)
    return fail(EGOPQ_ERR_INVALID_ARG, "bad sizes E=%lld I=%lld K=%lld", (long long)E, (long long)I,
                (long long)K);
  if (E > kMaxSets || I >= kMaxDim || E * 2 * I >= kMaxDim)
    return fail(EGOPQ_ERR_UNSUPPORTED_SHAPE, "E=%lld I=%lld: the experts' weight rows exceed the limits",
                (long long)E, (long long)I);
  int rc = check_w4_shape(0, I, K, group);
  if (rc) return rc;
  rc = check_ptrs(4, "w_q", w_q, "scale_f16", scale_f16, "zero", zero, "packed", packed);
  if (rc) return rc;
  if ((rc = check_arch())) return rc;
  cudaError_t e = launch_pack_gate_up(w_q, scale_f16, zero, E, I, K, packed, (cudaStream_t)stream);
  return e == cudaSuccess ? EGOPQ_OK : cuda_fail(e, "moe_pack_gate_up launch");
}

size_t egopq_moe_experts_workspace_bytes(int64_t T, int k, int E, int64_t H, int64_t I, int group,
                                         int variant, int path) {
  if (check_experts_shape(T, k, E, H, I, group, variant) != EGOPQ_OK || T == 0) return 0;
  ExpertsArgs a{};
  a.variant = variant;
  a.T = T;
  a.k = k;
  a.E = E;
  a.H = H;
  a.I = I;
  // enough for every smaller batch too, whichever way it takes
  size_t most = 0;
  for (ExpertsWay way : {kExpertsStream, kExpertsTensor}) {
    if ((path == EGOPQ_PATH_GEMV && way == kExpertsTensor) ||
        (path == EGOPQ_PATH_TC && way != kExpertsTensor))
      continue;
    a.T = T;
    if (path == EGOPQ_PATH_AUTO && way == kExpertsStream && T * k > kStreamRows * E)
      a.T = kStreamRows * E / k;  // the largest batch that still streams
    a.way = way;
    const size_t need = carve_experts(nullptr, a);
    if (need > most) most = need;
  }
  return most;
}

int egopq_moe_experts(const uint16_t* x_bf16, const int32_t* ids, const float* weights,
                      const void* packed_gate_up, const void* packed_down, int64_t T, int k, int E,
                      int64_t H, int64_t I, int group, int variant, uint16_t* out_bf16,
                      void* workspace, size_t workspace_bytes, int path, egopq_stream_t stream) {
  int rc = check_experts_shape(T, k, E, H, I, group, variant);
  if (rc) return rc;
  if (path != EGOPQ_PATH_AUTO && path != EGOPQ_PATH_GEMV && path != EGOPQ_PATH_TC)
    return fail(EGOPQ_ERR_INVALID_ARG, "unknown path %d", path);
  if (T == 0) return EGOPQ_OK;
  rc = check_ptrs(5, "x_bf16", x_bf16, "packed_gate_up", packed_gate_up, "packed_down",
                  packed_down, "out_bf16", out_bf16, "workspace", workspace);
  if (rc) return rc;
  if ((rc = check_picks(ids, "ids")) || (rc = check_picks(weights, "weights"))) return rc;
  ExpertsArgs a{};
  a.variant = variant;
  a.T = T;
  a.H = H;
  a.I = I;
  a.E = E;
  a.k = k;
  a.way = experts_way(T, k, E, path);
  a.x = x_bf16;
  a.ids = ids;
  a.weights = weights;
  a.gate_up = static_cast<const uint8_t*>(packed_gate_up);
  a.down = static_cast<const uint8_t*>(packed_down);
  a.out = out_bf16;
  a.timeout_ns = kTimeoutNs;
  const size_t need = carve_experts(workspace, a);
  if (workspace_bytes < need)
    return fail(EGOPQ_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if ((rc = check_arch())) return rc;
  cudaError_t e = launch_experts(a, (cudaStream_t)stream);
  if (e == cudaErrorNotSupported)
    return fail(EGOPQ_ERR_UNSUPPORTED_SHAPE, "too many rows for the requested path");
  return e == cudaSuccess ? EGOPQ_OK : cuda_fail(e, "moe_experts launch");
}

size_t egopq_lora_workspace_bytes(int64_t M, int64_t N, int64_t K, int L, int r) {
  if (check_lora_shape(M, N, K, L, r) != EGOPQ_OK || M == 0) return 0;
  LoraArgs a{};
  a.M = M;
  a.K = K;
  a.L = L;
  a.r = r;
  return carve_lora(nullptr, a);
}

int egopq_lora_add(const uint16_t* y_in, const uint16_t* x_bf16, const uint16_t* A_bf16,
                   const uint16_t* B_bf16, const float* scale, const int32_t* ranks,
                   const int32_t* ids, int64_t M, int64_t N, int64_t K, int L, int r,
                   uint16_t* y_out, void* workspace, size_t workspace_bytes,
                   egopq_stream_t stream) {
  int rc = check_lora_shape(M, N, K, L, r);
  if (rc) return rc;
  if (M == 0) return EGOPQ_OK;
  rc = check_ptrs(7, "y_in", y_in, "x_bf16", x_bf16, "A_bf16", A_bf16, "B_bf16", B_bf16, "scale",
                  scale, "y_out", y_out, "workspace", workspace);
  if (rc) return rc;
  if ((rc = check_picks(ids, "ids"))) return rc;
  if ((rc = check_aligned(ranks, 16, "ranks"))) return rc;
  LoraArgs a{};
  a.y_in = y_in;
  a.x = x_bf16;
  a.A = A_bf16;
  a.B = B_bf16;
  a.scale = scale;
  a.ranks = ranks;
  a.ids = ids;
  a.M = M;
  a.N = N;
  a.K = K;
  a.L = L;
  a.r = r;
  a.y_out = y_out;
  const size_t need = carve_lora(workspace, a);
  if (workspace_bytes < need)
    return fail(EGOPQ_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if ((rc = check_lora_overlap(a))) return rc;
  if ((rc = check_arch())) return rc;
  return lora_result(launch_lora(a, (cudaStream_t)stream), M);
}

size_t egopq_w4a8_linear_lora_workspace_bytes(int64_t M, int64_t N, int64_t K, int group, int L,
                                              int r, int path) {
  const size_t lora = egopq_lora_workspace_bytes(M, N, K, L, r);
  const size_t lin = egopq_w4a8_linear_workspace_bytes(M, K, group, path);
  return lora && lin ? lora + (lin + 255) / 256 * 256 : 0;
}

int egopq_w4a8_linear_lora(const uint16_t* x_bf16, const void* packed, const uint16_t* A_bf16,
                           const uint16_t* B_bf16, const float* scale, const int32_t* ranks,
                           const int32_t* ids, int64_t M, int64_t N, int64_t K, int group, int L,
                           int r, uint16_t* y_bf16, void* workspace, size_t workspace_bytes,
                           int path, egopq_stream_t stream) {
  int rc = check_w4_shape(M, N, K, group);
  if (rc) return rc;
  if ((rc = check_lora_shape(M, N, K, L, r))) return rc;
  if (path != EGOPQ_PATH_AUTO && path != EGOPQ_PATH_GEMV && path != EGOPQ_PATH_TC)
    return fail(EGOPQ_ERR_INVALID_ARG, "unknown path %d", path);
  if (M == 0) return EGOPQ_OK;
  // every argument of both halves is checked before the first launch
  rc = check_ptrs(7, "x_bf16", x_bf16, "packed", packed, "A_bf16", A_bf16, "B_bf16", B_bf16,
                  "scale", scale, "y_bf16", y_bf16, "workspace", workspace);
  if (rc) return rc;
  if ((rc = check_picks(ids, "ids"))) return rc;
  if ((rc = check_aligned(ranks, 16, "ranks"))) return rc;
  const size_t lin = egopq_w4a8_linear_workspace_bytes(M, K, group, path);
  const size_t lin_up = (lin + 255) / 256 * 256;
  const size_t need = lin_up + egopq_lora_workspace_bytes(M, N, K, L, r);
  if (workspace_bytes < need)
    return fail(EGOPQ_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  LoraArgs a{};
  a.y_in = y_bf16;
  a.x = x_bf16;
  a.A = A_bf16;
  a.B = B_bf16;
  a.scale = scale;
  a.ranks = ranks;
  a.ids = ids;
  a.M = M;
  a.N = N;
  a.K = K;
  a.L = L;
  a.r = r;
  a.y_out = y_bf16;
  carve_lora(static_cast<uint8_t*>(workspace) + lin_up, a);
  if ((rc = check_lora_overlap(a))) return rc;
  if ((rc = check_arch())) return rc;
  const cudaStream_t st = (cudaStream_t)stream;
  rc = run_linear(x_bf16, packed, M, N, K, y_bf16, static_cast<uint8_t*>(workspace),
                  auto_path(M, kW4A8, path), st, &a);
  return rc ? rc : lora_result(launch_lora(a, st, true), M);
}

}  // extern "C"
