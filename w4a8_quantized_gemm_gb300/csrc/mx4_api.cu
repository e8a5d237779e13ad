// mx4_api.cu -- C ABI of the microscaled 4-bit linears: argument checks and
// workspace layout only; nothing is allocated here.
#include <initializer_list>

#include "mx4_internal.h"

using namespace egopq;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s per bounded wait

bool known_format(int format) {
  return format == EGOPQ_MX4_E8M0 || format == EGOPQ_MX4_E4M3;
}

int check_format(int format) {
  return known_format(format) ? EGOPQ_OK
                              : fail(EGOPQ_ERR_INVALID_ARG, "unknown 4-bit format %d", format);
}

int check_type(int type, const char* name) {
  if (type != EGOPQ_TYPE_BF16 && type != EGOPQ_TYPE_F16 && type != EGOPQ_TYPE_F32)
    return fail(EGOPQ_ERR_INVALID_ARG, "unknown %s %d", name, type);
  return EGOPQ_OK;
}

// Sizes of M rows, N weight rows (of each of `sets` weights) and K columns.
int check_shape(int64_t M, int64_t sets, int64_t N, int64_t K) {
  if (M < 0 || sets <= 0 || N <= 0 || K <= 0)
    return fail(EGOPQ_ERR_INVALID_ARG, "bad sizes M=%lld sets=%lld N=%lld K=%lld", (long long)M,
                (long long)sets, (long long)N, (long long)K);
  if (M >= kMaxDim || N >= kMaxDim || K >= kMaxDim / 2)
    return fail(EGOPQ_ERR_UNSUPPORTED_SHAPE, "sizes M=%lld N=%lld K=%lld are too large",
                (long long)M, (long long)N, (long long)K);
  if (sets > kMaxSets)
    return fail(EGOPQ_ERR_UNSUPPORTED_SHAPE, "at most %d sets (got %lld)", kMaxSets,
                (long long)sets);
  if (K % 32)
    return fail(EGOPQ_ERR_UNSUPPORTED_SHAPE, "K (%lld) must be a multiple of 32", (long long)K);
  return EGOPQ_OK;
}

// A pointer that may be null, 4-byte aligned (scales, offsets, an index).
int check_words(const void* p, const char* name) {
  if (reinterpret_cast<uintptr_t>(p) & 3u)
    return fail(EGOPQ_ERR_MISALIGNED, "%s is not 4-byte aligned", name);
  return EGOPQ_OK;
}
int check_optional(const void* p, const char* name) {
  if (reinterpret_cast<uintptr_t>(p) & 15u)
    return fail(EGOPQ_ERR_MISALIGNED, "%s is not 16-byte aligned", name);
  return EGOPQ_OK;
}
// E8M0 has no tensor scale: one given would not be applied by everything.
int check_scales(int format, const float* a, const float* w) {
  if (format == EGOPQ_MX4_E8M0 && (a || w))
    return fail(EGOPQ_ERR_INVALID_ARG, "E8M0 blocks have no tensor scale");
  if (int rc = check_words(a, "the rows' tensor scale")) return rc;
  return check_words(w, "the weights' tensor scale");
}

int64_t type_bytes(int type) { return type == EGOPQ_TYPE_F32 ? 4 : 2; }

// A buffer, or none.
struct Span {
  const char* name;
  const void* at;
  int64_t bytes;
};
// What a call writes lies apart from what it reads: other blocks may still read it.
int check_apart(const Span& out, std::initializer_list<Span> in) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(out.at);
  for (const Span& s : in) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(s.at);
    if (out.at && s.at && a < b + (uintptr_t)s.bytes && b < a + (uintptr_t)out.bytes)
      return fail(EGOPQ_ERR_INVALID_ARG, "%s overlaps %s", out.name, s.name);
  }
  return EGOPQ_OK;
}

size_t operand_bytes(int64_t blocks, int64_t K, int format) {
  return (size_t)blocks * (size_t)mx4_kblocks(K) * (size_t)mx4_record_bytes(format);
}

int launched(cudaError_t e, const char* what) {
  if (e == cudaErrorNotSupported)
    return fail(EGOPQ_ERR_UNSUPPORTED_SHAPE, "%s: too large for one call", what);
  return e == cudaSuccess ? EGOPQ_OK : cuda_fail(e, what);
}

// Many rows gathered from at most a quarter as many are quantized once and gathered
// in 4 bits. Directly / so, us, whole calls of 32 sets: 8192 rows from 1024, K 3584,
// 28.5 / 21.7 (E4M3 34.1 / 24.6), 4096 from 512 19.9 / 16.8 (22.6 / 17.8); K 1024,
// 8192 from 1024, 14.1 / 15.6 (15.5 / 16.3).
bool gathers(int64_t rows, int64_t x_rows, int64_t K) {
  return x_rows <= rows / 4 && rows * K >= (3 << 22);
}
// Codes and scales of that many, behind the operand (a multiple of 16 bytes each).
size_t gather_bytes(int64_t x_rows, int64_t K, int format) {
  return (size_t)x_rows * (size_t)(K / 2 + K / mx4_block(format)) + 16;
}

// Quantization and product of a call whose arguments have been checked.
int run(Mx4QuantArgs& q, Mx4GemmArgs& g, cudaStream_t st) {
  q.early = true;  // (only the product behind it reads the workspace, after its wait)
  if (mx4_own_rows(g, q)) return launched(launch_mx4_own(g, q, st), "mx4 product launch");
  if (q.index && gathers(q.M, q.x_rows, q.K)) {
    Mx4QuantArgs once = q;
    once.M = q.x_rows;
    once.offsets = nullptr;
    once.index = nullptr;
    once.operand = nullptr;
    once.codes = q.operand + operand_bytes(mx4_row_blocks(q.M, q.sets), q.K, q.format);
    once.scales = once.codes + q.x_rows * (q.K / 2);
    if (q.x_rows > 0)
      if (int rc = launched(launch_mx4_quant(once, st), "mx4 quantization launch")) return rc;
    q.codes = once.codes;
    q.scales = once.scales;
    if (int rc = launched(launch_mx4_gather(q, st), "mx4 gather launch")) return rc;
    return launched(launch_mx4_gemm(g, st), "mx4 product launch");
  }
  if (int rc = launched(launch_mx4_quant(q, st), "mx4 quantization launch")) return rc;
  return launched(launch_mx4_gemm(g, st), "mx4 product launch");
}

}  // namespace

extern "C" {

size_t egopq_mx4_operand_bytes(int64_t M, int64_t K, int format) {
  if (!known_format(format) || M <= 0 || check_shape(M, 1, 1, K) != EGOPQ_OK) return 0;
  return operand_bytes((M + 127) / 128, K, format);
}

size_t egopq_mx4_packed_bytes(int64_t sets, int64_t N, int64_t K, int format) {
  if (!known_format(format) || check_shape(0, sets, N, K) != EGOPQ_OK) return 0;
  return operand_bytes(sets * ((N + 127) / 128), K, format);
}

int egopq_mx4_quant(const void* x, int x_type, int64_t M, int64_t K, int format,
                    const float* tensor_scale, int gated, uint8_t* codes, uint8_t* scales,
                    void* operand, egopq_stream_t stream) {
  int rc = check_shape(M, 1, 1, K);
  if (rc) return rc;
  if ((rc = check_format(format)) || (rc = check_type(x_type, "x_type"))) return rc;
  if (M == 0) return EGOPQ_OK;
  if ((rc = check_ptrs(1, "x", x))) return rc;
  if (!codes != !scales)
    return fail(EGOPQ_ERR_INVALID_ARG, "codes and scales are written together");
  if (!codes && !operand)
    return fail(EGOPQ_ERR_INVALID_ARG, "neither codes and scales nor operand is asked for");
  if ((rc = check_optional(codes, "codes")) || (rc = check_optional(scales, "scales")) ||
      (rc = check_optional(operand, "operand")) ||
      (rc = check_scales(format, tensor_scale, nullptr)))
    return rc;
  const Span from{"x", x, M * K * (gated ? 2 : 1) * type_bytes(x_type)};
  if ((rc = check_apart({"codes", codes, M * (K / 2)}, {from})) ||
      (rc = check_apart({"scales", scales, M * (K / mx4_block(format))}, {from})) ||
      (rc = check_apart({"operand", operand, (int64_t)operand_bytes((M + 127) / 128, K, format)},
                        {from})))
    return rc;
  if ((rc = check_arch())) return rc;
  Mx4QuantArgs a{};
  a.x = x;
  a.type = x_type;
  a.format = format;
  a.M = a.x_rows = M;
  a.K = K;
  a.gated = gated != 0;
  a.tensor_scale = tensor_scale;
  a.codes = codes;
  a.scales = scales;
  a.operand = static_cast<uint8_t*>(operand);
  a.early = !operand;
  return launched(launch_mx4_quant(a, (cudaStream_t)stream), "mx4_quant launch");
}

int egopq_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, int format,
                      const float* tensor_scale, int y_type, void* y, egopq_stream_t stream) {
  int rc = check_shape(M, 1, 1, K);
  if (rc) return rc;
  if ((rc = check_format(format)) || (rc = check_type(y_type, "y_type"))) return rc;
  if (M == 0) return EGOPQ_OK;
  if ((rc = check_ptrs(3, "codes", codes, "scales", scales, "y", y))) return rc;
  if ((rc = check_scales(format, tensor_scale, nullptr))) return rc;
  if ((rc = check_apart({"y", y, M * K * type_bytes(y_type)},
                        {{"codes", codes, M * (K / 2)},
                         {"scales", scales, M * (K / mx4_block(format))}})))
    return rc;
  if ((rc = check_arch())) return rc;
  return launched(launch_mx4_dequant(codes, scales, M, K, format, tensor_scale, y_type, y,
                                     (cudaStream_t)stream),
                  "mx4_dequant launch");
}

int egopq_mx4_pack(const uint8_t* codes, const uint8_t* scales, int64_t sets, int64_t N, int64_t K,
                   int format, void* packed, egopq_stream_t stream) {
  int rc = check_shape(0, sets, N, K);
  if (rc) return rc;
  if ((rc = check_format(format))) return rc;
  if ((rc = check_ptrs(3, "codes", codes, "scales", scales, "packed", packed))) return rc;
  const int64_t rows = sets * N, bytes = (int64_t)egopq_mx4_packed_bytes(sets, N, K, format);
  if ((rc = check_apart({"packed", packed, bytes},
                        {{"codes", codes, rows * (K / 2)},
                         {"scales", scales, rows * (K / mx4_block(format))}})))
    return rc;
  if ((rc = check_arch())) return rc;
  return launched(launch_mx4_pack(codes, scales, sets, N, K, format, packed, (cudaStream_t)stream),
                  "mx4_pack launch");
}

int egopq_mx4_unpack(const void* packed, int64_t sets, int64_t N, int64_t K, int format,
                     uint8_t* codes, uint8_t* scales, egopq_stream_t stream) {
  int rc = check_shape(0, sets, N, K);
  if (rc) return rc;
  if ((rc = check_format(format))) return rc;
  if ((rc = check_ptrs(3, "packed", packed, "codes", codes, "scales", scales))) return rc;
  const int64_t rows = sets * N;
  const Span from{"packed", packed, (int64_t)egopq_mx4_packed_bytes(sets, N, K, format)};
  if ((rc = check_apart({"codes", codes, rows * (K / 2)}, {from})) ||
      (rc = check_apart({"scales", scales, rows * (K / mx4_block(format))}, {from})))
    return rc;
  if ((rc = check_arch())) return rc;
  return launched(launch_mx4_unpack(packed, sets, N, K, format, codes, scales, (cudaStream_t)stream),
                  "mx4_unpack launch");
}

int egopq_mx4_gemm(const void* operand, const void* packed, const float* a_scale,
                   const float* w_scale, int64_t M, int64_t N, int64_t K, int format, int y_type,
                   void* y, egopq_stream_t stream) {
  int rc = check_shape(M, 1, N, K);
  if (rc) return rc;
  if ((rc = check_format(format)) || (rc = check_type(y_type, "y_type"))) return rc;
  if (M == 0) return EGOPQ_OK;
  if ((rc = check_ptrs(3, "operand", operand, "packed", packed, "y", y))) return rc;
  if ((rc = check_scales(format, a_scale, w_scale))) return rc;
  if ((rc = check_apart({"y", y, M * N * type_bytes(y_type)},
                        {{"operand", operand, (int64_t)operand_bytes((M + 127) / 128, K, format)},
                         {"packed", packed, (int64_t)operand_bytes((N + 127) / 128, K, format)}})))
    return rc;
  if ((rc = check_arch())) return rc;
  Mx4GemmArgs g{};
  g.format = format;
  g.M = M;
  g.N = N;
  g.K = K;
  g.operand = static_cast<const uint8_t*>(operand);
  g.packed = static_cast<const uint8_t*>(packed);
  g.a_scale = a_scale;
  g.w_scale = w_scale;
  g.sets = 1;
  g.type = y_type;
  g.y = y;
  g.timeout_ns = kTimeoutNs;
  return launched(launch_mx4_gemm(g, (cudaStream_t)stream), "mx4_gemm launch");
}

size_t egopq_mx4_linear_workspace_bytes(int64_t rows, int64_t sets, int64_t K, int format) {
  if (!known_format(format) || rows <= 0 || sets < 0 ||
      check_shape(rows, sets ? sets : 1, 1, K) != EGOPQ_OK)
    return 0;
  if (!sets) return operand_bytes((rows + 127) / 128, K, format);
  return operand_bytes(mx4_row_blocks(rows, sets), K, format) + gather_bytes(rows / 4, K, format);
}

// What both linears check once their own shape has been accepted.
static int check_linear(const Mx4QuantArgs& q, const Mx4GemmArgs& g, int64_t ws_sets,
                        const void* workspace, size_t workspace_bytes) {
  int rc = q.x_rows > 0 ? check_ptrs(1, "x", q.x) : EGOPQ_OK;  // (none: nothing to read)
  if (rc || (rc = check_ptrs(3, "packed", g.packed, "y", g.y, "workspace", workspace))) return rc;
  if ((rc = check_scales(g.format, g.a_scale, g.w_scale))) return rc;
  const size_t need = egopq_mx4_linear_workspace_bytes(g.M, ws_sets, g.K, g.format);
  if (workspace_bytes < need)
    return fail(EGOPQ_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  // (few rows are quantized by the blocks that need them, others writing y meanwhile)
  const Span x{"x", q.x, q.x_rows * g.K * (q.gated ? 2 : 1) * type_bytes(q.type)};
  const Span y{"y", g.y, g.M * g.N * type_bytes(g.type)};
  const Span w{"packed", g.packed,
               (int64_t)operand_bytes(g.sets * ((g.N + 127) / 128), g.K, g.format)};
  const Span offsets{"offsets", g.offsets, 4 * ((int64_t)g.sets + 1)}, index{"index", q.index, 4 * q.M};
  if ((rc = check_apart({"the workspace", workspace, (int64_t)need}, {x, y, w, offsets, index})) ||
      (rc = check_apart(y, {x, w, offsets, index})))
    return rc;
  return check_arch();
}

int egopq_mx4_linear(const void* x, int x_type, int64_t M, int64_t N, int64_t K, int gated,
                     const float* a_scale, const void* packed, const float* w_scale, int format,
                     int y_type, void* y, void* workspace, size_t workspace_bytes,
                     egopq_stream_t stream) {
  int rc = check_shape(M, 1, N, K);
  if (rc) return rc;
  if ((rc = check_format(format)) || (rc = check_type(x_type, "x_type")) ||
      (rc = check_type(y_type, "y_type")))
    return rc;
  if (M == 0) return EGOPQ_OK;
  Mx4QuantArgs q{};
  q.x = x;
  q.type = x_type;
  q.format = format;
  q.M = q.x_rows = M;
  q.K = K;
  q.gated = gated != 0;
  q.tensor_scale = a_scale;
  q.operand = static_cast<uint8_t*>(workspace);
  Mx4GemmArgs g{};
  g.format = format;
  g.M = M;
  g.N = N;
  g.K = K;
  g.operand = q.operand;
  g.packed = static_cast<const uint8_t*>(packed);
  g.a_scale = a_scale;
  g.w_scale = w_scale;
  g.sets = 1;
  g.type = y_type;
  g.y = y;
  g.timeout_ns = kTimeoutNs;
  if ((rc = check_linear(q, g, 0, workspace, workspace_bytes))) return rc;
  return run(q, g, (cudaStream_t)stream);
}

int egopq_mx4_linear_ragged(const void* x, int x_type, int64_t x_rows, const int32_t* index,
                            const int32_t* offsets, int64_t rows, int64_t sets, int64_t N,
                            int64_t K, int gated, const float* a_scale, const void* packed,
                            const float* w_scale, int format, int y_type, void* y, void* workspace,
                            size_t workspace_bytes, egopq_stream_t stream) {
  int rc = check_shape(rows, sets, N, K);
  if (rc) return rc;
  if ((rc = check_format(format)) || (rc = check_type(x_type, "x_type")) ||
      (rc = check_type(y_type, "y_type")))
    return rc;
  if (x_rows < 0 || x_rows >= kMaxDim)
    return fail(EGOPQ_ERR_INVALID_ARG, "bad number of rows of x (%lld)", (long long)x_rows);
  if (!index && x_rows != rows)
    return fail(EGOPQ_ERR_INVALID_ARG, "%lld rows of x for %lld rows, and no index",
                (long long)x_rows, (long long)rows);
  if (rows == 0) return EGOPQ_OK;
  if (!offsets) return fail(EGOPQ_ERR_INVALID_ARG, "offsets is NULL");
  if ((rc = check_words(offsets, "offsets")) || (rc = check_words(index, "index"))) return rc;
  Mx4QuantArgs q{};
  q.x = x;
  q.type = x_type;
  q.format = format;
  q.M = rows;
  q.x_rows = x_rows;
  q.K = K;
  q.gated = gated != 0;
  q.tensor_scale = a_scale;
  q.offsets = offsets;
  q.index = index;
  q.sets = (int)sets;
  q.operand = static_cast<uint8_t*>(workspace);
  Mx4GemmArgs g{};
  g.format = format;
  g.M = rows;
  g.N = N;
  g.K = K;
  g.operand = q.operand;
  g.packed = static_cast<const uint8_t*>(packed);
  g.a_scale = a_scale;
  g.w_scale = w_scale;
  g.offsets = offsets;
  g.sets = (int)sets;
  g.type = y_type;
  g.y = y;
  g.timeout_ns = kTimeoutNs;
  if ((rc = check_linear(q, g, sets, workspace, workspace_bytes))) return rc;
  return run(q, g, (cudaStream_t)stream);
}

}  // extern "C"
