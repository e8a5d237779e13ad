// egopq_internal.h -- launchers shared between the kernel files and the C ABI.
#pragma once

#include <atomic>
#include <cstdint>
#include <mutex>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/egopq.h"
#include "egopq_common.cuh"

namespace egopq {

// kW16A16: dense bf16 weights through the W4A16 tensor-core pipeline (the
// same roles, buffers and per-group drains; the converters copy instead of
// unpacking) -- a yardstick, not a quantized path.
enum Variant { kW4A8 = 0, kW4A16 = 1, kW8A16 = 2, kW8A8 = 3, kW16A16 = 4 };

// Launch state that depends on the device (shared-memory opt-ins, SM counts)
// is kept per device ordinal, up to this many devices.
constexpr int kMaxDevices = 64;

// Host-side checks shared by the entry points; each records its message as the
// calling thread's last error and returns a negative egopq_status on failure.
// Shape gate of the packed int4 weight (and the size limit of every call).
int check_w4_shape(int64_t M, int64_t N, int64_t K, int group);
// The current device is an sm_103 (cached per device).
int check_arch();

// Ordinal of the calling thread's current device, or -1 if cudaGetDevice
// fails or the ordinal is kMaxDevices or more.
int current_device();
// SM count of the current device (cached per device; 0 if it cannot be read).
int device_sm_count();

// A kernel's dynamic shared-memory opt-in, kept per device: cudaFuncSetAttribute
// applies to the current device only, so each device gets its own call. ensure()
// raises the opt-in to at least `bytes` (never lowers it); thread-safe.
class SmemOptIn {
 public:
  template <typename Kernel>
  cudaError_t ensure(Kernel kern, size_t bytes) {
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    if (done_[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
    std::lock_guard<std::mutex> lock(mu_);
    if (done_[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    done_[dev].store(bytes, std::memory_order_release);
    return cudaSuccess;
  }

 private:
  std::mutex mu_;
  std::atomic<size_t> done_[kMaxDevices] = {};
};

// 32 packed int4 codes of one weight row (one 16-byte unit of the record:
// K offsets 0..31 of a 32-wide slice, nibble order as packed) -> 16 words of
// a matrix instruction's A operand, zero point folded in: fp16 (w - z) pairs for
// W4A8, bf16 pairs for W4A16; both exact.
template <int VARIANT>
__device__ __forceinline__ void cvt_w4_unit(const uint4& v, uint32_t z, uint32_t (&o)[16]) {
  const uint32_t wv[4] = {v.x, v.y, v.z, v.w};
  if constexpr (VARIANT == kW4A8) {
    // fp16: 0x6400|e = 1024+e, 0x6400|(e<<4) = 1024+16e (exact)
    const __half2 zlo = __half2half2(__ushort_as_half((uint16_t)(0x6400u | z)));
    const __half2 nzhi = __half2half2(__float2half_rn(-64.0f - (float)z));
    const __half2 sixteenth = __float2half2_rn(0.0625f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = wv[j], w2 = wv[j] >> 8;
      uint32_t h0 = lop3_and_or(w, 0x000F000Fu, 0x64006400u);
      uint32_t h1 = lop3_and_or(w, 0x00F000F0u, 0x64006400u);
      uint32_t h2 = lop3_and_or(w2, 0x000F000Fu, 0x64006400u);
      uint32_t h3 = lop3_and_or(w2, 0x00F000F0u, 0x64006400u);
      __half2 r0 = __hsub2(*reinterpret_cast<__half2*>(&h0), zlo);
      __half2 r1 = __hfma2(*reinterpret_cast<__half2*>(&h1), sixteenth, nzhi);
      __half2 r2 = __hsub2(*reinterpret_cast<__half2*>(&h2), zlo);
      __half2 r3 = __hfma2(*reinterpret_cast<__half2*>(&h3), sixteenth, nzhi);
      o[j * 4 + 0] = *reinterpret_cast<uint32_t*>(&r0);
      o[j * 4 + 1] = *reinterpret_cast<uint32_t*>(&r1);
      o[j * 4 + 2] = *reinterpret_cast<uint32_t*>(&r2);
      o[j * 4 + 3] = *reinterpret_cast<uint32_t*>(&r3);
    }
  } else {
    // bf16: 0x4300|e = 128+e (exact for e < 128)
    const __nv_bfloat162 zz = __bfloat162bfloat162(__ushort_as_bfloat16((uint16_t)(0x4300u | z)));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t h = lop3_and_or(wv[j] >> (4 * q), 0x000F000Fu, 0x43004300u);
        __nv_bfloat162 rr = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&h), zz);
        o[j * 4 + q] = *reinterpret_cast<uint32_t*>(&rr);
      }
    }
  }
}

// Sibling linears that read the same activations, run as one launch: the
// output tiles (128 weight rows each) of linear j are the global tiles
// [tile0[j], tile0[j + 1]); a single linear is the table with count 1.
constexpr int kMaxSegs = 8;
struct SegTable {
  int count;
  int tile0[kMaxSegs + 1];
  const uint8_t* packed[kMaxSegs];  // packed int4 weight of linear j
  uint16_t* y[kMaxSegs];            // its bf16 output [M][N[j]]
  int64_t N[kMaxSegs];
};

// Global tile `nt` resolved to its linear: the packed record (tile, group 0)
// (records of one tile are consecutive, 8512 bytes apart), the output, its row
// count and the tile's first output row. Compile-time indexes only, so the
// table stays in the parameter space.
struct TileRef {
  const uint8_t* rec0;
  uint16_t* y;
  int64_t N;
  int64_t n0;
  int seg;  // which linear
};
__device__ __forceinline__ TileRef tile_ref(const SegTable& s, int nt, int G) {
  const uint8_t* pk = s.packed[0];
  uint16_t* y = s.y[0];
  int64_t N = s.N[0];
  int t0 = 0, seg = 0;
#pragma unroll
  for (int j = 1; j < kMaxSegs; ++j) {
    if (j < s.count && nt >= s.tile0[j]) {
      pk = s.packed[j];
      y = s.y[j];
      N = s.N[j];
      t0 = s.tile0[j];
      seg = j;
    }
  }
  const int64_t lt = nt - t0;
  return TileRef{pk + lt * G * 8512, y, N, lt * 128, seg};
}

// Operands of one GEMM call, already validated by the ABI layer.
struct GemmArgs {
  int variant;
  int64_t M, N, K;
  // activation codes (W4A8, W8A8; a_gsum W4A8 only)
  const int8_t* a_q;
  const void* a_tc;  // tensor-core operand form of a_q (see kTcFp8MaxM)
  const float* a_s;
  const int32_t* a_gsum;
  // W4A16 / W8A16
  const uint16_t* x;
  // packed int4 weight (W4A8, W4A16)
  const uint8_t* packed;
  // int8 weight and per-channel scale (W8A16, W8A8)
  const int8_t* w8;
  const uint16_t* s8;
  // dense bf16 weight [N][K] (W16A16)
  const uint16_t* w16;
  // outputs
  uint16_t* y;
  int32_t* partials;  // non-null: write group partials instead of y (W4A8 only)
  uint64_t timeout_ns;
  // packed int4 variants: sibling linears sharing the activations (null: one
  // linear, packed / y / N above)
  const SegTable* segs;
};

// The segment table of a call: `a.segs`, or the one linear of packed / y / N.
inline SegTable seg_table(const GemmArgs& a) {
  if (a.segs) return *a.segs;
  SegTable t{};
  t.count = 1;
  t.tile0[0] = 0;
  t.tile0[1] = (int)(a.N / 128);
  t.packed[0] = a.packed;
  t.y[0] = a.y;
  t.N[0] = a.N;
  return t;
}

cudaError_t launch_quant_act(const uint16_t* x, int64_t M, int64_t K, int8_t* a_q, float* a_s,
                             int32_t* a_gsum, void* a_tc, cudaStream_t st);
cudaError_t launch_pack_w4(const uint8_t* w_q, const uint16_t* s, const uint8_t* z, int64_t N,
                           int64_t K, void* packed, cudaStream_t st);
cudaError_t launch_unpack_w4(const void* packed, int64_t N, int64_t K, uint8_t* w_q, uint16_t* s,
                             uint8_t* z, cudaStream_t st);
cudaError_t launch_pack_w4_gptq(const int32_t* qweight, const int32_t* qzeros,
                               const uint16_t* scales, int64_t N, int64_t K, int zero_offset,
                               void* packed, cudaStream_t st);
cudaError_t launch_dequant_w4(const void* packed, int64_t N, int64_t K, uint16_t* w,
                              cudaStream_t st);

// ---- rows that pick their own weights (experts, adapters) -------------------------
// Host-side failure reporting of the entry points: records the calling thread's
// last error and returns `code` (an egopq_status).
int fail(int code, const char* fmt, ...);
int cuda_fail(cudaError_t e, const char* what);
// (name, pointer) pairs that must be non-null and 16-byte aligned.
int check_ptrs(int n, ...);

// A launch configuration whose grid may start while the preceding one drains
// (its kernel waits with griddepcontrol.wait before it touches memory).
struct PdlConfig {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  PdlConfig(dim3 grid, unsigned threads, size_t smem, cudaStream_t st) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

constexpr int kMaxSets = 1024;  // weight sets (experts, adapters) of one call

// Where a plan of n slots over S sets lies in a workspace (device memory):
//   head   [0] slots that picked a set, [1] entries of the tile table
//   order  [n] slots sorted by set (slot order inside a set); those without a
//          set come last
//   pos    [n] sorted position of each slot, -1 without a set (may be null)
//   offset [S + 1] first sorted position of each set (set s has the slots
//          [offset[s], offset[s + 1]) of order)
//   tiles  {set, first sorted position, rows} of each tile of at most bt rows
//          of one set; some entries are empty (rows = 0). Not written with
//          bt = 0.
struct RowPlan {
  int* head;
  int32_t* order;
  int32_t* pos;
  int32_t* offset;
  int4* tiles;
};
// Entries the tile table can have (its allocation, and the grid over it).
inline int64_t plan_max_tiles(int64_t n, int S, int bt) { return n / bt + (S < n ? S : n); }

struct RouteArgs {
  const void* logits;
  const float* bias;
  float* weights;
  int32_t* ids;
  int64_t T;
  int E, k, n_group, topk_group, bf16, sigmoid, top2, renorm;
  float scale;
};
cudaError_t launch_route(const RouteArgs& a, cudaStream_t st);
//
// An early kernel (here, quant_rows_kernel, lora_kernel) does its work, or the
// first part of it, before it waits for the kernel in front of it, whose results
// it does not read. It may where every block of that kernel waits first thing:
// then all that was in the stream before is done, and what it reads of that it
// reads past L1.
cudaError_t launch_plan(const int32_t* ids, int64_t n, int S, int bt, const RowPlan& plan,
                        cudaStream_t st, bool early = false);

// How a call's products run (experts.cu).
enum ExpertsWay { kExpertsFew, kExpertsStream, kExpertsTensor };
// (AUTO: the tcgen05 products from more than kStreamRows picks an expert;
// streamed / on the tensor cores, us, 14 and 16 picks an expert: 64 experts, 8
// picks, 3584 x 1280, W4A16 156 / 170 and 169 / 169, W4A8 175 / 186 and 192 /
// 186; 32 experts, 4 picks, 2048 x 1024, W4A16 54.7 / 57.2 and 58.0 / 57.6, W4A8
// 59.3 / 62.5 and 64.8 / 62.6)
constexpr int64_t kStreamRows = 15;
ExpertsWay experts_way(int64_t T, int k, int E, int path);

// Experts: one call's operands and workspace parts, validated by the ABI layer.
struct ExpertsArgs {
  int variant;  // kW4A8 or kW4A16
  int64_t T, H, I;
  int E, k;
  ExpertsWay way;
  const uint16_t* x;
  const int32_t* ids;
  const float* weights;
  const uint8_t* gate_up;
  const uint8_t* down;
  uint16_t* out;
  RowPlan plan;
  uint16_t* x_q;   // x [T][H] in the streaming products' form: fp16 codes and
                   // their scales (W4A8, few and stream), bf16 (W4A16, stream)
  float* x_s;
  uint16_t* rows;  // activations in sorted order [T*k][H], fp16 (tensor), and
  float* rows_s;   // their scales
  void* h;         // gated values [T*k][I], bf16; fp32 (W4A16, tensor)
  uint16_t* h_q;   // fp16 codes of h and their scales (W4A8, and tensor)
  float* h_s;
  void* y;         // [T*k][H], fp32 (stream) or bf16 (tensor)
  uint64_t timeout_ns;
};
cudaError_t launch_experts(const ExpertsArgs& a, cudaStream_t st);
// One tcgen05 product over sorted rows: h = silu(gate) * up, or the down
// projection.
struct RaggedArgs {
  bool gate_up;
  bool exact;           // gate and up: every group's sum exact (tc_experts.cu)
  bool wide;            // tiles of 128 rows (exact: 192), else 64
  int64_t rows_max;     // rows of `act` (T * k)
  int64_t N, K;         // weight rows and columns of one set
  int E;
  const uint16_t* act;  // fp16 [rows_max][K], sorted rows
  const float* a_s;     // scales of the sorted rows
  const uint8_t* packed;
  void* y;              // bf16; of the folded gate and up products fp32
  RowPlan plan;
  uint64_t timeout_ns;
};
cudaError_t launch_ragged(const RaggedArgs& a, cudaStream_t st);

struct LoraArgs {
  const uint16_t* y_in;
  const uint16_t* x;
  const uint16_t* A;
  const uint16_t* B;
  const float* scale;
  const int32_t* ranks;  // may be null: r everywhere
  const int32_t* ids;
  int64_t M, N, K;
  int L, r;
  uint16_t* y_out;
  RowPlan plan;
  float* h;  // [lora_h_rows][r]: [parts of K][M][r] sums of A x, sorted rows
};
// Whether M rows run without a plan (and without a workspace).
bool lora_few(int64_t M);
constexpr int kLoraTile = 32;  // rows of the smallest tile of a planned batch
// Rows of r fp32 sums that lie in memory between two kernels, at most.
int64_t lora_h_rows(int64_t M);
// The plan of a batch that has one, early (see launch_plan); launch_lora then
// gets `beside`: the adapters' product begins beside the kernels in front of it,
// which write y_in but not the rest.
cudaError_t launch_lora_plan(const LoraArgs& a, cudaStream_t st);
cudaError_t launch_lora(const LoraArgs& a, cudaStream_t st, bool beside = false);
int run_linear(const uint16_t* x_bf16, const void* packed, int64_t M, int64_t N, int64_t K,
               uint16_t* y_bf16, uint8_t* ws, int use, cudaStream_t st,
               const LoraArgs* lora = nullptr);

// Weights [E][2I][K] with I gate rows and then I up rows a set, packed with
// the two interleaved sixteen rows at a time.
cudaError_t launch_pack_gate_up(const uint8_t* w_q, const uint16_t* s, const uint8_t* z, int64_t E,
                                int64_t I, int64_t K, void* packed, cudaStream_t st);

// Each kernel unit's device error word, read and cleared (see egopq_common.cuh).
cudaError_t take_error_word_quant_pack(unsigned* out);
cudaError_t take_error_word_gemv(unsigned* out);
cudaError_t take_error_word_tc_gemm(unsigned* out);
cudaError_t take_error_word_tc_experts(unsigned* out);
cudaError_t take_error_word_mx4_gemm(unsigned* out);
cudaError_t take_error_word_mx4_pair(unsigned* out);
// Debug builds: the packed-record read limit of each unit that reads records
// (cudaErrorNotSupported in release builds).
cudaError_t set_record_limit_gemv(unsigned long long bytes);
cudaError_t set_record_limit_tc_gemm(unsigned long long bytes);
cudaError_t set_record_limit_tc_experts(unsigned long long bytes);
cudaError_t set_record_limit_mx4_gemm(unsigned long long bytes);
cudaError_t set_record_limit_mx4_pair(unsigned long long bytes);

// Byte size of the packed records of one linear with N rows and G groups.
__host__ __device__ inline uint64_t packed_record_bytes(int64_t N, int G) {
  return (uint64_t)(N / 128) * (uint64_t)G * 8512u;
}

// CUDA-core GEMV (small M). Returns cudaErrorNotSupported for shapes it does
// not take.
cudaError_t launch_gemv(const GemmArgs& a, cudaStream_t st);
// tcgen05 tensor-core GEMM (any M).
cudaError_t launch_tc_gemm(const GemmArgs& a, cudaStream_t st);
// Token tile (MMA N) the tensor-core GEMM runs an M x N x K call of `variant`
// with: 16, 32 or 64 up to 64 tokens; above, 128 or 192 (per-group variants,
// chosen from the grid each makes) or 128.
int tc_token_tile(int variant, int64_t M, int64_t N, int64_t K);
// Kernel launches of the tensor-core GEMM of that shape: 1, or 2 when the
// persistent grid's short last round runs as a split-K second launch.
int tc_launches(int variant, int64_t M, int64_t N, int64_t K);
// Bounded-wait self test.
cudaError_t launch_selftest_timeout(uint64_t timeout_ns, cudaStream_t st);

// Tensor-core W4A8 operand form: up to this many tokens the activation codes
// are staged as two e4m3 planes (a_q >> 4, a_q & 15) and the MMAs run
// kind::f8f6f4 at K = 32 (token tiles of at most 64); above it as fp16 codes
// for kind::f16 MMAs (128-token tiles).
constexpr int kTcFp8MaxM = 64;
// Largest M per W4A8 GEMV launch (larger M run as several launches).
constexpr int kGemvMaxRows = 16;
// AUTO path: W4A8, W4A16 and W8A16 batches up to this many tokens take the GEMV.
constexpr int kGemvAutoMaxM = 4;

// The kernel path a call takes: `path` itself unless it is EGOPQ_PATH_AUTO,
// which resolves by token count -- W4A8, W4A16 and W8A16 on the CUDA-core
// GEMVs up to kGemvAutoMaxM tokens, W8A8 on its GEMV up to kTcFp8MaxM (its
// tensor-core form exists only above), everything else on the tensor cores.
inline int auto_path(int64_t M, int variant, int path) {
  if (path != EGOPQ_PATH_AUTO) return path;
  if (variant == kW8A8) return M <= kTcFp8MaxM ? EGOPQ_PATH_GEMV : EGOPQ_PATH_TC;
  if (variant == kW16A16) return EGOPQ_PATH_TC;  // (no GEMV form)
  // W4A8, W4A16, W8A16: the GEMV up to kGemvAutoMaxM tokens (measured on
  // GB300: W4A16 3072 x 3072 at one token 5.5 us on the GEMV, 12.3 us on
  // 16-token tensor-core tiles; from 8 tokens the tiles win on every shape)
  return M <= kGemvAutoMaxM ? EGOPQ_PATH_GEMV : EGOPQ_PATH_TC;
}

}  // namespace egopq
