// mx4_internal.h -- layouts and launchers of the microscaled 4-bit linears.
//
// Values are e2m1 codes (sign, two exponent bits, one mantissa bit: 0, .5, 1,
// 1.5, 2, 3, 4, 6). A block of them along K shares a scale: 32 values a power of
// two (E8M0), or 16 values an e4m3 number under one fp32 scale of the tensor
// (E4M3). Both sides of a product, weights and rows, lie in the same records, so
// that one plain bulk copy stages everything 128 rows need for 256 values of K:
//   [0, 16384)   codes: row r's 128 bytes (low nibble first) at 128r, its
//                16-byte chunk c at chunk c ^ (r & 7) -- the tensor cores'
//                128-byte swizzle, as a tiled copy would have left it
//   [16384, ..)  scales, in atoms of 512 bytes: atom j holds scales 4j..4j+3 of
//                every row, row r's at 16 (r % 32) + 4 (r / 32) -- the order in
//                which tcgen05.cp brings them to Tensor Memory
// Record (block of 128 rows, block of 256 K) at (row block * KB + K block).
#pragma once

#include "egopq_internal.h"

namespace egopq {

enum Mx4Type { kMx4Bf16 = 0, kMx4F16 = 1, kMx4F32 = 2 };

constexpr int kMx4Codes = 16384;  // bytes of a record's codes
__host__ __device__ constexpr int mx4_block(int format) {
  return format == EGOPQ_MX4_E4M3 ? 16 : 32;
}
__host__ __device__ constexpr int mx4_record_bytes(int format) {
  return kMx4Codes + 128 * 256 / mx4_block(format);
}
__host__ __device__ constexpr int64_t mx4_kblocks(int64_t K) { return (K + 255) / 256; }
// Tiles of bt rows of one set each that `rows` rows of `sets` sets can make.
inline int64_t mx4_tiles(int64_t rows, int64_t sets, int bt) {
  return rows / bt + (sets < rows ? sets : rows);
}
// Blocks of 128 rows that they can take in the records, each set's first row at
// the start of one.
inline int64_t mx4_row_blocks(int64_t rows, int64_t sets) { return mx4_tiles(rows, sets, 128); }

struct Mx4QuantArgs {
  const void* x;
  int type;              // Mx4Type
  int format;
  int64_t M, K;          // rows that come out, values of each
  bool gated;            // x rows are [gate | up], 2K wide
  const float* tensor_scale;  // may be null: 1
  // ragged: set e's rows are [offsets[e], offsets[e + 1]); row r is x's row
  // index[r] (null: r); rows of x
  const int32_t* offsets;
  const int32_t* index;
  int sets;
  int64_t x_rows;
  uint8_t* codes;        // [M][K / 2], may be null
  uint8_t* scales;       // [M][K / block], may be null
  uint8_t* operand;      // records, may be null
  // The next kernel may begin while this one writes. Not where the operand is the
  // caller's: it may be the weight of the next call, which is read before that waits.
  bool early;
};
cudaError_t launch_mx4_quant(const Mx4QuantArgs& a, cudaStream_t st);
// Rows index[r] of codes [x_rows][K / 2] and scales to the operand's records.
cudaError_t launch_mx4_gather(const Mx4QuantArgs& a, cudaStream_t st);
cudaError_t launch_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K,
                               int format, const float* tensor_scale, int type, void* y,
                               cudaStream_t st);
cudaError_t launch_mx4_pack(const uint8_t* codes, const uint8_t* scales, int64_t sets, int64_t N,
                            int64_t K, int format, void* packed, cudaStream_t st);
cudaError_t launch_mx4_unpack(const void* packed, int64_t sets, int64_t N, int64_t K, int format,
                              uint8_t* codes, uint8_t* scales, cudaStream_t st);

struct Mx4GemmArgs {
  int format;
  int64_t M, N, K;
  const uint8_t* operand;
  const uint8_t* packed;
  const float* a_scale;  // [1], may be null
  const float* w_scale;  // [sets], may be null
  const int32_t* offsets;  // null: one set of M rows
  int sets;
  int type;
  void* y;               // [M][N]
  uint64_t timeout_ns;
};
// cudaErrorNotSupported: more work than one launch's counters hold.
cudaError_t launch_mx4_gemm(const Mx4GemmArgs& a, cudaStream_t st);
cudaError_t launch_mx4_pair(const Mx4GemmArgs& a, cudaStream_t st);  // (of many rows)
// A linear of so few rows that the product's kernel quantizes them itself, and it.
bool mx4_own_rows(const Mx4GemmArgs& a, const Mx4QuantArgs& q);
cudaError_t launch_mx4_own(const Mx4GemmArgs& a, const Mx4QuantArgs& q, cudaStream_t st);

// ---- ragged rows ---------------------------------------------------------------
// One warp: where each set's rows begin (clamped to [0, M] and to the sets
// before, so that no value of offsets leads outside a buffer), and how many
// 128-row blocks and tiles of bt rows lie before it (bt at most 128 and a divisor
// of it, or a multiple). Each array has sets + 1 entries; tile may be null.
// Offsets are read past L1 (the caller may run before the kernel in front of it
// has ended).
__device__ __forceinline__ void mx4_scan_sets(const int32_t* offsets, int sets, int64_t M, int bt,
                                              int* first, int* block, int* tile) {
  const int lane = threadIdx.x & 31;
  int low = 0, blocks = 0, tiles = 0;  // of the sets before this pass
  for (int e0 = 0; e0 <= sets; e0 += 32) {
    const int e = e0 + lane;
    int v = 0;
    if (e <= sets) v = (int)min((int64_t)max(__ldcg(offsets + e), 0), M);
    v = max(v, low);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, up);
    }
    // the next set's first row: the neighbour's, or the next pass's lowest
    int next = __shfl_down_sync(0xffffffffu, v, 1);
    if (lane == 31) {
      next = v;
      if (e < sets) next = max(v, (int)min((int64_t)max(__ldcg(offsets + e + 1), 0), M));
    }
    const int rows = e < sets ? next - v : 0;
    const int own_b = (rows + 127) >> 7, own_t = (rows + bt - 1) / bt;
    int b = own_b, t = own_t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ub = __shfl_up_sync(0xffffffffu, b, o), ut = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) {
        b += ub;
        t += ut;
      }
    }
    if (e <= sets) {
      first[e] = v;
      block[e] = blocks + b - own_b;
      if (tile) tile[e] = tiles + t - own_t;
    }
    low = __shfl_sync(0xffffffffu, v, 31);
    blocks += __shfl_sync(0xffffffffu, b, 31);
    tiles += __shfl_sync(0xffffffffu, t, 31);
  }
}
// The set whose entries of the rising array `at` hold q: the last with at[e] <= q.
__device__ __forceinline__ int mx4_find_set(const int* at, int sets, int q) {
  int lo = 0, hi = sets;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= q) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace egopq
