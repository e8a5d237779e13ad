// experts.cu -- the gated linears of a mixture of experts on packed int4
// weights: the products for few rows an expert, and the row moves and sums
// around the products.
//
//   out[t] = sum_j w[t,j] * D_e( silu(G_e x_t) * (U_e x_t) ),  e = ids[t,j]
//
// G, U and D are packed int4 weights s * (q - z) (group 128); activations are
// bf16 (W4A16) or per-token int8 codes (W4A8, h quantized again as bf16).
//
// Three ways, by the number of rows an expert has (experts_way):
//   few     up to 8 tokens: the matrix instruction's 8 columns are the tokens
//           themselves, every CTA finds the picked experts in the ids alone,
//           and the down product sums over the experts in registers: no plan,
//           no per-pick output
//   stream  rows sorted by expert (RowPlan), tiles of up to 16 rows of one
//   tensor  the tcgen05 products of tc_experts.cu over sorted rows
#include "egopq_internal.h"

namespace egopq {

// ---- products for few rows an expert --------------------------------------------
// A warp takes 32 packed weight rows of one expert (16 gate and the 16 up rows
// of the same outputs, or 32 rows of the down projection) times up to 8 * NT
// rows: the CTA's four warps four such blocks each with all of K, or, where that
// would leave SMs without work, one block with K split between them, whose sums
// they add through shared memory in warp order.
//
// The products run on mma.m16n8k16 with the weights as the 16-row operand. A
// thread of the fragment (row r = lane / 4, columns by lane % 4) reads the
// 16-byte unit of row r, chunk lane % 4 of a packed record: its 32 codes are
// the thread's operand of all eight K steps of the group, once K is taken in
// the order (step, lane % 4) -> 32 * (lane % 4) + 4 * step, which the
// activations follow: word j (8 values) of a thread's 32 belongs to the steps 2j
// and 2j + 1. So no shuffle and no transposition stands between memory and the
// matrix instruction. Rows of activations are stored in that order where this
// file writes them: values 32 t + 8 j + i of a group of 128 at 32 j + 8 t + i
// (unit_place), so that a load reads 64 contiguous bytes of a row.
//
// The weights stream from HBM once: each warp keeps kStages - 1 groups of its
// rows in flight (2.1 KB each) with cp.async into a ring of its own, which no
// other warp waits for. Bound by HBM where the rows are few; the conversion of
// the codes (2.5 instructions a pair in W4A8, 3.5 in W4A16) and the matrix
// instructions (W4A8: 45 % of their pipe) are next. 33 tokens of 64 experts (8
// picks, 3584 x 1280) touch 56 experts on average, 404 MB: W4A8 95 us, 4.2 TB/s of
// the 6.8 a copy reaches, W4A16 100; one token 20.4 us (W4A8 24.0), of which the
// weights' 57 MB are 8.4 and the rest the kernels' starts and ends.
constexpr int kStages = 4;
constexpr int kStageBytes = 2176;  // 4 x 512 codes, 64 scales, 16 zero points, padding
constexpr int kWarps = 4;          // of a CTA: parts of K, or blocks of rows
constexpr int kFewWarps = 16;      // the few-token down product's
constexpr int kFewTokens = 8;
constexpr int kFewSlots = 128;     // picks of a few-token batch

template <int VARIANT>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (VARIANT == kW4A8) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// Where the 8 values (16 bytes) that are number u of their row go.
__host__ __device__ __forceinline__ int64_t unit_place(int64_t u) {
  return (u & ~(int64_t)15) | ((u & 3) << 2) | ((u >> 2) & 3);
}

struct StreamParams {
  const uint16_t* act;     // bf16, or fp16 codes (see quant_rows_kernel) [rows][K]
  const float* a_s;        // scales of those rows (W4A8)
  const uint8_t* packed;   // [E] packed weights of N rows
  uint16_t* h;             // gate and up products: bf16 [sorted row or slot][N / 2]
  float* y;                // down product: fp32 [sorted row][N]
  uint16_t* out;           // few tokens, down product: bf16 [T][N]
  const int* head;         // plan
  const int4* tiles;
  const int32_t* order;
  const int32_t* ids;      // few tokens
  const float* weights;
  int T, k, E, N, G;
};

// A copy of weights, which are read once a call: they leave L2 before what the
// kernels hand on to each other does (layers from HBM: 33 tokens of 64 experts,
// W4A8, 99.1 -> 96.1 us, one token 21.1 -> 20.7; a layer of 100 MB that stays in
// L2 from call to call loses 5 % at 12 tokens).
__device__ __forceinline__ uint64_t weights_policy() {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void cp_async16_weights(uint32_t dst, const void* src,
                                                   uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The four operand words of one word of packed codes.
//   W4A8: the masked nibbles themselves are fp16 numbers below the smallest
//   normal one, q * 2^-24 (words 0 and 2) and q * 2^-20 (words 1 and 3, whose
//   activations come divided by 16: see quant_rows_kernel); every product and
//   sum is a whole multiple of 2^-24, below 2^24 of them, so the group's sum is
//   exact, and the zero point is subtracted from it, as z times the sum of the
//   activations, which one more row tile of ones gives in the same fragment
//   layout.
//   W4A16: q - z, exact, from 128 + q and 128 + z (zz: a pair) as bf16. The products are
//   summed in 32 bits, where a sum is as good as its largest terms: with the
//   zero point taken from the sum, an activation of 1e4 that meets weights of
//   zero (q = z) cost its neighbours of size 1 more than the bf16 result's
//   rounding.
template <int VARIANT>
__device__ __forceinline__ void raw_w4_word(uint32_t w, __nv_bfloat162 zz, uint32_t (&o)[4]) {
  if constexpr (VARIANT == kW4A8) {
    const uint32_t w2 = w >> 8;
    o[0] = w & 0x000F000Fu;
    o[1] = w & 0x00F000F0u;
    o[2] = w2 & 0x000F000Fu;
    o[3] = w2 & 0x00F000F0u;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t h = lop3_and_or(w >> (4 * q), 0x000F000Fu, 0x43004300u);
      const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&h), zz);
      o[q] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int j) {
  return j == 0 ? v.x : (j == 1 ? v.y : (j == 2 ? v.z : v.w));
}

// A warp's stream of units (one group of its 32 weight rows from rbase, times
// the activations of up to 8 NT rows), through a ring of kStages records.
// PLACED: rows in the order of unit_place, else as they come (a thread's 32
// values contiguous).
template <int VARIANT, int NT, bool PLACED>
struct Stream {
  static constexpr int kLane = PLACED ? 8 : 32;  // first value of thread column 1
  static constexpr int kWord = PLACED ? 4 : 1;   // 16-byte units from word to word
  uint32_t ring_at;
  const uint8_t* ring;
  int w_off, m_off;  // this lane's bytes of a record
  int put = 0;
  uint64_t policy = weights_policy();

  __device__ __forceinline__ Stream(uint8_t* r, int rbase) : ring(r) {
    const int lane = threadIdx.x & 31;
    ring_at = smem_u32(r);
    // row `lane`'s 16 bytes of each chunk (a copy is 512 contiguous bytes a
    // warp: with the lanes in fragment order, 32 bytes of four chunks a quarter
    // warp, the copies issued four times slower and one token's gate and up
    // products took 14 instead of 9 us), and of five lanes 16 of the 32 rows'
    // scales and zero points (all past L1: the products that begin early prime
    // their rings before their wait)
    w_off = (rbase + lane) * 16;
    m_off = lane < 4 ? 8192 + 2 * rbase + lane * 16 : 8448 + rbase / 2;
  }

  template <typename Rec>
  __device__ __forceinline__ void issue(bool live, Rec& next_rec) {
    if (live) {
      const int lane = threadIdx.x & 31;
      const uint8_t* rec = next_rec();
      const uint32_t st = ring_at + put * kStageBytes;
#pragma unroll
      for (int c = 0; c < 4; ++c)  // (rows of chunk c exchanged: conflict-free fragments)
        cp_async16_weights(st + (c * 32 + (lane ^ (2 * c))) * 16, rec + w_off + 2048 * c, policy);
      if (lane < 5) cp_async16(st + 2048 + lane * 16, rec + m_off);
      put = put + 1 == kStages ? 0 : put + 1;
    }
    cp_async_commit();
  }

  // The first records on their way (weights depend on no earlier kernel).
  template <typename Rec>
  __device__ __forceinline__ void prime(int n_units, Rec next_rec) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i < n_units, next_rec);
  }

  // sum += the products of the n_units units. next_rec(): the next unit's
  // record (after those primed); next_x(nt): this lane's 32 activations of
  // column tile nt of the next unit, or null; each called once a unit, in
  // order; after(): once a unit is in `sum`.
  template <typename Rec, typename NextX, typename After>
  __device__ __forceinline__ void run(int n_units, Rec next_rec, NextX next_x, After after,
                                      float (&sum)[2][NT][4]) {
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    uint4 x[NT][4];  // word j: the K steps 2j and 2j + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint4* src = n_units > 0 ? next_x(nt) : nullptr;
#pragma unroll
      for (int j = 0; j < 4; ++j) x[nt][j] = src ? __ldg(src + j * kWord) : make_uint4(0, 0, 0, 0);
    }
    int get = 0;
    for (int i = 0; i < n_units; ++i) {
      cp_async_wait<kStages - 2>();
      __syncwarp();  // unit i has landed, and every lane has read unit i - 1
      const uint8_t* st = ring + get * kStageBytes;
      get = get + 1 == kStages ? 0 : get + 1;
      uint4 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = *reinterpret_cast<const uint4*>(
            st + (tig * 32 + ((gid + 8 * q) ^ (2 * tig))) * 16);
      const uint4 zw = *reinterpret_cast<const uint4*>(st + 2112);
      uint16_t sh[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        sh[q] = *reinterpret_cast<const uint16_t*>(st + 2048 + 2 * (gid + 8 * q));
      issue(i + kStages - 1 < n_units, next_rec);
      const uint4* src[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) src[nt] = i + 1 < n_units ? next_x(nt) : nullptr;
      // zero points: rows 8q .. 8q + 7 are the nibbles of word q
      uint32_t z4[4];
      __nv_bfloat162 zz[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        z4[q] = (word_of(zw, q) >> (4 * gid)) & 0xFu;
        zz[q] = __bfloat162bfloat162(__ushort_as_bfloat16((uint16_t)(0x4300u | z4[q])));
      }
      float acc[2][NT][4], ones[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[0][nt][q] = acc[1][nt][q] = ones[nt][q] = 0.f;
      // (independent chains of matrix instructions a column tile: two, and W4A8's
      // ones)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t a[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) raw_w4_word<VARIANT>(word_of(w[q], j), zz[q], a[q]);
        // ones (words 1 and 3: 16, to undo the activations' division)
        constexpr uint32_t kOne = 0x3C003C00u, kOne16 = 0x4C004C00u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint4 b = x[nt][j];
          mma_16816<VARIANT>(acc[0][nt], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
          mma_16816<VARIANT>(acc[1][nt], a[2][0], a[3][0], a[2][1], a[3][1], b.x, b.y);
          if constexpr (VARIANT == kW4A8)
            mma_16816<VARIANT>(ones[nt], kOne, kOne, kOne16, kOne16, b.x, b.y);
          mma_16816<VARIANT>(acc[0][nt], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
          mma_16816<VARIANT>(acc[1][nt], a[2][2], a[3][2], a[2][3], a[3][3], b.z, b.w);
          if constexpr (VARIANT == kW4A8)
            mma_16816<VARIANT>(ones[nt], kOne, kOne, kOne16, kOne16, b.z, b.w);
          // the next unit's word, a unit ahead of its use
          if (src[nt]) x[nt][j] = __ldg(src[nt] + j * kWord);
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float s = f16_bits_to_f32(sh[q]);
        // W4A8: the sums are scaled by 2^-24, and -z 2^-24 as a float is 2^23 + z
        // under a sign, plus 2^23, times that
        const float z = (__uint_as_float(0xCB000000u | z4[q]) + 8388608.f) * 0x1p-24f;
        const float sz = VARIANT == kW4A8 ? s * 0x1p24f : s;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v = acc[q >> 1][nt][(q & 1) * 2 + c];
            if constexpr (VARIANT == kW4A8) v = fmaf(z, ones[nt][c], v);  // (exact)
            float& t = sum[q >> 1][nt][(q & 1) * 2 + c];
            t = fmaf(sz, v, t);
          }
      }
      after();
    }
  }
};

// A warp's share of the work of the gate and up or down products: a block of 32
// weight rows (of blockIdx.y's four, or blockIdx.y itself) and groups of K
// first, first + step, ... , `units` of them -- all of K, or a part that the
// block's other warps complete.
struct Share {
  int block, first, step, units;
  __device__ __forceinline__ Share(bool split, int warp, int G) {
    block = split ? blockIdx.y : blockIdx.y * kWarps + warp;
    first = split ? warp : 0;
    step = split ? kWarps : 1;
    units = first < G ? (G - first + step - 1) / step : 0;
  }
};

// The warp's 32 x 8 NT sums into its rows of `red` ([32][LD] a warp).
template <int NT, int LD>
__device__ __forceinline__ void put_sums(float* red, const float (&sum)[2][NT][4]) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[(mt * 16 + (q >> 1) * 8 + gid) * LD + nt * 8 + tig * 2 + (q & 1)] = sum[mt][nt][q];
}

template <int NT>
__device__ __forceinline__ void zero_sums(float (&sum)[2][NT][4]) {
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int q = 0; q < 4; ++q) sum[mt][nt][q] = 0.f;
}

// ---- few tokens: the picked experts, from the ids alone -----------------------------
// Every warp reads the (at most 128) ids, four a lane, and marks the picked
// experts in a bit set of its own; expert number b is the b-th set bit.
struct FewPicks {
  int id[4];        // ids of slots lane, lane + 32, ...; -1: none or no expert
  uint32_t seen;    // experts 32 lane ..
  int before;       // picked experts of the lanes below
  int count;        // picked experts

  __device__ __forceinline__ FewPicks(const StreamParams& p, uint32_t* bits) {
    const int lane = threadIdx.x & 31, n = p.T * p.k;
    bits[lane] = 0;
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = q * 32 + lane;
      id[q] = i < n ? __ldcg(p.ids + i) : -1;  // (L2: see experts_few_down_kernel)
      if (id[q] < 0 || id[q] >= p.E) id[q] = -1;
      else atomicOr(&bits[id[q] >> 5], 1u << (id[q] & 31));
    }
    __syncwarp();
    seen = bits[lane];
    int incl = __popc(seen);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    before = incl - __popc(seen);
    count = __shfl_sync(0xffffffffu, incl, 31);
  }
  // Expert number b (below the count).
  __device__ __forceinline__ int expert(int b) const {
    const int own = b - before;
    const bool here = own >= 0 && own < __popc(seen);
    uint32_t m = seen;
    for (int i = 0; here && i < own; ++i) m &= m - 1;
    const uint32_t who = __ballot_sync(0xffffffffu, here);
    return __shfl_sync(0xffffffffu, (threadIdx.x & 31) * 32 + __ffs(m) - 1, __ffs(who) - 1);
  }
  // The slots that picked expert e, as 128 bits.
  __device__ __forceinline__ void slots(int e, uint32_t (&m)[4]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) m[q] = __ballot_sync(0xffffffffu, id[q] == e);
  }
};

// Token t's first slot among the 128 bits m (slots t k .. t k + k - 1), or -1.
__device__ __forceinline__ int few_slot(const uint32_t (&m)[4], int t, int T, int k) {
  int found = -1;
  const int lo = t * k, hi = t < T ? lo + k : lo;
#pragma unroll
  for (int q = 3; q >= 0; --q) {
    const int a = max(lo - 32 * q, 0), b = min(hi - 32 * q, 32);
    if (a < b) {
      const uint32_t w = m[q] & (0xffffffffu >> (32 - b)) & (0xffffffffu << a);
      if (w) found = 32 * q + __ffs(w) - 1;
    }
  }
  return found;
}

// ---- h = silu(G x) * (U x) -----------------------------------------------------------
// h is rounded to bf16 once: W4A8's codes are those of bf16 values by definition,
// and W4A16's down product takes bf16 operands.
template <int VARIANT, int NT, bool FEW, bool SPLIT>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 ? 5 : 4)
experts_gate_up_kernel(const StreamParams p) {
  constexpr int LD = 8 * NT + 1;  // padded row of the partial sums
  static_assert(kWarps * kStages * kStageBytes >= kWarps * 32 * LD * 4, "sums reuse the ring");
  __shared__ __align__(128) uint8_t ring[kWarps][kStages * kStageBytes];
  __shared__ uint32_t bits[FEW ? kWarps : 1][32];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int G = p.G, K = G * 128;
  int set, rows, first = 0;  // the expert, its rows here, the first one's sorted position
  uint32_t picked[4];        // few tokens: the expert's slots
  if constexpr (FEW) {
    const FewPicks few(p, bits[warp]);
    if ((int)blockIdx.x >= few.count) return;
    set = few.expert(blockIdx.x);
    few.slots(set, picked);
    rows = p.T;
  } else {
    if ((int)blockIdx.x >= p.head[1]) return;
    const int4 tile = __ldg(p.tiles + blockIdx.x);
    set = tile.x;
    first = tile.y;
    rows = tile.z;
    if (rows == 0) return;
  }
  using S = Stream<VARIANT, NT, !(FEW && VARIANT == kW4A16)>;
  const Share sh(SPLIT, warp, G);
  S stream(ring[warp], (sh.block & 3) * 32);
  const uint8_t* rec =
      p.packed + (((int64_t)set * (p.N >> 7) + (sh.block >> 2)) * G + sh.first) * 8512;
  auto next_rec = [&] {
    const uint8_t* r = rec;
    rec += sh.step * 8512;
    return r;
  };
  stream.prime(sh.units, next_rec);
  const uint16_t* xp[NT];  // this lane's next activations of column gid of each tile, or null
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int j = nt * 8 + gid;
    bool live = j < rows;
    int64_t row = gid;
    if constexpr (FEW) live = few_slot(picked, gid, p.T, p.k) >= 0;
    else row = live ? __ldg(p.order + first + j) / p.k : 0;
    xp[nt] = live ? p.act + row * K + sh.first * 128 + S::kLane * tig : nullptr;
  }
  float sum[2][NT][4];
  zero_sums<NT>(sum);
  stream.run(
      sh.units, next_rec,
      [&](int nt) {
        const uint16_t* x = xp[nt];
        if (x) xp[nt] += sh.step * 128;
        return reinterpret_cast<const uint4*>(x);
      },
      [] {}, sum);
  const int I = p.N >> 1;
  auto put = [&](int j, int at, float gate, float up) {  // output `at` of column j
    const int64_t to = FEW ? few_slot(picked, j, p.T, p.k) : first + j;
    if (to < 0) return;
    if constexpr (VARIANT == kW4A8) {
      const float as = __ldg(p.a_s + (FEW ? j : __ldg(p.order + first + j) / p.k));
      gate *= as;
      up *= as;
    }
    p.h[to * I + unit_place(at >> 3) * 8 + (at & 7)] = f32_to_bf16_bits(gated(gate, up));
  };
  if constexpr (!SPLIT) {
    // this warp's sums are whole: row q >> 1 of each pair, column q & 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int j = nt * 8 + tig * 2 + (q & 1);
        if (j < rows)
          put(j, sh.block * 16 + gid + (q >> 1) * 8, sum[0][nt][q], sum[1][nt][q]);
      }
    return;
  }
  __syncthreads();  // every warp is done with its ring
  float* red = reinterpret_cast<float*>(ring[0]);
  put_sums<NT, LD>(red + warp * 32 * LD, sum);
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * 8 * NT; i += 32 * kWarps) {
    const int c = i & 15, j = i >> 4;
    if (j >= rows) break;
    float gate = 0.f, up = 0.f;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) {
      gate += red[(q * 32 + c) * LD + j];
      up += red[(q * 32 + 16 + c) * LD + j];
    }
    put(j, sh.block * 16 + c, gate, up);
  }
}

// ---- y = D h, a sorted row at a time ----------------------------------------------------
template <int VARIANT, int NT, bool SPLIT>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 ? 5 : 4)
experts_down_kernel(const StreamParams p) {
  constexpr int LD = 8 * NT + 1;
  __shared__ __align__(128) uint8_t ring[kWarps][kStages * kStageBytes];
  // the plan is older than the kernel before this one, every block of which
  // waited for it before it let this grid start: the weights may be on their
  // way before the gated values are there (read past L1, which this grid's own
  // wait has not yet made current)
  if ((int)blockIdx.x >= __ldcg(p.head + 1)) {
    griddep_wait();
    return;
  }
  const int4 tile = __ldcg(p.tiles + blockIdx.x);
  const int rows = tile.z;
  if (rows == 0) {
    griddep_wait();
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int G = p.G, K = G * 128;
  const Share sh(SPLIT, warp, G);
  Stream<VARIANT, NT, true> stream(ring[warp], (sh.block & 3) * 32);
  const uint8_t* rec =
      p.packed + (((int64_t)tile.x * (p.N >> 7) + (sh.block >> 2)) * G + sh.first) * 8512;
  auto next_rec = [&] {
    const uint8_t* r = rec;
    rec += sh.step * 8512;
    return r;
  };
  stream.prime(sh.units, next_rec);
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const uint16_t* xp[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int j = nt * 8 + gid;
    xp[nt] = j < rows ? p.act + (int64_t)(tile.y + j) * K + sh.first * 128 + 8 * tig : nullptr;
  }
  float sum[2][NT][4];
  zero_sums<NT>(sum);
  stream.run(
      sh.units, next_rec,
      [&](int nt) {
        const uint16_t* x = xp[nt];
        if (x) xp[nt] += sh.step * 128;
        return reinterpret_cast<const uint4*>(x);
      },
      [] {}, sum);
  auto put = [&](int j, int at, float v) {
    if constexpr (VARIANT == kW4A8) v *= __ldg(p.a_s + tile.y + j);
    p.y[(int64_t)(tile.y + j) * p.N + at] = v;
  };
  if constexpr (!SPLIT) {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j = nt * 8 + tig * 2 + (q & 1);
          if (j < rows) put(j, sh.block * 32 + mt * 16 + gid + (q >> 1) * 8, sum[mt][nt][q]);
        }
    return;
  }
  __syncthreads();
  float* red = reinterpret_cast<float*>(ring[0]);
  put_sums<NT, LD>(red + warp * 32 * LD, sum);
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * 8 * NT; i += 32 * kWarps) {
    const int c = i & 31, j = i >> 5;
    if (j >= rows) break;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) v += red[(q * 32 + c) * LD + j];
    put(j, sh.block * 32 + c, v);
  }
}

// ---- few tokens: out = sum over the experts of w * D h ----------------------------------
// One CTA a block of 32 output columns; its warps share the (expert, group)
// units of all picked experts, and since column t is token t for every expert,
// the weighted sums over the experts stay in registers.
template <int VARIANT>
__global__ void __launch_bounds__(32 * kFewWarps, 1)
experts_few_down_kernel(const StreamParams p) {
  constexpr int LD = kFewTokens + 1;
  extern __shared__ __align__(128) uint8_t few_ring[];  // [kFewWarps][kStages * kStageBytes]
  __shared__ uint32_t bits[kFewWarps][32];
  __shared__ int slot[kFewSlots][kFewTokens];      // token's row of h, -1: not picked
  __shared__ float weight[kFewSlots][kFewTokens];  // its weight (and the row's scale)
  // the ids and the router's weights are older than the kernel before this one,
  // every block of which waited for them before it let this grid start: the
  // experts can be found, and their weights be on their way, before the gated
  // values are there (ids and weights are read past L1, which this grid's own
  // wait has not yet made current)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int G = p.G, K = G * 128;
  const FewPicks few(p, bits[warp]);
  const int units = few.count * G;
  const int n_units = warp < units ? (units - warp + kFewWarps - 1) / kFewWarps : 0;
  // three walks over this warp's units (expert b, group g), kFewWarps units a
  // step: the records run ahead of the activations, these of the sums
  struct Walk {
    int b, g;
    __device__ __forceinline__ bool step(int G) {  // whether b moved
      g += kFewWarps;
      if (g < G) return false;
      do {
        g -= G;
        ++b;
      } while (g >= G);
      return true;
    }
  };
  Walk rw{warp / G, warp % G}, xw = rw, sw = rw;
  const uint8_t* blk = p.packed + (int64_t)(blockIdx.x >> 2) * G * 8512;
  const int64_t per_set = (int64_t)(p.N >> 7) * G * 8512;
  int rec_set = n_units > 0 ? few.expert(rw.b) : 0;
  auto next_rec = [&] {
    const uint8_t* r = blk + rec_set * per_set + rw.g * 8512;
    if (rw.step(G) && rw.b < few.count) rec_set = few.expert(rw.b);
    return r;
  };
  Stream<VARIANT, 1, true> stream(few_ring + warp * kStages * kStageBytes, (blockIdx.x & 3) * 32);
  stream.prime(n_units, next_rec);
  for (int b = warp; b < few.count; b += kFewWarps) {
    uint32_t picked[4];
    few.slots(few.expert(b), picked);
    if (lane < kFewTokens) {
      const int s = few_slot(picked, lane, p.T, p.k);
      float w = 0.f;
      // (a token that lists an expert twice: h is in the first slot, the
      // weights add up)
      for (int j = s; j >= 0 && j < (lane + 1) * p.k; ++j)
        if ((picked[j >> 5] >> (j & 31)) & 1) w += __ldcg(p.weights + j);
      slot[b][lane] = s;
      weight[b][lane] = w;
    }
  }
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  __syncthreads();
  if constexpr (VARIANT == kW4A8) {
    for (int i = threadIdx.x; i < few.count * kFewTokens; i += 32 * kFewWarps) {
      const int s = slot[i / kFewTokens][i % kFewTokens];
      if (s >= 0) weight[i / kFewTokens][i % kFewTokens] *= p.a_s[s];
    }
    __syncthreads();
  }
  float sum[2][1][4], total[2][1][4];
  zero_sums<1>(sum);
  zero_sums<1>(total);
  stream.run(
      n_units, next_rec,
      [&](int) {
        const int s = slot[xw.b][gid];
        const uint16_t* x =
            s >= 0 ? p.act + (int64_t)s * K + xw.g * 128 + 8 * tig : nullptr;
        xw.step(G);
        return reinterpret_cast<const uint4*>(x);
      },
      [&] {
        // (every unit adds its weighted sum: eight multiply-adds)
        const float w0 = weight[sw.b][2 * tig], w1 = weight[sw.b][2 * tig + 1];
        sw.step(G);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            total[mt][0][q] = fmaf((q & 1) ? w1 : w0, sum[mt][0][q], total[mt][0][q]);
            sum[mt][0][q] = 0.f;
          }
      },
      sum);
  __syncthreads();
  float* red = reinterpret_cast<float*>(few_ring);
  put_sums<1, LD>(red + warp * 32 * LD, total);
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * kFewTokens; i += 32 * kFewWarps) {
    const int c = i & 31, t = i >> 5;
    if (t >= p.T) break;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kFewWarps; ++q) v += red[(q * 32 + c) * LD + t];
    p.out[(int64_t)t * p.N + blockIdx.x * 32 + c] = f32_to_bf16_bits(v);
  }
}

// ---- the picks' outputs summed -----------------------------------------------------
// out[t] = sum_j w[t,j] * y[pos[t,j]] in fp32, j in order; a dropped pick adds
// nothing. A thread holds eight columns. Bound by y: 4096 tokens of 8 picks and
// 3584 columns read 235 MB in 46 us (5.1 TB/s).
constexpr int kCombineThreads = 128;

template <typename Y>  // float or uint16_t (bf16)
__global__ void __launch_bounds__(kCombineThreads)
combine_kernel(const Y* __restrict__ y, const float* __restrict__ weights,
               const int32_t* __restrict__ pos, int k, int64_t H, uint16_t* __restrict__ out) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const int64_t v = (int64_t)blockIdx.y * kCombineThreads + threadIdx.x;
  if (v * 8 >= H) return;
  float acc[8] = {};
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int at = __ldg(pos + t * k + j);
    if (at < 0) continue;
    const float w = __ldg(weights + t * k + j);
    if constexpr (sizeof(Y) == 4) {
      const float4* src = reinterpret_cast<const float4*>(y + (int64_t)at * H) + 2 * v;
      const float4 a = __ldg(src), b = __ldg(src + 1);
      const float q[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, q[i], acc[i]);
    } else {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(y + (int64_t)at * H) + v);
      const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] = fmaf(w, __uint_as_float(q[i] << 16), acc[2 * i]);
        acc[2 * i + 1] = fmaf(w, __uint_as_float(q[i] & 0xFFFF0000u), acc[2 * i + 1]);
      }
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = (uint32_t)f32_to_bf16_bits(acc[2 * i]) |
           ((uint32_t)f32_to_bf16_bits(acc[2 * i + 1]) << 16);
  reinterpret_cast<uint4*>(out + t * H)[v] = make_uint4(o[0], o[1], o[2], o[3]);
}

// ---- rows quantized, and rows in sorted order -----------------------------------------
// Codes of a bf16 row as egopq_quant_act_i8 defines them (fp32 scale
// absmax / 127, fp32 quotient rounded half to even) as exact fp16 numbers: the
// integers themselves (tensor), or every second pair of them divided by 16, the
// form the streaming products' operand words ask for, in the order of
// unit_place, which their input may have already (kStreamPlaced) or not. The
// tensor products take W4A16's activations as fp16 as well: kPowerForm is the
// value over a power of two that brings the row's largest to [2^14, 2^15).
enum QuantForm { kTensorForm, kStreamForm, kStreamPlaced, kPowerForm };

// A row's scale from its largest magnitude.
template <QuantForm FORM>
__device__ __forceinline__ float row_scale(float a) {
  if constexpr (FORM == kPowerForm) {
    // 2^(exponent of a - 14), at least 2^-100 (so that its inverse is a number:
    // smaller rows lose bits below 2^-124); 1 for a row of zeros, infinities or
    // NaNs
    const int e = (int)(__float_as_uint(a) >> 23);
    if (a == 0.f || e == 255) return 1.f;
    return __uint_as_float((uint32_t)max(e - 14, 27) << 23);
  } else {
    return __fdiv_rn(a, 127.0f);
  }
}
// Eight neighbouring values of a row, bf16 or fp32, as they lie in memory.
template <typename X>
struct Eight {
  uint4 v[sizeof(X) / 2];
  // early: past L1 (see launch_plan)
  __device__ __forceinline__ void load(const X* row, int64_t i, bool early) {
#pragma unroll
    for (int q = 0; q < (int)sizeof(X) / 2; ++q) {
      const uint4* at = reinterpret_cast<const uint4*>(row) + i * (sizeof(X) / 2) + q;
      v[q] = early ? __ldcg(at) : __ldg(at);
    }
  }
  __device__ __forceinline__ float value(int j) const {
    if constexpr (sizeof(X) == 4) return __uint_as_float(word_of(v[j >> 2], j & 3));
    const uint32_t w = word_of(v[0], j >> 1);
    return __uint_as_float((j & 1) ? w & 0xFFFF0000u : w << 16);
  }
  __device__ __forceinline__ float absmax(float m) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(value(j)));
    return m;
  }
};
// Eight values of a row of scale s (inv: its inverse for the form, 0 in a row
// of zeros) as eight fp16.
template <QuantForm FORM, typename X>
__device__ __forceinline__ uint4 row_f16(const Eight<X>& v, float s, float inv, bool zero) {
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float q0 = v.value(2 * j), q1 = v.value(2 * j + 1);
    if constexpr (FORM == kPowerForm) {
      q0 *= inv;
      q1 *= inv;
    } else {
      const float f = FORM != kTensorForm && (j & 1) ? 0.0625f : 1.f;
      q0 = zero ? 0.f : quant_code(q0, s, inv) * f;
      q1 = zero ? 0.f : quant_code(q1, s, inv) * f;
    }
    const __half2 h = __floats2half2_rn(q0, q1);
    o[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
template <QuantForm FORM>
__device__ __forceinline__ float row_inverse(float s) {
  return FORM == kPowerForm ? __frcp_rn(s) : quant_recip(s);
}

// Maximum over the R threads of a row (R = 32, or the whole block).
template <int R>
__device__ __forceinline__ float row_max(float m, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if constexpr (R > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = part[0];
#pragma unroll
    for (int i = 1; i < R / 32; ++i) m = fmaxf(m, part[i]);
  }
  return m;
}

constexpr int kRowThreads = 128;

// Rows [0, rows) (or those below head[0], where head is given) of x [.][K].
// early: see launch_plan.
template <int R, QuantForm FORM, typename X>
__global__ void __launch_bounds__(kRowThreads)
quant_rows_kernel(const X* __restrict__ x, const int* __restrict__ head, int64_t rows, int64_t K,
                  uint16_t* __restrict__ codes, float* __restrict__ scales, bool early) {
  // eights of its row a thread keeps (a block a row has few: every test of one
  // that is not there costs a small batch: 8 instead of 4 are 0.4 us)
  constexpr int kRowVecs = R > 32 ? 4 : sizeof(X) == 4 ? 6 : 8;
  __shared__ float part[kRowThreads / 32];
  if (!early) griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int64_t m = (int64_t)blockIdx.x * (kRowThreads / R) + threadIdx.x / R;
  if (head) rows = head[0];
  if (m >= rows) return;  // (a whole warp, or the whole block)
  const int t = threadIdx.x % R;
  const X* src = x + m * K;
  const int64_t nvec = K / 8;
  Eight<X> v[kRowVecs];
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < kRowVecs; ++i)
    if (t + i * R < nvec) v[i].load(src, t + i * R, early);
#pragma unroll
  for (int i = 0; i < kRowVecs; ++i)
    if (t + i * R < nvec) a = v[i].absmax(a);
  for (int64_t i = t + kRowVecs * R; i < nvec; i += R) {
    Eight<X> u;
    u.load(src, i, early);
    a = u.absmax(a);
  }
  a = row_max<R>(a, part);
  const float s = row_scale<FORM>(a), inv = row_inverse<FORM>(s);
  if (t == 0) scales[m] = s;
  auto put = [&](const Eight<X>& u, int64_t i) {
    reinterpret_cast<uint4*>(codes + m * K)[FORM == kStreamForm ? unit_place(i) : i] =
        row_f16<FORM>(u, s, inv, a == 0.f);
  };
#pragma unroll
  for (int i = 0; i < kRowVecs; ++i)
    if (t + i * R < nvec) put(v[i], t + i * R);
  for (int64_t i = t + kRowVecs * R; i < nvec; i += R) {
    Eight<X> u;
    u.load(src, i, early);
    put(u, i);
  }
  if (early) griddep_wait();  // (a grid's end follows that of the one before)
}

// bf16 rows in the order of unit_place (W4A16, stream); early: see launch_plan.
__global__ void __launch_bounds__(kRowThreads)
place_rows_kernel(const uint16_t* __restrict__ x, int64_t K, uint16_t* __restrict__ out) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int64_t at = (int64_t)blockIdx.x * K;
  for (int64_t i = threadIdx.x; i < K / 8; i += kRowThreads)
    reinterpret_cast<uint4*>(out + at)[unit_place(i)] =
        __ldcg(reinterpret_cast<const uint4*>(x + at) + i);
  griddep_wait();  // (a grid's end follows that of the one before)
}

// rows[pos[t, j]] = token t's activations as fp16 and rows_s their scale, for
// each of its picks that has an expert. One CTA a token: x is read from memory
// once, each copy written once. Early (see launch_plan) until the picks' places
// are asked for; the grid behind it reads the plan before its own wait, and so
// must not begin before this one has waited. Bound by its writes: 4096 tokens of 8
// picks and 3584 values write 235 MB in about 45 us.
template <QuantForm FORM>
__global__ void __launch_bounds__(kRowThreads)
scatter_rows_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ pos, int k,
                    int64_t K, uint16_t* __restrict__ rows, float* __restrict__ rows_s) {
  constexpr int kKeep = 4;  // eights of its row a thread keeps
  __shared__ float part[kRowThreads / 32];
  const int64_t m = blockIdx.x;
  const uint16_t* src = x + m * K;
  const int nvec = (int)(K / 8), t = threadIdx.x, lane = t & 31;
  uint4 kept[kKeep];
  float a = 0.f;
  {
    Eight<uint16_t> v[kKeep];
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (t + i * kRowThreads < nvec) v[i].load(src, t + i * kRowThreads, true);
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (t + i * kRowThreads < nvec) a = v[i].absmax(a);
    for (int i = t + kKeep * kRowThreads; i < nvec; i += kRowThreads) {
      Eight<uint16_t> u;
      u.load(src, i, true);
      a = u.absmax(a);
    }
    a = row_max<kRowThreads>(a, part);
    const float s = row_scale<FORM>(a), inv = row_inverse<FORM>(s);
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (t + i * kRowThreads < nvec) kept[i] = row_f16<FORM>(v[i], s, inv, a == 0.f);
  }
  const float s = row_scale<FORM>(a), inv = row_inverse<FORM>(s);
  griddep_wait();
  if (t == 0) griddep_launch_dependents();
  for (int j0 = 0; j0 < k; j0 += 32) {
    const int mine = j0 + lane < k ? __ldcg(pos + m * k + j0 + lane) : -1;
    for (int j = 0; j < 32 && j0 + j < k; ++j) {
      const int at = __shfl_sync(0xffffffffu, mine, j);
      if (at < 0) continue;
      if (t == 0) rows_s[at] = s;
      uint4* to = reinterpret_cast<uint4*>(rows + (int64_t)at * K);
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        if (t + i * kRowThreads < nvec) to[t + i * kRowThreads] = kept[i];
      for (int i = t + kKeep * kRowThreads; i < nvec; i += kRowThreads) {
        Eight<uint16_t> u;
        u.load(src, i, false);
        to[i] = row_f16<FORM>(u, s, inv, a == 0.f);
      }
    }
  }
}

// ---- launches -----------------------------------------------------------------------
template <QuantForm FORM, typename X>
static cudaError_t launch_quant_rows(const X* x, const int* head, int64_t rows, int64_t K,
                                     uint16_t* codes, float* scales, cudaStream_t st,
                                     bool early = false) {
  // a warp a row where there are rows for every warp of the GPU (32768 x 1280:
  // a block a row leaves most of its threads without work), else a block
  if (rows >= 4096 && K <= 2048) {
    PdlConfig c(dim3((unsigned)((rows + 3) / 4), 1, 1), kRowThreads, 0, st);
    return cudaLaunchKernelEx(&c.cfg, quant_rows_kernel<32, FORM, X>, x, head, rows, K, codes,
                              scales, early);
  }
  PdlConfig c(dim3((unsigned)rows, 1, 1), kRowThreads, 0, st);
  return cudaLaunchKernelEx(&c.cfg, quant_rows_kernel<kRowThreads, FORM, X>, x, head, rows, K, codes,
                            scales, early);
}

template <typename Y>
static cudaError_t launch_combine(const ExpertsArgs& a, const Y* y, cudaStream_t st) {
  PdlConfig c(dim3((unsigned)a.T, (unsigned)((a.H / 8 + kCombineThreads - 1) / kCombineThreads), 1),
              kCombineThreads, 0, st);
  return cudaLaunchKernelEx(&c.cfg, combine_kernel<Y>, y, a.weights, (const int32_t*)a.plan.pos,
                            a.k, a.H, a.out);
}

// Many rows an expert: the rows in sorted order, then the tcgen05 products.
template <int VARIANT>
static cudaError_t run_tensor(const ExpertsArgs& a, cudaStream_t st) {
  constexpr QuantForm kForm = VARIANT == kW4A8 ? kTensorForm : kPowerForm;
  const int64_t n = a.T * a.k;
  cudaError_t e = launch_plan(a.ids, n, a.E, 0, a.plan, st);
  if (e != cudaSuccess) return e;
  PdlConfig c(dim3((unsigned)a.T, 1, 1), kRowThreads, 0, st);
  e = cudaLaunchKernelEx(&c.cfg, scatter_rows_kernel<kForm>, a.x, (const int32_t*)a.plan.pos, a.k,
                         a.H, a.rows, a.rows_s);
  if (e != cudaSuccess) return e;
  RaggedArgs r{};
  r.gate_up = true;
  r.wide = n > 64 * (int64_t)a.E;  // (see tc_experts.cu)
  r.exact = VARIANT == kW4A8;
  r.rows_max = n;
  r.N = 2 * a.I;
  r.K = a.H;
  r.E = a.E;
  r.act = a.rows;
  r.a_s = a.rows_s;
  r.packed = a.gate_up;
  r.y = a.h;
  r.plan = a.plan;
  r.timeout_ns = a.timeout_ns;
  if ((e = launch_ragged(r, st)) != cudaSuccess) return e;
  if (VARIANT == kW4A8)
    e = launch_quant_rows<kForm>(static_cast<const uint16_t*>(a.h), a.plan.head, n, a.I, a.h_q,
                                 a.h_s, st);
  else
    e = launch_quant_rows<kForm>(static_cast<const float*>(a.h), a.plan.head, n, a.I, a.h_q, a.h_s,
                                 st);
  if (e != cudaSuccess) return e;
  r.gate_up = false;
  r.N = a.H;
  r.K = a.I;
  r.act = a.h_q;
  r.a_s = a.h_s;
  r.packed = a.down;
  r.y = a.y;
  if ((e = launch_ragged(r, st)) != cudaSuccess) return e;
  return launch_combine(a, (const uint16_t*)a.y, st);
}

// Whether the products of `tiles` row tiles with N weight rows split K between
// the warps of a CTA: with all of K a warp there have to be about seven CTAs an
// SM (64 experts, 8 picks, 3584 x 1280, W4A16, split / whole: 1 token 19.1 /
// 32.9 us, 4 tokens 48.6 / 55.1, 8 tokens 75.1 / 72.3, 33 tokens 104 / 99; 32
// experts, 4 picks, 2048 x 1024: 24 tokens 30 / 37).
static bool split_k(int64_t tiles, int64_t N) {
  return tiles * (N / 128) < 7 * (int64_t)device_sm_count();
}

template <int VARIANT, int NT, bool FEW>
static cudaError_t launch_gate_up(const StreamParams& p, int64_t tiles, int64_t sets,
                                  cudaStream_t st) {
  const bool split = split_k(sets, p.N);
  PdlConfig c(dim3((unsigned)tiles, (unsigned)(p.N / (split ? 32 : 128)), 1), 32 * kWarps, 0, st);
  return split ? cudaLaunchKernelEx(&c.cfg, experts_gate_up_kernel<VARIANT, NT, FEW, true>, p)
               : cudaLaunchKernelEx(&c.cfg, experts_gate_up_kernel<VARIANT, NT, FEW, false>, p);
}

template <int VARIANT>
static cudaError_t run_few(const ExpertsArgs& a, StreamParams p, cudaStream_t st) {
  const int64_t n = a.T * a.k;
  const int64_t most = n < a.E ? n : a.E;
  cudaError_t e = launch_gate_up<VARIANT, 1, true>(p, most, most, st);
  if (e != cudaSuccess) return e;
  if (VARIANT == kW4A8) {
    // (a slot without an expert holds no row: its codes are never read)
    e = launch_quant_rows<kStreamPlaced>(p.h, nullptr, n, a.I, a.h_q, a.h_s, st);
    if (e != cudaSuccess) return e;
  }
  p.act = VARIANT == kW4A8 ? a.h_q : p.h;
  p.a_s = a.h_s;
  p.packed = a.down;
  p.N = (int)a.H;
  p.G = (int)(a.I / 128);
  constexpr size_t kSmem = (size_t)kFewWarps * kStages * kStageBytes;
  static SmemOptIn opt_in;
  if ((e = opt_in.ensure(experts_few_down_kernel<VARIANT>, kSmem)) != cudaSuccess) return e;
  PdlConfig d(dim3((unsigned)(a.H / 32), 1, 1), 32 * kFewWarps, kSmem, st);
  return cudaLaunchKernelEx(&d.cfg, experts_few_down_kernel<VARIANT>, p);
}

template <int VARIANT, int NT>
static cudaError_t run_stream(const ExpertsArgs& a, StreamParams p, cudaStream_t st) {
  const int64_t n = a.T * a.k;
  const int64_t tiles = plan_max_tiles(n, a.E, 8 * NT);
  const int64_t sets = n < a.E ? n : a.E;  // tiles that multiply, at least about
  cudaError_t e = launch_gate_up<VARIANT, NT, false>(p, tiles, sets, st);
  if (e != cudaSuccess) return e;
  if (VARIANT == kW4A8) {
    e = launch_quant_rows<kStreamPlaced>(p.h, a.plan.head, n, a.I, a.h_q, a.h_s, st);
    if (e != cudaSuccess) return e;
  }
  p.act = VARIANT == kW4A8 ? a.h_q : p.h;
  p.a_s = a.h_s;
  p.packed = a.down;
  p.N = (int)a.H;
  p.G = (int)(a.I / 128);
  const bool split = split_k(sets, p.N);
  PdlConfig d(dim3((unsigned)tiles, (unsigned)(p.N / (split ? 32 : 128)), 1), 32 * kWarps, 0, st);
  e = split ? cudaLaunchKernelEx(&d.cfg, experts_down_kernel<VARIANT, NT, true>, p)
            : cudaLaunchKernelEx(&d.cfg, experts_down_kernel<VARIANT, NT, false>, p);
  if (e != cudaSuccess) return e;
  return launch_combine(a, (const float*)a.y, st);
}

template <int VARIANT>
static cudaError_t run_experts(const ExpertsArgs& a, cudaStream_t st) {
  if (a.way == kExpertsTensor) return run_tensor<VARIANT>(a, st);
  const int64_t n = a.T * a.k;
  StreamParams p{};
  p.act = VARIANT == kW4A8 ? a.x_q : a.x;
  p.a_s = a.x_s;
  p.packed = a.gate_up;
  p.h = static_cast<uint16_t*>(a.h);
  p.y = static_cast<float*>(a.y);
  p.out = a.out;
  p.head = a.plan.head;
  p.tiles = a.plan.tiles;
  p.order = a.plan.order;
  p.ids = a.ids;
  p.weights = a.weights;
  p.T = (int)a.T;
  p.k = a.k;
  p.E = a.E;
  p.N = (int)(2 * a.I);
  p.G = (int)(a.H / 128);
  // rows of a tile, 8 or 16: an expert with more rows takes several tiles, whose
  // weights then come from L2, but a tile of 16 multiplies twice as much per
  // record, and W4A8 half as much again for its zero points. Tiles of 8 / of 16,
  // us, by picks an expert: 64 experts, 8 picks, 3584 x 1280, W4A16 6: 115 / 118,
  // 7: 125 / 120, W4A8 14: 175 / 178, 16: 192 / 192; 32 experts, 4 picks, 2048 x
  // 1024, W4A16 6: 38.7 / 41.8, 10: 47.3 / 47.3, W4A8 14: 59.3 / 59.9, 16: 64.8 /
  // 64.1
  const int nt = n <= (int64_t)(VARIANT == kW4A8 ? 15 : 6) * a.E ? 1 : 2;
  cudaError_t e = cudaSuccess;
  if (a.way == kExpertsStream) e = launch_plan(a.ids, n, a.E, 8 * nt, a.plan, st);
  // (the rows do not depend on the plan: they are quantized, or placed, beside it)
  if (e == cudaSuccess && VARIANT == kW4A8)
    e = launch_quant_rows<kStreamForm>(a.x, nullptr, a.T, a.H, a.x_q, a.x_s, st,
                                       a.way == kExpertsStream);
  if (e == cudaSuccess && VARIANT == kW4A16 && a.way == kExpertsStream) {
    PdlConfig c(dim3((unsigned)a.T, 1, 1), kRowThreads, 0, st);
    e = cudaLaunchKernelEx(&c.cfg, place_rows_kernel, a.x, a.H, a.x_q);
    p.act = a.x_q;
  }
  if (e != cudaSuccess) return e;
  if (a.way == kExpertsFew) return run_few<VARIANT>(a, p, st);
  return nt == 1 ? run_stream<VARIANT, 1>(a, p, st) : run_stream<VARIANT, 2>(a, p, st);
}

cudaError_t launch_experts(const ExpertsArgs& a, cudaStream_t st) {
  return a.variant == kW4A8 ? run_experts<kW4A8>(a, st) : run_experts<kW4A16>(a, st);
}

ExpertsWay experts_way(int64_t T, int k, int E, int path) {
  if (path == EGOPQ_PATH_TC) return kExpertsTensor;
  const int64_t n = T * k;
  if (path == EGOPQ_PATH_AUTO && n > kStreamRows * E) return kExpertsTensor;
  return T <= kFewTokens && n <= kFewSlots ? kExpertsFew : kExpertsStream;
}

}  // namespace egopq
