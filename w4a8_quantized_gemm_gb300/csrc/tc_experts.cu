// tc_experts.cu -- the experts' products on the tensor cores (tcgen05), for
// many rows an expert.
//
//   y[p] = a_s[p] * W_e a[p]   (or silu(gate) * up of interleaved rows),
//   W = s * (q - z),  rows p sorted by expert e
//
// Activations come as fp16 numbers with one fp32 scale a row: the int8 codes of
// W4A8, or for W4A16 the bf16 values over a power of two (fp16 holds their
// eight bits exactly from 2^-29 of the row's largest up). The weights enter in
// one of two ways:
//   folded  s * (q - z) as fp16, rounded once (2^-11 of it at most, and
//           independently a weight, where the bf16 result's rounding is 2^-8): a
//           whole row of K accumulates in Tensor Memory and is read once a tile.
//           A product of 65520 and more becomes infinite
//   exact   q - z: every group's sum is the exact integer, read a group at a
//           time and scaled and added in fp32. For the gate and up products of
//           W4A8, whose bf16 results are quantized again: the folded weights'
//           rounding moves about one int8 code of a hundred by one, which
//           doubles the distance of the layer's output from its definition.
//
// A persistent CTA an SM walks units (expert, 128 weight rows, up to BT rows of
// the expert), whose number only the device knows; all row tiles of a weight
// block in turn. The 128 weight rows are the MMA's M and lie in Tensor Memory
// as the A operand, the BT rows its N, from shared memory:
//   records producer   one 8512-byte bulk copy a group (codes, scales, zeros)
//   rows producer      one TMA copy a group (BT x 128 fp16, 128-byte swizzle)
//   2 converter sets   of four warps, taking groups in turn: codes -> fp16
//                      weights -> one of four A buffers (64 columns each)
//   2 issuers          taking groups in turn, folded ones into an accumulator of
//                      its own (two threads' MMAs into one would need an order
//                      between them). They meet the converters on named
//                      barriers, since an mbarrier test queues behind the MMAs
//                      just issued
//   2 drain warpgroups half of the BT columns each: accumulators added, scaled,
//                      gated, staged in shared memory, stored by rows (keep
//                      their work short: 20 instructions more a value for
//                      fp16 gated values over powers of two took 430 us where
//                      fp32 ones of twice the memory take 372, 2977 tokens)
// Tensor Memory: 256 columns of accumulators (folded: two an issuer at BT = 64,
// so a tile's reading runs beside the next one's MMAs, one at 128; exact: four
// groups'), 256 of A buffers.
//
// What a group costs (measured, 64 experts of 3584 x 1280, cycles): with every
// weight used once ~800 at 64 rows, ~1050 at 128, ~1150 at 160, ~1330 at 192;
// with weights shared by several row tiles ~780 at 128. The eight MMAs alone
// take ~760, for an MMA with A in Tensor Memory costs ~95 cycles for any N up to
// 176; beyond, rows are written to and read from shared memory at 128 bytes a
// cycle, four cycles a row and group. So tiles have 64 rows up to 64 rows an
// expert and 128 above. Deeper rings (14 records), four converter sets, four
// issuers, one issuer (exact, 128 rows) changed none of this or cost time.
// All three kernels of a layer: 4096 tokens of 64 experts (8 picks, 3584 x 1280,
// W4A8) take 891 us, 1012 TFLOP/s, half of cuBLAS's bf16 rate: gate and up (in
// 192-row exact tiles, tc_kernel.cuh) 500, down 250, the rest the rows' ways in
// and out. 2977 tokens of 64 experts (6 picks, 2048 x 1408, W4A16) 367 us, 842
// TFLOP/s (reading an accumulator only when it is needed next cost 394); 509
// tokens of 32 experts (4 picks, 2048 x 1024) 71 us.
// Every wait on an mbarrier is bounded; after one gives up, every warp still
// makes its remaining named-barrier meetings and skips the work.
#include "tc_kernel.cuh"

namespace egopq {

template <int BT, bool EXACT>
struct RgCfg {
  static constexpr int kIssuers = 2;
  static constexpr int kNumA = 4;
  // accumulators: folded, of so many tiles (each issuer its own); exact, of so
  // many groups
  static constexpr int kSlots = EXACT ? 4 : (BT == 64 ? 2 : 1);
  static_assert(!EXACT || BT == 64, "exact tiles have 64 rows");
  static constexpr int kConvSets = 2;
  static constexpr int kDrainWarps = 8;
  static constexpr int kConvWarp0 = kDrainWarps;
  static constexpr int kRecWarp = kDrainWarps + 4 * kConvSets;
  static constexpr int kRowWarp = kRecWarp + 1;
  static constexpr int kMmaWarp = kRowWarp + 1;
  static constexpr int kThreads = 32 * (kMmaWarp + kIssuers);
  static constexpr int kRowBytes = BT * 256;  // a group's rows
  static constexpr int kHalfBytes = BT * 128;
  static constexpr int kRowStages = BT == 64 ? 7 : 4;
  static constexpr int kRecStages = 6;
  static constexpr int kHB = BT / 2;  // columns of a drain warpgroup
  static constexpr int kRound = 32;   // columns it stages at a time
  // shared memory, from a 1024-byte boundary
  static constexpr int kRecAt = kRowStages * kRowBytes;
  static constexpr int kOutAt = kRecAt + (kRecStages * 8512 + 1023) / 1024 * 1024;
  static constexpr int kOutBytes = 2 * kRound * 128 * 2;  // staged results, both warpgroups
  static constexpr int kAsAt = kOutAt + kOutBytes;
  static constexpr int kBarAt = kAsAt + BT * 4;
  static constexpr int kFirstAt = kBarAt + 512;  // row tiles below each set
  static constexpr int kOffsetAt = kFirstAt + (kMaxSets + 4) * 4;  // rows below each set
  static constexpr int kSmem = kOffsetAt + (kMaxSets + 4) * 4 + 1024;
  static_assert(kSmem <= kMaxSmem && kSmem > kMaxSmem / 2, "shared memory of one CTA an SM");
};

struct RgParams {
  const float* a_s;
  const uint8_t* packed;
  void* y;                // bf16, or fp32 (folded gate and up) [sorted rows][columns]
  const int32_t* offset;  // first sorted row of each set, [sets + 1]
  int sets, n_tiles, G;   // weight blocks of 128 rows a set, groups of K
  uint64_t timeout_ns;
};

// Codes of one 16-byte unit -> 16 words of s * (q - z) as fp16 pairs.
__device__ __forceinline__ void scaled_w4_unit(const uint4& v, uint32_t z, __half2 s,
                                               uint32_t (&o)[16]) {
  cvt_w4_unit<kW4A8>(v, z, o);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&o[i]), s);
    o[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <int BT, bool GATE_UP, bool EXACT>
__global__ void __launch_bounds__(RgCfg<BT, EXACT>::kThreads, 1)
ragged_kernel(const __grid_constant__ CUtensorMap row_map, const __grid_constant__ RgParams p) {
  using C = RgCfg<BT, EXACT>;
  constexpr int XS = C::kRowStages, RS = C::kRecStages, NA = C::kNumA, HB = C::kHB;
  constexpr int kCols = GATE_UP ? 64 : 128;  // output columns of a weight block
  // W4A16's gated values stay fp32 until their row's scale is known (rounding
  // them to bf16 first would be the largest error of the layer but its output's)
  using Y = std::conditional_t<GATE_UP && !EXACT, float, uint16_t>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_addr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.G;

  // ---- barriers, Tensor Memory, the units' table ----------------------------------
  const uint32_t bar0 = base + C::kBarAt;
  auto xfull = [&](int s) { return bar0 + 8u * s; };
  auto xempty = [&](int s) { return bar0 + 8u * (XS + s); };
  auto wfull = [&](int r) { return bar0 + 8u * (2 * XS + r); };
  auto wempty = [&](int r) { return bar0 + 8u * (2 * XS + RS + r); };
  auto aempty = [&](int b) { return bar0 + 8u * (2 * XS + 2 * RS + b); };
  // folded: 2 slot + issuer of the unit's accumulators, and 2 (unit mod 4) +
  // issuer of those that were read: four units, because a converter set may wait
  // for every fourth unit only (one group a tile), and must not miss a phase of
  // its barrier; exact: slot of the group's accumulator for both
  auto dfull = [&](int s) { return bar0 + 8u * (2 * XS + 2 * RS + NA + s); };
  auto dempty = [&](int s) { return bar0 + 8u * (2 * XS + 2 * RS + NA + 4 + s); };
  auto fin = [&](int q) { return bar0 + 8u * (2 * XS + 2 * RS + NA + 12 + q); };
  static_assert(8 * (2 * XS + 2 * RS + NA + 14) <= 496, "barrier region");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarAt + 496);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBarAt + 500);
  int* first_tile = reinterpret_cast<int*>(smem + C::kFirstAt);
  int* offset = reinterpret_cast<int*>(smem + C::kOffsetAt);

  if (threadIdx.x == 0) {
    for (int s = 0; s < XS; ++s) {
      mbar_init(xfull(s), 1);
      mbar_init(xempty(s), 1);
    }
    for (int r = 0; r < RS; ++r) {
      mbar_init(wfull(r), 1);
      mbar_init(wempty(r), 4);
    }
    for (int b = 0; b < NA; ++b) mbar_init(aempty(b), 1);
    for (int s = 0; s < 4; ++s) mbar_init(dfull(s), 1);
    for (int s = 0; s < 8; ++s) mbar_init(dempty(s), C::kDrainWarps);
    for (int q = 0; q < 2; ++q) mbar_init(fin(q), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::kRowWarp && lane == 0) prefetch_tensormap(&row_map);
  if (warp == C::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // The plan was there before this kernel could begin (every block of the one in
  // front waits before it lets it), so the units and the weights need no wait;
  // the rows and their scales, and what this kernel writes, do (rows producer,
  // drains).
  if (warp == 0) {
    int below = 0;
    for (int e0 = 0; e0 < p.sets; e0 += 32) {
      const int e = e0 + lane;
      int t = 0;
      if (e < p.sets) {
        const int row = __ldcg(p.offset + e);
        offset[e] = row;
        t = (__ldcg(p.offset + e + 1) - row + BT - 1) / BT;
      }
      int incl = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      if (e < p.sets) first_tile[e] = below + incl - t;
      below += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      first_tile[p.sets] = below;
      offset[p.sets] = __ldcg(p.offset + p.sets);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t a_tmem = tmem + 256;
  const uint64_t tmo = p.timeout_ns;
  const int total = first_tile[p.sets] * p.n_tiles;
  const int n_units = (int)blockIdx.x < total
                          ? (total - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x
                          : 0;
  const int n_items = n_units * G;
  // unit k of this CTA: its expert, weight block and rows
  struct Unit {
    const uint8_t* rec0;
    int row0, rows, n0;
  };
  auto unit_at = [&](int k) {
    const int u = (int)blockIdx.x + k * (int)gridDim.x;
    const int q = u / p.n_tiles;  // the set whose tiles cover q: the last with first_tile <= q
    int lo = 0, hi = p.sets;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_tile[mid] <= q) lo = mid; else hi = mid;
    }
    const int first = first_tile[lo], tiles = first_tile[lo + 1] - first;
    const int local = u - first * p.n_tiles;
    const int t = local / tiles;
    Unit r;
    r.row0 = offset[lo] + (local - t * tiles) * BT;
    r.rows = min(BT, offset[lo + 1] - r.row0);
    r.n0 = t;
    r.rec0 = p.packed + ((int64_t)lo * p.n_tiles + t) * G * 8512;
    return r;
  };
  // all threads, at the end: no warp leaves while Tensor Memory or a copy is in use
  auto teardown = [&] {
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(C::kThreads) : "memory");
  };
  // group i's converters and its issuer, on the named barrier of its A buffer
  constexpr int kMeet = 32 * 5;  // a set and an issuer
  auto meet = [&](int i) {
    asm volatile("bar.sync %0, %1;" ::"r"(2 + i % NA), "n"(kMeet) : "memory");
  };

  auto rec_role = [&] {
    // ---------------------------------------------------------------- records
    if (lane == 0) {
      int issued = 0, gi = 0, k = 0;
      Unit un{};
      if (n_items > 0) un = unit_at(0);
      for (int i = 0; i < n_items; ++i) {
        const int r = i % RS;
        if (i >= RS && !mbar_wait(wempty(r), ((i / RS) & 1) ^ 1, abort_flag, tmo)) break;
        mbar_arrive_expect_tx(wfull(r), 8512);
        const uint8_t* src = un.rec0 + (int64_t)gi * 8512;
        if (!dbg_record_ok((uint64_t)(src - p.packed), 8512,
                           (uint64_t)p.sets * p.n_tiles * G * 8512u))
          src = p.packed;
        bulk_load(base + C::kRecAt + (uint32_t)(r * 8512), src, 8512, wfull(r));
        ++issued;
        if (++gi == G) {
          gi = 0;
          if (++k < n_units) un = unit_at(k);
        }
      }
      for (int i = (issued > RS ? issued - RS : 0); i < issued; ++i) {
        volatile int no_abort = 0;
        mbar_wait(wfull(i % RS), (i / RS) & 1, &no_abort, tmo);
      }
    }
    __syncwarp();
    teardown();
  };
  auto row_role = [&] {
    // ---------------------------------------------------------------- rows
    if (lane == 0) {
      griddep_wait();
      griddep_launch_dependents();
      int issued = 0, gi = 0, k = 0;
      Unit un{};
      if (n_items > 0) un = unit_at(0);
      for (int i = 0; i < n_items; ++i) {
        const int s = i % XS;
        if (i >= XS && !mbar_wait(xempty(s), ((i / XS) & 1) ^ 1, abort_flag, tmo)) break;
        mbar_arrive_expect_tx(xfull(s), C::kRowBytes);
        // (rows past the expert's last are another's: columns that are not stored)
        tma_load_3d(base + (uint32_t)(s * C::kRowBytes), &row_map, xfull(s), 0, un.row0, gi * 2);
        ++issued;
        if (++gi == G) {
          gi = 0;
          if (++k < n_units) un = unit_at(k);
        }
      }
      for (int i = (issued > XS ? issued - XS : 0); i < issued; ++i) {
        volatile int no_abort = 0;
        mbar_wait(xfull(i % XS), (i / XS) & 1, &no_abort, tmo);
      }
    }
    __syncwarp();
    teardown();
  };
  auto mma_role = [&] {
    // ---------------------------------------------------------------- issuers
    const int q = warp - C::kMmaWarp;
    constexpr int kStep = C::kIssuers;
    constexpr uint32_t idesc = idesc_f16(128, BT, 0);
    bool any = false;
    int gi = q, k = 0;  // item i = unit k, group gi
    while (gi >= G) {
      gi -= G;
      ++k;
    }
    for (int i = q; i < n_items; i += kStep) {
      meet(i);
      if (!__shfl_sync(0xffffffffu, *abort_flag != 0 ? 1 : 0, 0)) {
        if (lane == 0) {
          const int s = i % XS, b = i % NA;
          const int slot = (EXACT ? i : k) % C::kSlots;
          const uint32_t d = tmem + (EXACT ? slot * BT : slot * 128 + q * BT);
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t b_addr =
                base + (uint32_t)(s * C::kRowBytes + (j >> 2) * C::kHalfBytes + (j & 3) * 32);
            tc_mma_f16_ts(d, a_tmem + b * 64 + j * 8, sdesc_kmajor_sw128(b_addr), idesc,
                          (j > 0 || (!EXACT && gi >= kStep)) ? 1u : 0u);
          }
          tc_commit(xempty(s));
          tc_commit(aempty(b));
          // (folded: at this issuer's last group of the tile)
          if (EXACT || gi + kStep >= G) tc_commit(dfull(EXACT ? slot : slot * 2 + q));
        }
        any = true;
      }
      __syncwarp();
      gi += kStep;
      while (gi >= G) {
        gi -= G;
        ++k;
      }
    }
    if (lane == 0 && any) {  // let this issuer's MMAs finish before teardown
      tc_commit(fin(q));
      volatile int no_abort = 0;
      mbar_wait(fin(q), 0, &no_abort, tmo);
    }
    __syncwarp();
    teardown();
    if (warp == C::kMmaWarp) {
      tc_fence_after();
      tmem_dealloc(tmem, 512);
    }
  };
  auto conv_role = [&] {
    // ---------------------------------------------------------------- converters
    const int r = (warp & 3) * 32 + lane;  // weight row == TMEM lane
    const int set = (warp - C::kConvWarp0) >> 2;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const bool gate_warp = (warp & 3) == 0;
    int gi = set, k = 0;  // item i = unit k, group gi
    while (gi >= G) {
      gi -= G;
      ++k;
    }
    // (whole warps wait and give up together: Tensor Memory's stores are a warp's)
    auto wait = [&](uint32_t bar, int phase) {
      return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, abort_flag, tmo)) != 0;
    };
    auto convert = [&](int i) -> bool {
      const int w = i % RS, b = i % NA, s = i % XS;
      if (!wait(wfull(w), i / RS)) return false;
      const uint8_t* rec = smem + C::kRecAt + w * 8512;
      uint4 v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        v[c] = *reinterpret_cast<const uint4*>(rec + c * 2048 + r * 16);
      const uint16_t sh = *reinterpret_cast<const uint16_t*>(rec + 8192 + 2 * r);
      const uint32_t zb = rec[8448 + (r >> 1)];
      __syncwarp();
      if (lane == 0) mbar_arrive(wempty(w));
      const uint32_t z = (r & 1) ? (zb >> 4) : (zb & 0xF);
      const __half2 s2 = __half2half2(__ushort_as_half(sh));
      // A buffer b is free once the MMAs of the item before in it have completed
      const uint32_t dst = a_tmem + lane_base + b * 64;
      uint32_t out[16];
      auto weights = [&](const uint4& u) {
        if constexpr (EXACT) cvt_w4_unit<kW4A8>(u, z, out);
        else scaled_w4_unit(u, z, s2, out);
      };
      weights(v[0]);
      if (!wait(aempty(b), (i / NA) ^ 1)) return false;
      tc_fence_after();
      tmem_st16(dst, out);
#pragma unroll
      for (int c = 1; c < 4; ++c) {
        weights(v[c]);
        tmem_st16(dst + c * 16, out);
      }
      if (gate_warp) {
        // the rows have landed, and the accumulator has been read: of the tile
        // kSlots before (at a tile's first groups), or of the group kSlots before
        if (!wait(xfull(s), i / XS)) return false;
        if constexpr (EXACT) {
          if (!wait(dempty(i % C::kSlots), (i / C::kSlots) ^ 1)) return false;
        } else {
          const int v_unit = k - C::kSlots;
          if (gi < 2 && v_unit >= 0 && !wait(dempty(v_unit % 4 * 2 + set), v_unit / 4)) return false;
        }
      }
      tmem_wait_st();
      return true;
    };
    bool ok = true;
    for (int i = set; i < n_items; i += C::kConvSets) {
      if (ok) ok = convert(i);
      tc_fence_before();
      __syncwarp();
      meet(i);
      gi += C::kConvSets;
      while (gi >= G) {
        gi -= G;
        ++k;
      }
    }
    __syncwarp();
    teardown();
  };
  auto drain_role = [&] {
    // ---------------------------------------------------------------- drains
    griddep_wait();
    const int r = (warp & 3) * 32 + lane;
    const int wg = warp >> 2;
    const int col0 = wg * HB;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    Y* out = reinterpret_cast<Y*>(smem + C::kOutAt + wg * C::kRound * 256);
    float* as = reinterpret_cast<float*>(smem + C::kAsAt) + col0;
    const int64_t ld = (int64_t)p.n_tiles * kCols;
    bool ok = true;
    // columns [c0, c0 + kRound) of the unit, given as v: scaled, gated, staged
    // and stored (all four warps; two barriers, whatever happened)
    auto put = [&](const Unit& un, int c0, const float (&v)[C::kRound]) {
      constexpr int RD = C::kRound;
      const float* as_c = as + c0;
      if constexpr (GATE_UP) {
        // lanes 16 apart hold gate and up of one output; of two tokens each
        // takes one
        const bool up = (lane & 16) != 0;
        const int col = (warp & 3) * 16 + (lane & 15);
#pragma unroll
        for (int c = 0; c < RD; c += 2) {
          const float2 a2 = *reinterpret_cast<const float2*>(as_c + c);
          const float v0 = v[c] * a2.x, v1 = v[c + 1] * a2.y;
          const float other = __shfl_xor_sync(0xffffffffu, up ? v0 : v1, 16);
          const float h = up ? gated(other, v1) : gated(v0, other);
          if constexpr (sizeof(Y) == 4) out[(c + (up ? 1 : 0)) * kCols + col] = h;
          else out[(c + (up ? 1 : 0)) * kCols + col] = f32_to_bf16_bits(h);
        }
      } else {
        // (a pick's output is rounded to bf16 once before the picks are summed in
        // fp32: written and read again once a pick, it is half of fp32's memory,
        // 235 MB at 4096 tokens of 8 picks and 3584 columns)
#pragma unroll
        for (int c = 0; c < RD; c += 2) {
          const float2 a2 = *reinterpret_cast<const float2*>(as_c + c);
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[c] * a2.x, v[c + 1] * a2.y);
          out[c * kCols + r] = __bfloat16_as_ushort(h.x);
          out[(c + 1) * kCols + r] = __bfloat16_as_ushort(h.y);
        }
      }
      asm volatile("bar.sync %0, 128;" ::"r"(6 + wg) : "memory");
      const int rows = ok ? min(RD, un.rows - col0 - c0) : 0;
      constexpr int kPer = 16 / sizeof(Y), kVec = kCols / kPer;  // 16-byte vectors of a row
      const uint4* src = reinterpret_cast<const uint4*>(out);
      Y* dst = static_cast<Y*>(p.y) + (int64_t)(un.row0 + col0 + c0) * ld + un.n0 * kCols;
#pragma unroll 4
      for (int i = r; i < rows * kVec; i += 128)
        *reinterpret_cast<uint4*>(dst + (int64_t)(i / kVec) * ld + (i % kVec) * kPer) = src[i];
      asm volatile("bar.sync %0, 128;" ::"r"(6 + wg) : "memory");  // the staging rows are free
    };
    for (int k = 0; k < n_units; ++k) {
      const Unit un = unit_at(k);
      float my_as = 0.f;
      if (r < HB && col0 + r < un.rows) my_as = __ldg(p.a_s + un.row0 + col0 + r);
      if constexpr (EXACT) {
        float R[HB];
#pragma unroll
        for (int q = 0; q < HB; ++q) R[q] = 0.f;
        // this row's scales, fetched a group ahead
        const uint8_t* sp = un.rec0 + 8192 + 2 * r;
        uint16_t s_next = __ldg(reinterpret_cast<const uint16_t*>(sp));
        for (int gi = 0; gi < G; ++gi) {
          const int i = k * G + gi, slot = i % C::kSlots;
          const uint64_t s2 = f32x2_splat(f16_bits_to_f32(s_next));
          if (gi + 1 < G)
            s_next = __ldg(reinterpret_cast<const uint16_t*>(sp + (int64_t)(gi + 1) * 8512));
          if (ok) ok = mbar_wait(dfull(slot), (i / C::kSlots) & 1, abort_flag, tmo);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + lane_base + slot * BT + col0;
          constexpr int kLd = HB;  // columns on their way at once
#pragma unroll
          for (int c = 0; c < HB; c += kLd) {
            uint32_t v[kLd / 16][16];
#pragma unroll
            for (int q = 0; q < kLd / 16; ++q) tmem_ld16(d + c + q * 16, v[q]);
            tmem_wait_ld();
            if (c + kLd >= HB) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(dempty(slot));
            }
#pragma unroll
            for (int q = 0; q < kLd; q += 2)
              fma_f32x2(R[c + q], R[c + q + 1], s2, v[q / 16][q % 16], v[q / 16][q % 16 + 1]);
          }
        }
        if (r < HB) as[r] = my_as;
        asm volatile("bar.sync %0, 128;" ::"r"(6 + wg) : "memory");
#pragma unroll
        for (int c0 = 0; c0 < HB; c0 += C::kRound) {
          float v[C::kRound];
#pragma unroll
          for (int q = 0; q < C::kRound; ++q) v[q] = R[c0 + q];
          put(un, c0, v);
        }
      } else {
        const int slot = k % C::kSlots;
        if (r < HB) as[r] = my_as;
        asm volatile("bar.sync %0, 128;" ::"r"(6 + wg) : "memory");
        // Both issuers' accumulators, the one whose last group comes first first:
        // it is the one the next tile begins with, whose MMAs wait for its
        // columns to be read but for nothing that is done with them (a tile of
        // one group has one accumulator, its issuer's).
        constexpr int kRounds = HB / C::kRound;
        const int last = ((k + 1) * G - 1) & 1;
        float v[kRounds][C::kRound];
#pragma unroll
        for (int c = 0; c < kRounds; ++c)
#pragma unroll
          for (int q = 0; q < C::kRound; ++q) v[c][q] = 0.f;
        for (int n = G < 2 ? 1 : 0; n < 2; ++n) {
          const int q = n ? last : last ^ 1;
          if (ok)
            ok = mbar_wait(dfull(slot * 2 + q), (G < 2 ? k / 2 : k / C::kSlots) & 1, abort_flag, tmo);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + lane_base + slot * 128 + q * BT + col0;
#pragma unroll
          for (int c = 0; c < kRounds; ++c) {
            uint32_t u[C::kRound / 16][16];
#pragma unroll
            for (int b = 0; b < C::kRound / 16; ++b) tmem_ld16(d + c * C::kRound + b * 16, u[b]);
            tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < C::kRound; ++b) v[c][b] += __uint_as_float(u[b / 16][b % 16]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(dempty(k % 4 * 2 + q));
            if (G < 2) mbar_arrive(dempty(k % 4 * 2 + (q ^ 1)));
          }
        }
#pragma unroll
        for (int c = 0; c < kRounds; ++c) put(un, c * C::kRound, v[c]);
      }
    }
    __syncwarp();
    teardown();
  };
  if (warp == C::kRecWarp) rec_role();
  else if (warp == C::kRowWarp) row_role();
  else if (warp >= C::kMmaWarp) mma_role();
  else if (warp >= C::kConvWarp0) conv_role();
  else drain_role();
}

template <int BT, bool GATE_UP, bool EXACT>
static cudaError_t launch_ragged_bt(const RaggedArgs& a, cudaStream_t st) {
  using C = RgCfg<BT, EXACT>;
  CUtensorMap map;
  if (!make_act_map_3d(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.act, a.rows_max, a.K, BT))
    return cudaErrorInvalidValue;
  RgParams p;
  p.a_s = a.a_s;
  p.packed = a.packed;
  p.y = a.y;
  p.offset = a.plan.offset;
  p.sets = a.E;
  p.n_tiles = (int)(a.N / 128);
  p.G = (int)(a.K / 128);
  p.timeout_ns = a.timeout_ns;
  // units at most (the device counts them): as many CTAs as SMs, or fewer
  const int64_t most = plan_max_tiles(a.rows_max, a.E, BT) * p.n_tiles;
  const int sms = device_sm_count();
  if (sms < 1) return cudaErrorInvalidConfiguration;
  if (most >= (1LL << 31) || (most / sms + 1) * p.G >= (1LL << 31)) return cudaErrorNotSupported;
  auto kern = ragged_kernel<BT, GATE_UP, EXACT>;
  static SmemOptIn opt_in;
  if (cudaError_t e = opt_in.ensure(kern, C::kSmem); e != cudaSuccess) return e;
  PdlConfig c(dim3((unsigned)(most < sms ? most : sms), 1, 1), C::kThreads, C::kSmem, st);
  return cudaLaunchKernelEx(&c.cfg, kern, map, p);
}

// The exact gate and up products of many rows: the linears' kernel in its ragged
// mode (192 rows, every group's sum exact).
static cudaError_t launch_exact_wide(const RaggedArgs& a, cudaStream_t st) {
  using C = TcCfg<kW4A8, kFullBT>;
  constexpr size_t kSmem = C::kSmemBytes + (kTcMaxSets + 4) * sizeof(int);
  static_assert(kSmem <= kMaxSmem, "shared memory of the ragged products");
  CUtensorMap act_map, none;
  memset(&none, 0, sizeof(none));
  YMaps ymaps;
  memset(&ymaps, 0, sizeof(ymaps));
  if (!make_act_map_3d(&act_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.act, a.rows_max, a.K, kFullBT))
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
  p.seg.y[0] = static_cast<uint16_t*>(a.y);
  p.seg.N[0] = a.N;
  p.set_offset = a.plan.offset;
  p.sets = a.E;
  const int64_t most = plan_max_tiles(a.rows_max, a.E, kFullBT) * p.n_tiles;
  const int sms = device_sm_count();
  if (sms < 1) return cudaErrorInvalidConfiguration;
  if (most >= (1LL << 31) || (most / sms + 1) * p.G >= (1LL << 31)) return cudaErrorNotSupported;
  auto kern = tc_gemm_kernel<kW4A8, kFullBT, false, kTcGateUp>;
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
  if (a.gate_up && a.exact)
    return a.wide ? launch_exact_wide(a, st) : launch_ragged_bt<64, true, true>(a, st);
  if (a.gate_up)
    return a.wide ? launch_ragged_bt<128, true, false>(a, st)
                  : launch_ragged_bt<64, true, false>(a, st);
  return a.wide ? launch_ragged_bt<128, false, false>(a, st)
                : launch_ragged_bt<64, false, false>(a, st);
}

cudaError_t take_error_word_tc_experts(unsigned* out) { return take_local_error_word(out); }
cudaError_t set_record_limit_tc_experts(unsigned long long bytes) {
  return set_local_record_limit(bytes);
}

}  // namespace egopq
