// route.cu -- the router of a mixture of experts, and the plan that sorts the
// rows of a batch by the weight set each picks (an expert, an adapter).
//
// Router (egopq_moe_route), per token t over E experts:
//   s_e = exp(l_e - max) / sum exp, or 1 / (1 + exp(-l_e))
//   c_e = s_e + bias_e                      (the choice, not the weight)
//   group score = max of c, or the sum of its two largest, over a group's
//   experts; only the topk_group best groups' experts may be chosen
//   ids = the k largest c, w_j = s[ids_j] (/ (sum + 1e-20)) * scale
// Ties go to the lowest index everywhere. All arithmetic is fp32.
#include "egopq_internal.h"

namespace egopq {

// ---- router ------------------------------------------------------------------
// One warp a token; lane l holds the V experts from V l, so that the lowest lane
// of a tie has its lowest expert. Choices are compared as unsigned keys that
// keep the order of the floats (0: not to be chosen; 1: masked off by its logit,
// behind every number, whatever the bias). A group whose experts are
// whole lanes, a power of two of them, is scored by exchanges inside its lanes,
// others by one lane a group out of shared memory. A lane sorts its keys once,
// so that a pick is a maximum over the lanes and a shift (without the sort, a
// search of every lane's V keys a pick: 19.3 us where this took 17.1). The
// weights are formed last, for the picks alone. Bound by the instructions a
// token takes, about a thousand: 16384 tokens of 256 experts in 8 groups, 8
// picks, move 18 MB in 17.5 us (1.0 TB/s); one token takes 2 us.
constexpr int kRouteWarps = 4;
constexpr uint32_t kMaskedKey = 1;  // (the lowest number's, -inf's, is 0x007FFFFF)

__device__ __forceinline__ uint32_t order_key(float c) {
  const uint32_t u = __float_as_uint(c + 0.f);  // (-0 + 0 = +0: they tie)
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}

struct RouteParams {
  const void* logits;
  const float* bias;
  float* weights;
  int32_t* ids;
  int64_t T;
  int E, k, n_group, topk_group, per_group;
  int group_lanes;  // lanes of a group, a power of two; 0: groups are not whole lanes
  int bf16, vec, sigmoid, top2, renorm;
  float scale;
};

// A logit as a finite number or -inf (an expert masked off): NaN reads as -inf
// and +inf as the largest finite value.
__device__ __forceinline__ float clean_logit(float l) {
  return l != l ? -INFINITY : fminf(l, 3.402823466e38f);
}
__device__ __forceinline__ float sigmoid_rn(float l) { return __frcp_rn(1.f + expf(-l)); }

// A lane's keys, largest first (Batcher's merge exchange).
template <int V>
__device__ __forceinline__ void sort_down(uint32_t (&v)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2) {
#pragma unroll
    for (int k = p; k >= 1; k /= 2) {
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k) {
#pragma unroll
        for (int i = 0; i < k; ++i) {
          const int a = i + j, b = a + k;
          if (b < V && a / (2 * p) == b / (2 * p)) {
            const uint32_t hi = max(v[a], v[b]);
            v[b] = min(v[a], v[b]);
            v[a] = hi;
          }
        }
      }
    }
  }
}

template <int V>
__global__ void __launch_bounds__(32 * kRouteWarps)
route_kernel(const RouteParams p) {
  __shared__ uint32_t group_keys[kRouteWarps][V == 1 ? 32 : 32 * V];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (t >= p.T) return;
  const int e0 = lane * V;
  const float* row32 = static_cast<const float*>(p.logits) + t * p.E;
  const uint16_t* row16 = static_cast<const uint16_t*>(p.logits) + t * p.E;
  float s[V];
  bool loaded = false;
  if constexpr (V % 4 == 0) {
    // whole 16-byte (fp32) or 8-byte (bf16) vectors: E a multiple of 4
    if (p.vec) {
      loaded = true;
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (e0 + i < p.E) {
          if (p.bf16) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(row16 + e0 + i));
            v = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                            __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
          } else {
            v = __ldg(reinterpret_cast<const float4*>(row32 + e0 + i));
          }
        }
        s[i] = v.x;
        s[i + 1] = v.y;
        s[i + 2] = v.z;
        s[i + 3] = v.w;
      }
    }
  }
  if (!loaded) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = -INFINITY;
      if (e0 + i < p.E) s[i] = p.bf16 ? bf16_bits_to_f32(__ldg(row16 + e0 + i)) : __ldg(row32 + e0 + i);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = clean_logit(s[i]);
  uint32_t live = 0;  // bit i: expert e0 + i is there and not masked off
#pragma unroll
  for (int i = 0; i < V; ++i) live |= (s[i] > -INFINITY ? 1u : 0u) << i;
  float mx = 0.f, inv_sum = 1.f;
  // the softmax without a bias chooses by the logits, whose order it keeps
  // (groups by their two best: by the scores, which are added)
  const bool by_score = p.bias || p.top2;
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = sigmoid_rn(s[i]);
  } else {
    mx = s[0];
#pragma unroll
    for (int i = 1; i < V; ++i) mx = fmaxf(mx, s[i]);
    mx = key_value(__reduce_max_sync(0xffffffffu, order_key(mx)));
    if (mx == -INFINITY) mx = 0.f;  // every expert masked off: scores of zero
    float sum = 0.f, ex[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ex[i] = expf(s[i] - mx);
      sum += ex[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    inv_sum = sum > 0.f ? __fdiv_rn(1.f, sum) : 0.f;
    if (by_score) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = ex[i] * inv_sum;
    }
  }
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = 0;
    if (e0 + i < p.E) {
      float c = s[i];
      if (p.bias) {
        c += __ldg(p.bias + e0 + i);
        if (c != c) c = -INFINITY;  // a NaN choice ranks last
      }
      key[i] = (live >> i) & 1 ? order_key(c) : kMaskedKey;
    }
  }
  if (p.topk_group < p.n_group) {
    // a group's score from its largest key and, for the two best, the second
    // (where there is one that is not masked off)
    auto score_of = [&](uint32_t m1, uint32_t m2) {
      return p.top2 && m2 > kMaskedKey ? order_key(key_value(m1) + key_value(m2)) : m1;
    };
    uint32_t m1 = 0, m2 = 0;
    if (p.group_lanes) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        m2 = max(m2, min(m1, key[i]));
        m1 = max(m1, key[i]);
      }
      for (int o = 1; o < p.group_lanes; o <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(0xffffffffu, m1, o);
        const uint32_t o2 = __shfl_xor_sync(0xffffffffu, m2, o);
        m2 = max(max(m2, o2), min(m1, o1));
        m1 = max(m1, o1);
      }
      const uint32_t mine = score_of(m1, m2);
      // my group is kept if fewer than topk_group groups are better (or as good
      // and lower)
      const int g = lane / p.group_lanes;
      int better = 0;
      for (int q = 0; q < p.n_group; ++q) {
        const uint32_t other = __shfl_sync(0xffffffffu, mine, q * p.group_lanes);
        better += other > mine || (other == mine && q < g);
      }
      if (better >= p.topk_group) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = 0;
      }
    } else {
      uint32_t* keys = group_keys[warp];
#pragma unroll
      for (int i = 0; i < V; ++i) keys[e0 + i] = key[i];
      __syncwarp();
      uint32_t mine = 0;  // lane g: group g's score
      if (lane < p.n_group) {
        for (int i = 0; i < p.per_group; ++i) {
          const uint32_t kk = keys[lane * p.per_group + i];
          m2 = max(m2, min(m1, kk));
          m1 = max(m1, kk);
        }
        mine = score_of(m1, m2);
      }
      int better = 0;
      for (int q = 0; q < p.n_group; ++q) {
        const uint32_t other = __shfl_sync(0xffffffffu, mine, q);
        better += other > mine || (other == mine && q < lane);
      }
      const uint32_t keep =
          __ballot_sync(0xffffffffu, lane < p.n_group && better < p.topk_group);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i < p.E && !((keep >> ((e0 + i) / p.per_group)) & 1)) key[i] = 0;
    }
  }
  // k times the best of the lanes' best; lane j remembers pick j's key and lane
  // (and, of equal keys in a row out of one lane, which of them it is)
  uint32_t best[V];
#pragma unroll
  for (int i = 0; i < V; ++i) best[i] = key[i];
  sort_down<V>(best);
  uint32_t my_key = 0, last = 0;
  int my_lane = 0, my_nth = 0, from = -1, nth = 0;
  for (int j = 0; j < p.k; ++j) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, best[0]);
    const int who = __ffs(__ballot_sync(0xffffffffu, best[0] == top)) - 1;
    nth = top == last && who == from ? nth + 1 : 0;
    last = top;
    from = who;
    if (lane == j) {
      my_key = top;
      my_lane = who;
      my_nth = nth;
    }
    if (lane == who) {
#pragma unroll
      for (int i = 0; i + 1 < V; ++i) best[i] = best[i + 1];
      best[V - 1] = 0;
    }
  }
  uint32_t equal = 0;  // the picked lane's experts of that key
#pragma unroll
  for (int i = 0; i < V; ++i)
    equal |= (__shfl_sync(0xffffffffu, key[i], my_lane) == my_key ? 1u : 0u) << i;
  for (; my_nth > 0; --my_nth) equal &= equal - 1;
  const int my_id = lane < p.k ? my_lane * V + __ffs(equal) - 1 : 0;
  float w = 0.f;
  if (lane < p.k) {
    const float l = clean_logit(p.bf16 ? bf16_bits_to_f32(__ldg(row16 + my_id)) : __ldg(row32 + my_id));
    w = p.sigmoid ? sigmoid_rn(l) : expf(l - mx) * inv_sum;
  }
  if (p.renorm) {
    float sum = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = __fdiv_rn(w, sum + 1e-20f);
  }
  if (lane < p.k) {
    p.weights[t * p.k + lane] = w * p.scale;
    p.ids[t * p.k + lane] = my_id;
  }
}

template <int V>
static cudaError_t launch_route_v(RouteParams p, cudaStream_t st) {
  const int lanes = p.per_group % V ? 0 : p.per_group / V;
  p.group_lanes = lanes && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  PdlConfig c(dim3((unsigned)((p.T + kRouteWarps - 1) / kRouteWarps), 1, 1), 32 * kRouteWarps, 0,
              st);
  return cudaLaunchKernelEx(&c.cfg, route_kernel<V>, p);
}

cudaError_t launch_route(const RouteArgs& a, cudaStream_t st) {
  RouteParams p;
  p.logits = a.logits;
  p.bias = a.bias;
  p.weights = a.weights;
  p.ids = a.ids;
  p.T = a.T;
  p.E = a.E;
  p.k = a.k;
  p.n_group = a.n_group;
  p.topk_group = a.topk_group;
  p.per_group = a.E / a.n_group;
  p.group_lanes = 0;
  p.bf16 = a.bf16;
  p.vec = a.E % 4 == 0;
  p.sigmoid = a.sigmoid;
  p.top2 = a.top2;
  p.renorm = a.renorm;
  p.scale = a.scale;
  if (a.E <= 32) return launch_route_v<1>(p, st);
  if (a.E <= 64) return launch_route_v<2>(p, st);
  if (a.E <= 128) return launch_route_v<4>(p, st);
  // (five experts a lane: 160 in 8 groups of 20 are then four whole lanes a group.
  // Five / eight a lane, 16384 tokens: 160 experts in 8 groups 12.1 / 20.4 us, in
  // 4 11.8 / 21.3, in one 9.9 / 12.6, 140 in 4 17.0 / 21.3; one token of 160 in 8
  // groups 2.6 / 4.0)
  if (a.E <= 160 && p.per_group % 5 == 0) return launch_route_v<5>(p, st);
  if (a.E <= 256) return launch_route_v<8>(p, st);
  return launch_route_v<16>(p, st);
}

// ---- plan ----------------------------------------------------------------------
// One CTA a weight set, and one more for the rows that pick none. Each CTA
// reads all n picks (out of L2), so it knows its own first sorted position --
// the picks of lower sets -- and the number of non-empty lower sets without
// hearing from another CTA, and the whole plan is one launch. A thread holds
// PT consecutive picks in registers, so one scan over the threads keeps the
// slots of a set in order; more than PT * 1024 picks go in rounds. Bound by that
// scan and its barriers: 264 picks of 64 sets take 4 us, 32768 take 10 (with the
// picks read again for the second pass, 55).
constexpr int kPlanThreads = 1024;

template <int PT>
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const int32_t* __restrict__ ids, int n, int S, int bt, RowPlan plan, bool early) {
  if (!early) griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  __shared__ uint32_t seen[kMaxSets / 32];  // bit s: set s has a row
  __shared__ int warp_eq[32], warp_lt[32];
  const int set = blockIdx.x;  // S: the rows without a set
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nthr = blockDim.x, nwarp = nthr >> 5;
  if (bt) {
    for (int i = tid; i < kMaxSets / 32; i += nthr) seen[i] = 0;
    __syncthreads();
  }
  int v[PT];
  const bool vec = (reinterpret_cast<uintptr_t>(ids) & 15) == 0;  // (a slice's need not be)
  // picks [i0, i0 + PT) as set numbers; past the end: S + 1
  auto load = [&](int64_t i0) {
#pragma unroll
    for (int q = 0; q < PT; q += 4) {
      int4 u = make_int4(S + 1, S + 1, S + 1, S + 1);
      const int64_t i = i0 + q;
      if (vec && i + 3 < n) {
        u = __ldcg(reinterpret_cast<const int4*>(ids + i));
      } else if (i < n) {
        u.x = __ldcg(ids + i);
        if (i + 1 < n) u.y = __ldcg(ids + i + 1);
        if (i + 2 < n) u.z = __ldcg(ids + i + 2);
        if (i + 3 < n) u.w = __ldcg(ids + i + 3);
      }
      v[q] = u.x;
      v[q + 1] = u.y;
      v[q + 2] = u.z;
      v[q + 3] = u.w;
    }
#pragma unroll
    for (int q = 0; q < PT; ++q) {
      if (i0 + q >= n) v[q] = S + 1;
      else if (v[q] < 0 || v[q] >= S) v[q] = S;
    }
  };
  const int64_t round = (int64_t)nthr * PT;
  int eq = 0, lt = 0, mine = 0;
  for (int64_t c0 = 0; c0 < n; c0 += round) {
    load(c0 + (int64_t)tid * PT);
    mine = 0;
    int last = -1;
#pragma unroll
    for (int q = 0; q < PT; ++q) {
      mine += v[q] == set;
      lt += v[q] < set;
      if (bt && v[q] < S && v[q] != last) {
        last = v[q];
        const uint32_t bit = 1u << (last & 31);
        if (!(*(volatile uint32_t*)&seen[last >> 5] & bit)) atomicOr(&seen[last >> 5], bit);
      }
    }
    eq += mine;
  }
  const int all_eq = __reduce_add_sync(0xffffffffu, eq);
  lt = __reduce_add_sync(0xffffffffu, lt);
  if (lane == 0) {
    warp_eq[warp] = all_eq;
    warp_lt[warp] = lt;
  }
  __syncthreads();
  // totals, and (one round) the slots of the warps before this one
  int count = warp_eq[lane < nwarp ? lane : 0], base = warp_lt[lane < nwarp ? lane : 0];
  if (lane >= nwarp) count = base = 0;
  int before = lane < warp ? count : 0;
  count = __reduce_add_sync(0xffffffffu, count);
  base = __reduce_add_sync(0xffffffffu, base);
  before = __reduce_add_sync(0xffffffffu, before);
  // the slots in order: the thread's come after those of the threads before it
  auto write = [&](int64_t i0, int at) {
#pragma unroll
    for (int q = 0; q < PT; ++q) {
      if (v[q] == set) {
        plan.order[at] = (int)(i0 + q);
        if (plan.pos) plan.pos[i0 + q] = set < S ? at : -1;
        ++at;
      }
    }
  };
  auto lanes_before = [&](int m) {
    int incl = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    return incl - m;
  };
  if (n <= round) {
    if (all_eq) write((int64_t)tid * PT, base + before + lanes_before(mine));
  } else {
    int done = 0;
    for (int64_t c0 = 0; c0 < n && done < count; c0 += round) {
      load(c0 + (int64_t)tid * PT);
      mine = 0;
#pragma unroll
      for (int q = 0; q < PT; ++q) mine += v[q] == set;
      const int in_warp = __reduce_add_sync(0xffffffffu, mine);
      __syncthreads();
      if (lane == 0) warp_eq[warp] = in_warp;
      __syncthreads();
      int sum = lane < nwarp ? warp_eq[lane] : 0;
      const int below = __reduce_add_sync(0xffffffffu, lane < warp ? sum : 0);
      sum = __reduce_add_sync(0xffffffffu, sum);
      if (in_warp) write(c0 + (int64_t)tid * PT, base + done + below + lanes_before(mine));
      done += sum;
    }
  }
  if (tid == 0) {
    plan.offset[set] = base;
    if (set == S) plan.head[0] = base;  // rows that have a set
  }
  if (early) griddep_wait();  // (a grid's end follows that of the one before)
  if (!bt) return;
  // tiles of at most bt rows: set s takes the entries from base / bt + rank up
  // to the next set's first, (base + count) / bt + rank + 1: as many as it
  // needs, or one more, which is then empty (rank: non-empty sets below)
  int rank = 0;
  for (int w = 0; w < (set + 31) / 32; ++w) {
    uint32_t m = seen[w];
    if (w == set / 32) m &= (1u << (set & 31)) - 1;
    rank += __popc(m);
  }
  if (set < S) {
    if (count > 0) {
      const int t0 = base / bt + rank, t1 = (base + count) / bt + rank + 1;
      for (int t = t0 + tid; t < t1; t += nthr) {
        const int r0 = (t - t0) * bt;
        const int rows = max(0, min(bt, count - r0));
        plan.tiles[t] = make_int4(set, base + r0, rows, 0);
      }
    }
  } else if (tid == 0) {
    plan.head[1] = base / bt + rank;  // entries of the tile table
  }
}

cudaError_t launch_plan(const int32_t* ids, int64_t n, int S, int bt, const RowPlan& plan,
                        cudaStream_t st, bool early) {
  // four picks a thread while that fits one round, else 32
  const bool small = n <= 4 * kPlanThreads;
  const int64_t want = small ? (n + 3) / 4 : kPlanThreads;
  PdlConfig c(dim3((unsigned)(S + 1), 1, 1), (unsigned)((want + 31) / 32 * 32), 0, st);
  return small ? cudaLaunchKernelEx(&c.cfg, plan_kernel<4>, ids, (int)n, S, bt, plan, early)
               : cudaLaunchKernelEx(&c.cfg, plan_kernel<32>, ids, (int)n, S, bt, plan, early);
}

}  // namespace egopq
