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
// One warp a token; expert e lives in lane e % 32, register e / 32. Choices
// are compared as unsigned keys that keep the order of the floats (0: not to
// be chosen), so one redux.sync finds a maximum and a second one the lowest
// index that has it.
constexpr int kRouteWarps = 4;

__device__ __forceinline__ uint32_t order_key(float c) {
  if (c != c) c = -INFINITY;                  // a NaN choice ranks last
  const uint32_t u = __float_as_uint(c + 0.f);  // (-0 + 0 = +0: they tie)
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k);
}

struct RouteParams {
  const void* logits;
  const float* bias;
  float* weights;
  int32_t* ids;
  int64_t T;
  int E, k, n_group, topk_group, per_group;
  int bf16, sigmoid, top2, renorm;
  float scale;
};

template <int V>  // registers a lane: E <= 32 * V
__global__ void __launch_bounds__(32 * kRouteWarps)
route_kernel(const RouteParams p) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (t >= p.T) return;
  float s[V];
  // logits as finite numbers or -inf (an expert masked off): NaN reads as
  // -inf and +inf as the largest finite value
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 32 + lane;
    float l = -INFINITY;
    if (e < p.E) {
      l = p.bf16 ? bf16_bits_to_f32(__ldg(static_cast<const uint16_t*>(p.logits) + t * p.E + e))
                 : __ldg(static_cast<const float*>(p.logits) + t * p.E + e);
      if (l != l) l = -INFINITY;
      l = fminf(l, 3.402823466e38f);
    }
    s[i] = l;
  }
  uint32_t key[V];
  float inv_sum = 1.f, mx = 0.f;
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = __fdiv_rn(1.f, 1.f + expf(-s[i]));
  } else {
    // the softmax keeps its logits until the weights are formed: without a
    // bias they are the choice (the softmax keeps their order)
    mx = s[0];
#pragma unroll
    for (int i = 1; i < V; ++i) mx = fmaxf(mx, s[i]);
    mx = key_value(__reduce_max_sync(0xffffffffu, order_key(mx)));
    if (mx == -INFINITY) mx = 0.f;  // every expert masked off: scores of zero
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += expf(s[i] - mx);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    inv_sum = sum > 0.f ? __fdiv_rn(1.f, sum) : 0.f;
    if (p.bias || p.top2) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = expf(s[i] - mx) * inv_sum;
    }
  }
  const bool by_logit = !p.sigmoid && !(p.bias || p.top2);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 32 + lane;
    key[i] = 0;
    if (e < p.E) key[i] = order_key(p.bias ? s[i] + __ldg(p.bias + e) : s[i]);
  }
  if (p.topk_group < p.n_group) {
    // lane g gets group g's score
    uint32_t gkey = 0;
    for (int g = 0; g < p.n_group; ++g) {
      const int lo = g * p.per_group, hi = lo + p.per_group;
      uint32_t m1 = 0, m2 = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        const uint32_t kk = (e >= lo && e < hi) ? key[i] : 0u;
        m2 = max(m2, min(m1, kk));
        m1 = max(m1, kk);
      }
      const uint32_t best = __reduce_max_sync(0xffffffffu, m1);
      uint32_t gk = best;
      if (p.top2) {
        // the second best: of the best's first holder its own second, of the
        // other lanes their first
        const int holder = __ffs(__ballot_sync(0xffffffffu, m1 == best)) - 1;
        const uint32_t second = __reduce_max_sync(0xffffffffu, lane == holder ? m2 : m1);
        const float sum = second ? key_value(best) + key_value(second) : key_value(best);
        gk = order_key(sum);
      }
      if (lane == g) gkey = gk;
    }
    uint32_t keep = 0;
    for (int j = 0; j < p.topk_group; ++j) {
      const uint32_t best = __reduce_max_sync(0xffffffffu, gkey);
      const int g = __ffs(__ballot_sync(0xffffffffu, gkey == best)) - 1;
      keep |= 1u << g;
      if (lane == g) gkey = 0;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      if (e < p.E && !((keep >> (e / p.per_group)) & 1)) key[i] = 0;
    }
  }
  float my_w = 0.f;
  int my_id = 0;
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = key[0];
    int bi = 0;
    float bs = s[0];
#pragma unroll
    for (int i = 1; i < V; ++i) {
      if (key[i] > best) {
        best = key[i];
        bi = i;
        bs = s[i];
      }
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const unsigned e = best == top ? (unsigned)(bi * 32 + lane) : 0xffffffffu;
    const unsigned win = __reduce_min_sync(0xffffffffu, e);
    const float ws = __shfl_sync(0xffffffffu, bs, win & 31);
    if (lane == j) {
      my_w = ws;
      my_id = (int)win;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((unsigned)(i * 32 + lane) == win) key[i] = 0;
  }
  if (by_logit && lane < p.k) my_w = expf(my_w - mx) * inv_sum;
  if (p.renorm) {
    float sum = lane < p.k ? my_w : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    my_w = __fdiv_rn(my_w, sum + 1e-20f);
  }
  if (lane < p.k) {
    p.weights[t * p.k + lane] = my_w * p.scale;
    p.ids[t * p.k + lane] = my_id;
  }
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
  p.bf16 = a.bf16;
  p.sigmoid = a.sigmoid;
  p.top2 = a.top2;
  p.renorm = a.renorm;
  p.scale = a.scale;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.T + kRouteWarps - 1) / kRouteWarps), 1, 1);
  cfg.blockDim = dim3(32 * kRouteWarps, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.E <= 64) return cudaLaunchKernelEx(&cfg, route_kernel<2>, p);
  if (a.E <= 128) return cudaLaunchKernelEx(&cfg, route_kernel<4>, p);
  if (a.E <= 256) return cudaLaunchKernelEx(&cfg, route_kernel<8>, p);
  return cudaLaunchKernelEx(&cfg, route_kernel<16>, p);
}

// ---- plan ----------------------------------------------------------------------
// One CTA a weight set, and one more for the rows that pick none. Each CTA
// reads all n picks (out of L2), so it knows its own first sorted position --
// the picks of lower sets -- and the number of non-empty lower sets without
// hearing from another CTA, and the whole plan is one launch. A thread holds
// PT consecutive picks in registers, so one scan over the threads keeps the
// slots of a set in order; more than PT * 1024 picks go in rounds.
constexpr int kPlanThreads = 1024;

template <int PT>
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const int32_t* __restrict__ ids, int n, int S, int bt, RowPlan plan) {
  griddep_wait();
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
  // picks [i0, i0 + PT) as set numbers; past the end: S + 1
  auto load = [&](int64_t i0) {
#pragma unroll
    for (int q = 0; q < PT; q += 4) {
      int4 u = make_int4(S + 1, S + 1, S + 1, S + 1);
      const int64_t i = i0 + q;
      if (i + 3 < n) {
        u = __ldg(reinterpret_cast<const int4*>(ids + i));
      } else if (i < n) {
        u.x = __ldg(ids + i);
        if (i + 1 < n) u.y = __ldg(ids + i + 1);
        if (i + 2 < n) u.z = __ldg(ids + i + 2);
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
                        cudaStream_t st) {
  // four picks a thread while that fits one round, else 32
  const bool small = n <= 4 * kPlanThreads;
  const int64_t want = small ? (n + 3) / 4 : kPlanThreads;
  PdlConfig c(dim3((unsigned)(S + 1), 1, 1), (unsigned)((want + 31) / 32 * 32), 0, st);
  return small ? cudaLaunchKernelEx(&c.cfg, plan_kernel<4>, ids, (int)n, S, bt, plan)
               : cudaLaunchKernelEx(&c.cfg, plan_kernel<32>, ids, (int)n, S, bt, plan);
}

}  // namespace egopq
