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
// reads all n picks (out of L2, once: in registers up to 32 a thread), so it
// knows its own first sorted position -- the picks of lower sets -- and the
// number of non-empty lower sets without hearing from another CTA, and the
// whole plan is one launch. A thread holds consecutive picks, so a scan over
// the threads keeps the slots of a set in order.
constexpr int kPlanThreads = 1024;
constexpr int kPlanPerThread = 32;  // picks a thread holds at once

__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const int32_t* __restrict__ ids, int n, int S, int bt, RowPlan plan) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  __shared__ uint32_t seen[kMaxSets / 32];  // bit s: set s has a row
  __shared__ int warp_eq[32], warp_lt[32];
  const int set = blockIdx.x;  // S: the rows without a set
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nthr = blockDim.x, nwarp = nthr >> 5;
  for (int i = tid; i < kMaxSets / 32; i += nthr) seen[i] = 0;
  __syncthreads();
  const int chunk = nthr * kPlanPerThread;
  // pass 1 counts picks of this set and of lower ones
  auto set_of = [&](int i) { const int v = __ldg(ids + i); return (v < 0 || v >= S) ? S : v; };
  int eq = 0, lt = 0;
  for (int c0 = 0; c0 < n; c0 += chunk) {
    const int i0 = c0 + tid;
#pragma unroll 8
    for (int j = 0; j < kPlanPerThread; ++j) {
      const int i = i0 + j * nthr;
      if (i >= n) break;
      const int v = set_of(i);
      eq += v == set;
      lt += v < set;
      if (v < S) {
        const uint32_t bit = 1u << (v & 31);
        if (!(*(volatile uint32_t*)&seen[v >> 5] & bit)) atomicOr(&seen[v >> 5], bit);
      }
    }
  }
  eq = __reduce_add_sync(0xffffffffu, eq);
  lt = __reduce_add_sync(0xffffffffu, lt);
  if (lane == 0) {
    warp_eq[warp] = eq;
    warp_lt[warp] = lt;
  }
  __syncthreads();
  int count = 0, base = 0;
  for (int w = 0; w < nwarp; ++w) {
    count += warp_eq[w];
    base += warp_lt[w];
  }
  int rank = 0;  // non-empty sets below this one
  for (int w = 0; w < (set + 31) / 32; ++w) {
    uint32_t m = seen[w];
    if (w == set / 32) m &= (1u << (set & 31)) - 1;
    rank += __popc(m);
  }
  // pass 2 writes the slots in order, a chunk of consecutive picks a thread
  int done = 0;
  for (int c0 = 0; c0 < n && done < count; c0 += nthr) {
    const int i = c0 + tid;
    const bool mine = i < n && set_of(i) == set;
    const uint32_t b = __ballot_sync(0xffffffffu, mine);
    __syncthreads();
    if (lane == 0) warp_eq[warp] = __popc(b);
    __syncthreads();
    int before = done, total = 0;
    for (int w = 0; w < nwarp; ++w) {
      if (w < warp) before += warp_eq[w];
      total += warp_eq[w];
    }
    if (mine) {
      const int at = base + before + __popc(b & ((1u << lane) - 1));
      plan.order[at] = i;
      if (plan.pos) plan.pos[i] = set < S ? at : -1;
    }
    done += total;
  }
  // tiles of at most bt rows: set s takes the entries from base / bt + rank up
  // to the next set's first, (base + count) / bt + rank + 1: as many as it
  // needs, or one more, which is then empty
  if (tid == 0) plan.offset[set] = base;
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
    plan.head[0] = base;              // rows that have a set
    plan.head[1] = base / bt + rank;  // entries of the tile table
  }
}

cudaError_t launch_plan(const int32_t* ids, int64_t n, int S, int bt, const RowPlan& plan,
                        cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(S + 1), 1, 1);
  cfg.blockDim = dim3(n <= 256 ? 128 : (n <= 4096 ? 512 : kPlanThreads), 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_kernel, ids, (int)n, S, bt, plan);
}

}  // namespace egopq
