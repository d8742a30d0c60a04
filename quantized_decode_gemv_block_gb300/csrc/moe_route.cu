// Routing to experts, and the plan of the experts' rows.
//
// Routing: scores s = softmax(x) or 1 / (1 + exp(-x)) of a token's E logits, choices c = s + bias, of which the k largest
// are taken in falling order, ties to the lowest expert; with groups, first the top_group groups of experts by their
// largest choice or the sum of their two largest. Weights are the chosen experts' s, divided by their sum on request.
//
// Choices are those of 64-bit scores. Without a bias the logits are in the same order as the scores, and they are compared
// as they are. With one, a warp orders fp32 choices and looks at the gaps that decide: where one is within what fp32 can be
// off, it does the token again in 64 bits (a few tokens in a thousand; all others need no 64-bit arithmetic, of which this
// GPU has little). Two experts of the same logit and bias are equal in either, so that bf16 logits' ties stay in fp32.
//
// One warp per token, logits and choices in registers, the maxima by the warp's integer reduction on keys in the order of
// the values. Plan: a stable counting sort; a warp takes its consecutive pairs 32 at a time and ranks those of one expert
// among them by a match, once to count and once to place, with the sums over warps (and up to eight CTAs of a
// cluster, through their shared memory) between.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <cfloat>
#include <cstdint>

#include "kq.h"
#include "kq_device.cuh"
#include "kq_internal.h"
#include "kq_launch.cuh"

namespace cg = cooperative_groups;

namespace kq {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kRouteWarps = 4;

struct RouteParams {
  MoeRouteArgs a;
  int per_group;  // experts of a group
  int row_bytes;  // shared memory of a warp: E logits, E choices in 64 bits
};

// Keys in the order of the values.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k); }

template <typename V>
__device__ __forceinline__ V low() { return -(V)INFINITY; }

// What fp32 scores and choices can be off by, with room: s is within a dozen roundings of 2^-24 (s |ln s| <= 0.37 covers
// the difference of logits), and adding the bias rounds once more.
__device__ __forceinline__ float off_by(float c) { return 1.9073486e-6f * (2.f + fabsf(c)); }

// The groups that stay, as a mask. choice: E values, -inf where an expert cannot be chosen. sure: cleared where the border
// is too narrow for fp32 (V = float, `exact` false).
template <typename V>
__device__ unsigned keep_groups(const V* choice, int G, int keep, int per_group, bool two, bool exact, bool* sure) {
  const int lane = threadIdx.x & 31;
  int lanes = 32;
  while (lanes * G > 32) lanes /= 2;  // lanes of a group
  const int mine = lane / lanes;
  V a = low<V>(), b = low<V>();
  if (mine < G) {
    for (int i = lane % lanes; i < per_group; i += lanes) {
      const V c = choice[mine * per_group + i];
      if (c > a) b = a, a = c;
      else if (c > b) b = c;
    }
  }
  for (int d = 1; d < lanes; d *= 2) {
    const V a2 = __shfl_xor_sync(kAll, a, d), b2 = __shfl_xor_sync(kAll, b, d);
    const V lo = a < a2 ? a : a2;
    b = b > b2 ? b : b2;
    b = b > lo ? b : lo;
    a = a > a2 ? a : a2;
  }
  const V score = two && b != low<V>() ? a + b : a;
  // lane g now takes group g
  const V s = __shfl_sync(kAll, score, (lane < G ? lane : 0) * lanes);
  int before = 0;
  for (int g = 0; g < G; ++g) {
    const V o = __shfl_sync(kAll, s, g);
    before += o > s || (o == s && g < lane);
  }
  const unsigned kept = __ballot_sync(kAll, lane < G && before < keep);
  if (!exact) {
    const float in = lane < G && (kept >> lane & 1) ? (float)s : INFINITY, out = lane < G && !(kept >> lane & 1) ? (float)s : -INFINITY;
    const float least = of_key(__reduce_min_sync(kAll, key_of(in))), most = of_key(__reduce_max_sync(kAll, key_of(out)));
    if (least - most <= 2.f * off_by(least)) *sure = false;
  }
  return kept;
}

template <int VPL>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_kernel(const RouteParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const MoeRouteArgs& a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  double* wide = reinterpret_cast<double*>(smem + warp * p.row_bytes);
  float* xs = reinterpret_cast<float*>(wide + a.E);
  const long long t = (long long)blockIdx.x * kRouteWarps + warp;
  grid_launch_dependents();
  grid_dependency_wait();
  if (t >= a.T) return;

  float x[VPL], c[VPL];  // expert 32 i + lane
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = 32 * i + lane;
    float v = -INFINITY;
    if (e < a.E) {
      v = a.x_dtype == KQ_F32 ? static_cast<const float*>(a.x)[t * a.xs + e]
                              : __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.x)[t * a.xs + e] << 16);
      v = v == v ? fminf(v, FLT_MAX) : -INFINITY;  // NaN: not to be chosen; +inf: the largest
      xs[e] = v;
    }
    x[i] = v;
    top = fmaxf(top, v);
  }
  top = of_key(__reduce_max_sync(kAll, key_of(top)));
  __syncwarp();

  const bool by_score = a.bias || (a.n_group > 1 && a.two);  // else logits are in the scores' order
  float sum = 0.f;
  if (a.softmax && (by_score || !a.renorm) && top > -INFINITY) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) sum += x[i] > -INFINITY ? expf(x[i] - top) : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(kAll, sum, d);
  }
  auto score = [&](float v) { return v == -INFINITY ? 0.f : a.softmax ? expf(v - top) / sum : 1.f / (1.f + expf(-v)); };
  auto bias = [&](int e) { return a.bias ? a.bias[e] : 0.f; };
  // an expert that can be chosen has a logit, and a bias that is not -inf or NaN
  auto choice_of = [&](float v, int e) {
    const float s = score(v) + bias(e);
    return v == -INFINITY || !(s > -INFINITY) ? -INFINITY : s;
  };

  // c: what is compared
  bool sure = true;
  unsigned groups = kAll;
#pragma unroll
  for (int i = 0; i < VPL; ++i) c[i] = by_score && 32 * i + lane < a.E ? choice_of(x[i], 32 * i + lane) : x[i];
  if (a.n_group > 1) {
    float* cs = reinterpret_cast<float*>(wide);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (32 * i + lane < a.E) cs[32 * i + lane] = c[i];
    __syncwarp();
    groups = keep_groups<float>(cs, a.n_group, a.top_group, p.per_group, a.two, !by_score, &sure);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = 32 * i + lane;
      if (e < a.E && !(groups >> e / p.per_group & 1)) c[i] = x[i] = -INFINITY;
      else if (!a.bias) c[i] = x[i];
    }
  }

  int id = -1;  // lane j holds choice j
  if (sure) {
    float last = INFINITY;
    int last_e = 0;
    const int rounds = a.bias ? min(a.k + 1, a.E) : a.k;  // one more, for the last gap
    for (int j = 0; j < rounds; ++j) {
      float m = c[0];
      int e = lane;
#pragma unroll
      for (int i = 1; i < VPL; ++i)
        if (c[i] > m) m = c[i], e = 32 * i + lane;
      const uint32_t key = __reduce_max_sync(kAll, key_of(m));
      const float most = of_key(key);
      if (most == -INFINITY) break;
      e = (int)__reduce_min_sync(kAll, key_of(m) == key ? (unsigned)e : kAll);
      if (a.bias && j > 0 && last - most <= 2.f * off_by(last) && !(xs[last_e] == xs[e] && a.bias[last_e] == a.bias[e])) {
        sure = false;
        break;
      }
      if (lane == j) id = e;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (32 * i + lane == e) c[i] = -INFINITY;
      last = most;
      last_e = e;
    }
    if (a.bias && lane >= a.k) id = -1;
  }
  if (!sure) {  // again in 64 bits
    double z = 0.0;
    id = -1;
    if (a.softmax) {
      for (int e = lane; e < a.E; e += 32) z += xs[e] > -INFINITY ? exp((double)xs[e] - (double)top) : 0.0;
#pragma unroll
      for (int d = 16; d > 0; d /= 2) z += __shfl_xor_sync(kAll, z, d);
    }
    __syncwarp();
    for (int e = lane; e < a.E; e += 32) {
      const double v = xs[e], s = a.softmax ? exp(v - (double)top) / z : 1.0 / (1.0 + exp(-v));
      const double w = s + (double)bias(e);
      wide[e] = v == low<double>() || !(w > low<double>()) ? low<double>() : w;
    }
    __syncwarp();
    if (a.n_group > 1) {
      bool unused = true;
      groups = keep_groups<double>(wide, a.n_group, a.top_group, p.per_group, a.two, true, &unused);
      __syncwarp();
      for (int e = lane; e < a.E; e += 32) {
        if (!(groups >> e / p.per_group & 1)) wide[e] = low<double>();
        else if (!a.bias) wide[e] = xs[e];
      }
      __syncwarp();
    }
    for (int j = 0; j < a.k; ++j) {
      double m = low<double>();
      int best = a.E;
      for (int e = lane; e < a.E; e += 32)
        if (wide[e] > m) m = wide[e], best = e;
#pragma unroll
      for (int d = 16; d > 0; d /= 2) {
        const double m2 = __shfl_xor_sync(kAll, m, d);
        const int e2 = __shfl_xor_sync(kAll, best, d);
        if (m2 > m || (m2 == m && e2 < best)) m = m2, best = e2;
      }
      if (best == a.E) break;
      if (lane == j) id = best;
      if (lane == best % 32) wide[best] = low<double>();
      __syncwarp();
    }
  }

  const float v = id >= 0 ? xs[id] : -INFINITY;
  float w;
  if (a.softmax && a.renorm) {  // softmax over the chosen: no sum over all experts to underflow against
    const float most = of_key(__reduce_max_sync(kAll, key_of(v)));
    w = id >= 0 ? expf(v - most) : 0.f;
  } else {
    w = id >= 0 ? score(v) : 0.f;
  }
  if (a.renorm) {
    float s = w;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(kAll, s, d);
    w = s > 0.f ? w / s : 0.f;
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = id;
    a.weights[t * a.k + lane] = w * a.scale;
  }
}

// ---------------------------------------------------------------- plan

constexpr int kPlanWarps = 32;
constexpr int kPlanCluster = 8;

struct PlanParams {
  const int* ids;
  int n, E;
  int segment;  // pairs of a warp, a multiple of 32
  int warps;    // warps of a CTA that have pairs
  int ctas;
  int *offsets, *order;
};

__global__ void __launch_bounds__(kPlanWarps * 32) moe_plan_kernel(const PlanParams p) {
  extern __shared__ int counts[];  // [warps][E], then E totals
  __shared__ int sums[32];
  int* total = counts + p.warps * p.E;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, tid = threadIdx.x;
  int rank = 0;
  if (p.ctas > 1) rank = (int)cg::this_cluster().block_rank();
  for (int i = tid; i < p.warps * p.E; i += kPlanWarps * 32) counts[i] = 0;
  grid_launch_dependents();
  grid_dependency_wait();
  __syncthreads();

  // pairs [p0, p1) are this warp's
  const long long p0 = ((long long)rank * p.warps + warp) * p.segment;
  const long long p1 = warp < p.warps ? min(p0 + p.segment, (long long)p.n) : p0;
  int* mine = counts + warp * p.E;
  for (long long b = p0; b < p1; b += 32) {
    const int id = b + lane < p1 ? p.ids[b + lane] : -1;
    const unsigned same = __match_any_sync(kAll, id);
    if (id >= 0 && id < p.E && (same & ((1u << lane) - 1)) == 0) mine[id] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  int all = 0, before = 0;
  if (tid < p.E) {  // E <= threads
    int run = 0;
    for (int w = 0; w < p.warps; ++w) {
      const int c = counts[w * p.E + tid];
      counts[w * p.E + tid] = run;
      run += c;
    }
    total[tid] = run;
    all = run;
  }
  if (p.ctas > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (tid < p.E) {
      all = 0;
      for (int r = 0; r < p.ctas; ++r) {
        const int c = cluster.map_shared_rank(total, r)[tid];
        if (r < rank) before += c;
        all += c;
      }
    }
    cluster.sync();  // totals are read everywhere before they are overwritten
  }
  // exclusive sums over the experts
  int scan = all;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(kAll, scan, d);
    if (lane >= d) scan += o;
  }
  if (lane == 31) sums[warp] = scan;
  __syncthreads();
  if (warp == 0) {
    int s = sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int o = __shfl_up_sync(kAll, s, d);
      if (lane >= d) s += o;
    }
    sums[lane] = s;
  }
  __syncthreads();
  const int start = scan - all + (warp > 0 ? sums[warp - 1] : 0), live = sums[31];
  if (tid < p.E) {
    total[tid] = start + before;
    if (rank == 0) p.offsets[tid] = start;
  }
  if (rank == 0 && tid == 0) p.offsets[p.E] = live;
  __syncthreads();
  for (long long b = p0; b < p1; b += 32) {
    const int id = b + lane < p1 ? p.ids[b + lane] : -1;
    const unsigned same = __match_any_sync(kAll, id), lower = same & ((1u << lane) - 1);
    const bool ok = id >= 0 && id < p.E;
    if (ok) p.order[total[id] + mine[id] + __popc(lower)] = (int)(b + lane);
    __syncwarp();
    if (ok && lower == 0) mine[id] += __popc(same);
    __syncwarp();
  }
  for (long long i = (long long)live + rank * (kPlanWarps * 32) + tid; i < p.n; i += p.ctas * (kPlanWarps * 32)) p.order[i] = -1;
}

template <int VPL>
int launch_route(const RouteParams& p, cudaStream_t s, std::string* err) {
  static SmemAllowed allowed;
  if (allow_smem(allowed, moe_route_kernel<VPL>, (size_t)kRouteWarps * 12 * 32 * VPL, "moe_route", err)) return -1;
  const unsigned grid = (unsigned)((p.a.T + kRouteWarps - 1) / kRouteWarps);
  return launch_pdl(moe_route_kernel<VPL>, dim3(grid), dim3(kRouteWarps * 32), (size_t)kRouteWarps * p.row_bytes, s, p, "moe_route", err);
}

}  // namespace

int launch_moe_route(const MoeRouteArgs& a, cudaStream_t s, std::string* err) {
  RouteParams p;
  p.a = a;
  p.per_group = a.E / a.n_group;
  p.row_bytes = 12 * ((a.E + 1) / 2 * 2);
  const int vpl = (a.E + 31) / 32;
  if (vpl <= 1) return launch_route<1>(p, s, err);
  if (vpl <= 2) return launch_route<2>(p, s, err);
  if (vpl <= 4) return launch_route<4>(p, s, err);
  if (vpl <= 8) return launch_route<8>(p, s, err);
  if (vpl <= 16) return launch_route<16>(p, s, err);
  return launch_route<32>(p, s, err);
}

int launch_moe_plan(const int* ids, long long n, int E, int* offsets, int* order, cudaStream_t s, std::string* err) {
  PlanParams p;
  p.ids = ids;
  p.n = (int)n;
  p.E = E;
  p.offsets = offsets;
  p.order = order;
  // one CTA up to what its warps take in a few turns; a cluster's two barriers cost about a microsecond
  p.ctas = n > 4 * 32 * kPlanWarps ? kPlanCluster : 1;
  const long long warps = (n + 31) / 32;
  p.warps = (int)(warps < 1 ? 1 : warps < kPlanWarps ? warps : kPlanWarps);
  const long long each = (n + (long long)p.ctas * p.warps - 1) / ((long long)p.ctas * p.warps);
  p.segment = (int)((each + 31) / 32 * 32);
  const size_t smem = ((size_t)p.warps + 1) * E * 4;
  static SmemAllowed allowed;
  if (allow_smem(allowed, moe_plan_kernel, (size_t)(kPlanWarps + 1) * KQ_MOE_MAX_EXPERTS * 4, "moe_plan", err)) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(kPlanWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.ctas > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, moe_plan_kernel, p);
  if (e != cudaSuccess) {
    *err = std::string("moe_plan launch: ") + cudaGetErrorString(e);
    return -1;
  }
  return 0;
}

}  // namespace kq
