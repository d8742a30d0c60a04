// Routing to experts, and the plan of the experts' rows.
//
// Routing: scores s = softmax(x) or 1 / (1 + exp(-x)) of a token's E logits, choices c = s + bias, of which the k largest
// are taken in falling order, ties to the lowest expert; with groups, first the top_group groups of experts by their
// largest choice or the sum of their two largest. Weights are the chosen experts' s, divided by their sum on request.
//
// Choices are those of 64-bit scores. Without a bias the logits are in the same order as the scores, and they are compared
// as they are. With one, a warp orders fp32 choices and looks at the gaps that decide: where one is within what fp32 can be
// off, it forms the choices that can be concerned in 64 bits, a lane for each (one token in a hundred needs that, but with
// all 256 experts in 64 bits that token alone took 13 us of the call's 28: this GPU has little 64-bit arithmetic). Two
// experts of the same logit and bias are equal in either, so that bf16 logits' ties stay in fp32; where they stand on both sides of the
// last gap, the one behind all of them is what it is measured to.
//
// One warp per token, logits and choices in registers. Bound by the instructions: up to 256 experts a lane sorts its own (a
// network of 19 exchanges for eight) and a choice takes the largest of the lanes' heads by the warp's integer reduction, on
// keys in the order of the values.
// Plan: a stable counting sort. A warp holds up to 256 consecutive pairs and ranks those of one expert among 32 by ballots over
// the ids' bits; counts go to the warp's own counters, and the sums over warps (and the eight CTAs of a cluster, through
// their shared memory) give each pair its place. Bound by latency: loads, two turns of shared memory, two cluster barriers.
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
  int magic;      // e / per_group = e * magic >> 20, for e < 1024
  int row_bytes;  // shared memory of a warp: E times keys of 64-bit choices, logits, fp32 choices, a list
};

// Keys in the order of the values (-0 as 0).
__device__ __forceinline__ uint32_t key_of(float v) {
  const int b = __float_as_int(v + 0.f);
  return (uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k ^ ((uint32_t)((int)~k >> 31) | 0x80000000u)); }
constexpr uint32_t kNone = 0x007FFFFFu;  // the key of -inf

// A lane's choices, largest first, equal ones by the lower expert. Up to eight are sorted once by exchanges of neighbours, which
// keep equal keys in their order, and then move up; more of them are looked through for each choice (at 16 sorting
// would take 120 exchanges).
template <int N>
struct Lane {
  static constexpr bool kSorted = N <= 8;
  uint32_t key[N];
  int at[kSorted ? N : 1];

  __device__ __forceinline__ void ready() {
    if constexpr (kSorted) {
#pragma unroll
      for (int i = 0; i < N; ++i) at[i] = i;
#pragma unroll
      for (int r = 0; r < N; ++r) {
#pragma unroll
        for (int i = r & 1; i + 1 < N; i += 2) {
          const bool swap = key[i + 1] > key[i];
          const uint32_t k = key[i];
          const int a = at[i];
          key[i] = swap ? key[i + 1] : k, key[i + 1] = swap ? k : key[i + 1];
          at[i] = swap ? at[i + 1] : a, at[i + 1] = swap ? a : at[i + 1];
        }
      }
    }
  }
  __device__ __forceinline__ void head(uint32_t& k, int& i) const {
    if constexpr (kSorted) {
      k = key[0], i = at[0];
    } else {
      k = key[0];
#pragma unroll
      for (int n = 1; n < N; ++n) k = max(k, key[n]);
      i = 0;
#pragma unroll
      for (int n = N - 1; n >= 0; --n) i = key[n] == k ? n : i;
    }
  }
  __device__ __forceinline__ void pop(int i) {
    if constexpr (kSorted) {
#pragma unroll
      for (int n = 0; n + 1 < N; ++n) key[n] = key[n + 1], at[n] = at[n + 1];
      key[N - 1] = kNone;
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n) key[n] = n == i ? kNone : key[n];
    }
  }
};

// 64-bit values are compared as whole numbers in their order: this GPU's 64-bit unit takes 32 cycles for a warp.
constexpr long long kLeast = (long long)0x8000000000000000ull;  // -inf
__device__ __forceinline__ long long key64_of(double v) {
  const long long b = __double_as_longlong(v + 0.0);
  return v > -(double)INFINITY ? b ^ ((b >> 63) & 0x7FFFFFFFFFFFFFFFll) : kLeast;
}
__device__ __forceinline__ double of_key64(long long k) { return __longlong_as_double(k ^ ((k >> 63) & 0x7FFFFFFFFFFFFFFFll)); }

__device__ __forceinline__ float least(float) { return -INFINITY; }
__device__ __forceinline__ long long least(long long) { return kLeast; }
__device__ __forceinline__ float plus(float a, float b) { return fmaxf(a + b, -FLT_MAX); }  // -inf stands for none
__device__ __forceinline__ long long plus(long long a, long long b) { return key64_of(of_key64(a) + of_key64(b)); }

// What a choice formed from fast fp32 scores can be off by: __expf is within (2 + 1.2 |d|) 2^-23 of its value e^-|d|, so
// within 2.5 * 2^-23; the sum of up to 1024 of them (32 of a lane, 5 levels) within 21 * 2^-23 of itself, the division, the
// product and the addition of the bias two roundings each: under 32 * 2^-23 for s <= 1, and a rounding of |c|.
__device__ __forceinline__ float off_by(float c) { return 3.8146973e-6f * (1.f + 0.5f * fabsf(c)); }

// The groups that stay, as a mask. choice: E values (float, or keys of 64-bit ones), the least where an expert cannot be
// chosen. sure: NULL, or cleared where the border is too narrow for fp32; *edge is then what the lane's group (lane / lanes of a
// group) scores by at least: its second largest choice or its largest.
template <typename V>
__device__ unsigned keep_groups(const V* choice, int G, int keep, int per_group, bool two, bool* sure, V* edge) {
  const int lane = threadIdx.x & 31;
  int lanes = 32;
  while (lanes * G > 32) lanes /= 2;  // lanes of a group
  const int mine = lane / lanes;
  const V none = least(V());
  V a = none, b = none;
  if (mine < G) {
#pragma unroll 1
    for (int i = lane % lanes; i < per_group; i += lanes) {
      const V c = choice[mine * per_group + i], lo = a < c ? a : c;
      a = a > c ? a : c;
      b = b > lo ? b : lo;
    }
  }
#pragma unroll 1
  for (int d = 1; d < lanes; d *= 2) {
    const V a2 = __shfl_xor_sync(kAll, a, d), b2 = __shfl_xor_sync(kAll, b, d);
    const V lo = a < a2 ? a : a2;
    b = b > b2 ? b : b2;
    b = b > lo ? b : lo;
    a = a > a2 ? a : a2;
  }
  const V score = two && b != none ? plus(a, b) : a;
  if (edge) *edge = two && b != none ? b : a;
  // lane g now takes group g
  const V s = __shfl_sync(kAll, score, (lane < G ? lane : 0) * lanes);
  int before = 0;
#pragma unroll 1
  for (int g = 0; g < G; ++g) {
    const V o = __shfl_sync(kAll, s, g);
    before += o > s || (o == s && g < lane);
  }
  const unsigned kept = __ballot_sync(kAll, lane < G && before < keep);
  if constexpr (sizeof(V) == 4) {
    if (sure) {
      // a sum is off by what its two choices are, which can be far larger than it is
      const float o = __shfl_sync(kAll, off_by(a) + (two && b != none ? off_by(b) : 0.f), (lane < G ? lane : 0) * lanes);
      const bool in = lane < G && (kept >> lane & 1);
      const float off = fabsf(s) < INFINITY ? o : 0.f;
      const float low = of_key(__reduce_min_sync(kAll, key_of(in ? s - off : INFINITY)));
      const float high = of_key(__reduce_max_sync(kAll, key_of(lane < G && !in ? s + off : -INFINITY)));
      if (low <= high && high > -INFINITY) *sure = false;
    }
  }
  return kept;
}

// The 64-bit choices of the experts whose fp32 one is within reach of `edge` (of lane (group * lanes)'s edge where lanes > 0), as
// keys; the others' are the fp32 ones, which decide nothing. All lanes take part. Out of line, as most tokens pass by.
__device__ __noinline__ void exact_choices(const RouteParams& p, long long* keys, float top, float edge, int lanes) {
  const MoeRouteArgs& a = p.a;
  const float* xs = reinterpret_cast<const float*>(keys + a.E);
  const float* cs = xs + a.E;
  int* list = reinterpret_cast<int*>(keys + 2 * a.E);
  const int lane = threadIdx.x % 32;
  int n = 0;
  for (int b = 0; b < a.E; b += 32) {
    const int e = b + lane;
    const float at = __shfl_sync(kAll, edge, lanes && e < a.E ? (e * p.magic >> 20) * lanes : 0);
    const float f = e < a.E ? cs[e] : -INFINITY;
    const bool in = f > -INFINITY && f >= at - 2.f * off_by(at);
    if (e < a.E) keys[e] = key64_of((double)f);
    const unsigned ins = __ballot_sync(kAll, in);
    if (in) list[n + __popc(ins & ((1u << lane) - 1))] = e;
    n += __popc(ins);
  }
  double per_z = 1.0;
  if (a.softmax) {
    double z = 0.0;
    for (int e = lane; e < a.E; e += 32) z += exp((double)xs[e] - (double)top);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) z += __shfl_xor_sync(kAll, z, d);
    per_z = 1.0 / z;
  }
  __syncwarp();
  for (int j = lane; j < n; j += 32) {
    const int e = list[j];
    const double v = xs[e];
    double s = exp(a.softmax ? v - (double)top : -fabs(v)) * per_z;
    if (!a.softmax) {  // u / (1 + u) or 1 / (1 + u) of u = exp(-|v|) <= 1: a reciprocal in [1/2, 1] by two Newton steps
      const double y = 1.0 + s;
      double r = (double)__frcp_rn((float)y);
      r = fma(r, fma(-y, r, 1.0), r);
      r = fma(r, fma(-y, r, 1.0), r);
      s = v < 0.0 ? s * r : r;
    }
    keys[e] = key64_of(s + (a.bias ? (double)a.bias[e] : 0.0));
  }
  __syncwarp();
}

// The largest fp32 choice up to expert id's that is not its equal by logit and bias. All lanes take part; out of line, as few tokens
// have equals at the border.
__device__ __noinline__ float next_other(const float* xs, const float* cs, const float* bias, int E, int id) {
  const float x = xs[id], b = bias[id], c = cs[id];
  float most = -INFINITY;
  for (int e = threadIdx.x % 32; e < E; e += 32) {
    const float f = cs[e];
    if (f <= c && !(xs[e] == x && bias[e] == b)) most = fmaxf(most, f);
  }
  return of_key(__reduce_max_sync(kAll, key_of(most)));
}

// Lane j gets the expert of the j-th largest key, -1 where there is none; the keys are used up.
__device__ __noinline__ int largest_keys(long long* keys, int E, int k) {
  const int lane = threadIdx.x % 32;
  int id = -1;
  for (int j = 0; j < k; ++j) {
    long long m = kLeast;
    int best = E;
#pragma unroll 4
    for (int e = lane; e < E; e += 32)
      if (keys[e] > m) m = keys[e], best = e;
    const int hi = __reduce_max_sync(kAll, (int)(m >> 32));
    const unsigned lo = __reduce_max_sync(kAll, (int)(m >> 32) == hi ? (unsigned)m : 0u);
    const bool mine = (int)(m >> 32) == hi && (unsigned)m == lo;
    best = (int)__reduce_min_sync(kAll, mine ? (unsigned)best : kAll);
    if (best == E) break;
    if (lane == j) id = best;
    if (lane == (best & 31)) keys[best] = kLeast;
    __syncwarp();
  }
  return id;
}

template <typename X, int VPL>
__global__ void __launch_bounds__(kRouteWarps * 32, VPL <= 8 ? 8 : 1) moe_route_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const MoeRouteArgs& a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  long long* keys = reinterpret_cast<long long*>(smem + warp * p.row_bytes);
  float* xs = reinterpret_cast<float*>(keys + a.E);
  float* cs = xs + a.E;
  const long long t = (long long)blockIdx.x * kRouteWarps + warp;
  grid_launch_dependents();
  grid_dependency_wait();
  if (t >= a.T) return;

  float x[VPL], b[VPL];  // of expert 32 i + lane: logit, and bias, asked for together
  const X* row = static_cast<const X*>(a.x) + t * a.xs + lane;
  uint32_t most = kNone;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    float v = -INFINITY;
    if (32 * i + lane < a.E) {
      if constexpr (sizeof(X) == 4) v = row[32 * i];
      else v = __uint_as_float((uint32_t)row[32 * i] << 16);
    }
    x[i] = v;
    b[i] = a.bias && 32 * i + lane < a.E ? a.bias[32 * i + lane] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    x[i] = x[i] == x[i] ? fminf(x[i], FLT_MAX) : -INFINITY;  // NaN: not to be chosen; +inf: the largest
    if (32 * i + lane < a.E) xs[32 * i + lane] = x[i];
    most = max(most, key_of(x[i]));
  }
  const float top = of_key(__reduce_max_sync(kAll, most));
  __syncwarp();

  const bool by_score = a.bias || (a.n_group > 1 && a.two);  // else logits are in the scores' order
  float sum = 0.f;
  if (a.softmax && (by_score || !a.renorm) && top > -INFINITY) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) sum += expf(x[i] - top);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(kAll, sum, d);
  }

  // c: what is compared; an expert that can be chosen has a logit, and a bias that is not -inf or NaN
  Lane<VPL> c;
  if (by_score) {
    const float rest = a.softmax ? __fdividef(1.f, sum) : 1.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = 32 * i + lane;
      const float s = a.softmax ? __expf(x[i] - top) * rest : __fdividef(1.f, 1.f + __expf(-x[i]));
      float f = -INFINITY;
      if (e < a.E) {
        f = x[i] > -INFINITY ? s + b[i] : -INFINITY;
        f = f > -INFINITY ? f : -INFINITY;  // NaN
        cs[e] = f;
      }
      c.key[i] = key_of(f);
    }
    __syncwarp();
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) c.key[i] = key_of(x[i]);
  }
  if (a.n_group > 1) {
    bool sure = true;
    float edge = -INFINITY;
    unsigned groups = keep_groups<float>(by_score ? cs : xs, a.n_group, a.top_group, p.per_group, a.two, by_score ? &sure : nullptr, &edge);
    if (!sure) {
      int lanes = 32;
      while (lanes * a.n_group > 32) lanes /= 2;
      exact_choices(p, keys, top, edge, lanes);
      groups = keep_groups<long long>(keys, a.n_group, a.top_group, p.per_group, a.two, nullptr, nullptr);
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const bool in = groups >> ((32 * i + lane) * p.magic >> 20 & 31) & 1;
      if (!a.bias) c.key[i] = key_of(x[i]);
      else if (!in && 32 * i + lane < a.E) cs[32 * i + lane] = -INFINITY;
      if (!in) c.key[i] = kNone;
    }
  }

  int id = -1;  // lane j holds choice j and its key; with a bias one more is taken, for the last gap
  uint32_t mine = kNone, next = kNone;
  int next_e = 0;
  c.ready();
  const int rounds = a.bias ? min(a.k + 1, a.E) : a.k;
  for (int j = 0; j < rounds; ++j) {
    uint32_t k;
    int i;
    c.head(k, i);
    const uint32_t key = __reduce_max_sync(kAll, k);
    if (key == kNone) break;
    const int e = (int)__reduce_min_sync(kAll, k == key ? (unsigned)(32 * i + lane) : kAll);
    if (j == a.k) next = key, next_e = e;
    else if (lane == j) id = e, mine = key;
    if (lane == (e & 31)) c.pop(i);
  }
  bool sure = true;
  uint32_t last = kNone;  // the last choice's key
  if (a.bias) {
    const uint32_t k = __shfl_down_sync(kAll, mine, 1);
    const int e = __shfl_down_sync(kAll, id, 1);
    last = __reduce_min_sync(kAll, id >= 0 ? mine : kAll);
    if (lane < a.k - 1) next = k, next_e = e;
    const float f = of_key(mine);
    float g = of_key(next);
    const bool gap = id >= 0 && lane < a.k && next != kNone;
    bool equal = gap && xs[id] == xs[next_e] && a.bias[id] == a.bias[next_e];
    // equals on both sides of the border: what decides is whether one behind them can be larger than they are
    if (__shfl_sync(kAll, equal, a.k - 1)) {
      __syncwarp();
      const float o = next_other(xs, cs, a.bias, a.E, __shfl_sync(kAll, id, a.k - 1));
      if (lane == a.k - 1) g = o, equal = o == -INFINITY;
    }
    sure = !__any_sync(kAll, gap && !equal && f - g <= 2.f * off_by(f));
  }
  if (!sure) {  // a.bias: again from the exact choices down to the last one's reach
    __syncwarp();
    exact_choices(p, keys, top, of_key(last), 0);
    id = largest_keys(keys, a.E, a.k);
  }

  const float v = id >= 0 ? xs[id] : -INFINITY;
  float w = 0.f;
  if (a.softmax && a.renorm) {  // softmax over the chosen: no sum over all experts to underflow against
    const float most = of_key(__reduce_max_sync(kAll, key_of(v)));
    if (id >= 0) w = expf(v - most);
  } else if (id >= 0) {
    w = a.softmax ? expf(v - top) / sum : 1.f / (1.f + expf(-v));
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
constexpr int kHold = 8;  // pairs of a lane at a time

struct PlanParams {
  const int* ids;
  int n, E;
  int bits;     // of an id, and of E, which stands for none
  int segment;  // pairs of a warp, a multiple of 32
  int warps;    // warps of a CTA that have pairs
  int ctas;
  int *offsets, *order;
};

// The next 32 * kHold pairs of a warp from b on: their ids (E: none), and for each the lanes that have the same one.
__device__ __forceinline__ void take_pairs(const PlanParams& p, long long b, long long end, int (&id)[kHold], unsigned (&same)[kHold]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const long long q = b + 32 * i + lane;
    id[i] = q < end ? p.ids[q] : -1;
  }
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    if ((unsigned)id[i] >= (unsigned)p.E) id[i] = p.E;
    same[i] = kAll;
  }
  for (int bit = 0; bit < p.bits; ++bit) {
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const bool set = id[i] >> bit & 1;
      const unsigned v = __ballot_sync(kAll, set);
      same[i] &= set ? v : ~v;
    }
  }
}

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

  // pairs [p0, p1) are this warp's
  const long long p0 = ((long long)rank * p.warps + warp) * p.segment;
  const long long p1 = warp < p.warps ? min(p0 + p.segment, (long long)p.n) : p0;
  int* mine = counts + warp * p.E;
  const unsigned below = (1u << lane) - 1;
  int id[kHold];
  unsigned same[kHold];
  if (p0 < p1) take_pairs(p, p0, p1, id, same);
  __syncthreads();
  for (long long b = p0; b < p1; b += 32 * kHold) {
    if (b > p0) take_pairs(p, b, p1, id, same);
#pragma unroll
    for (int i = 0; i < kHold; ++i)  // additions of whole numbers: their order does not matter
      if (id[i] < p.E && !(same[i] & below)) atomicAdd(mine + id[i], __popc(same[i]));
  }
  __syncthreads();
  int all = 0, before = 0;
  if (tid < p.E) {  // E <= threads
    int run = 0;
#pragma unroll 8
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
      int c[kPlanCluster];
#pragma unroll
      for (int r = 0; r < kPlanCluster; ++r) c[r] = cluster.map_shared_rank(total, r)[tid];
      all = 0;
#pragma unroll
      for (int r = 0; r < kPlanCluster; ++r) {
        before += r < rank ? c[r] : 0;
        all += c[r];
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
  for (long long b = p0; b < p1; b += 32 * kHold) {
    if (p.segment > 32 * kHold) take_pairs(p, b, p1, id, same);
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      int place = 0;  // of the first lane with this id, which holds the counter's turn
      const bool first = !(same[i] & below);
      if (id[i] < p.E && first) {
        place = total[id[i]] + mine[id[i]];
        mine[id[i]] += __popc(same[i]);
      }
      place = __shfl_sync(kAll, place, __ffs(same[i]) - 1) + __popc(same[i] & below);
      if (id[i] < p.E) p.order[place] = (int)(b + 32 * i + lane);
      __syncwarp();
    }
  }
  for (long long i = (long long)live + rank * (kPlanWarps * 32) + tid; i < p.n; i += p.ctas * (kPlanWarps * 32)) p.order[i] = -1;
}

template <typename X, int VPL>
int launch_route(const RouteParams& p, cudaStream_t s, std::string* err) {
  static SmemAllowed allowed;
  if (allow_smem(allowed, moe_route_kernel<X, VPL>, (size_t)kRouteWarps * 20 * 32 * VPL, "moe_route", err)) return -1;
  const unsigned grid = (unsigned)((p.a.T + kRouteWarps - 1) / kRouteWarps);
  return launch_pdl(moe_route_kernel<X, VPL>, dim3(grid), dim3(kRouteWarps * 32), (size_t)kRouteWarps * p.row_bytes, s, p, "moe_route", err);
}
template <typename X>
int launch_route_of(const RouteParams& p, cudaStream_t s, std::string* err) {
  const int n = (p.a.E + 31) / 32;
  if (n <= 1) return launch_route<X, 1>(p, s, err);
  if (n <= 2) return launch_route<X, 2>(p, s, err);
  if (n <= 4) return launch_route<X, 4>(p, s, err);
  if (n <= 8) return launch_route<X, 8>(p, s, err);
  if (n <= 16) return launch_route<X, 16>(p, s, err);
  return launch_route<X, 32>(p, s, err);
}

}  // namespace

int launch_moe_route(const MoeRouteArgs& a, cudaStream_t s, std::string* err) {
  RouteParams p;
  p.a = a;
  p.per_group = a.E / a.n_group;
  p.row_bytes = 20 * ((a.E + 1) / 2 * 2);
  p.magic = (1 << 20) / p.per_group + 1;  // off by less than e / 2^20 < 1 / per_group
  return a.x_dtype == KQ_F32 ? launch_route_of<float>(p, s, err) : launch_route_of<uint16_t>(p, s, err);
}

int launch_moe_plan(const int* ids, long long n, int E, int* offsets, int* order, cudaStream_t s, std::string* err) {
  PlanParams p;
  p.ids = ids;
  p.n = (int)n;
  p.E = E;
  p.bits = 32 - __builtin_clz(E);
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
