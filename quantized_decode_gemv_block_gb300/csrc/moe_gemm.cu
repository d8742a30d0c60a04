// Products of the experts' block-quantized matrices with the rows that were routed to them.
//
// Expert e of E has N x K weights W_e; the plan lists the pairs (token, choice) expert by expert. For each pair p,
//     kq_moe_gate_up:  act[p] = silu(g) * u,  [g u] = W_e x[token of p]          (N = 2 F rows: gate, then up)
//     kq_moe_down:     y[t] = add[t] + sum_j weight[t, j] * (W_e act[t k + j])   (join: the token's choices in order)
//
// moe_stream_kernel, the streaming product: an expert's rows in chunks of up to 16 tokens, its weights in tiles of 16 rows.
// All (chunk, tile) items of the call, chunk by chunk, are cut into equal ranges, one per cluster of C CTAs, so that few
// experts are spread over all SMs and many are walked through by each. A CTA stages a chunk's activations once (fp16 under
// an exact power of two per 256 values, or bf16), its warps take the range's tiles in turn and stream them through
// rings of tensor copies that run ahead across chunks; mma.sync multiplies 16 weight rows by 8 or 16 tokens. A tile's
// K is summed by one warp in order, K above 2560 in C parts added in order, so a pair's bits depend on its own row and expert
// only. Bound by the weights' bytes where an expert has few tokens.
#include <cooperative_groups.h>
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "gemv_formats.cuh"
#include "kq_device.cuh"
#include "kq_internal.h"
#include "kq_launch.cuh"
#include "moe.cuh"

namespace cg = cooperative_groups;

namespace kq {

__device__ unsigned int g_moe_errors = 0;  // bit 0: a bounded wait gave up; bit 1: a plan out of bounds

namespace {
using namespace gemv;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 256;           // weights per K-unit
constexpr int kMaxChunk = 16;        // tokens of a chunk
constexpr int kMaxSliceUnits = 10;   // K-units of activations a CTA stages
constexpr int kMaxCluster = 8;       // K up to 20480
constexpr int kMaxJoinTiles = 24;    // tiles whose parts meet across a cluster at a time
constexpr int kStreamSmem = kSmemCap - 512;  // of a CTA, beside its static memory
constexpr uint64_t kWaitLimitNs = 2000000000ull;

struct StreamParams {
  const uint8_t* w;
  const uint16_t* x;
  long long xs;       // elements between rows of x
  int div;            // pairs per row of x
  const int *offsets, *order;
  int E, P;           // experts, pairs
  int N, K, half;     // rows of an expert; half: F of a gate | up matrix, 0 otherwise
  float* y;           // half == 0: P x N
  uint16_t* act;      // half != 0: P x half
  long long row_bytes;
  int units, tiles, C, G;
  int chunk;          // tokens of a chunk at most
  int su, depth, row_stride, unit_bytes, xstride, xts, s2ts;
  int off_ss, off_aux, off_res, off_bar, off_start, off_ring;
};

// A chunk's activations for the fp16 staging: this thread's 32-value groups into registers (finish() converts and stores
// them), the row of zeros that absent tokens read, and their scales.
template <class F, class Row>
__device__ void load_rows(StageQ4KH<kThreads, F>& st, Row row, int M, int k0, int S, uint8_t* xh, int xts, uint8_t* s2, int s2ts,
                          float* iv) {
#pragma unroll
  for (int it = 0; it < StageQ4KH<kThreads, F>::kItems; ++it) {
    const int i = threadIdx.x + it * kThreads;
    if (i < M * S * 8) {
      const int tok = i / (S * 8), grp = i - tok * (S * 8);
      const uint16_t* src = row(tok) + (long long)k0 * kUnit + grp * 32;
#pragma unroll
      for (int v = 0; v < 4; ++v) st.u[it][v] = ldg128(src + 8 * v);
    }
  }
  for (int i = threadIdx.x; i < S * 32; i += kThreads) *reinterpret_cast<uint4*>(xh + M * xts + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
  for (int i = threadIdx.x; i < S * 4; i += kThreads) *reinterpret_cast<uint2*>(s2 + M * s2ts + 8 * i) = make_uint2(0u, 0u);
  for (int i = threadIdx.x; i < S * 16; i += kThreads)
    if ((i & 15) >= M) iv[i] = 0.f;
}

// bf16 activations of a chunk into shared memory in fragment order, and the fp32 sum of each 32 values (affine4).
template <class F, int T, class Row>
__device__ void stage_bf16(Row row, int M, int xstride, uint16_t* xs, float* ss, int k0, int S) {
  const int per_tok = S * 32;  // 16-byte vectors
  for (int i = threadIdx.x; i < M * per_tok; i += kThreads) {
    const int tok = i / per_tok, v = i - tok * per_tok;
    const uint4 o = ldg128(row(tok) + (long long)k0 * kUnit + v * 8);
    // (e0 e1 e2 e3) -> (e0 e2 e1 e3) within each group of four
    *reinterpret_cast<uint4*>(xs + tok * xstride + v * 8) =
        make_uint4(prmt(o.x, o.y, 0x5410u), prmt(o.x, o.y, 0x7632u), prmt(o.z, o.w, 0x5410u), prmt(o.z, o.w, 0x7632u));
  }
  for (int i = threadIdx.x; i < T * S * 8; i += kThreads) {
    const int grp = i / T, tok = i - grp * T;
    float s = 0.f;
    if (tok < M) {
      const uint16_t* src = row(tok) + (long long)k0 * kUnit + grp * 32;
      float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const uint4 u = ldg128(src + 8 * v);
        a[0] += bf16_lo(u.x); a[1] += bf16_hi(u.x); a[2] += bf16_lo(u.y); a[3] += bf16_hi(u.y);
        a[0] += bf16_lo(u.z); a[1] += bf16_hi(u.z); a[2] += bf16_lo(u.w); a[3] += bf16_hi(u.w);
      }
      s = (a[0] + a[1]) + (a[2] + a[3]);
    }
    ss[grp * T + tok] = s;
  }
}

// A stretch of a cluster's range: tiles [t0, t0 + nt) of one chunk.
struct Stretch {
  long long next;  // the range's first item behind it
  int e, chunk, t0, nt;
};

template <class F>
struct Stream {
  const StreamParams& p;
  const CUtensorMap* tmap;
  uint8_t* smem;
  const int* start;  // first chunk of each expert, E + 1
  int warp, lane, k0, S;
  long long i1;      // end of the cluster's range
  uint8_t* ring;
  uint64_t* bars;

  // The stretch that begins at item i (< i1), in expert e or a later one.
  __device__ Stretch stretch(long long i, int e) const {
    Stretch s;
    s.chunk = (int)(i / p.tiles);
    s.t0 = (int)(i - (long long)s.chunk * p.tiles);
    while (start[e + 1] <= s.chunk) ++e;
    s.e = e;
    long long n = min((long long)(p.tiles - s.t0), i1 - i);
    if (p.C > 1) n = min(n, (long long)kMaxJoinTiles);
    s.nt = (int)n;
    s.next = i + n;
    return s;
  }

  // Producer: the warp's stages in order, tiles warp, warp + 8, ... of each stretch.
  Stretch ps;
  int pj, pu;  // its tile in the stretch and unit
  __device__ bool more() const { return pj < ps.nt; }
  __device__ void settle() {  // on to the next stretch where this one has no tile left for the warp
    while (pj >= ps.nt && ps.next < i1) {
      ps = stretch(ps.next, ps.e);
      pj = warp;
    }
  }
  __device__ void issue(int slot) {
    const int nu = min(p.su, S - pu);
    uint8_t* dst = ring + (size_t)slot * 16 * p.row_stride;
    const long long row0 = (long long)ps.e * p.N;
    if constexpr (F::kRowCopies) {
      // one bulk copy per row: the 16-byte-aligned span over the row's units (the buffer ends on such a boundary)
      const int r = p.half ? (ps.t0 + pj) * 8 + (lane & 7) : (ps.t0 + pj) * 16 + lane;
      const bool in = lane < 16 && r < (p.half ? p.half : p.N);
      uint32_t bytes = 0;
      long long a0 = 0;
      if (in) {
        const long long a = (row0 + (p.half && lane >= 8 ? p.half + r : r)) * p.row_bytes + (long long)(k0 + pu) * F::kUnitBytes;
        a0 = a & ~15ll;
        bytes = (uint32_t)(((a + (long long)nu * F::kUnitBytes + 15) & ~15ll) - a0);
      }
      const uint32_t total = __reduce_add_sync(0xFFFFFFFFu, bytes);
      if (lane == 0) mbar_arrive_expect_tx(&bars[slot], total);
      __syncwarp();
      if (bytes) bulk_g2s(dst + (size_t)lane * p.row_stride, p.w + a0, bytes, &bars[slot]);
    } else if (lane == 0) {
      mbar_arrive_expect_tx(&bars[slot], 16u * (uint32_t)p.row_stride);
      const int col = (k0 + pu) * (p.unit_bytes / 4);
      if (p.half) {
        const int r = (int)row0 + (ps.t0 + pj) * 8;
        tma_load_2d(dst, tmap, col, r, &bars[slot]);
        tma_load_2d(dst + (size_t)8 * p.row_stride, tmap, col, r + p.half, &bars[slot]);
      } else {
        tma_load_2d(dst, tmap, col, (int)row0 + (ps.t0 + pj) * 16, &bars[slot]);
      }
    }
    pu += nu;
    if (pu == S) {
      pu = 0;
      pj += kWarps;
      settle();
    }
  }

  // Consumer.
  int slot = 0;
  uint32_t parity = 0;
  bool ok = true;

  template <int NT>
  __device__ void tiles_of(const Stretch& s, int M, const int* rows) {
    constexpr int T = 8 * NT;
    const int g = lane >> 2, q = lane & 3;
    float* res = reinterpret_cast<float*>(smem + p.off_res);
    int xo[NT], so[NT], io[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int tok = 8 * t + g, row = tok < M ? tok : M;
      if constexpr (F::kHalfX) {
        xo[t] = row * p.xts + F::kXq * q;
        so[t] = row * p.s2ts + 8 * q;
      } else {
        xo[t] = so[t] = 0;
      }
      io[t] = 8 * t + 2 * q;
    }
    for (int j = warp; j < s.nt; j += kWarps) {
      float acc[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
      const int tile = s.t0 + j;
      for (int u = 0; u < S;) {
        const int nu = min(p.su, S - u);
        if (ok && !mbar_wait_bounded(&bars[slot], parity, kWaitLimitNs)) {
          ok = false;
          if (lane == 0) atomicOr(&g_moe_errors, 1u);
        }
        ok = __all_sync(0xFFFFFFFFu, ok);  // the products and copies need every lane
        if (ok) {
          const uint8_t* sa = ring + ((size_t)slot * 16 + g) * p.row_stride;
          const uint8_t* sb = sa + (size_t)8 * p.row_stride;
          if constexpr (F::kRowCopies) {  // where each row's copy put the stage's first unit; modulo 2^32 keeps modulo 16
            const uint32_t u0 = (uint32_t)(k0 + u) * F::kUnitBytes, rb = (uint32_t)p.row_bytes;
            const uint32_t r0 = (uint32_t)s.e * (uint32_t)p.N + (uint32_t)(p.half ? tile * 8 : tile * 16) + g;
            sa += (r0 * rb + u0) & 15u;
            sb += ((r0 + (uint32_t)(p.half ? p.half : 8)) * rb + u0) & 15u;
          }
          for (int i = 0; i < nu; ++i) {
            typename F::Raw raw;
            F::template load<LdShared>(raw, sa + i * p.unit_bytes, sb + i * p.unit_bytes, q);
            if constexpr (F::kHalfX)
              F::template compute<NT>(raw, acc, smem + (u + i) * 512, xo, smem + p.off_ss + (u + i) * 32, so,
                                      reinterpret_cast<const float*>(smem + p.off_aux) + (u + i) * 16, io, lane);
            else
              F::template compute<NT>(raw, acc, reinterpret_cast<const uint16_t*>(smem) + (u + i) * kUnit, p.xstride,
                                      reinterpret_cast<const float*>(smem + p.off_ss) + (u + i) * 8 * T, lane, M);
          }
        }
        __syncwarp();
        u += nu;
        if (ok && more()) {
          fence_proxy_async_smem();
          issue(slot);
        }
        if (++slot == p.depth) slot = 0, parity ^= 1u;
      }
      if (p.C == 1) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          put(tile, g, 8 * t + 2 * q, M, rows, acc[t][0], acc[t][2]);
          put(tile, g, 8 * t + 2 * q + 1, M, rows, acc[t][1], acc[t][3]);
        }
      } else {
        float* r = res + (size_t)j * 16 * T;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int j0 = 8 * t + 2 * q;
          r[g * T + j0] = acc[t][0];
          r[g * T + j0 + 1] = acc[t][1];
          r[(g + 8) * T + j0] = acc[t][2];
          r[(g + 8) * T + j0 + 1] = acc[t][3];
        }
      }
    }
    if (p.C == 1) return;
    // the ranks' parts of the stretch's tiles, added in order; each rank takes its share of the (row pair, token)s
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const int total = s.nt * 8 * M, rank = (int)cluster.block_rank();
    for (int i = rank * kThreads + threadIdx.x; i < total; i += p.C * kThreads) {
      const int row = i & 7, tok = (i >> 3) % M, j = (i >> 3) / M;
      float a[kMaxCluster], b[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        const float* src = r < p.C ? cluster.map_shared_rank(res, r) + ((size_t)j * 16 + row) * T + tok : res;
        a[r] = r < p.C ? src[0] : 0.f;
        b[r] = r < p.C ? src[8 * T] : 0.f;
      }
      float va = 0.f, vb = 0.f;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < p.C) va += a[r], vb += b[r];
      put(s.t0 + j, row, tok, M, rows, va, vb);
    }
    cluster.sync();
  }

  // Results of rows g and g + 8 of a tile for a token of the chunk.
  __device__ void put(int tile, int g, int tok, int M, const int* rows, float a, float b) {
    if (tok >= M) return;
    const int pair = rows[tok];
    if (pair < 0) return;
    if (p.half) {
      const int i = tile * 8 + g;
      if (i < p.half) p.act[(long long)pair * p.half + i] = silu_mul(a, b);
    } else {
      const int n = tile * 16 + g;
      float* o = p.y + (long long)pair * p.N + n;
      if (n < p.N) o[0] = a;
      if (n + 8 < p.N) o[8] = b;
    }
  }
};

template <class F>
__global__ void __launch_bounds__(kThreads, 1) moe_stream_kernel(const __grid_constant__ CUtensorMap tmap, const StreamParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int rows[kMaxChunk], sums[kWarps + 1];
  int* start = reinterpret_cast<int*>(smem + p.off_start);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int rank = 0;
  if (p.C > 1) rank = (int)cg::this_cluster().block_rank();
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.off_bar) + warp * p.depth;
  if (lane == 0) {
    for (int s = 0; s < p.depth; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  grid_launch_dependents();
  grid_dependency_wait();

  // Chunks of the experts before each one. A plan out of bounds leaves its experts without any.
  constexpr int kPer = (KQ_MOE_MAX_EXPERTS + kThreads - 1) / kThreads;
  int n[kPer], mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    n[i] = 0;
    if (e < p.E) {
      const int a = p.offsets[e], b = p.offsets[e + 1];
      if (a < 0 || b < a || b > p.P) {
        if (rank == 0 && blockIdx.x == 0) atomicOr(&g_moe_errors, 2u);
      } else {
        n[i] = (b - a + p.chunk - 1) / p.chunk;
      }
    }
    mine += n[i];
  }
  int scan = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, scan, d);
    if (lane >= d) scan += o;
  }
  if (lane == 31) sums[warp] = scan;
  __syncthreads();
  int before = scan - mine, chunks = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sums[w];
    chunks += sums[w];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    if (e <= p.E) start[e] = before;
    before += n[i];
  }
  if (threadIdx.x == 0) start[p.E] = chunks;
  __syncthreads();

  const long long items = (long long)chunks * p.tiles;
  const int cid = blockIdx.x / p.C;
  const long long i0 = items * cid / p.G, i1 = items * (cid + 1) / p.G;
  if (i0 >= i1) return;  // the same for all of a cluster
  const int k0 = (int)((long long)rank * p.units / p.C), k1 = (int)((long long)(rank + 1) * p.units / p.C);

  // the first expert with chunk i0 / tiles
  int e0 = 0;
  {
    const int c = (int)(i0 / p.tiles);
    int hi = p.E;
    while (hi - e0 > 1) {
      const int mid = (e0 + hi) / 2;
      if (start[mid] <= c) e0 = mid;
      else hi = mid;
    }
  }
  Stream<F> st{p, &tmap, smem, start, warp, lane, k0, k1 - k0, i1, smem + p.off_ring + (size_t)warp * p.depth * 16 * p.row_stride, bars};
  Stretch s = st.stretch(i0, e0);
  st.ps = s;
  st.pj = warp;
  st.pu = 0;
  st.settle();
  int ahead = 0;
  for (; ahead < p.depth && st.more(); ++ahead) st.issue(ahead);

  int staged = -1;  // chunk whose activations are staged
  int M = 0;
  for (;;) {
    if (s.chunk != staged) {
      __syncthreads();  // every warp is done with the chunk before
      const int first = p.offsets[s.e] + (s.chunk - start[s.e]) * p.chunk;
      M = min(p.chunk, p.offsets[s.e + 1] - first);
      if (threadIdx.x < M) {
        int pair = p.order[first + threadIdx.x];
        if (pair < 0 || pair >= p.P) {
          atomicOr(&g_moe_errors, 2u);
          pair = -1;
        }
        rows[threadIdx.x] = pair;
      }
      __syncthreads();
      auto row = [&](int tok) { return p.x + (long long)(max(rows[tok], 0) / p.div) * p.xs; };
      if constexpr (F::kHalfX) {
        StageQ4KH<kThreads, F> stq;
        float* iv = reinterpret_cast<float*>(smem + p.off_aux);
        load_rows<F>(stq, row, M, k0, st.S, smem, p.xts, smem + p.off_ss, p.s2ts, iv);
        stq.finish(M, st.S, smem, p.xts, smem + p.off_ss, p.s2ts, iv);
      } else if (M <= 8) {
        stage_bf16<F, 8>(row, M, p.xstride, reinterpret_cast<uint16_t*>(smem), reinterpret_cast<float*>(smem + p.off_ss), k0, st.S);
      } else {
        stage_bf16<F, 16>(row, M, p.xstride, reinterpret_cast<uint16_t*>(smem), reinterpret_cast<float*>(smem + p.off_ss), k0, st.S);
      }
      __syncthreads();
      staged = s.chunk;
    }
    if (M <= 8) st.template tiles_of<1>(s, M, rows);
    else st.template tiles_of<2>(s, M, rows);
    if (s.next >= i1) break;
    s = st.stretch(s.next, s.e);
  }
  if (!st.ok) {  // let this warp's copies in flight land before the CTA can exit
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
}

// y[t] = add[t] + sum_j weight[t, j] * part[t k + j], j in order, choices without an expert left out. A part that a wait gave
// up on or a plan left out is what the workspace held.
struct JoinParams {
  const float *part, *weights, *add;
  const int* ids;
  void* y;
  long long add_stride, y_stride;
  int T, k, H, E, y_dtype;
};
template <int V>
__global__ void __launch_bounds__(256) moe_join_kernel(const JoinParams p) {
  grid_launch_dependents();
  grid_dependency_wait();
  const long long per = p.H / V, n = per * p.T;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    const long long t = i / per;
    const int h = (int)(i - t * per) * V;
    float s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = p.add ? p.add[t * p.add_stride + h + v] : 0.f;
    // eight choices at a time, all read without a condition so that the reads are in flight together (the rows are in the
    // workspace whatever they hold); a choice without an expert adds nothing
    for (int j0 = 0; j0 < p.k; j0 += 8) {
      float w[8], r[8][V];
      int id[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const long long pair = t * p.k + min(j0 + j, p.k - 1);
        id[j] = p.ids[pair];
        w[j] = p.weights[pair];
        const float* src = p.part + pair * p.H + h;
        if constexpr (V == 4) {
          const float4 a = __ldcs(reinterpret_cast<const float4*>(src));
          r[j][0] = a.x, r[j][1] = a.y, r[j][2] = a.z, r[j][3] = a.w;
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v) r[j][v] = src[v];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < p.k && id[j] >= 0 && id[j] < p.E) {
#pragma unroll
          for (int v = 0; v < V; ++v) s[v] = __fmaf_rn(w[j], r[j][v], s[v]);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (p.y_dtype == KQ_F32) static_cast<float*>(p.y)[t * p.y_stride + h + v] = s[v];
      else static_cast<uint16_t*>(p.y)[t * p.y_stride + h + v] = f32_to_bf16_rn(s[v]);
    }
  }
}

int unit_bytes_of(int fmt) {
  return fmt == FMT_Q4_K ? 144 : fmt == FMT_Q5_K ? 176 : fmt == FMT_Q6_K ? 210 : fmt == FMT_Q8_0 ? 272 : 160;
}

// Shared memory: staged activations, their sums, scales, the cluster's partial tiles, barriers, chunk starts, the rings.
bool stream_layout(int fmt, StreamParams* p, size_t* smem) {
  auto al = [](size_t v) { return (v + 127) & ~size_t(127); };
  const bool half_x = fmt != FMT_AFFINE4;
  const int S = (p->units + p->C - 1) / p->C, T = p->chunk > 8 ? 16 : 8, ub = unit_bytes_of(fmt);
  p->xts = p->s2ts = p->xstride = 0;
  size_t off;
  if (half_x) {  // the tokens' rows and one of zeros
    p->xts = S * 512 + 64;
    p->s2ts = 32 * (S | 1);
    p->off_ss = (int)al((size_t)(p->chunk + 1) * p->xts);
    off = al(p->off_ss + (size_t)(p->chunk + 1) * p->s2ts);
  } else {
    p->xstride = S * kUnit + 32;
    p->off_ss = (int)al((size_t)T * p->xstride * 2);
    off = al(p->off_ss + (size_t)S * 8 * T * 4);
  }
  p->off_aux = (int)off;
  off = al(off + (size_t)kMaxSliceUnits * 16 * 4);
  p->off_res = (int)off;
  if (p->C > 1) off = al(off + (size_t)kMaxJoinTiles * 16 * T * 4);
  p->off_bar = (int)off;
  off = al(off + kWarps * 8 * 8);
  p->off_start = (int)off;
  off = al(off + (size_t)(p->E + 1) * 4);
  p->off_ring = (int)off;
  for (int su = std::min(S, fmt == FMT_Q8_0 ? 2 : 4); su >= 1; --su) {
    int stride = fmt == FMT_Q6_K ? (su * ub + 30 + 15) / 16 * 16 : su * ub;  // + the span's alignment slack
    if (half_x && fmt != FMT_Q8_0) {  // 16-byte loads of a quad at 16 + 32q: rows differ by 16 mod 32 bytes
      while (stride % 32 != 16) stride += 16;
    } else {  // 8-byte loads of 4 rows a phase: rows differ by 32 or 96 mod 128
      while (stride % 128 != 32 && stride % 128 != 96) stride += 16;
    }
    if (fmt != FMT_Q6_K && stride / 4 > 256) continue;  // a tensor copy's box
    const size_t stage = (size_t)kWarps * 16 * stride;
    const int depth = off >= (size_t)kStreamSmem ? 0 : (int)std::min<size_t>(8, ((size_t)kStreamSmem - off) / stage);
    if (depth < 2) continue;
    p->su = su;
    p->depth = depth;
    p->row_stride = stride;
    p->unit_bytes = ub;
    *smem = off + (size_t)depth * stage;
    return true;
  }
  return false;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                   const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled_fn() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult qr;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &qr) == cudaSuccess &&
                    qr == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<EncodeTiledFn>(f) : nullptr;
  }();
  return fn;
}

template <class F>
int launch_stream(const CUtensorMap& tm, StreamParams& p, size_t smem, int num_sms, cudaStream_t s, std::string* err) {
  auto kernel = moe_stream_kernel<F>;
  static std::atomic<unsigned long long> ready{0};
  static std::atomic<int> resident[64][4];  // clusters of 1, 2, 4, 8 CTAs that fit the device at once
  int dev = 0, ci = 0;
  while ((1 << ci) < p.C) ++ci;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev > 63 || !(ready.load() >> dev & 1))) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem);
    if (e == cudaSuccess && dev < 64) ready.fetch_or(1ull << dev);
  }
  if (e != cudaSuccess) {
    *err = std::string("moe product: ") + cudaGetErrorString(e);
    return -1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kStreamSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = dev < 64 ? resident[dev][ci].load() : 0;
  if (n == 0) {
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = std::max(1, num_sms / p.C);
    }
    if (dev < 64) resident[dev][ci].store(n);
  }
  p.G = n;
  cfg.gridDim = dim3(p.G * p.C);
  cfg.dynamicSmemBytes = smem;
  if (p.C == 1) attr[0] = attr[1];
  cfg.numAttrs = p.C == 1 ? 1 : 2;
  e = cudaLaunchKernelEx(&cfg, kernel, tm, p);
  if (e != cudaSuccess) {
    *err = std::string("moe product launch: ") + cudaGetErrorString(e);
    return -1;
  }
  return 0;
}

// From KQ_MOE_TC_ROWS rows per expert on average the tensor-core product is faster: 128 experts of 2 x 768 x 2048, rows per expert
// (streaming, tensor cores) 28: 151, 172 us; 32: 168, 174; 36: 185, 175; 128: 535, 218; 60 of 2 x 1408 x 2048, 32: 138, 142; 40:
// 171, 143; 8 of 2 x 2048 x 4096, 24: 67, 70; 32: 78, 70; down, 128 of 2048 x 768, 32: 106, 103.
bool by_tensor_cores(int fmt, int T, int k, int E) { return fmt == FMT_Q4_K && (long long)T * k >= (long long)KQ_MOE_TC_ROWS * E; }

// ws: of the tensor-core product
int launch_products(const MoeGemmArgs& a, bool gate_up, float* parts, void* ws, int num_sms, cudaStream_t s, std::string* err) {
  if (by_tensor_cores(a.fmt, a.T, a.k, a.E)) return launch_moe_tc(a, gate_up, parts, ws, num_sms, s, err);
  StreamParams p = {};
  p.w = static_cast<const uint8_t*>(a.w);
  p.x = static_cast<const uint16_t*>(a.x);
  p.xs = a.xs;
  p.div = gate_up ? a.k : 1;
  p.offsets = a.offsets;
  p.order = a.order;
  p.E = a.E;
  p.P = a.T * a.k;
  p.N = gate_up ? 2 * a.N : a.N;
  p.half = gate_up ? a.N : 0;
  p.K = a.K;
  p.y = parts;
  p.act = static_cast<uint16_t*>(a.act);
  p.row_bytes = (long long)kq_row_bytes(a.fmt, a.K);
  p.units = a.K / kUnit;
  p.tiles = gate_up ? (a.N + 7) / 8 : (a.N + 15) / 16;
  p.C = 1;
  while ((p.units + p.C - 1) / p.C > kMaxSliceUnits) p.C *= 2;
  p.chunk = std::min(kMaxChunk, a.T);  // a token chooses an expert once; where it does twice there are more chunks
  size_t smem = 0;
  bool fits = p.C <= kMaxCluster && stream_layout(a.fmt, &p, &smem);
  if (fits && p.chunk > 8 && p.P <= 4 * a.E) {
    // few rows per expert: chunks of eight where that leaves room for longer stages (37 tokens, 4 of 60 experts in Q8_0, 2560 x
    // 1280: stages of one unit 82 us, of two 69)
    StreamParams q = p;
    q.chunk = 8;
    size_t n = 0;
    if (stream_layout(a.fmt, &q, &n) && q.su > p.su) p = q, smem = n;
  }
  if (!fits) {
    *err = "internal: the product does not fit shared memory";
    return -1;
  }
  CUtensorMap tm;
  std::memset(&tm, 0, sizeof(tm));
  if (a.fmt != FMT_Q6_K) {
    // all experts' rows as a 2-D tensor of 4-byte words
    const EncodeTiledFn enc = encode_tiled_fn();
    const cuuint64_t dim[2] = {(cuuint64_t)(p.row_bytes / 4), (cuuint64_t)p.E * p.N}, stride[1] = {(cuuint64_t)p.row_bytes};
    const cuuint32_t box[2] = {(cuuint32_t)(p.row_stride / 4), gate_up ? 8u : 16u}, es[2] = {1u, 1u};
    const CUresult cr = enc ? enc(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(a.w), dim, stride, box, es,
                                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE)
                            : CUDA_ERROR_NOT_FOUND;
    if (cr != CUDA_SUCCESS) {
      *err = "cuTensorMapEncodeTiled failed (" + std::to_string((int)cr) + ")";
      return -1;
    }
  }
  switch (a.fmt) {
    case FMT_Q4_K: return launch_stream<FmtQ4KH>(tm, p, smem, num_sms, s, err);
    case FMT_Q5_K: return launch_stream<FmtQ5KH>(tm, p, smem, num_sms, s, err);
    case FMT_Q6_K: return launch_stream<FmtQ6KH>(tm, p, smem, num_sms, s, err);
    case FMT_Q8_0: return launch_stream<FmtQ8_0H>(tm, p, smem, num_sms, s, err);
    case FMT_AFFINE4: return launch_stream<FmtAffine4>(tm, p, smem, num_sms, s, err);
  }
  *err = "unsupported format";
  return -1;
}

}  // namespace

size_t moe_gate_up_workspace(int fmt, int T, int k, int E, int F, int K) {
  (void)F;
  return by_tensor_cores(fmt, T, k, E) ? moe_tc_workspace(T * k, K) : 0;
}
// The pairs' products, then the tensor-core product's own.
static size_t down_parts(int T, int k, int H) { return ((size_t)T * k * H * 4 + 255) / 256 * 256; }
size_t moe_down_workspace(int fmt, int T, int k, int E, int H, int K) {
  return down_parts(T, k, H) + (by_tensor_cores(fmt, T, k, E) ? moe_tc_workspace(T * k, K) : 0);
}

int launch_moe_gate_up(const MoeGemmArgs& a, int num_sms, cudaStream_t s, std::string* err) {
  return launch_products(a, true, nullptr, a.ws, num_sms, s, err);
}

int launch_moe_down(const MoeGemmArgs& a, int num_sms, cudaStream_t s, std::string* err) {
  float* parts = static_cast<float*>(a.ws);
  if (launch_products(a, false, parts, static_cast<uint8_t*>(a.ws) + down_parts(a.T, a.k, a.N), num_sms, s, err)) return -1;
  JoinParams p = {parts, a.weights, a.add, a.ids, a.y, a.add_stride, a.y_stride, a.T, a.k, a.N, a.E, a.y_dtype};
  const int V = a.N % 4 == 0 ? 4 : 1;
  const long long n = (long long)a.T * (a.N / V);
  const dim3 grid((unsigned)std::min<long long>((n + 255) / 256, (long long)num_sms * 16));
  return V == 4 ? launch_pdl(moe_join_kernel<4>, grid, dim3(256), 0, s, p, "moe_down join", err)
                : launch_pdl(moe_join_kernel<1>, grid, dim3(256), 0, s, p, "moe_down join", err);
}

unsigned int take_moe_errors() {
  unsigned int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_moe_errors, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  cudaMemcpyToSymbol(g_moe_errors, &z, sizeof(z));
  return v;
}

}  // namespace kq
