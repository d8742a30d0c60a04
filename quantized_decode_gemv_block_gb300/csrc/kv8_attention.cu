// Attention over the paged 8-bit KV cache: single tokens, verify windows and prompts of a batch
// of requests of uneven length, grouped-query heads.
//
//   o = sum_p w_p v_p / sum_p w_p,  w_p = 2^(x_p - max x),  x_p = log2(e) scale q.k_p
// over the positions p that the row sees. k_p = (c + 1/2) s with int8 codes c and one scale s per
// (page, kv head), so q.k_p = s (q.c + sum(q) / 2), and v's halves add sum_p w_p s_p / 2 to every
// dim: the tensor cores multiply the codes alone, exact in fp16 (two byte permutes and one
// subtraction per pair; the cache's byte order is that of the MMA operands, see kv8.cuh).
//
// Products: S^T = K q^T and O^T = V^T w^T on mma.sync.m16n8k16 with the cache as the A operand:
// 16 tokens (or dims) by 8 query rows, so a lone token's few rows pad to 8 and not to 16. w^T goes
// from the accumulators of S^T to the B operand by one movmatrix per 8x8 block. q is scaled per row
// by the power of two that puts its largest value in [2^14, 2^15) and rounded to fp16: exact for
// bf16 values within 2^-28 of the row's largest; for fp32 queries a relative 2^-12, below the
// rounding of a bf16 output. For fp32 outputs q and w are split into fp16 hi + lo parts (22 bits).
// The weights that enter a product are those against the page's largest score, up by 2^15 (fp16
// then holds weights down to 2^-29 of the page's largest in full, and an absolute 2^-40 below), and
// the accumulators take the page's share of the softmax and its v scale in fp32: pages whose scales
// lie far apart lose nothing to one another.
//
// Work: a tile is 256 positions, 64 per warp. The positions of a request are cut into segments of
// 1, 2, 4 .. tiles (at most 128 segments; a function of its own length, so a row's bits depend on
// its request and its window alone, never on the batch). An item is (request, block of query rows,
// segment, kv head); a persistent grid walks the items, each CTA finding its requests in prefix
// sums that it forms itself from the lengths, so nothing is planned on the host and the call can be
// captured. Each warp brings its 64 positions' K and V by bulk copies of whole 16-token groups (2 KB
// at D = 128), all requested before the first is used, and works on them alone; the four warps meet
// in shared memory once per item. A request of one segment writes its output there; others write
// partials that a second kernel adds in segment order. Windows of more than 32 tokens are not cut.
//
// Bound by DRAM: every code of the context is read once per block of query rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cstdint>

#include "kq.h"
#include "kq_device.cuh"
#include "kq_internal.h"
#include "kq_launch.cuh"
#include "kv8.cuh"

namespace kq {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kWarpPos = 64, kTile = kWarps * kWarpPos;
constexpr int kMaxSegments = 128;
constexpr int kSplitTokens = 32;  // windows up to this many tokens are cut along the context
constexpr int kMaxRows = 32;      // query rows of an item
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kCombThreads = 256;

__device__ unsigned int g_kv8_errors = 0;  // bit 0: a bounded wait gave up; bit 1: bad lengths or page ids

struct AttnKV8Params {
  const void* q;
  long long qs;  // elements between tokens
  void* o;
  long long os;
  int q_f32, o_f32;
  const int8_t *kc, *vc;
  const float *ks, *vs;
  const int* table;
  int max_blocks;
  const int *ctx, *fresh;
  const uint32_t* mask;
  int B, T, max_new, max_len, n_pages, log2p, n_kv, group;
  float scale_log2e;
  float* part;      // [slot][n_kv][row_cap][D]
  float2* part_ml;  // [slot][n_kv][row_cap]: largest x, sum of weights
  int slots, row_cap;
};

__device__ __forceinline__ int segment_tiles(int len) {  // tiles per segment: a power of two
  const int tiles = (len + kTile - 1) / kTile;
  int n = 1;
  while ((tiles + n - 1) / n > kMaxSegments) n <<= 1;
  return n;
}
__device__ __forceinline__ int segments(int len) {
  const int n = segment_tiles(len) * kTile;
  return (len + n - 1) / n;
}

// A request whose lengths do not fit the call's bounds takes no part.
__device__ __forceinline__ bool request_ok(const AttnKV8Params& p, int c, int n) {
  return c >= 0 && n >= 0 && n <= p.max_new && c <= p.max_len - n && (p.mask == nullptr || n <= kSplitTokens) &&
         ((c + n + (1 << p.log2p) - 1) >> p.log2p) <= p.max_blocks;
}

// Prefix sums over the requests in shared memory: its first token, work item and partial slot.
// ITEMS: items of the attention kernel; otherwise tokens of requests that the combine finishes.
template <int THREADS, bool ITEMS>
__device__ __forceinline__ void scan_requests(const AttnKV8Params& p, int row_block, int* tok, int* item, int* slot, int* sm) {
  constexpr int W = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  long long ct = 0;
  int ci = 0, cs = 0;
  bool bad = false;
  for (int base = 0; base < p.B; base += THREADS) {
    const int r = base + tid;
    int a = 0, b = 0, c = 0;
    if (r < p.B) {
      const int ctx = p.ctx[r], n = p.fresh[r];
      a = n > 0 ? min(n, p.T + 1) : 0;
      if (request_ok(p, ctx, n)) {
        if (n > 0) {
          const bool cut = n <= kSplitTokens;
          const int nseg = cut ? segments(ctx + n) : 1;
          if (ITEMS) b = (n * p.group + row_block - 1) / row_block * nseg;
          else b = nseg > 1 ? n : 0;
          c = nseg > 1 ? nseg : 0;
        }
      } else {
        bad = true;
      }
    }
    const int a0 = a, b0 = b, c0 = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int xa = __shfl_up_sync(~0u, a, o), xb = __shfl_up_sync(~0u, b, o), xc = __shfl_up_sync(~0u, c, o);
      if (lane >= o) {
        a += xa;
        b += xb;
        c += xc;
      }
    }
    __syncthreads();
    if (lane == 31) {
      sm[w] = a;
      sm[W + w] = b;
      sm[2 * W + w] = c;
    }
    __syncthreads();
    int pa = 0, pb = 0, pc = 0, ta = 0, tb = 0, tc = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int xa = sm[i], xb = sm[W + i], xc = sm[2 * W + i];
      if (i < w) {
        pa += xa;
        pb += xb;
        pc += xc;
      }
      ta += xa;
      tb += xb;
      tc += xc;
    }
    if (r < p.B) {
      tok[r] = (int)min(ct + pa + a - a0, (long long)INT_MAX);
      item[r] = ci + pb + b - b0;
      slot[r] = cs + pc + c - c0;
    }
    ct += ta;
    ci += tb;
    cs += tc;
  }
  if (tid == 0) {
    tok[p.B] = (int)min(ct, (long long)INT_MAX);
    item[p.B] = ct > p.T ? 0 : ci;  // more tokens than q has rows: nothing is done
    slot[p.B] = cs;
  }
  if (bad || ct > p.T) atomicOr(&g_kv8_errors, 2u);
  __syncthreads();
}

__device__ __forceinline__ int find_request(const int* s, int B, int x) {  // largest r with s[r] <= x
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// Four int8 codes -> fp16 pairs: 1024 + (c + 128) by a byte permute under 0x64, minus 1152.
__device__ __forceinline__ void codes_to_h2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = h2_sub(prmt(u, 0x64646464u, 0x4140), 0x64806480u);
  hi = h2_sub(prmt(u, 0x64646464u, 0x4342), 0x64806480u);
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Largest of the eight lanes that hold one query row's scores.
__device__ __forceinline__ float max_over_rows(float v) {
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, x));
  return v;
}

template <int D, int NT, bool WIDE>
struct AttnSmem {
  static constexpr int RB = 8 * NT;
  static constexpr int kStage = kWarpPos * D;          // bytes of K (and of V) per warp
  static constexpr int kOut = RB * (D + 4) * 4;        // a warp's output rows, 4 floats of padding
  static constexpr int kWarpBytes = (2 * kStage > kOut ? 2 * kStage : kOut + 127) / 128 * 128;
  static constexpr int kQ = NT * D * 16;               // fp16 query operands (hi); the lo parts follow
  static constexpr size_t bytes(int B) { return (size_t)kWarps * kWarpBytes + (WIDE ? 2 : 1) * kQ + (size_t)3 * (B + 1) * 4; }
};

template <int D, int NT, bool WIDE>
__global__ void __launch_bounds__(kThreads) attn_kv8_kernel(const AttnKV8Params p) {
  using S = AttnSmem<D, NT, WIDE>;
  constexpr int RB = S::RB, C32 = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t sm_bar[kWarps][2];
  __shared__ float sm_hq[RB], sm_rf[RB], sm_m[kWarps][RB], sm_l[kWarps][RB], sm_h[kWarps][RB];
  __shared__ int sm_lim[RB], sm_scan[3 * kWarps];
  __shared__ uint32_t sm_mask[RB];
  uint32_t* sm_q = reinterpret_cast<uint32_t*>(smem + kWarps * S::kWarpBytes);  // [hi/lo][NT][C32][32][4]
  int* sm_tok = reinterpret_cast<int*>(smem + kWarps * S::kWarpBytes + (WIDE ? 2 : 1) * S::kQ);
  int* sm_item = sm_tok + p.B + 1;
  int* sm_slot = sm_item + p.B + 1;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, t4 = lane & 3;
  uint8_t* kst = smem + w * S::kWarpBytes;
  uint8_t* vst = kst + S::kStage;
  if (lane == 0) {
    mbar_init(&sm_bar[w][0], 1);
    mbar_init(&sm_bar[w][1], 1);
    fence_mbar_init();
  }
  grid_dependency_wait();
  scan_requests<kThreads, true>(p, RB, sm_tok, sm_item, sm_slot, sm_scan);
  grid_launch_dependents();
  const long long total = (long long)sm_item[p.B] * p.n_kv;
  const int P = 1 << p.log2p, page_groups = P >= kWarpPos ? 4 : P >> 4;
  uint32_t phase = 0;
  bool dead = false;
  for (long long it = blockIdx.x; it < total; it += gridDim.x) {
    const int h = (int)(it % p.n_kv), wi = (int)(it / p.n_kv);
    const int r = find_request(sm_item, p.B, wi);
    const int ctx = p.ctx[r], n = p.fresh[r], len = ctx + n, rows = n * p.group;
    const bool cut = n <= kSplitTokens;
    const int seg_tiles = cut ? segment_tiles(len) : 0, nseg = cut ? segments(len) : 1;
    const int local = wi - sm_item[r], rb = local / nseg, seg = local - rb * nseg;
    const int row0 = rb * RB, tok0 = sm_tok[r];
    // tiles: the segment's, and none past what the block's last token sees
    const int last_row = min(row0 + RB, rows) - 1;
    const int end = p.mask ? len : ctx + last_row / p.group + 1;  // exclusive
    const int tile0 = cut ? seg * seg_tiles : 0;
    const int tile1 = cut ? min(tile0 + seg_tiles, (end + kTile - 1) / kTile) : (end + kTile - 1) / kTile;

    // ---- this warp's copies of one tile: K and V of its 64 positions
    int page = -1;  // lane j < 4: page of group j
    auto request = [&](int tile) {
      const int pos = tile * kTile + w * kWarpPos + 16 * lane;
      page = -1;
      if (lane < 4 && (pos & -P) < end) {  // also groups past the end of a page that holds positions: its scale is theirs
        page = p.table[(long long)r * p.max_blocks + (pos >> p.log2p)];
        if (page < 0 || page >= p.n_pages) {
          page = -2;
          atomicOr(&g_kv8_errors, 2u);
        }
      }
      const bool live = page >= 0 && pos < end;
      const unsigned any = __ballot_sync(~0u, live);
      if (lane == 0) {
        const uint32_t bytes = __popc(any) * 16 * D;
        mbar_arrive_expect_tx(&sm_bar[w][0], bytes);
        mbar_arrive_expect_tx(&sm_bar[w][1], bytes);
      }
      __syncwarp();
      if (live) {
        const long long off = (((long long)page * p.n_kv + h) << p.log2p) * D + (pos & (P - 1)) * D;
        bulk_g2s(kst + lane * 16 * D, p.kc + off, 16 * D, &sm_bar[w][0]);
        bulk_g2s(vst + lane * 16 * D, p.vc + off, 16 * D, &sm_bar[w][1]);
      }
    };
    if (tile0 < tile1) request(tile0);

    // ---- query operands: warp w takes rows w, w + 4, ...
    for (int rr = w; rr < RB; rr += kWarps) {
      const int row = row0 + rr, i = row / p.group;
      const bool live = row < rows;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (live && 4 * lane < D) {
        const long long at = (tok0 + i) * p.qs + (long long)(h * p.group + row - i * p.group) * D + 4 * lane;
        if (p.q_f32) {
          const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at);
          v[0] = x.x;
          v[1] = x.y;
          v[2] = x.z;
          v[3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + at);
          v[0] = __uint_as_float(x.x << 16);
          v[1] = __uint_as_float(x.x & 0xFFFF0000u);
          v[2] = __uint_as_float(x.y << 16);
          v[3] = __uint_as_float(x.y & 0xFFFF0000u);
        }
      }
      unsigned top = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
      top = __reduce_max_sync(~0u, top);
      // 2^e with the largest |q| 2^e in [2^14, 2^15); 1 for zero rows and for rows that are not finite
      const int ex = (int)(top >> 23);
      const int e2 = top == 0 || ex == 0xFF ? 0 : max(-126, min(126, 14 - (ex - 127)));
      const float up = __uint_as_float((unsigned)(127 + e2) << 23), down = __uint_as_float((unsigned)(127 - e2) << 23);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= up;
      const uint32_t h0 = f2_to_h2(v[0], v[1]), h1 = f2_to_h2(v[2], v[3]);
      float f[4] = {h_lo_to_f(h0), h_lo_to_f(h0 >> 16), h_lo_to_f(h1), h_lo_to_f(h1 >> 16)};
      const int c = lane >> 3, s = (lane >> 2) & 1, at = (((rr >> 3) * C32 + c) * 32 + (rr & 7) * 4 + t4) * 4 + 2 * s;
      if (4 * lane < D) {
        sm_q[at] = h0;
        sm_q[at + 1] = h1;
      }
      if (WIDE) {
        const uint32_t l0 = f2_to_h2(v[0] - f[0], v[1] - f[1]), l1 = f2_to_h2(v[2] - f[2], v[3] - f[3]);
        f[0] += h_lo_to_f(l0);
        f[1] += h_lo_to_f(l0 >> 16);
        f[2] += h_lo_to_f(l1);
        f[3] += h_lo_to_f(l1 >> 16);
        if (4 * lane < D) {
          sm_q[S::kQ / 4 + at] = l0;
          sm_q[S::kQ / 4 + at + 1] = l1;
        }
      }
      float sum = (f[0] + f[1]) + (f[2] + f[3]);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
      if (lane == 0) {
        sm_hq[rr] = 0.5f * sum;
        sm_rf[rr] = down * p.scale_log2e;
        sm_lim[rr] = live ? ctx + i : -1;
        sm_mask[rr] = live && p.mask ? p.mask[tok0 + i] : 0u;
      }
    }
    __syncthreads();

    float o[C32][2][NT][4], m[NT][2], l[NT][2], hv[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        m[nt][k] = -INFINITY;
        l[nt][k] = hv[nt][k] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < C32; ++c)
#pragma unroll
        for (int s = 0; s < 2; ++s) o[c][s][nt][0] = o[c][s][nt][1] = o[c][s][nt][2] = o[c][s][nt][3] = 0.f;
    }
    const int tok_pos = 4 * (g >> 1) + (g & 1);  // token of operand row g in its group; row g + 8 is two further

    for (int tile = tile0; tile < tile1; ++tile) {
      const int base = tile * kTile + w * kWarpPos;
      if (base < end) {
        float ksc = 0.f, vsc = 0.f;
        if (lane < 4 && page != -1) {
          const float nan = __uint_as_float(0x7FC00000u);
          ksc = page >= 0 ? p.ks[(long long)page * p.n_kv + h] : nan;
          vsc = page >= 0 ? p.vs[(long long)page * p.n_kv + h] : nan;
        }
        // ---- scores
        if (!dead && !mbar_wait_bounded(&sm_bar[w][0], phase, kWaitNs)) dead = true;
        float sc[4][NT][4];
#pragma unroll
        for (int st = 0; st < 4; ++st)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) sc[st][nt][0] = sc[st][nt][1] = sc[st][nt][2] = sc[st][nt][3] = 0.f;
#pragma unroll
        for (int c = 0; c < C32; ++c) {
          uint4 qh[NT], ql[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            qh[nt] = lds128(sm_q + ((nt * C32 + c) * 32 + lane) * 4);
            if (WIDE) ql[nt] = lds128(sm_q + S::kQ / 4 + ((nt * C32 + c) * 32 + lane) * 4);
          }
#pragma unroll
          for (int st = 0; st < 4; ++st) {
            const uint4 x = lds128(kst + st * 16 * D + c * 512 + lane * 16);
            uint32_t a0[4], a1[4];
            codes_to_h2(x.x, a0[0], a0[2]);
            codes_to_h2(x.y, a0[1], a0[3]);
            codes_to_h2(x.z, a1[0], a1[2]);
            codes_to_h2(x.w, a1[1], a1[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16_16816(sc[st][nt], a0, qh[nt].x, qh[nt].y, sc[st][nt]);
              mma_f16_16816(sc[st][nt], a1, qh[nt].z, qh[nt].w, sc[st][nt]);
              if (WIDE) {
                mma_f16_16816(sc[st][nt], a0, ql[nt].x, ql[nt].y, sc[st][nt]);
                mma_f16_16816(sc[st][nt], a1, ql[nt].z, ql[nt].w, sc[st][nt]);
              }
            }
          }
        }
        float kf[4], vf[4];
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          kf[st] = __shfl_sync(~0u, ksc, st);
          vf[st] = __shfl_sync(~0u, vsc, st);
        }
        // ---- weights: rows 2 t4 and 2 t4 + 1 of each block of 8, operand rows g and g + 8 (tokens)
        uint32_t wb[4][NT][2], wlo[WIDE ? 4 : 1][NT][2];
        float fv[4][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int rr = nt * 8 + 2 * t4;
          const float2 hq = lds_f2(sm_hq + rr), rf = lds_f2(sm_rf + rr);
          const int lim0 = sm_lim[rr], lim1 = sm_lim[rr + 1];
          const uint32_t mk0 = sm_mask[rr], mk1 = sm_mask[rr + 1];
          auto sees = [&](int pos, int lim, uint32_t mk) {
            if (p.mask == nullptr) return pos <= lim;
            const int j = pos - ctx;
            return lim >= 0 && pos < len && (j < 0 || (mk >> (j & 31) & 1u) != 0);
          };
          float gx[4][2];  // largest score of each group, then of each page
#pragma unroll
          for (int st = 0; st < 4; ++st) {
            const int p0 = base + 16 * st + tok_pos, p1 = p0 + 2;
            float* s = sc[st][nt];
            s[0] = sees(p0, lim0, mk0) ? (s[0] + hq.x) * (rf.x * kf[st]) : -INFINITY;
            s[1] = sees(p0, lim1, mk1) ? (s[1] + hq.y) * (rf.y * kf[st]) : -INFINITY;
            s[2] = sees(p1, lim0, mk0) ? (s[2] + hq.x) * (rf.x * kf[st]) : -INFINITY;
            s[3] = sees(p1, lim1, mk1) ? (s[3] + hq.y) * (rf.y * kf[st]) : -INFINITY;
            gx[st][0] = fmaxf(s[0], s[2]);
            gx[st][1] = fmaxf(s[1], s[3]);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (page_groups == 4) {
              gx[0][k] = gx[1][k] = gx[2][k] = gx[3][k] = max_over_rows(fmaxf(fmaxf(gx[0][k], gx[1][k]), fmaxf(gx[2][k], gx[3][k])));
            } else if (page_groups == 2) {
              gx[0][k] = gx[1][k] = max_over_rows(fmaxf(gx[0][k], gx[1][k]));
              gx[2][k] = gx[3][k] = max_over_rows(fmaxf(gx[2][k], gx[3][k]));
            } else {
#pragma unroll
              for (int st = 0; st < 4; ++st) gx[st][k] = max_over_rows(gx[st][k]);
            }
          }
          const float mx0 = fmaxf(fmaxf(gx[0][0], gx[1][0]), fmaxf(gx[2][0], gx[3][0]));
          const float mx1 = fmaxf(fmaxf(gx[0][1], gx[1][1]), fmaxf(gx[2][1], gx[3][1]));
          const float n0 = fmaxf(m[nt][0], mx0), n1 = fmaxf(m[nt][1], mx1);
          const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;
          const float al0 = fast_exp2(m[nt][0] - b0), al1 = fast_exp2(m[nt][1] - b1);
          m[nt][0] = n0;
          m[nt][1] = n1;
          if (tile > tile0) {
            l[nt][0] *= al0;
            l[nt][1] *= al1;
            hv[nt][0] *= al0;
            hv[nt][1] *= al1;
#pragma unroll
            for (int c = 0; c < C32; ++c)
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                o[c][s][nt][0] *= al0;
                o[c][s][nt][1] *= al1;
                o[c][s][nt][2] *= al0;
                o[c][s][nt][3] *= al1;
              }
          }
#pragma unroll
          for (int st = 0; st < 4; ++st) {
            float* s = sc[st][nt];
            // weights against the page's largest score, up by 2^15 into fp16's range
            const float c0 = gx[st][0] == -INFINITY ? 0.f : gx[st][0] - 15.f, c1 = gx[st][1] == -INFINITY ? 0.f : gx[st][1] - 15.f;
            s[0] = fast_exp2(s[0] - c0);
            s[1] = fast_exp2(s[1] - c1);
            s[2] = fast_exp2(s[2] - c0);
            s[3] = fast_exp2(s[3] - c1);
            const float up0 = gx[st][0] == -INFINITY ? 0.f : fast_exp2(c0 - b0), up1 = gx[st][1] == -INFINITY ? 0.f : fast_exp2(c1 - b1);
            float f0 = vf[st] * up0, f1 = vf[st] * up1;
            if (!(fabsf(vf[st]) <= 3.402823466e38f)) {  // a broken scale reaches the rows that see its page alone
              const int p0 = base + 16 * st + tok_pos, p1 = p0 + 2;
              int any = (sees(p0, lim0, mk0) || sees(p1, lim0, mk0) ? 1 : 0) | (sees(p0, lim1, mk1) || sees(p1, lim1, mk1) ? 2 : 0);
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) any |= __shfl_xor_sync(~0u, any, x);
              if (!(any & 1)) f0 = 0.f;
              if (!(any & 2)) f1 = 0.f;
            }
            fv[st][nt][0] = f0;
            fv[st][nt][1] = f1;
            const float w0 = s[0] + s[2], w1 = s[1] + s[3];
            l[nt][0] += w0 * up0;
            l[nt][1] += w1 * up1;
            hv[nt][0] += w0 * f0;
            hv[nt][1] += w1 * f1;
            const uint32_t e0 = f2_to_h2(s[0], s[1]), e1 = f2_to_h2(s[2], s[3]);
            wb[st][nt][0] = movmatrix(e0);
            wb[st][nt][1] = movmatrix(e1);
            if (WIDE) {
              wlo[st][nt][0] = movmatrix(f2_to_h2(s[0] - h_lo_to_f(e0), s[1] - h_lo_to_f(e0 >> 16)));
              wlo[st][nt][1] = movmatrix(f2_to_h2(s[2] - h_lo_to_f(e1), s[3] - h_lo_to_f(e1 >> 16)));
            }
          }
        }
        // ---- values: the groups of one page are added up before its scale
        if (!dead && !mbar_wait_bounded(&sm_bar[w][1], phase, kWaitNs)) dead = true;
#pragma unroll
        for (int c = 0; c < C32; ++c) {
          float acc[2][NT][4];
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[s][nt][0] = acc[s][nt][1] = acc[s][nt][2] = acc[s][nt][3] = 0.f;
#pragma unroll
          for (int st = 0; st < 4; ++st) {
            const uint4 x = lds128(vst + st * 16 * D + c * 512 + lane * 16);
            uint32_t a0[4], a1[4];
            codes_to_h2(x.x, a0[0], a0[2]);
            codes_to_h2(x.y, a0[1], a0[3]);
            codes_to_h2(x.z, a1[0], a1[2]);
            codes_to_h2(x.w, a1[1], a1[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16_16816(acc[0][nt], a0, wb[st][nt][0], wb[st][nt][1], acc[0][nt]);
              mma_f16_16816(acc[1][nt], a1, wb[st][nt][0], wb[st][nt][1], acc[1][nt]);
              if (WIDE) {
                mma_f16_16816(acc[0][nt], a0, wlo[st][nt][0], wlo[st][nt][1], acc[0][nt]);
                mma_f16_16816(acc[1][nt], a1, wlo[st][nt][0], wlo[st][nt][1], acc[1][nt]);
              }
            }
            if (((st + 1) & (page_groups - 1)) == 0) {
#pragma unroll
              for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  o[c][s][nt][0] += fv[st][nt][0] * acc[s][nt][0];
                  o[c][s][nt][1] += fv[st][nt][1] * acc[s][nt][1];
                  o[c][s][nt][2] += fv[st][nt][0] * acc[s][nt][2];
                  o[c][s][nt][3] += fv[st][nt][1] * acc[s][nt][3];
                  acc[s][nt][0] = acc[s][nt][1] = acc[s][nt][2] = acc[s][nt][3] = 0.f;
                }
            }
          }
        }
      } else if (!dead) {  // nothing was copied: the empty phase still completes
        if (!mbar_wait_bounded(&sm_bar[w][0], phase, kWaitNs) || !mbar_wait_bounded(&sm_bar[w][1], phase, kWaitNs)) dead = true;
      }
      phase ^= 1;
      if (tile + 1 < tile1) {
        __syncwarp();  // every lane has read the staged codes
        request(tile + 1);
      }
    }

    // ---- the four warps' results meet
    __syncwarp();
    float* out = reinterpret_cast<float*>(kst);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float a = l[nt][k], b = hv[nt][k];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          a += __shfl_xor_sync(~0u, a, x);
          b += __shfl_xor_sync(~0u, b, x);
        }
        if (g == 0) {
          sm_m[w][nt * 8 + 2 * t4 + k] = m[nt][k];
          sm_l[w][nt * 8 + 2 * t4 + k] = a;
          sm_h[w][nt * 8 + 2 * t4 + k] = 0.5f * b;
        }
      }
      float* o0 = out + (nt * 8 + 2 * t4) * (D + 4) + g;
#pragma unroll
      for (int c = 0; c < C32; ++c)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          o0[32 * c + 16 * s] = o[c][s][nt][0];
          o0[32 * c + 16 * s + D + 4] = o[c][s][nt][1];
          o0[32 * c + 16 * s + 8] = o[c][s][nt][2];
          o0[32 * c + 16 * s + 8 + D + 4] = o[c][s][nt][3];
        }
    }
    __syncthreads();
    const bool partial = nseg > 1;
    const long long slot = (long long)sm_slot[r] + seg;
    const bool room = !partial || (slot < p.slots && rows <= p.row_cap);
    if (!room && tid == 0) atomicOr(&g_kv8_errors, 2u);
    for (int x = tid; x < RB * (D / 4); x += kThreads) {
      const int rr = x / (D / 4), d = (x - rr * (D / 4)) * 4, row = row0 + rr;
      if (row >= rows || !room) continue;
      float mm = sm_m[0][rr];
#pragma unroll
      for (int i = 1; i < kWarps; ++i) mm = fmaxf(mm, sm_m[i][rr]);
      const float mb = mm == -INFINITY ? 0.f : mm;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float den = 0.f, hs = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        if (sm_l[i][rr] == 0.f) continue;  // the warp's positions are none of the row's
        const float f = fast_exp2(sm_m[i][rr] - mb);
        const float4 v = *reinterpret_cast<const float4*>(smem + i * S::kWarpBytes + (rr * (D + 4) + d) * 4);
        sum.x += f * v.x;
        sum.y += f * v.y;
        sum.z += f * v.z;
        sum.w += f * v.w;
        den += f * sm_l[i][rr];
        hs += f * sm_h[i][rr];
      }
      sum.x += hs;
      sum.y += hs;
      sum.z += hs;
      sum.w += hs;
      if (partial) {
        const long long at = (slot * p.n_kv + h) * p.row_cap + row;
        *reinterpret_cast<float4*>(p.part + at * D + d) = sum;
        if (d == 0) p.part_ml[at] = make_float2(mm, den);
      } else {
        const float inv = den == 0.f ? 0.f : 1.f / den;
        const int i = row / p.group;
        const long long at = (tok0 + i) * p.os + (long long)(h * p.group + row - i * p.group) * D + d;
        if (p.o_f32) {
          *reinterpret_cast<float4*>(static_cast<float*>(p.o) + at) = make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
        } else {
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + at) =
              make_uint2((uint32_t)f32_to_bf16_rn(sum.x * inv) | (uint32_t)f32_to_bf16_rn(sum.y * inv) << 16,
                         (uint32_t)f32_to_bf16_rn(sum.z * inv) | (uint32_t)f32_to_bf16_rn(sum.w * inv) << 16);
        }
      }
    }
    fence_proxy_async_smem();  // the next copies overwrite what was read above
    __syncthreads();
  }
  if (dead) atomicOr(&g_kv8_errors, 1u);
}

// The segments of a request added in order: one CTA per (token, query head), its eight warps each
// taking every eighth segment, then warp 0 the eight sums.
template <int D>
__global__ void __launch_bounds__(kCombThreads) attn_kv8_combine_kernel(const AttnKV8Params p) {
  constexpr int W = kCombThreads / 32, E = D / 32;
  extern __shared__ int sm_req[];
  __shared__ int sm_scan[3 * W];
  __shared__ float sm_o[W][D], sm_mx[W], sm_sum[W];
  int *sm_tok = sm_req, *sm_item = sm_tok + p.B + 1, *sm_slot = sm_item + p.B + 1;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  grid_dependency_wait();
  scan_requests<kCombThreads, false>(p, 1, sm_tok, sm_item, sm_slot, sm_scan);
  const int n_q = p.n_kv * p.group;
  const long long total = (long long)sm_item[p.B] * n_q;
  for (long long it = blockIdx.x; it < total; it += gridDim.x) {
    const int ti = (int)(it / n_q), hq = (int)(it - (long long)ti * n_q);
    const int r = find_request(sm_item, p.B, ti), i = ti - sm_item[r];
    const int n = p.fresh[r], nseg = segments(p.ctx[r] + n), h = hq / p.group, row = i * p.group + hq - h * p.group;
    if ((long long)sm_slot[r] + nseg > p.slots || n * p.group > p.row_cap) continue;
    const long long first = ((long long)sm_slot[r] * p.n_kv + h) * p.row_cap + row, step = (long long)p.n_kv * p.row_cap;
    float mx = -INFINITY;
    for (int s = lane; s < nseg; s += 32) mx = fmaxf(mx, p.part_ml[first + s * step].x);
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, x));
    const float mb = mx == -INFINITY ? 0.f : mx;
    float acc[E], den = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int s = w; s < nseg; s += W) {
      const float2 ml = p.part_ml[first + s * step];
      const float* src = p.part + (first + s * step) * D + lane * E;
      const float f = ml.y == 0.f ? 0.f : fast_exp2(ml.x - mb);
      den += f * ml.y;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += f * src[e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[w][lane * E + e] = acc[e];
    if (lane == 0) sm_sum[w] = den;
    __syncthreads();
    if (tid < D) {
      float v = 0.f, dn = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        v += sm_o[k][tid];
        dn += sm_sum[k];
      }
      const float res = dn == 0.f ? 0.f : v * (1.f / dn);  // as a request of one segment
      const long long at = (sm_tok[r] + i) * p.os + (long long)hq * D + tid;
      if (p.o_f32) static_cast<float*>(p.o)[at] = res;
      else static_cast<uint16_t*>(p.o)[at] = f32_to_bf16_rn(res);
    }
    __syncthreads();
  }
}

template <int D, int NT, bool WIDE>
int launch_typed(const AttnKV8Params& p, int num_sms, cudaStream_t s, std::string* err) {
  const size_t smem = AttnSmem<D, NT, WIDE>::bytes(p.B);
  auto* kernel = attn_kv8_kernel<D, NT, WIDE>;
  // CTAs per SM at this shared-memory size, asked for once per host thread, device and size
  static thread_local int known_dev = -1, per_sm = 0;
  static thread_local size_t known_smem = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev != known_dev || smem != known_smem)) {
    per_sm = 0;
    known_dev = -1;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, smem);
    if (e == cudaSuccess && per_sm > 0) {
      known_dev = dev;
      known_smem = smem;
    }
  }
  if (e != cudaSuccess || per_sm < 1) {
    *err = std::string("attention_kv8: ") + (e != cudaSuccess ? cudaGetErrorString(e) : "the kernel does not fit an SM");
    return -1;
  }
  if (launch_pdl(kernel, dim3(num_sms * per_sm), dim3(kThreads), smem, s, p, "attention_kv8", err) != 0) return -1;
  if (p.max_len <= kTile) return 0;  // no request can have two segments
  const long long tasks = (long long)p.T * p.n_kv * p.group;
  const int grid = (int)(tasks < (long long)num_sms * 8 ? tasks : (long long)num_sms * 8);
  return launch_pdl(attn_kv8_combine_kernel<D>, dim3(grid), dim3(kCombThreads), (size_t)3 * (p.B + 1) * 4, s, p,
                    "attention_kv8 combine", err);
}

template <int D>
int launch_dim(const AttnKV8Params& p, int num_sms, cudaStream_t s, std::string* err) {
  const long long rows = (long long)p.max_new * p.group;
  if (p.o_f32) return rows <= 8 ? launch_typed<D, 1, true>(p, num_sms, s, err) : launch_typed<D, 2, true>(p, num_sms, s, err);
  return rows <= 8 ? launch_typed<D, 1, false>(p, num_sms, s, err)
       : rows <= 16 ? launch_typed<D, 2, false>(p, num_sms, s, err) : launch_typed<D, 4, false>(p, num_sms, s, err);
}

size_t part_rows(int max_new, int n_q, int n_kv) { return (size_t)(n_q / n_kv) * (max_new < kSplitTokens ? max_new : kSplitTokens); }
size_t part_slots(int B, long long total_len) { return (size_t)(total_len / kTile) + B; }

}  // namespace

unsigned int take_kv8_errors() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv8_errors, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (cudaMemcpyToSymbol(g_kv8_errors, &zero, sizeof(zero)) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
}

size_t attention_kv8_workspace(int B, long long total_len, int max_new, int n_q, int n_kv, int D) {
  return part_slots(B, total_len) * n_kv * part_rows(max_new, n_q, n_kv) * (D + 2) * sizeof(float);
}

int launch_attention_kv8(const KV8Args& c, const AttnKV8Args& a, int num_sms, cudaStream_t s, std::string* err) {
  AttnKV8Params p = {};
  p.q = a.q;
  p.qs = a.qs;
  p.o = a.o;
  p.os = a.os;
  p.q_f32 = a.q_dtype == KQ_F32;
  p.o_f32 = a.o_dtype == KQ_F32;
  p.kc = c.k;
  p.vc = c.v;
  p.ks = c.k_scale;
  p.vs = c.v_scale;
  p.table = a.table;
  p.max_blocks = a.max_blocks;
  p.ctx = a.ctx;
  p.fresh = a.fresh;
  p.mask = a.mask;
  p.B = a.B;
  p.T = a.T;
  p.max_new = a.max_new;
  p.max_len = a.max_len;
  p.n_pages = c.n_pages;
  p.log2p = c.log2p;
  p.n_kv = c.n_kv;
  p.group = a.n_q / c.n_kv;
  p.scale_log2e = a.scale * 1.4426950408889634f;
  p.slots = (int)part_slots(a.B, a.total_len);
  p.row_cap = (int)part_rows(a.max_new, a.n_q, c.n_kv);
  p.part = static_cast<float*>(a.ws);
  p.part_ml = reinterpret_cast<float2*>(p.part + (size_t)p.slots * c.n_kv * p.row_cap * c.D);
  return c.D == 64 ? launch_dim<64>(p, num_sms, s, err) : launch_dim<128>(p, num_sms, s, err);
}

}  // namespace kq
