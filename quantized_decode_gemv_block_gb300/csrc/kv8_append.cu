// Append to the paged 8-bit KV cache: quantize the new tokens' k and v into their slots.
//
// One fp32 scale s per (page, kv head), for k and for v: s = 2^(floor(log2 max|x|) - 6) over the
// page's tokens, so |x| < 128 s, the code floor(x / s) fits int8, and (code + 1/2) s is within s / 2
// of x. When new tokens raise the scale by 2^n the page's codes are shifted right by n:
// floor(floor(x / s) / 2^n) = floor(x / (2^n s)), so the page always holds what quantizing all of
// its tokens at once would give, however they were grouped into calls. x / s is exact (a power of
// two), so every code follows exactly from the inputs.
//
// Bound by DRAM for prompts (k, v in once, one byte per value out), by latency for single tokens.
// The rows of one call that share a page (a run) stand behind one another, with skipped rows between them at most; the CTA
// whose token range holds a run's first row takes the whole run, for one head's k or v or for several of them where a page
// has few values. A row begins a run if the last one before it that has a slot is of another page, so that no two CTAs
// take one page. Nearly every run is rows in a row at consecutive slots, seen whole in the slots that a CTA loads first. Only
// where a skipped row stands before its first or behind its last one, or another slot of the page follows, the CTA looks
// further and takes what comes row by row, one after the other, which gives what coding the run at once gives.
//   A thread holds 4 tokens x 8 dims of the page in registers between the pass for max|x| and the coding, so k and v
// are read once; the codes of such a tile are whole words of the cache's order (kv8.cuh), both for k (4 dims of a token) and for v
// (4 tokens of a dim), so a thread shares no word with another and rewrites the ones that it must
// shift without any exchange. A word's four codes are the low bytes of fma(x, 1 / s, 1.5 * 2^23)
// rounded down: floor(x / s) in one instruction. No CTA waits for another and no atomics meet in
// memory, so results never vary.
// Measured: 28000 tokens of 8 heads of 128 in bf16 (174 MB) in 35.1 us, 5.0 TB/s, the arithmetic and
// byte permutes at 55 % of their pipe and the issue slots at 64 %; 108 us with both passes over global memory and codes of v
// gathered one by one, 57 with one of k and v per thread, 38.5 without the path for whole words. 64
// tokens of as many requests: 4.1 us, latency: the slots, the values, the maximum, the codes. Looking further costs about
// 1 us: the same 64 tokens with three skipped rows behind each 7.1 us (6.3 without it), and with 777 skipped rows
// at the end 8.6 (8.4).
#include <cuda_bf16.h>

#include <climits>
#include <cstdint>

#include "kq.h"
#include "kq_device.cuh"
#include "kq_internal.h"
#include "kq_launch.cuh"
#include "kv8.cuh"

namespace kq {
namespace {

constexpr int kThreads = 256;
constexpr int kSeek = 4;  // slots that a thread reads at once when it looks beyond the first ones

__device__ unsigned int g_kv8_append_errors = 0;  // bit 1: a slot beyond the cache's pages

struct AppendParams {
  const void* x[2];  // k, v
  long long xs[2];   // elements between tokens
  int8_t* codes[2];
  float* scale[2];
  const int* slot;
  int T, log2p, n_pages, n_kv, range;
};

// Eight dims of a token, raw.
struct RowF32 {
  uint4 a, b;
};
struct RowBf16 {
  uint4 a;
};
__device__ __forceinline__ void load_row(RowF32& r, const float* p) {
  r.a = reinterpret_cast<const uint4*>(p)[0];
  r.b = reinterpret_cast<const uint4*>(p)[1];
}
__device__ __forceinline__ void load_row(RowBf16& r, const uint16_t* p) { r.a = *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void clear_row(RowF32& r) { r.a = r.b = make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ void clear_row(RowBf16& r) { r.a = make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ unsigned top4(const uint4& v) {
  constexpr unsigned M = 0x7FFFFFFFu;
  return max(max(v.x & M, v.y & M), max(v.z & M, v.w & M));
}
// Largest |x| of the row by its fp32 bits: a NaN or infinity is above every finite value.
__device__ __forceinline__ unsigned top_of(const RowF32& r) { return max(top4(r.a), top4(r.b)); }
__device__ __forceinline__ unsigned top_of(const RowBf16& r) {
  constexpr unsigned M = 0x7FFF7FFFu;
  const unsigned m = __vmaxu2(__vmaxu2(r.a.x & M, r.a.y & M), __vmaxu2(r.a.z & M, r.a.w & M));
  return max(m & 0xFFFF0000u, m << 16);
}
__device__ __forceinline__ void values(float (&v)[8], const RowF32& r) {
  const unsigned w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void values(float (&v)[8], const RowBf16& r) {
  const unsigned w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// floor(x * inv) in the low byte; inv is a power of two, or 0 (code 0).
__device__ __forceinline__ uint32_t code(float x, float inv) { return __float_as_uint(__fmaf_rd(x, inv, 12582912.f)); }
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return prmt(prmt(a, b, 0x0040), prmt(c, d, 0x0040), 0x5410);
}

// Each byte of w shifted right arithmetically by n (0..7).
__device__ __forceinline__ uint32_t shift_bytes(uint32_t w, int n) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) r |= ((uint32_t)((int)(int8_t)(w >> (8 * i)) >> n) & 0xFFu) << (8 * i);
  return r;
}

// The page of a slot, or -1 where the token is skipped: no slot, or one beyond the cache.
__device__ __forceinline__ int page_of(int slot, int log2p, int n_pages) {
  const int page = slot >> log2p;
  return page < n_pages ? max(page, -1) : -1;
}

// The nearest token from `from` on (step 1) or back from it (step -1) that has a page; -1 if there is none. For the
// whole CTA; `found` is two shared words. Out of line: it is seldom called, and the kernel keeps its registers.
__device__ __noinline__ int seek(const int* slot, int T, int log2p, int n_pages, int from, int step, int* found) {
  const int left = step > 0 ? T - from : from + 1;  // tokens to look through
  __syncthreads();  // the words are read no more from a call before
  if (threadIdx.x < 2) found[threadIdx.x] = INT_MAX;
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i * kSeek * kThreads < left; ++i) {
    int best = INT_MAX;
#pragma unroll
    for (int u = kSeek - 1; u >= 0; --u) {
      const int d = (i * kSeek + u) * kThreads + (int)threadIdx.x;
      if (d < left && page_of(slot[from + step * d], log2p, n_pages) >= 0) best = d;
    }
    best = __reduce_min_sync(~0u, best);
    if ((threadIdx.x & 31) == 0 && best != INT_MAX) atomicMin(&found[i & 1], best);
    __syncthreads();
    const int d = found[i & 1];  // the other word is the next turn's
    if (d != INT_MAX) return from + step * d;
  }
  return -1;
}

// n rows from token t on, at consecutive slots of the page from offset `at`. D dims. A thread holds two tiles of 4 tokens x
// 8 dims: one place of k and of v, or, for pages of more than 256 tiles (BIG), two places of one of them. A barrier
// has to follow before shared memory or the page is used again.
template <typename X, typename Row, int D, bool BIG>
__device__ __forceinline__ void take_run(const AppendParams& p, int t, int n, int page, int at, unsigned (*sm_max)[kThreads / 32]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = 1 << p.log2p;
  const int owners = BIG ? kThreads : (P / 4) * (D / 8);  // threads of one (page, head): whole warps
  const int sub = tid / owners, tile0 = tid - sub * owners;
  const int unit = blockIdx.y * (kThreads / owners) + sub;  // head; BIG: k's heads, then v's
  const bool mine = unit < (BIG ? 2 : 1) * p.n_kv;
  const int big_v = BIG && unit >= p.n_kv, h = big_v ? unit - p.n_kv : unit;
  // this thread's values of the page and the largest of all
  Row rows[2][4];
  unsigned top[2];
  float old[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool v = BIG ? big_v : i == 1;
    const long long xs = v ? p.xs[1] : p.xs[0];
    const X* x = static_cast<const X*>(v ? p.x[1] : p.x[0]) + t * xs + (long long)h * D;
    const int tile = tile0 + (BIG ? i * kThreads : 0), d = tile % (D / 8) * 8, j0 = tile / (D / 8) * 4 - at;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (mine && j0 + b >= 0 && j0 + b < n) load_row(rows[i][b], x + (j0 + b) * xs + d);
      else clear_row(rows[i][b]);
    }
    // a row at offset 0 starts the page afresh
    old[i] = mine && at ? (v ? p.scale[1] : p.scale[0])[(long long)page * p.n_kv + h] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    top[i] = max(max(top_of(rows[i][0]), top_of(rows[i][1])), max(top_of(rows[i][2]), top_of(rows[i][3])));
    top[i] = __reduce_max_sync(~0u, top[i]);
    if (lane == 0) sm_max[i][warp] = top[i];
  }
  __syncthreads();  // also: every thread has read the old scales
  for (int i = 0; i < owners / 32; ++i) {
    top[0] = max(top[0], sm_max[0][sub * (owners / 32) + i]);
    top[1] = max(top[1], sm_max[1][sub * (owners / 32) + i]);
  }
  if (BIG) top[0] = top[1] = max(top[0], top[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool v = BIG ? big_v : i == 1;
    const unsigned ex = top[i] >> 23;
    float need = top[i] == 0 ? 0.f : __uint_as_float((ex > 6 ? ex - 6 : 1u) << 23);  // never below 2^-126
    if (ex == 0xFF) need = __uint_as_float(0x7FC00000u);
    const bool broken = old[i] != old[i] || need != need;
    const float now = broken ? __uint_as_float(0x7FC00000u) : fmaxf(old[i], need);
    const float inv = broken || now == 0.f ? 0.f : __uint_as_float((254u - (__float_as_uint(now) >> 23)) << 23);
    int shift = 0;
    if (!broken && old[i] > 0.f && now > old[i])
      shift = min((int)(__float_as_uint(now) >> 23) - (int)(__float_as_uint(old[i]) >> 23), 7);
    if (mine && tile0 == 0 && !(BIG && i == 1)) (v ? p.scale[1] : p.scale[0])[(long long)page * p.n_kv + h] = now;
    const int tile = tile0 + (BIG ? i * kThreads : 0), e = tile % (D / 8), quad = tile / (D / 8), j0 = quad * 4 - at;
    unsigned in = 0;  // which of the four tokens are the run's
#pragma unroll
    for (int b = 0; b < 4; ++b) in |= (j0 + b >= 0 && j0 + b < n ? 1u : 0u) << b;
    if (!mine || (in == 0 && shift == 0)) continue;
    uint32_t c[4][8];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      float val[8];
      values(val, rows[i][b]);
#pragma unroll
      for (int k = 0; k < 8; ++k) c[b][k] = code(val[k], inv);
    }
    // (group of 16 tokens, 32 dims, word of 4 tokens or of 4 dims): see kv8.cuh
    int8_t* base = (v ? p.codes[1] : p.codes[0]) + ((long long)page * p.n_kv + h) * P * D + (quad >> 2) * 16 * D + (e >> 2) * 512;
    // k: words (2 o + k') of tokens o, o + 2 (adjacent), dims 8 e + 4 k'; v: words k of dim 8 e + k
    int8_t* k_at = base + (quad & 3) * 128 + (e & 1) * 32 + (e >> 1 & 1) * 8;
    int8_t* v_at = base + (quad & 3) * 16 + (e >> 1 & 1) * 8 + (e & 1) * 4;
    if (in == 15u) {  // whole words, whatever stood there
      if (!v) {
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<uint2*>(k_at + o * 64 + k * 16) =
                make_uint2(pack4(c[o][4 * k], c[o][4 * k + 1], c[o][4 * k + 2], c[o][4 * k + 3]),
                           pack4(c[o + 2][4 * k], c[o + 2][4 * k + 1], c[o + 2][4 * k + 2], c[o + 2][4 * k + 3]));
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) *reinterpret_cast<uint32_t*>(v_at + k * 64) = pack4(c[0][k], c[1][k], c[2][k], c[3][k]);
      }
    } else if (!v) {
#pragma unroll
      for (int o = 0; o < 4; ++o)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t* dst = reinterpret_cast<uint32_t*>(k_at + (o & 1) * 64 + k * 16 + (o >> 1) * 4);
          if (in >> o & 1) *dst = pack4(c[o][4 * k], c[o][4 * k + 1], c[o][4 * k + 2], c[o][4 * k + 3]);
          else if (shift) *dst = shift_bytes(*dst, shift);
        }
    } else {
      const uint32_t in4 = (in & 1 ? 0xFFu : 0u) | (in & 2 ? 0xFF00u : 0u) | (in & 4 ? 0xFF0000u : 0u) | (in & 8 ? 0xFF000000u : 0u);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t word = pack4(c[0][k], c[1][k], c[2][k], c[3][k]);
        uint32_t* dst = reinterpret_cast<uint32_t*>(v_at + k * 64);
        if (shift) {
          *dst = (shift_bytes(*dst, shift) & ~in4) | (word & in4);
        } else {
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (in >> b & 1) reinterpret_cast<uint8_t*>(dst)[b] = (uint8_t)(word >> (8 * b));
        }
      }
    }
  }
}

template <typename X, typename Row, int D, bool BIG>
__global__ void __launch_bounds__(kThreads, sizeof(Row) == 16 ? 4 : 2) kv8_append_kernel(const AppendParams p) {
  __shared__ unsigned sm_max[2][kThreads / 32], sm_lead[4], sm_ends[8];
  __shared__ int sm_slot[257];  // slots from token t0 - 1 to range + P - 1 behind t0
  __shared__ int sm_found[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = 1 << p.log2p;
  grid_dependency_wait();
  const int t0 = blockIdx.x * p.range, nt = min(p.range, p.T - t0);  // range <= 128
  for (int i = tid; i <= p.range + P; i += kThreads) {
    const int t = t0 - 1 + i;
    sm_slot[i] = t >= 0 && t < p.T ? p.slot[t] : -1;
  }
  __syncthreads();
  // the runs that begin in this CTA's tokens; the tokens where rows at consecutive slots end
  {
    const int s = sm_slot[1 + min(tid, p.range + P - 2)], before = sm_slot[min(tid, p.range + P - 2)];
    const bool follows = s >= 0 && before == s - 1 && (s & (P - 1)) != 0;
    bool lead = false;
    if (tid < nt && s >= 0) {
      const bool inside = (s >> p.log2p) < p.n_pages;
      if (!inside) atomicOr(&g_kv8_append_errors, 2u);
      lead = inside && !follows && before >> p.log2p != s >> p.log2p;
    }
    const unsigned leads = __ballot_sync(~0u, lead), ends = __ballot_sync(~0u, !follows);
    if (lane == 0) {
      if (warp < 4) sm_lead[warp] = leads;
      sm_ends[warp] = ends;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
#pragma unroll 1
    for (unsigned bits = sm_lead[q]; bits; bits &= bits - 1) {
      const int at_token = 32 * q + __ffs(bits) - 1;
      const int s0 = sm_slot[1 + at_token], page = s0 >> p.log2p;
      int t = t0 + at_token, at = s0 & (P - 1);
      // rows in a row, up to the page's end: to the first token that does not follow
      int n = min(P - at, p.T - t);
      for (int i = (at_token + 1) >> 5, from = (at_token + 1) & 31; i < 8 && 32 * i < at_token + n; ++i, from = 0) {
        const unsigned e = sm_ends[i] >> from << from;
        if (e) {
          n = min(n, 32 * i + __ffs(e) - 1 - at_token);
          break;
        }
      }
      // it may go on where a skipped row comes next, or another slot of the page
      const int next = page_of(sm_slot[1 + at_token + n], p.log2p, p.n_pages);
      bool open = t + n < p.T && (next < 0 || next == page);
#pragma unroll 1
      for (int look = t > 0 && page_of(sm_slot[at_token], p.log2p, p.n_pages) < 0 ? -1 : 0;; look = 1) {
        if (look) {  // behind skipped rows: does the page's run begin before them? at its end: does it go on behind them?
          const int u = seek(p.slot, p.T, p.log2p, p.n_pages, look < 0 ? t - 1 : t + n, look, sm_found), s = u < 0 ? -1 : p.slot[u];
          if ((s >> p.log2p == page) == (look < 0)) break;
          if (look > 0) {
            t = u;
            at = s & (P - 1);
            n = 1;
            open = t + 1 < p.T;
          }
        }
        take_run<X, Row, D, BIG>(p, t, n, page, at, sm_max);
        __syncthreads();  // the shared words are used again; the page's scale and codes are read again
        if (!open) break;
      }
    }
  }
}

template <typename X, typename Row>
int launch_typed(const AppendParams& p, int D, dim3 grid, bool two, cudaStream_t s, std::string* err) {
  if (two) return launch_pdl(kv8_append_kernel<X, Row, 128, true>, grid, dim3(kThreads), 0, s, p, "kv8_append", err);
  return D == 64 ? launch_pdl(kv8_append_kernel<X, Row, 64, false>, grid, dim3(kThreads), 0, s, p, "kv8_append", err)
                 : launch_pdl(kv8_append_kernel<X, Row, 128, false>, grid, dim3(kThreads), 0, s, p, "kv8_append", err);
}

}  // namespace

unsigned int take_kv8_append_errors() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv8_append_errors, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (cudaMemcpyToSymbol(g_kv8_append_errors, &zero, sizeof(zero)) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
}

int launch_kv8_append(const KV8Args& c, int x_dtype, const void* k, long long ks, const void* v, long long vs,
                      const int* slot, int T, int num_sms, cudaStream_t s, std::string* err) {
  AppendParams p = {};
  p.x[0] = k;
  p.x[1] = v;
  p.xs[0] = ks;
  p.xs[1] = vs;
  p.codes[0] = c.k;
  p.codes[1] = c.v;
  p.scale[0] = c.k_scale;
  p.scale[1] = c.v_scale;
  p.slot = slot;
  p.T = T;
  p.log2p = c.log2p;
  p.n_pages = c.n_pages;
  p.n_kv = c.n_kv;
  // tokens per CTA: one while the grid is small (runs are short: single tokens in parallel), up to a page
  const int tiles = (1 << c.log2p) / 4 * (c.D / 8), heads = tiles < kThreads ? kThreads / tiles : 1;
  const bool two = tiles > kThreads;  // pages of 128 tokens of 128 dims
  const unsigned gy = two ? 2u * c.n_kv : (unsigned)((c.n_kv + heads - 1) / heads);
  const long long range = (long long)T * gy / ((long long)num_sms * 8);
  p.range = (int)(range < 1 ? 1 : range > (1 << c.log2p) ? (1 << c.log2p) : range);
  const dim3 grid((unsigned)((T + p.range - 1) / p.range), gy);
  return x_dtype == KQ_F32 ? launch_typed<float, RowF32>(p, c.D, grid, two, s, err)
                           : launch_typed<uint16_t, RowBf16>(p, c.D, grid, two, s, err);
}

}  // namespace kq
