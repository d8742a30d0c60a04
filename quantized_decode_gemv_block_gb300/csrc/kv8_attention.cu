// Attention over the paged 8-bit KV cache: single tokens, verify windows and prompts of a batch
// of requests of uneven length, grouped-query heads.
//
//   o = sum_p w_p v_p / sum_p w_p,  w_p = 2^(x_p - r),  x_p = log2(e) scale q.k_p
// over the positions p that the row sees; r is a reference that follows the row's largest x_p.
// k_p = (c + 1/2) s with int8 codes c and one scale s per (page, kv head), so q.k_p =
// s (q.c + sum(q) / 2), and v's halves add sum_p w_p s_p / 2 to every dim: the tensor cores multiply
// the codes alone, exact in fp16 (a LOP3 and a subtraction per pair; the cache's byte order is that of
// the MMA operands, see kv8.cuh).
//
// Precision. q is scaled per row by the power of two that puts its largest value in [2^14, 2^15)
// and rounded to fp16: exact for bf16 values within 2^-28 of the row's largest. fp32 queries, and all of them where
// the output is fp32, are split into fp16 hi + lo parts (QP = 2, 22 bits): rounded to one they would move a score by
// 2^-12 of sum_d |scale q_d k_d|, and the weights by as much, which passes a bf16 output's 2^-9 from scores of 8 on. The
// second part costs, with bf16 outputs, 84 -> 92 us for 16 requests x 8 tokens over 1000 to 9000 positions in pages of 32, 94 -> 105
// for 64 tokens over 1 to 8191, 374 -> 435 for 2 x 2048 (32 / 8 heads of 128), 10.2 -> 11.2 for one token over 4096 (16 / 4 heads).
// Weights are one fp16 part (2^-12 of themselves) for bf16 outputs, two (WP = 2) for fp32 ones. The weights that enter a product are those against the largest score of
// their page (of up to 32 positions of it), up by 2^15: fp16 then holds weights down to 2^-29 of that in
// full, and an absolute 2^-40 below. The accumulators take the page's share of the softmax and its v scale
// in fp32, so pages whose scales lie far apart lose nothing to one another. Weight sums are products with
// ones, of the same rounded weights. References, sums and outputs are fp32.
//
// Products, on mma.sync.m16n8k16 with the codes converted in registers (the codes would have to be
// written to shared memory twice as wide to reach tcgen05, and a few query rows leave its 128-row
// operand empty). Up to 8 query rows per kv head: the cache is the A operand, S^T = K q^T and
// O^T = V^T w^T, 16 tokens (or dims) by 8 rows, so that a lone token's few rows pad to 8 and not to
// 16; the weights turn from accumulators into the B operand by one movmatrix per 8x8 block. More rows
// (R16): the rows are the A operand, 16 at a time, and the weights become operands where they stand.
// With 16 rows in the first form (two blocks of 8) a batch of windows of 32 rows of 64 took 48.7 us
// in place of 41, and 32 rows at a time 79.
//
// Work. The positions of a request are cut into segments, where they end being a matter of the position alone: 64 of
// 512 (256 for one or two kv heads), then 32 of each doubled size; and they are joined in an order that their number
// does not change. So a row's bits depend on its own request alone, and not on the tokens behind it. An item is
// (request, block of rows, segment, kv head). A persistent grid walks the items; each CTA finds them in prefix sums
// that it forms itself from the lengths on the device, so the host plans nothing and the call can be captured. In a
// CTA four warps multiply and a fifth copies: it reads page ids and scales 512 positions at a time and fills a ring
// of slots, each a step of 128 positions of K or of V, by bulk copies of whole pages, across items. Each of the four
// takes 32 positions of a step through both products alone, and they meet in shared memory once per item. A request
// of one segment writes its output there; others write partials that a second kernel joins.
//   Windows of more than 32 tokens (prompts) run in a launch of their own, where max_new allows them: blocks of 64
// rows, 16 for each warp, which takes its rows over all positions and writes them alone. Over contexts from 4096
// positions on a request is cut so that it alone gives every CTA one item, or two where that comes out more even.
// One request over 131k positions, 32 / 8 heads of 128: 395 us for 32 tokens, 511 for 33, 648 for 64, 2388 for 200
// (616, 761 and 3012 with 32 items per kv head, 530, 678 and 2421 with 76, each rounded up to 512 positions); 4 / 1
// heads: 79 us for 33. What it costs: 16 requests of 64 tokens over 6000 positions, which fill the machine
// together, 614 us in place of 566. In the windows' form 2 x 2048 tokens took 437 us in place of 368, 38 requests
// of 155 to 311 tokens (fp32, 16 / 8 heads) 221 in place of 163. Codes converted once for all warps into shared
// memory: with 8 warps and 128 rows 374 and 198 us, with 4 warps 393 and 198 us; the barriers cost more than the
// conversions.
// Measured on the way: a CTA of four warps with nothing copied ahead across items 168 us on the decoding batch below;
// warps that share the second product by dims, with a barrier per step, 177 us; each warp with items and a ring of
// its own 112 to 132 us (its copies' and its items' bookkeeping weighed as much as its products); the fifth warp 100
// us. Segments of 256 positions 115 us and of 1024 100 us; one token over 4096 positions 9.6, 10.4 and 14.4 us with
// segments of 256, 512 and 1024 (queries of one part). Few heads leave CTAs idle, so that short segments win: one token over 4096
// positions, 16 / 2 heads, 8.7 us with segments of 256 (11.4 with 512); 63 tokens over 1030 to 2060, 2 / 1 heads of
// 64, 12 us (20); the other side, 64 tokens over 1 to 8191, 8 / 2 heads, 36.7 (35.4), and with four heads 62 (57).
//
// Bound by DRAM for single tokens: 64 requests of 1 to 8191 positions, 32 / 8 heads of 128, 543 MB in
// 98.4 us, 5.5 TB/s, of which 5 us are the join and about 10 the start and the end; four contexts of 128k
// positions 168 us, 6.2 TB/s (of 6.79 copied). Windows and prompts are bound by the multiplying warps'
// latency (two or three of them per scheduler): the conversions, the softmax and the products follow one
// another in each, 92 us for 16 requests x 8 tokens x 4 heads per kv head of 128 over 1000 to 9000
// positions, 178 MB, and 175 to 210 TFLOP/s for prompts.
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

constexpr int kWarps = 4;                          // warps that multiply; one more brings the codes
constexpr int kMath = 32 * kWarps, kThreads = kMath + 32;
constexpr int kWarpPos = 32, kStep = kWarps * kWarpPos;  // positions of a step, 32 per warp
constexpr int kSegLog2 = 9, kFewSegLog2 = 8;             // positions of a segment at least; for few kv heads
constexpr int kWindow = 32 * 16 / kStep;                 // steps whose page ids are read at once, a group of 16 tokens per lane
constexpr int kSplitTokens = 32;                         // windows up to this many tokens are cut as above
constexpr int kPromptRows = 64;                          // query rows of an item of larger windows (prompts)
constexpr int kFewHeads = 2;                             // kv heads that are few
constexpr int kLongContext = 4096, kShortest = 512;      // prompts over at least so many positions are cut; into at least so many
constexpr int kWaves = 2;                                // items per CTA that a prompt alone is cut into at most
constexpr float kLowest = -3e38f;  // below every finite score in use: keeps -inf out of differences
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kCombThreads = 256;

__device__ unsigned int g_kv8_errors = 0;  // bit 0: a bounded wait gave up; bit 1: bad lengths or page ids

// How a request's positions are cut: a function of its own lengths and the heads.
struct Cut {
  int len, count;  // positions of a segment (multiples of a step; 0: those of a window), segments
};
struct Cutter {
  int group, n_kv, seg_log2, wave;  // query heads per kv head; kv heads; windows' shortest segments; prompts' CTAs at once
  __host__ __device__ Cut operator()(int len, int n) const {
    if (n <= kSplitTokens) {
      const int u = len - 1, over = u >> (seg_log2 + 6);
      if (over == 0) return {0, (u >> seg_log2) + 1};
      int j = 0;  // floor(log2(over))
#ifdef __CUDA_ARCH__
      j = 31 - __clz(over);
#else
      while (over >> (j + 1)) ++j;
#endif
      return {0, 64 + 32 * j + (((u >> (seg_log2 + j)) - 64) >> 1) + 1};
    }
    // as many segments as give all CTAs one item, or two where that shares the work out better by 5 %
    const Cut whole = {1 << 29, 1};
    const int blocks = (n * group + kPromptRows - 1) / kPromptRows;
    if (len < kLongContext || blocks >= kWaves * wave) return whole;
    const int items = blocks * n_kv, two = kWaves * wave / items;
    int count = wave / items;
    if (20 * two > 21 * kWaves * count) count = two;
    count = count < len / kShortest ? count : len / kShortest;
    if (count <= 1) return whole;
    const int size = ((len + count - 1) / count + kStep - 1) / kStep * kStep;
    return {size, (len + size - 1) / size};
  }
  // Where a segment begins: in windows at a position of its own, whatever the length: 64 segments of the shortest, then
  // 32 of each doubled size.
  __host__ __device__ int begin(const Cut& c, int seg) const {
    if (c.len) return seg * c.len;
    if (seg < 64) return seg << seg_log2;
    const int t = seg - 64;
    return (64 + ((t & 31) << 1)) << (seg_log2 + (t >> 5));
  }
};
Cutter cutter_of(int n_kv, int group, int D) {
  return {group, n_kv, n_kv <= kFewHeads ? kFewSegLog2 : kSegLog2, 152 * (D == 64 ? 3 : 2)};
}

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
  Cutter cut;
  unsigned group_inv;  // 2^32 / group rounded up; 0 for a group of one
  float scale_log2e;
  float* part;          // a request's partial rows: [kv head][segment][row][D]
  float2* part_ml;      // [kv head][segment][row]: reference, sum of weights
  long long part_rows;  // room per kv head
};

// Warps that share a row of the combine: 8 segments each, and up to 8 warps.
__host__ __device__ constexpr int combine_warps(int nseg) { return nseg <= 8 ? 1 : nseg <= 16 ? 2 : nseg <= 32 ? 4 : 8; }

// row / group for rows below 2^26 (group <= 64): row * (group * group_inv - 2^32) < 2^32.
__device__ __forceinline__ int token_of(const AttnKV8Params& p, int row) { return p.group_inv ? (int)__umulhi((unsigned)row, p.group_inv) : row; }

// A request whose lengths do not fit the call's bounds takes no part.
__device__ __forceinline__ bool request_ok(const AttnKV8Params& p, int c, int n) {
  return c >= 0 && n >= 0 && n <= p.max_new && c <= p.max_len - n && (p.mask == nullptr || n <= kSplitTokens) &&
         ((c + n + (1 << p.log2p) - 1) >> p.log2p) <= p.max_blocks;
}

// The requests in shared memory: each one's first token, work item and partial row, and its cached
// length. Items: windows of up to 32 tokens (kWindows), larger ones (kPrompts), or CTA tasks of the combine.
enum Kind { kWindows, kPrompts, kCombine };
struct Request {
  int tok, item, ctx;
  long long part;
};
template <int THREADS, Kind KIND>
__device__ __forceinline__ void scan_requests(const AttnKV8Params& p, int row_block, Request* req, long long* sm) {
  constexpr int W = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int per = (p.B + THREADS - 1) / THREADS, r0 = min(tid * per, p.B), r1 = min(r0 + per, p.B);  // this thread's requests
  long long a = 0, c = 0;  // sums within them, then before them
  int b = 0;
  bool bad = false;
#pragma unroll 2
  for (int r = r0; r < r1; ++r) {
    const int n = p.fresh[r], ctx = p.ctx[r];
    req[r] = {(int)min(a, (long long)INT_MAX), b, ctx, c};
    a += n > 0 ? n : 0;
    if (!request_ok(p, ctx, n)) bad = true;
    else if (n > 0) {
      const int nseg = p.cut(ctx + n, n).count, rows = n * p.group;
      if (KIND != kCombine) b += (n <= kSplitTokens) == (KIND == kWindows) ? (rows + row_block - 1) / row_block * nseg : 0;
      else b += nseg <= 1 ? 0 : (rows * p.n_kv * combine_warps(nseg) + W - 1) / W;
      c += nseg > 1 ? (long long)nseg * rows : 0;
    }
  }
  const long long a0 = a, c0 = c;
  const int b0 = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long xa = __shfl_up_sync(~0u, a, o), xc = __shfl_up_sync(~0u, c, o);
    const int xb = __shfl_up_sync(~0u, b, o);
    if (lane >= o) {
      a += xa;
      b += xb;
      c += xc;
    }
  }
  if (lane == 31) {
    sm[w] = a;
    sm[W + w] = b;
    sm[2 * W + w] = c;
  }
  __syncthreads();
  long long ct = 0;
  int ci = 0;
  a -= a0;
  b -= b0;
  c -= c0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (i < w) {
      a += sm[i];
      b += (int)sm[W + i];
      c += sm[2 * W + i];
    }
    ct += sm[i];
    ci += (int)sm[W + i];
  }
  for (int r = r0; r < r1; ++r) {
    req[r].tok = (int)min(a + req[r].tok, (long long)INT_MAX);
    req[r].item += b;
    req[r].part += c;
  }
  // more tokens than q has rows, or too many items: nothing is done
  const bool over = ct > p.T || (long long)ci * p.n_kv > INT_MAX;
  if (tid == 0) req[p.B] = {(int)min(ct, (long long)INT_MAX), over ? 0 : ci, 0, 0};
  if (KIND != kCombine && (bad || over)) atomicOr(&g_kv8_errors, 2u);
  __syncthreads();
}

__device__ __forceinline__ int find_request(const Request* req, int B, int item) {  // the last r that starts at or before it
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (req[mid].item <= item) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// Four int8 codes -> the fp16 pairs (0, 2) and (1, 3): c + 128 under the byte 0x64 is 1152 + c - 128 in
// fp16 (1024 + u), one LOP3 per pair ((w & mask) ^ bits), minus 1152.
__device__ __forceinline__ void codes_to_h2(uint32_t w, uint32_t& even, uint32_t& odd) {
  uint32_t e, o;
  asm("lop3.b32 %0, %1, 0x00FF00FF, 0x64806480, 0x6A;" : "=r"(e) : "r"(w));
  asm("lop3.b32 %0, %1, 0x00FF00FF, 0x64806480, 0x6A;" : "=r"(o) : "r"(w >> 8));
  even = h2_sub(e, 0x64806480u);
  odd = h2_sub(o, 0x64806480u);
}
// Tokens (4 t, 4 t + 1) and (4 t + 2, 4 t + 3) of a row -> the pairs that codes_to_h2 makes.
__device__ __forceinline__ void weight_operand(uint32_t (&b)[4], uint32_t lo, uint32_t hi) {
  b[0] = prmt(lo, hi, 0x5410);
  b[1] = prmt(lo, hi, 0x7632);
  b[2] = b[3] = 0u;
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Largest over the lanes that hold one query row: eight for 8 rows, four for 16.
template <bool R16>
__device__ __forceinline__ float max_over_row(float v) {
#pragma unroll
  for (int x = R16 ? 1 : 4; x < (R16 ? 4 : 32); x <<= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, x));
  return v;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// The warps that multiply, without the one that copies.
__device__ __forceinline__ void math_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kMath) : "memory"); }

// Shared memory of a CTA: a ring of slots (a step's K or its V), the warps' outputs of an item, for 16
// query rows the item's query operands, the requests.
enum Form { kRows8, kRows16, kPrompt };
template <int D, Form FORM, int QP>
struct AttnSmem {
  static constexpr int RB = FORM == kPrompt ? kPromptRows : FORM == kRows16 ? 16 : 8;
  static constexpr int kDepth = D == 64 ? 6 : FORM == kPrompt ? 4 : 3;
  static constexpr int kSlot = kStep * D;
  static constexpr int kOut = kDepth * kSlot;                                            // [warp][RB][D + 4] floats
  static constexpr int kOutWarp = FORM == kPrompt ? 0 : RB * (D + 4);
  static constexpr int kQ = kOut + kWarps * kOutWarp * 4;                                // [part][D / 16][32 lanes][4 words]
  static constexpr int kQPart = FORM == kRows8 ? 0 : D / 16 * 512;
  static constexpr int kReq = kQ + (FORM == kPrompt ? kWarps : 1) * QP * kQPart;         // prompts: for each warp
  static constexpr size_t bytes(int B) { return kReq + (size_t)(B + 1) * sizeof(Request); }
};

struct Item {  // (request, kv head, block of query rows, segment)
  int r, h, row0, rows, seg, nseg, ctx, len, tok0;
  long long part;
  int step0, step1, end, seen;  // steps of kStep; positions from `end` on are seen by no row, those below `seen` by all
};

// kRows8: 8 query rows as the B operand (rows 2 t4, 2 t4 + 1 in a lane); the others: 16 as the A operand (rows
// g, g + 8). kRows8 and kRows16 give a row the same bits: every sum over dims, positions or lanes is the
// tensor cores' own, in the same order of k. kPrompt: windows of more than 32 tokens, 64 rows an item, 16 for
// each warp over all positions of a step, so that nothing is joined at the end. QP, WP: fp16 parts of queries and weights.
template <int D, Form FORM, int QP, int WP>
__global__ void __launch_bounds__(kThreads, FORM == kRows8 ? (D == 64 ? 4 : 3) : D == 64 ? 3 : 2) attn_kv8_kernel(const AttnKV8Params p) {
  constexpr bool R16 = FORM != kRows8, PR = FORM == kPrompt;
  using S = AttnSmem<D, FORM, QP>;
  constexpr int RB = S::RB, C32 = D / 32, K16 = D / 16, DEPTH = S::kDepth;
  constexpr int NV = R16 ? 4 : 2;              // scores of a row per lane and group of 16 tokens
  constexpr int NO = R16 ? 2 * K16 : K16;      // output tiles: 8 dims by 16 rows, or 16 dims by 8 rows
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t sm_full[DEPTH], sm_empty[DEPTH];
  __shared__ __align__(16) float sm_scale[4][2][kStep / 16];  // [step & 3][k, v][group]
  __shared__ long long sm_scan[3 * (kThreads / 32)];
  __shared__ __align__(16) float sm_hq[RB];  // written in pairs
  __shared__ float sm_rf[RB];
  __shared__ float sm_m[kWarps][PR ? 1 : RB], sm_l[kWarps][PR ? 1 : RB], sm_h[kWarps][PR ? 1 : RB];
  __shared__ int sm_lim[RB];
  __shared__ uint32_t sm_mask[RB];
  Request* req = reinterpret_cast<Request*>(smem + S::kReq);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int wrow = PR ? 16 * w : 0;  // the warp's first row of the item
  uint32_t* sm_q = reinterpret_cast<uint32_t*>(smem + S::kQ) + (PR ? w * QP * (S::kQPart / 4) : 0);
  if (tid == 0) {
    for (int k = 0; k < DEPTH; ++k) {
      mbar_init(&sm_full[k], 1);
      mbar_init(&sm_empty[k], kWarps);
    }
    fence_mbar_init();
  }
  grid_dependency_wait();
  scan_requests<kThreads, PR ? kPrompts : kWindows>(p, RB, req, sm_scan);
  grid_launch_dependents();
  const int total = req[p.B].item, P = 1 << p.log2p;
  // items x kv heads, a CTA's shares gridDim.x apart: (item, head) moves by (d_item, d_head)
  const int d_item = gridDim.x / p.n_kv, d_head = gridDim.x - d_item * p.n_kv;
  struct Place {
    int item, head;
  };
  const Place place0 = {(int)blockIdx.x / p.n_kv, (int)blockIdx.x % p.n_kv};
  auto move = [&](Place& at) {
    at.item += d_item;
    at.head += d_head;
    if (at.head >= p.n_kv) {
      at.head -= p.n_kv;
      ++at.item;
    }
  };

  auto item_of = [&](Place at) {
    Item x;
    x.h = at.head;
    x.r = find_request(req, p.B, at.item);
    const Request q = req[x.r];
    x.tok0 = q.tok;
    x.ctx = q.ctx;
    x.part = q.part;
    const int n = req[x.r + 1].tok - q.tok;
    x.len = q.ctx + n;
    x.rows = n * p.group;
    const Cut cut = p.cut(x.len, n);
    x.nseg = cut.count;
    int local = at.item - q.item, rb = 0;
    if (local >= x.nseg) {
      rb = local / x.nseg;
      local -= rb * x.nseg;
    }
    x.seg = local;
    x.row0 = rb * RB;
    x.end = p.mask || n == 1 ? x.len : x.ctx + token_of(p, min(x.row0 + RB, x.rows) - 1) + 1;
    x.seen = x.ctx + (p.mask ? 0 : token_of(p, x.row0) + 1);
    const int last = (x.end + kStep - 1) / kStep;
    static_assert((1 << kFewSegLog2) % kStep == 0 && kFewSegLog2 <= kSegLog2, "segments are cut into steps");
    x.step0 = p.cut.begin(cut, x.seg) / kStep;
    x.step1 = min(p.cut.begin(cut, x.seg + 1) / kStep, last);
    return x;
  };

  bool dead = false;
  auto wait = [&](uint64_t* bar, uint32_t phase) {
    if (!dead && !mbar_wait_bounded(bar, phase, kWaitNs)) dead = true;
  };
  int slot = 0;
  uint32_t phase = 0;
  auto next_slot = [&]() {
    if (++slot == DEPTH) {
      slot = 0;
      phase ^= 1;
    }
  };

  // ---- the last warp runs ahead over the CTA's steps, across its items, and fills the ring
  if (w == kWarps) {
    const int per = P >> 4, chunks = kStep >> p.log2p;  // groups of a page; pages of a step
    int steps = 0;
    for (Place at = place0; at.item < total; move(at)) {
      const Item x = item_of(at);
      for (int s0 = x.step0; s0 < x.step1; s0 += kWindow) {
        // page id and scales of this lane's group of 16 tokens; also of groups past the end of a page
        // that holds positions: its scale is theirs
        const int pos = s0 * kStep + 16 * lane;
        int page = -1;
        float ks = 0.f, vs = 0.f;
        if ((pos & -P) < x.end) {
          page = p.table[(long long)x.r * p.max_blocks + (pos >> p.log2p)];
          if ((unsigned)page < (unsigned)p.n_pages) {
            const long long sc = (long long)page * p.n_kv + x.h;
            ks = p.ks[sc];
            vs = p.vs[sc];
          } else {  // no page of this cache: nothing is copied, the rows that see it come out NaN
            page = -1;
            ks = vs = __uint_as_float(0x7FC00000u);
            atomicOr(&g_kv8_errors, 2u);
          }
        }
        const int n = min(kWindow, x.step1 - s0);
        for (int j = 0; j < n; ++j, ++steps) {
          const int c = lane < chunks ? lane : 0;  // lane c copies the step's c-th page
          const int c_page = __shfl_sync(~0u, page, 8 * j + c * per);
          const int left = x.end - ((s0 + j) * kStep + (c << p.log2p));
          const unsigned bytes = lane < chunks && c_page >= 0 && left > 0 ? min(per, (left + 15) >> 4) * 16 * D : 0;
          const unsigned all = __reduce_add_sync(~0u, bytes);
          const long long off = (((long long)c_page * p.n_kv + x.h) << p.log2p) * D;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            wait(&sm_empty[slot], phase ^ 1);
            if (half == 0 && (lane >> 3) == j) {
              sm_scale[steps & 3][0][lane & 7] = ks;
              sm_scale[steps & 3][1][lane & 7] = vs;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&sm_full[slot], all);
            __syncwarp();
            if (bytes) bulk_g2s(smem + slot * S::kSlot + (c << p.log2p) * D, (half ? p.vc : p.kc) + off, bytes, &sm_full[slot]);
            next_slot();
          }
        }
      }
    }
    if (dead && lane == 0) atomicOr(&g_kv8_errors, 1u);
    return;
  }

  auto free_slot = [&](int s) {  // its codes are used
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm_empty[s]);
  };
  int steps = 0;
  for (Place at = place0; at.item < total; move(at)) {
    const Item x = item_of(at);
    const int group = p.group;
    // ---- query operands: lane (g, t4) takes row g of a block of 8 at dims 16 s + 4 t4 .. + 3; rows past
    // the last are zeros that see nothing. 8 rows: each warp for itself, in registers; 16: warps 0 and 1
    // for all, in shared memory
    uint2 qh[R16 ? 1 : K16], ql[!R16 && QP == 2 ? K16 : 1];
    float hq[2], rf[2];
    int lim[2];
    uint32_t see[2];
#pragma unroll 1
    for (int nt = R16 && !PR ? w : 0; nt < (R16 ? 2 : 1); nt += R16 && !PR ? kWarps : 1) {
      const int row = x.row0 + wrow + 8 * nt + g, ti = token_of(p, row);
      const bool live = row < x.rows;
      float v[K16][4];
      const long long from = (x.tok0 + ti) * p.qs + (long long)(x.h * group + row - ti * group) * D + 4 * t4;
      if (p.q_f32) {
        const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + from);
#pragma unroll
        for (int s = 0; s < K16; ++s) {
          const float4 q = live ? src[4 * s] : make_float4(0.f, 0.f, 0.f, 0.f);
          v[s][0] = q.x;
          v[s][1] = q.y;
          v[s][2] = q.z;
          v[s][3] = q.w;
        }
      } else {
        const uint2* src = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + from);
#pragma unroll
        for (int s = 0; s < K16; ++s) {
          const uint2 q = live ? src[4 * s] : make_uint2(0u, 0u);
          v[s][0] = __uint_as_float(q.x << 16);
          v[s][1] = __uint_as_float(q.x & 0xFFFF0000u);
          v[s][2] = __uint_as_float(q.y << 16);
          v[s][3] = __uint_as_float(q.y & 0xFFFF0000u);
        }
      }
      unsigned top = 0;
#pragma unroll
      for (int s = 0; s < K16; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(v[s][e]) & 0x7FFFFFFFu);
      top = max(top, __shfl_xor_sync(~0u, top, 1));
      top = max(top, __shfl_xor_sync(~0u, top, 2));
      // 2^e with the largest |q| 2^e in [2^14, 2^15); 1 for zero rows and for rows that are not finite
      const int ex = (int)(top >> 23);
      const int e2 = top == 0 || ex == 0xFF ? 0 : max(-126, min(126, 14 - (ex - 127)));
      const float up = __uint_as_float((unsigned)(127 + e2) << 23);
      const float factor = __uint_as_float((unsigned)(127 - e2) << 23) * p.scale_log2e;
      // half of each row's sum, as the products below add it up: the codes' + 1/2
      float half[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t halves[4] = {0x38003800u, 0x38003800u, 0x38003800u, 0x38003800u};
#pragma unroll
      for (int s = 0; s < K16; ++s) {
        const float f[4] = {v[s][0] * up, v[s][1] * up, v[s][2] * up, v[s][3] * up};
        const uint2 hi = make_uint2(f2_to_h2(f[0], f[2]), f2_to_h2(f[1], f[3]));
        mma_f16_16816(half, halves, hi.x, hi.y, half);
        uint32_t* q16 = sm_q + (s * 32 + lane) * 4 + nt;  // rows g: words 0, 2; rows g + 8: words 1, 3
        if (R16) {
          q16[0] = hi.x;
          q16[2] = hi.y;
        } else {
          qh[R16 ? 0 : s] = hi;
        }
        if (QP == 2) {
          const uint2 lo = make_uint2(f2_to_h2(f[0] - h_lo_to_f(hi.x), f[2] - h_lo_to_f(hi.x >> 16)),
                                      f2_to_h2(f[1] - h_lo_to_f(hi.y), f[3] - h_lo_to_f(hi.y >> 16)));
          mma_f16_16816(half, halves, lo.x, lo.y, half);
          if (R16) {
            q16[S::kQPart / 4] = lo.x;
            q16[S::kQPart / 4 + 2] = lo.y;
          } else {
            ql[!R16 && QP == 2 ? s : 0] = lo;
          }
        }
      }
      const int last = live ? x.ctx + ti : -1;
      const uint32_t word = live && p.mask ? p.mask[x.tok0 + ti] : 0u;
      if (R16) {
        if (g == 0) *reinterpret_cast<float2*>(sm_hq + wrow + 8 * nt + 2 * t4) = make_float2(half[0], half[1]);
        if (t4 == 0) {
          sm_rf[wrow + 8 * nt + g] = factor;
          sm_lim[wrow + 8 * nt + g] = last;
          sm_mask[wrow + 8 * nt + g] = word;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          hq[k] = half[k];
          rf[k] = __shfl_sync(~0u, factor, 8 * t4 + 4 * k);
          lim[k] = __shfl_sync(~0u, last, 8 * t4 + 4 * k);
          see[k] = __shfl_sync(~0u, word, 8 * t4 + 4 * k);
        }
      }
    }
    if (R16) {
      if (PR) __syncwarp();
      else math_barrier();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        hq[k] = sm_hq[wrow + g + 8 * k];
        rf[k] = sm_rf[wrow + g + 8 * k];
        lim[k] = sm_lim[wrow + g + 8 * k];
        see[k] = sm_mask[wrow + g + 8 * k];
      }
    }

    // this lane's two rows: reference, sum of weights, sum of weights times v scales; output tiles
    float o[NO][4], m[2], l[2], hv[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      m[k] = -INFINITY;
      l[k] = hv[k] = 0.f;
    }
#pragma unroll
    for (int s = 0; s < NO; ++s) o[s][0] = o[s][1] = o[s][2] = o[s][3] = 0.f;

    // prompts: what this warp's rows see ends, and is seen by all of them, of its own
    const int w_end = PR ? x.ctx + token_of(p, max(min(x.row0 + wrow + 16, x.rows) - 1, 0)) + 1 : x.end;
    const int w_seen = PR ? x.ctx + token_of(p, x.row0 + wrow) + 1 : x.seen;
    for (int step = x.step0; step < x.step1; ++step, ++steps) {
      const int k_slot = slot;
      wait(&sm_full[slot], phase);
      next_slot();
      const int v_slot = slot;
      const uint32_t v_phase = phase;
      next_slot();
      if (PR) wait(&sm_full[v_slot], v_phase);
#pragma unroll 1
      for (int part32 = PR ? 0 : w; part32 < (PR ? kWarps : w + 1); ++part32) {  // 32 positions
      const int pos32 = step * kStep + part32 * kWarpPos;
      if (PR && (pos32 >= w_end || x.row0 + wrow >= x.rows)) break;
      const uint8_t* kst = smem + k_slot * S::kSlot + part32 * kWarpPos * D;
      // ---- scores: [group][R16: the group's token pairs 4 t, 4 t + 1 and 4 t + 2, 4 t + 3]
      float sc[2][R16 ? 2 : 1][4];
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int i = 0; i < (R16 ? 2 : 1); ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[st][i][e] = hq[R16 ? e >> 1 : e & 1];
      const float2 kf2 = lds_f2(&sm_scale[steps & 3][0][2 * part32]), vf2 = lds_f2(&sm_scale[steps & 3][1][2 * part32]);
      const float kf[2] = {kf2.x, kf2.y}, vf[2] = {vf2.x, vf2.y};
#pragma unroll
      for (int cc = 0; cc < C32; ++cc) {
        uint32_t qa[QP][2][4];
        if (R16) {
#pragma unroll
          for (int part = 0; part < QP; ++part)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint4 q = lds128(sm_q + part * (S::kQPart / 4) + ((2 * cc + i) * 32 + lane) * 4);
              qa[part][i][0] = q.x;
              qa[part][i][1] = q.y;
              qa[part][i][2] = q.z;
              qa[part][i][3] = q.w;
            }
        }
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          const uint4 k = lds128(kst + st * 16 * D + cc * 512 + lane * 16);
          uint32_t a[2][4];  // [16 dims][rows g, g + 8 of even pairs, then of odd ones]
          codes_to_h2(k.x, a[0][0], a[0][2]);
          codes_to_h2(k.y, a[0][1], a[0][3]);
          codes_to_h2(k.z, a[1][0], a[1][2]);
          codes_to_h2(k.w, a[1][1], a[1][3]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (R16) {
#pragma unroll
              for (int part = 0; part < QP; ++part) {
                mma_f16_16816(sc[st][0], qa[part][i], a[i][0], a[i][2], sc[st][0]);
                mma_f16_16816(sc[st][R16 ? 1 : 0], qa[part][i], a[i][1], a[i][3], sc[st][R16 ? 1 : 0]);
              }
            } else {
              const int s = R16 ? 0 : 2 * cc + i;
              mma_f16_16816(sc[st][0], a[i], qh[s].x, qh[s].y, sc[st][0]);
              if (QP == 2) mma_f16_16816(sc[st][0], a[i], ql[QP == 2 ? s : 0].x, ql[QP == 2 ? s : 0].y, sc[st][0]);
            }
          }
        }
      }
      if (!PR) free_slot(k_slot);
      // ---- weights against the page's largest score, up by 2^15 into fp16's range
      // value v of row k in group st is score sc[st][..] below, of position pos0 + 16 st + (R16 ? v : 2 v)
      const int pos0 = pos32 + (R16 ? 4 * t4 : 4 * (g >> 1) + (g & 1));
      float sv[2][2][NV];
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float r = rf[k] * kf[st];
#pragma unroll
          for (int v = 0; v < NV; ++v) sv[st][k][v] = r * (R16 ? sc[st][R16 ? v >> 1 : 0][2 * k + (v & 1)] : sc[st][0][k + 2 * (v & 1)]);
        }
      // all positions seen by every row: nothing to mask (rows past the last come along: nothing reads them)
      if (pos32 + kWarpPos > w_seen) {
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              const int pos = pos0 + 16 * st + (R16 ? v : 2 * v), j = pos - x.ctx;
              const bool sees = p.mask == nullptr ? pos <= lim[k]
                                                  : lim[k] >= 0 && pos < x.len && (j < 0 || (see[k] >> (j & 31) & 1u) != 0);
              if (!sees) sv[st][k][v] = -INFINITY;
            }
      }
      float al[2], up[2][2], fv[2][2];  // [group][row]: the page's weight against the row's reference; times its v scale
      bool moved = false;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float top[2];
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          top[st] = fmaxf(sv[st][k][0], sv[st][k][1]);
          if (R16) top[st] = fmaxf(top[st], fmaxf(sv[st][k][NV - 2], sv[st][k][NV - 1]));
        }
        if (P > 16) {
          top[0] = top[1] = max_over_row<R16>(fmaxf(top[0], top[1]));
        } else {
          top[0] = max_over_row<R16>(top[0]);
          top[1] = max_over_row<R16>(top[1]);
        }
        // the row's reference follows its largest score only when that is 2^16 weights above it
        const float both = fmaxf(top[0], top[1]), was = m[k], ref = both > was + 16.f ? both : was;
        al[k] = ref == was ? 1.f : fast_exp2(was - ref);
        moved |= ref != was;
        m[k] = ref;
        const float base = fmaxf(ref, kLowest);
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          if (st == 1 && P > 16) {  // one page
            up[1][k] = up[0][k];
            fv[1][k] = fv[0][k];
          } else {
            up[st][k] = fast_exp2(fmaxf(top[st], kLowest) - 15.f - base);
            // a group that the row sees nothing of has weights of 0 and takes nothing of its scale, even of a NaN
            fv[st][k] = top[st] == -INFINITY ? 0.f : up[st][k] * vf[st];
          }
          const float c = fmaxf(top[st], kLowest) - 15.f;
#pragma unroll
          for (int v = 0; v < NV; ++v) sv[st][k][v] = fast_exp2(sv[st][k][v] - c);
        }
      }
      // the weights as operands: pairs of tokens (4 t, 4 t + 2) and (4 t + 1, 4 t + 3), as codes_to_h2 makes them
      uint32_t wt[2][WP][4];  // 8 rows: two of the four
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        if (R16) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // row g + 8 (i & 1), even or odd pair
            const float a = sv[st][i & 1][i >> 1], b = sv[st][i & 1][R16 ? 2 + (i >> 1) : 0];
            const uint32_t hi = f2_to_h2(a, b);
            wt[st][0][i] = hi;
            if (WP == 2) wt[st][WP - 1][i] = f2_to_h2(a - h_lo_to_f(hi), b - h_lo_to_f(hi >> 16));
          }
        } else {
          const uint32_t e0 = f2_to_h2(sv[st][0][0], sv[st][1][0]), e1 = f2_to_h2(sv[st][0][1], sv[st][1][1]);
          weight_operand(wt[st][0], movmatrix(e0), movmatrix(e1));
          if (WP == 2)
            weight_operand(wt[st][WP - 1], movmatrix(f2_to_h2(sv[st][0][0] - h_lo_to_f(e0), sv[st][1][0] - h_lo_to_f(e0 >> 16))),
                           movmatrix(f2_to_h2(sv[st][0][1] - h_lo_to_f(e1), sv[st][1][1] - h_lo_to_f(e1 >> 16))));
        }
      }
      if (__any_sync(~0u, moved)) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          l[k] *= al[k];
          hv[k] *= al[k];
        }
#pragma unroll
        for (int s = 0; s < NO; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[s][e] *= al[R16 ? e >> 1 : e & 1];
      }
      // ---- sums of the weights, then values: a page's products are added up before its scale
      const uint8_t* vst = smem + v_slot * S::kSlot + part32 * kWarpPos * D;
      constexpr uint32_t kOnes = 0x3C003C00u;
      const uint32_t ones[4] = {kOnes, kOnes, kOnes, kOnes};
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int st = 0; st < 2; ++st) {
#pragma unroll
        for (int part = 0; part < WP; ++part) {
          if (R16) mma_f16_16816(acc, wt[st][part], kOnes, kOnes, acc);
          else mma_f16_16816(acc, ones, wt[st][part][0], wt[st][part][1], acc);
        }
        if (st == 1 || P == 16) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float sum = acc[R16 ? 2 * k : k];
            l[k] = __fmaf_rn(up[st][k], sum, l[k]);
            hv[k] = __fmaf_rn(fv[st][k], sum, hv[k]);
          }
          acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
        }
      }
      if (!PR) wait(&sm_full[v_slot], v_phase);
#pragma unroll
      for (int cc = 0; cc < C32; ++cc) {
        constexpr int NA = R16 ? 4 : 2;  // output tiles of 32 dims
        float av[NA][4];
#pragma unroll
        for (int s = 0; s < NA; ++s) av[s][0] = av[s][1] = av[s][2] = av[s][3] = 0.f;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          const uint4 v = lds128(vst + st * 16 * D + cc * 512 + lane * 16);
          uint32_t a[2][4];
          codes_to_h2(v.x, a[0][0], a[0][2]);
          codes_to_h2(v.y, a[0][1], a[0][3]);
          codes_to_h2(v.z, a[1][0], a[1][2]);
          codes_to_h2(v.w, a[1][1], a[1][3]);
#pragma unroll
          for (int part = 0; part < WP; ++part)
#pragma unroll
            for (int s = 0; s < NA; ++s) {
              if (R16) mma_f16_16816(av[s], wt[st][part], a[s >> 1][s & 1], a[s >> 1][2 + (s & 1)], av[s]);
              else mma_f16_16816(av[s], a[R16 ? 0 : s], wt[st][part][0], wt[st][part][1], av[s]);
            }
          if (st == 1 || P == 16) {
#pragma unroll
            for (int s = 0; s < NA; ++s)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float& oo = o[NA * cc + s][e];
                oo = __fmaf_rn(fv[st][R16 ? e >> 1 : e & 1], av[s][e], oo);
                if (st == 0) av[s][e] = 0.f;
              }
          }
        }
      }
      }
      if (PR) free_slot(k_slot);
      free_slot(v_slot);
    }

    const bool partial = x.nseg > 1;
    const bool room = !partial || x.part + (long long)x.nseg * x.rows <= p.part_rows;
    const long long part_row = x.part * p.n_kv + ((long long)x.h * x.nseg + x.seg) * x.rows;
    if (!room && tid == 0) atomicOr(&g_kv8_errors, 2u);
    if (PR) {  // this warp's rows are done
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = x.row0 + wrow + g + 8 * k, ti = token_of(p, row);
        if (row >= x.rows || !room) continue;
        const float half = 0.5f * hv[k], inv = partial ? 1.f : l[k] == 0.f ? 0.f : 1.f / l[k];
        const long long to = partial ? (part_row + row) * D : (x.tok0 + ti) * p.os + (long long)(x.h * group + row - ti * group) * D;
#pragma unroll
        for (int s = 0; s < NO; ++s) {  // dims 8 s + 2 t4, + 1
          const float v0 = (o[s][R16 ? 2 * k : 0] + half) * inv, v1 = (o[s][R16 ? 2 * k + 1 : 0] + half) * inv;
          const long long at_d = to + 8 * s + 2 * t4;
          if (partial) *reinterpret_cast<float2*>(p.part + at_d) = make_float2(v0, v1);
          else if (p.o_f32) *reinterpret_cast<float2*>(static_cast<float*>(p.o) + at_d) = make_float2(v0, v1);
          else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + at_d) = (uint32_t)f32_to_bf16_rn(v0) | (uint32_t)f32_to_bf16_rn(v1) << 16;
        }
        if (partial && t4 == 0) p.part_ml[part_row + row] = make_float2(m[k], l[k]);
      }
      continue;
    }
    // ---- the four warps' results meet
    float* out = reinterpret_cast<float*>(smem + S::kOut);
    float* mine = out + w * S::kOutWarp;
    if (R16 ? t4 == 0 : g == 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int rr = R16 ? g + 8 * k : 2 * t4 + k;
        sm_m[w][rr] = m[k];
        sm_l[w][rr] = l[k];
        sm_h[w][rr] = 0.5f * hv[k];
      }
    }
#pragma unroll
    for (int s = 0; s < NO; ++s) {
      if (R16) {  // dims 8 s + 2 t4, + 1 of rows g, g + 8
        *reinterpret_cast<float2*>(mine + g * (D + 4) + 8 * s + 2 * t4) = make_float2(o[s][0], o[s][1]);
        *reinterpret_cast<float2*>(mine + (g + 8) * (D + 4) + 8 * s + 2 * t4) = make_float2(o[s][2], o[s][3]);
      } else {    // dims 16 s + g, + 8 of rows 2 t4, + 1
#pragma unroll
        for (int e = 0; e < 4; ++e) mine[(2 * t4 + (e & 1)) * (D + 4) + 16 * s + 8 * (e >> 1) + g] = o[s][e];
      }
    }
    math_barrier();
    const int live_rows = room ? min(RB, x.rows - x.row0) : 0;
    for (int e = tid; e < live_rows * (D / 4); e += kMath) {
      const int rr = e / (D / 4), d = (e - rr * (D / 4)) * 4, row = x.row0 + rr;
      float mm = sm_m[0][rr];
#pragma unroll
      for (int i = 1; i < kWarps; ++i) mm = fmaxf(mm, sm_m[i][rr]);
      const float mb = mm == -INFINITY ? 0.f : mm;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float den = 0.f, hs = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float li = sm_l[i][rr], f = li == 0.f ? 0.f : fast_exp2(sm_m[i][rr] - mb);
        const float4 v = *reinterpret_cast<const float4*>(out + i * S::kOutWarp + rr * (D + 4) + d);
        sum.x += f * v.x;
        sum.y += f * v.y;
        sum.z += f * v.z;
        sum.w += f * v.w;
        den += f * li;
        hs += f * sm_h[i][rr];
      }
      sum.x += hs;
      sum.y += hs;
      sum.z += hs;
      sum.w += hs;
      if (partial) {
        const long long to = part_row + row;
        *reinterpret_cast<float4*>(p.part + to * D + d) = sum;
        if (d == 0) p.part_ml[to] = make_float2(mm, den);
      } else {
        const float inv = den == 0.f ? 0.f : 1.f / den;
        const int ti = token_of(p, row);
        const long long to = (x.tok0 + ti) * p.os + (long long)(x.h * group + row - ti * group) * D + d;
        if (p.o_f32)
          *reinterpret_cast<float4*>(static_cast<float*>(p.o) + to) = make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + to) =
              make_uint2((uint32_t)f32_to_bf16_rn(sum.x * inv) | (uint32_t)f32_to_bf16_rn(sum.y * inv) << 16,
                         (uint32_t)f32_to_bf16_rn(sum.z * inv) | (uint32_t)f32_to_bf16_rn(sum.w * inv) << 16);
      }
    }
    math_barrier();
  }
  if (dead && lane == 0) atomicOr(&g_kv8_errors, 1u);
}

// Sums 4, 2 and 1 apart of `COUNT` sums.
template <int COUNT, int N>
__device__ __forceinline__ void fold_sums(float (&acc)[COUNT][N]) {
#pragma unroll
  for (int h = COUNT / 2; h; h >>= 1)
#pragma unroll
    for (int q = 0; q < h; ++q)
#pragma unroll
      for (int e = 0; e < N; ++e) acc[q][e] += acc[q + h][e];
}

// The segments of a request added up in an order that does not depend on how many there are: eight sums, each of
// every eighth segment in order, then sums 4, 2 and 1 apart. K warps of a CTA share them: warp `sub` takes sums
// sub, sub + K, ... and joins its own. sum: D / 32 dims of this lane, and the weights'.
template <int K, int E>
__device__ __forceinline__ void join_segments(float (&sum)[E + 1], const AttnKV8Params& p, long long first, long long step, int nseg, int sub, float mb) {
  constexpr int SUMS = 8 / K;
  float acc[SUMS][E + 1];
#pragma unroll
  for (int q = 0; q < SUMS; ++q)
#pragma unroll
    for (int e = 0; e <= E; ++e) acc[q][e] = 0.f;
  for (int s0 = sub; s0 < nseg; s0 += 8 * K) {
    float2 ml[8];
    float v[8][E];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int s = s0 + u * K;
      const long long at = first + s * step;
      const float* src = p.part + at * 32 * E + (threadIdx.x & 31) * E;
      ml[u] = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) v[u][e] = 0.f;
      if (s < nseg) {
        ml[u] = p.part_ml[at];
        if (E == 4) {
          const float4 x = *reinterpret_cast<const float4*>(src);
          v[u][0] = x.x, v[u][1] = x.y, v[u][E - 2] = x.z, v[u][E - 1] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(src);
          v[u][0] = x.x, v[u][1] = x.y;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float f = ml[u].y == 0.f ? 0.f : fast_exp2(ml[u].x - mb);
      float(&to)[E + 1] = acc[u % SUMS];
#pragma unroll
      for (int e = 0; e < E; ++e) to[e] = __fmaf_rn(f, v[u][e], to[e]);
      to[E] = __fmaf_rn(f, ml[u].y, to[E]);
    }
  }
  fold_sums(acc);
#pragma unroll
  for (int e = 0; e <= E; ++e) sum[e] = acc[0][e];
}

// The other warps' sums, in shared memory behind this one's, joined with it.
template <int K, int D>
__device__ __forceinline__ void join_warps(float (&sum)[D / 32 + 1], const float (*sm_o)[D], const float* sm_sum) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  float acc[K][E + 1];
#pragma unroll
  for (int q = 0; q < K; ++q) {
#pragma unroll
    for (int e = 0; e < E; ++e) acc[q][e] = sm_o[q][lane * E + e];
    acc[q][E] = sm_sum[q];
  }
  fold_sums(acc);
#pragma unroll
  for (int e = 0; e <= E; ++e) sum[e] = acc[0][e];
}

template <int D>
__global__ void __launch_bounds__(kCombThreads, D == 64 ? 3 : 1) attn_kv8_combine_kernel(const AttnKV8Params p) {
  constexpr int W = kCombThreads / 32, E = D / 32;
  extern __shared__ __align__(16) int sm_req[];
  __shared__ long long sm_scan[3 * W];
  __shared__ __align__(16) float sm_o[W][D];
  __shared__ float sm_sum[W];
  Request* req = reinterpret_cast<Request*>(sm_req);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  // the lengths were written before the attention kernel passed its own wait, after which alone this
  // kernel can start
  scan_requests<kCombThreads, kCombine>(p, 1, req, sm_scan);
  grid_dependency_wait();
  const int n_q = p.n_kv * p.group, total = req[p.B].item;
  for (int it = blockIdx.x; it < total; it += gridDim.x) {
    const int r = find_request(req, p.B, it), local = it - req[r].item, tok0 = req[r].tok;
    const int n = req[r + 1].tok - tok0, nseg = p.cut(req[r].ctx + n, n).count;
    if (req[r].part + (long long)nseg * n * p.group > p.part_rows) continue;
    const int k = combine_warps(nseg), sub = w & (k - 1);
    const int task = (local * W + w) / k;  // (token, query head) of the request
    const bool live = task < n * n_q;
    const int i = task / n_q, hq = task - i * n_q, h = hq / p.group, row = i * p.group + hq - h * p.group;
    const long long step = (long long)n * p.group, first = req[r].part * p.n_kv + h * nseg * step + row;
    float sum[E + 1];  // the last: of the weights
#pragma unroll
    for (int e = 0; e <= E; ++e) sum[e] = 0.f;
    if (live) {
      float mx = -INFINITY;
      for (int s = lane; s < nseg; s += 32) mx = fmaxf(mx, p.part_ml[first + s * step].x);
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, x));
      const float mb = mx == -INFINITY ? 0.f : mx;
      if (k == 1) join_segments<1, E>(sum, p, first, step, nseg, sub, mb);
      else if (k == 2) join_segments<2, E>(sum, p, first, step, nseg, sub, mb);
      else if (k == 4) join_segments<4, E>(sum, p, first, step, nseg, sub, mb);
      else join_segments<8, E>(sum, p, first, step, nseg, sub, mb);
    }
    if (k > 1) {  // uniform in the CTA
#pragma unroll
      for (int e = 0; e < E; ++e) sm_o[w][lane * E + e] = sum[e];
      if (lane == 0) sm_sum[w] = sum[E];
      __syncthreads();
      if (sub == 0) {
        if (k == 2) join_warps<2, D>(sum, sm_o + w, sm_sum + w);
        else if (k == 4) join_warps<4, D>(sum, sm_o + w, sm_sum + w);
        else join_warps<8, D>(sum, sm_o + w, sm_sum + w);
      }
      __syncthreads();
    }
    const float den = sum[E];
    if (live && sub == 0) {
      const float inv = den == 0.f ? 0.f : 1.f / den;  // as a request of one segment
      const long long at = (tok0 + i) * p.os + (long long)hq * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float v0 = sum[e] * inv, v1 = sum[e + 1] * inv;
        if (p.o_f32) *reinterpret_cast<float2*>(static_cast<float*>(p.o) + at + e) = make_float2(v0, v1);
        else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + at + e) = (uint32_t)f32_to_bf16_rn(v0) | (uint32_t)f32_to_bf16_rn(v1) << 16;
      }
    }
  }
}

template <int D, Form FORM, int QP, int WP>
int launch_form(const AttnKV8Params& p, int num_sms, cudaStream_t s, std::string* err) {
  const size_t smem = AttnSmem<D, FORM, QP>::bytes(p.B);
  constexpr size_t kMost = AttnSmem<D, FORM, QP>::bytes(KQ_KV8_MAX_REQUESTS);
  static_assert(kMost + 2048 <= 227 * 1024, "with the kernel's static memory it fits an SM");
  auto* kernel = attn_kv8_kernel<D, FORM, QP, WP>;
  static SmemAllowed allowed;
  if (allow_smem(allowed, kernel, kMost, "attention_kv8", err) != 0) return -1;
  // CTAs per SM at this shared-memory size, asked for once per host thread, device and size
  static thread_local int known_dev = -1, per_sm = 0;
  static thread_local size_t known_smem = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev != known_dev || smem != known_smem)) {
    per_sm = 0;
    known_dev = -1;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, smem);
    if (e == cudaSuccess && per_sm > 0) {
      known_dev = dev;
      known_smem = smem;
    }
  }
  if (e != cudaSuccess || per_sm < 1) {
    *err = std::string("attention_kv8: ") + (e != cudaSuccess ? cudaGetErrorString(e) : "the kernel does not fit an SM");
    return -1;
  }
  return launch_pdl(kernel, dim3(num_sms * per_sm), dim3(kThreads), smem, s, p, "attention_kv8", err);
}

// Windows of up to 32 tokens, and, where max_new allows larger ones, those in a launch of their own: which
// form a request takes, and its bits, do not depend on the others.
template <int D, int QP, int WP>
int launch_all(const AttnKV8Params& p, int num_sms, cudaStream_t s, std::string* err) {
  const bool rows8 = (long long)p.max_new * p.group <= 8;
  if ((rows8 ? launch_form<D, kRows8, QP, WP>(p, num_sms, s, err) : launch_form<D, kRows16, QP, WP>(p, num_sms, s, err)) != 0) return -1;
  if (p.max_new > kSplitTokens && launch_form<D, kPrompt, QP, WP>(p, num_sms, s, err) != 0) return -1;
  if (p.max_len <= 1 << p.cut.seg_log2) return 0;  // no request can have two segments
  const long long tasks = (long long)p.T * p.n_kv * p.group;
  // no more CTAs than the longest request's rows would need: each forms the prefix sums
  const long long want = (tasks * combine_warps(p.cut(p.max_len, 1).count) + kCombThreads / 32 - 1) / (kCombThreads / 32);
  const int grid = (int)(want < (long long)num_sms * 8 ? want : (long long)num_sms * 8);
  static SmemAllowed allowed;
  if (allow_smem(allowed, attn_kv8_combine_kernel<D>, (KQ_KV8_MAX_REQUESTS + 1) * sizeof(Request), "attention_kv8 combine", err) != 0) return -1;
  return launch_pdl(attn_kv8_combine_kernel<D>, dim3(grid), dim3(kCombThreads), (size_t)(p.B + 1) * sizeof(Request), s, p,
                    "attention_kv8 combine", err);
}

template <int D>
int launch_dim(const AttnKV8Params& p, int num_sms, cudaStream_t s, std::string* err) {
  if (p.o_f32) return launch_all<D, 2, 2>(p, num_sms, s, err);
  return p.q_f32 ? launch_all<D, 2, 1>(p, num_sms, s, err) : launch_all<D, 1, 1>(p, num_sms, s, err);
}

// Partial rows at most: windows of up to 32 tokens have len / 512 + 1 segments, larger ones segments x rows
// <= items of 64 rows, where their context is long.
size_t part_rows(const Cutter& cut, int B, long long total_len, int max_new) {
  const int window = max_new < kSplitTokens ? max_new : kSplitTokens;
  const size_t rows = (size_t)cut.group * window * ((size_t)(total_len >> cut.seg_log2) + B);
  if (max_new <= kSplitTokens) return rows;
  const long long many = total_len / kLongContext < B ? total_len / kLongContext : B;
  const size_t by_items = (size_t)many * (kWaves * cut.wave / cut.n_kv) * kPromptRows;
  const size_t by_length = (size_t)(total_len / kShortest) * cut.group * max_new;
  return rows + (by_items < by_length ? by_items : by_length);
}

}  // namespace

unsigned int take_kv8_errors() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv8_errors, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (cudaMemcpyToSymbol(g_kv8_errors, &zero, sizeof(zero)) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
}

size_t attention_kv8_workspace(int B, long long total_len, int max_new, int n_q, int n_kv, int D) {
  return part_rows(cutter_of(n_kv, n_q / n_kv, D), B, total_len, max_new) * n_kv * (D + 2) * sizeof(float);
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
  p.cut = cutter_of(c.n_kv, p.group, c.D);
  p.group_inv = p.group == 1 ? 0u : (unsigned)(((1ull << 32) + p.group - 1) / p.group);
  p.scale_log2e = a.scale * 1.4426950408889634f;
  p.part_rows = (long long)part_rows(p.cut, a.B, a.total_len, a.max_new);
  p.part = static_cast<float*>(a.ws);
  p.part_ml = reinterpret_cast<float2*>(p.part + (size_t)p.part_rows * c.n_kv * c.D);
  return c.D == 64 ? launch_dim<64>(p, num_sms, s, err) : launch_dim<128>(p, num_sms, s, err);
}

}  // namespace kq
