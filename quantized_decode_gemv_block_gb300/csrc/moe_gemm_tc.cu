// Products of the experts' Q4_K matrices with many rows each, on the 5th-generation tensor cores (tcgen05).
//
// The arithmetic is that of the prefill product: with w = d_s (sc_b q) - dmin_s m_b,
//   y[n] = sum_s d_s (sum_{k in s} x[k] t[n][k])  -  sum_b (dmin m)_b S_b(x),      t = sc q <= 945, exact in fp16,
// x in fp16 under an exact power of two per row, S_b the sum of x over 32 values; both S_b / 64 and -64 dmin m enter as
// fp16 pairs hi + lo (products hi hi, lo hi, hi lo). Every product is exact, a super-block's sum is scaled by d_s in fp32.
//  * a pre-pass writes the experts' rows in the plan's order, as fp16 with their sums behind
//    them: per super-block eight S_hi, eight S_lo, eight S_hi, eight zeros;
//  * a cluster of two CTAs owns a tile of 256 weight rows x up to 256 rows of one expert (cta_group::2, M = 256,
//    N = 32 .. 256 by the expert's rows; rank r holds weight rows 128 r.. and half of the N rows); for gate | up
//    a CTA's 128 rows are 64 of each, 16 and 16 of a warp's 32 lanes, so that the epilogue forms silu(g) u by a shuffle;
//  * roles as in the prefill product: copies of rows, copies of raw blocks, MMA, four unpacking warps, eight epilogue warps that
//    add d_s times each finished super-block into registers.
// Tiles follow from the plan's offsets on the device: expert by expert, an expert's rows in equal parts of up to 256. The
// min-term tiles (two super-blocks each, [M_hi M_hi M_lo 0] per super-block) are formed by the unpacking warps from the
// blocks' headers and come last.
// 2048 tokens, 8 of 128 experts: gate | up (2 x 768 x 2048) 218 us, 470 TFLOP/s, pre-pass and all; down (2048 x 768) 159 us, 325. No
// part alone bounds it: gate | up without the unpacking takes 187 us, without the results' stores 197, without the MMAs 207, without
// unpacking and MMAs 174, the rest of which are the hand-overs between the roles (stage free, unpacked, both CTAs' arrival, MMA,
// commit), the epilogue and the pre-pass. On the way there: raw blocks through a warp of their own and one barrier per stage 5 %,
// results stored without branches 8 %, roles of one thread by elect 9 %.
// Every wait is bounded: a timeout records the error word and raises the abort flag of both CTAs; all roles then drain
// and return.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "kq_device.cuh"
#include "kq_internal.h"
#include "kq_launch.cuh"
#include "moe.cuh"

namespace cg = cooperative_groups;

namespace kq {

__device__ unsigned int g_moe_tc_errors = 0;  // bit 0: a bounded wait gave up; bit 1: a plan out of bounds; bit 2: a min past fp16

namespace {

constexpr int TM = 128;       // weight rows of a CTA, half of the pair's M
constexpr int TN = 256;       // rows of an expert in a tile at most; each CTA stages half
constexpr int BK = 64;        // k per stage: one 128-byte swizzle row of fp16
constexpr int kBoxRows = 32;  // rows of a token copy
constexpr int STAGES = 5;
constexpr int RAW_STAGES = 3;
constexpr int kWTileBytes = TM * BK * 2;
constexpr int kXTileBytes = (TN / 2) * BK * 2;
constexpr int kStageBytes = kWTileBytes + kXTileBytes;
constexpr int kRawBytes = TM * 144;  // one super-block of the CTA's weight rows
// Four warpgroups: 0-1 epilogue, 2 unpacking, 3 copies / MMA. The epilogue's 128 sums per thread need more registers than
// the 128 a 512-thread CTA starts with; the others hand theirs over.
constexpr int kEpiWarps = 8, kDqWarps = 4;
constexpr int kTmaWarp = kEpiWarps + kDqWarps, kMmaWarp = kTmaWarp + 1, kRawWarp = kTmaWarp + 2;
constexpr int kTcThreads = 16 * 32;
constexpr int kLaunchRegs = 128, kEpiRegs = 184, kDqRegs = 96, kCtlRegs = 48;
static_assert(2 * 128 * kEpiRegs + 128 * kDqRegs + 128 * kCtlRegs == kTcThreads * kLaunchRegs, "register split");
static_assert(kDqWarps <= STAGES, "an unpacking warp's previous wait was kDqWarps + STAGES k-tiles back");
constexpr int kTmemCols = 2 * TN;  // two accumulator groups in flight
constexpr int kBarBytes = 512;
constexpr int kListBytes = 2 * (KQ_MOE_MAX_EXPERTS + 1) * 4 + 8;  // tiles before each expert, and its first row
// A pair's first tiles are worked out before the roles part, for those that feed the tensor cores (2 us a tile in the MMAs' own
// thread; 65536 pairs of 1024 experts, 2 x 512 x 1024: 572 -> 557 us); further ones, of calls beyond about 600,000 rows of 512, as they come
constexpr int kTable = 64;
constexpr int kScaleGroups = 4;               // super-blocks whose d the epilogue may still need
constexpr int kScaleBytes = kScaleGroups * TM * 4;
constexpr int kTcSmem = STAGES * kStageBytes + RAW_STAGES * kRawBytes + kBarBytes + kScaleBytes + kListBytes + kTable * 16 + 1024 /*alignment*/;
constexpr uint32_t kNoPair = 0x80000000u;   // a tag of none: a column behind a tile's rows
constexpr uint32_t kBadPair = 0x80000001u;  // and of a place whose pair is out of bounds; nothing is stored from kNoPair on
constexpr uint64_t kTcWaitNs = 2000000000ull;
static_assert(kTcSmem <= 232448 - 256, "shared memory per CTA");

struct TcParams {
  const uint8_t* w;
  const uint32_t* tags;    // per place in the plan (see the pre-pass)
  const int *offsets, *order;
  int E, P;
  int N, K, half;          // weight rows of an expert; half: F of a gate | up matrix, 0 otherwise
  float* y;                // half == 0: P x N
  uint16_t* act;           // half != 0: P x half
  long long row_bytes;
  int n_ext;               // min-term k-tiles
  int row_tiles;           // of an expert
};

// A shared-memory operand: K-major, 128-byte swizzle, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16: fp32 sums, fp16 operands, both K-major, M = 256, N rows of the expert.
__device__ __forceinline__ uint32_t instr_desc(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)((2 * TM) >> 4) << 24); }

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void umma_pair_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on `bar` of both CTAs when every MMA issued so far by this thread has completed.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
__device__ __forceinline__ void mbar_arrive_local(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// 32 consecutive fp32 columns of the warp's 32 tensor-memory lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// A tensor copy into this CTA's shared memory, counted on a barrier of either CTA (shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const void* tmap, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Stores without a branch.
__device__ __forceinline__ void store_if(bool on, uint16_t* to, uint16_t v) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %2, 0;\n@p st.global.u16 [%0], %1;\n}" ::"l"(to), "h"(v), "r"((uint32_t)on) : "memory");
}
__device__ __forceinline__ void store_if(bool on, float* to, float v) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %2, 0;\n@p st.global.cs.f32 [%0], %1;\n}" ::"l"(to), "f"(v), "r"((uint32_t)on) : "memory");
}
// True for one lane of a whole warp. What it guards is known to be one thread's, so that descriptors and barriers stay in uniform
// registers: with lane == 0 in its place the MMAs' thread was the slowest role (2048 tokens, gate | up 239 us, now 218).
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(on));
  return on != 0;
}
// 16-byte chunk `c` of row r in a K-major 64-wide fp16 tile with the 128-byte swizzle.
__device__ __forceinline__ int sw128_off(int r, int c) { return (r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4); }

// The 64 values t = sc q of k-chunk kc (0..3) of a super-block into row r of the tile. b: the block; sub-blocks 2 kc (low
// nibbles, k = 0..31) and 2 kc + 1 (high nibbles): a pair of codes becomes 1024 + q or 1024 + 16 q in fp16, and one fma takes the
// offset off and multiplies by sc. The scales become fp16 by exponent bytes too: conversions run at a quarter of the rate. Returns
// the header's first word: d and dmin.
__device__ __forceinline__ uint32_t unpack_row(const uint8_t* b, int kc, uint8_t* tile, int r) {
  const uint4 h = lds128(b), qa = lds128(b + 16 + 32 * kc), qb = lds128(b + 32 + 32 * kc);
  // sc of the two sub-blocks in bytes 0 and 1: six bits of scales[2 kc], or four of scales[2 kc + 4] and two of scales[2 kc - 4]
  const int at = 16 * (kc & 1);
  const uint32_t s0 = h.y >> at, s2 = h.w >> at;
  const uint32_t sc = kc < 2 ? s0 & 0x3F3Fu : (s2 & 0x0F0Fu) | ((s0 >> 2) & 0x3030u);
  const uint32_t a_l = h2_sub(prmt(sc, 0x64646464u, 0x4040u), 0x64006400u), c_l = h2_mul(a_l, 0xE400E400u);  // sc, -1024 sc
  const uint32_t a_h = h2_sub(prmt(sc, 0x54545454u, 0x4141u), 0x54005400u), c_h = h2_mul(a_h, 0xE400E400u);  // sc / 16, -64 sc
  const uint32_t qw[8] = {qa.x, qa.y, qa.z, qa.w, qb.x, qb.y, qb.z, qb.w};
  uint32_t lo[16], hi[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t p01 = prmt(qw[i], 0u, 0x3120u), p23 = prmt(qw[i], 0u, 0x1302u);
    lo[2 * i] = h2_fma(and_or(p01, 0x000F000Fu, 0x64006400u), a_l, c_l);
    lo[2 * i + 1] = h2_fma(and_or(p23, 0x000F000Fu, 0x64006400u), a_l, c_l);
    hi[2 * i] = h2_fma(and_or(p01, 0x00F000F0u, 0x64006400u), a_h, c_h);
    hi[2 * i + 1] = h2_fma(and_or(p23, 0x00F000F0u, 0x64006400u), a_h, c_h);
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    *reinterpret_cast<uint4*>(tile + sw128_off(r, c)) = make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
    *reinterpret_cast<uint4*>(tile + sw128_off(r, c + 4)) = make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
  }
  return h.x;
}

// -64 dmin m of a super-block's eight sub-blocks (header h) as fp16 hi + lo, chunks 4 j .. 4 j + 3 of row r: hi, hi, lo, zeros.
// lo = -64 dmin m - hi is exact: what rounding 11 bits times 6 to 11 leaves has six bits, none below the last of dmin.
__device__ __forceinline__ void min_row(const uint4& h, int j, uint8_t* tile, int r) {
  const uint32_t dmin = prmt(h.x, 0u, 0x3232u);
  const uint32_t m[2] = {h.z & 0x3F3F3F3Fu, ((h.w >> 4) & 0x0F0F0F0Fu) | ((h.z >> 2) & 0x30303030u)};  // six bits a byte
  uint32_t hv[4], lv[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint32_t f = h2_mul(h2_sub(prmt(m[b / 2], 0x64646464u, b & 1 ? 0x4342u : 0x4140u), 0x64006400u), 0xD400D400u);  // -64 m
    hv[b] = h2_mul(dmin, f);
    lv[b] = h2_fma(dmin, f, hv[b] ^ 0x80008000u);
  }
  *reinterpret_cast<uint4*>(tile + sw128_off(r, 4 * j)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
  *reinterpret_cast<uint4*>(tile + sw128_off(r, 4 * j + 1)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
  *reinterpret_cast<uint4*>(tile + sw128_off(r, 4 * j + 2)) = make_uint4(lv[0], lv[1], lv[2], lv[3]);
  *reinterpret_cast<uint4*>(tile + sw128_off(r, 4 * j + 3)) = make_uint4(0u, 0u, 0u, 0u);
}

// Whether -64 dmin m of one of a header's sub-blocks is past fp16. Out of line, and asked only where dmin is 16.25 or more: below, no m
// of six bits gets there (asked of every header: 2048 tokens, gate | up 217 -> 223 us).
__device__ __noinline__ bool min_past(const uint4 h) {
  const float dmin = fabsf(half_bits_to_float(h.x >> 16));
  uint32_t most = 0u;
  for (int b = 0; b < 4; ++b) most = max(most, max(h.z >> 8 * b & 63u, (h.w >> (8 * b + 4) & 15u) | (h.z >> (8 * b + 2) & 48u)));
  return !(64.f * dmin * (float)most < 65520.f);
}

// A tile: `n` rows of expert e from place `first` of the plan on, its weight rows from row_tile on; h of the rows (a multiple of 16)
// are rank 0's, the others rank 1's.
struct Tile {
  int e, first, n, h, row_tile;
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTcThreads, 1)
    moe_q4k_tc_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap, const TcParams p) {
  extern __shared__ uint8_t tc_smem_raw[];
  __shared__ int scan_sums[16];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tc_smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* raw = smem + STAGES * kStageBytes;     // stage s: t tile, then this CTA's rows
  uint64_t* full = reinterpret_cast<uint64_t*>(raw + RAW_STAGES * kRawBytes);  // rank 0: copies landed, both CTAs' t tiles written
  uint64_t* empty = full + STAGES;                // each: the pair's MMAs read the stage
  uint64_t* acc_full = empty + STAGES;            // each [2]: group finished
  uint64_t* acc_empty = acc_full + 2;             // each [2]: the CTA's epilogue read the group (rank 0: and rank 1's)
  uint64_t* raw_full = acc_empty + 2;             // each [RAW_STAGES]: raw super-block landed
  uint64_t* raw_empty = raw_full + RAW_STAGES;    // each [RAW_STAGES]: the super-block's 4 k-tiles unpacked
  uint64_t* mma_done = raw_empty + RAW_STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  unsigned int* abort_flag = tmem_slot + 1;
  // d of the last four groups' super-blocks, by row: written by the unpacking warps, read by the epilogue. Unpacking group G starts
  // after the MMAs of group G - 2, which began when the epilogue had read group G - 4
  float* dscale = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(full) + kBarBytes);
  int* start = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(dscale) + kScaleBytes);  // E + 1: tiles before each expert
  int* place = start + KQ_MOE_MAX_EXPERTS + 1;                                          // E + 1: offsets
  int4* table = reinterpret_cast<int4*>(reinterpret_cast<uint8_t*>(start) + kListBytes);  // e, first, n and h, row_tile

  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank();
  const bool leader = rank == 0;
  const int pair = static_cast<int>(blockIdx.x >> 1), npairs = static_cast<int>(gridDim.x >> 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nsb = p.K / 256, kt_tile = p.n_ext + 4 * nsb;

  if (threadIdx.x == 0) {
    // rank 1's unpacking warps arrive at rank 0's barriers, its epilogue warps at their own, which one thread forwards
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 3);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kEpiWarps + (leader ? 1 : 0));
    }
    for (int r = 0; r < RAW_STAGES; ++r) {
      mbar_init(&raw_full[r], 1);
      mbar_init(&raw_empty[r], 4);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0u;
    fence_mbar_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(&xmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&wmap) : "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  grid_launch_dependents();
  grid_dependency_wait();

  // tiles before each expert, two experts per thread
  {
    int n[2], mine = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 2 * threadIdx.x + i;
      n[i] = 0;
      if (e < p.E) {
        const int a = p.offsets[e], b = p.offsets[e + 1];
        place[e] = a;
        if (e == p.E - 1) place[p.E] = b;
        if (a < 0 || b < a || b > p.P) {
          if (blockIdx.x == 0) atomicOr(&g_moe_tc_errors, 2u);
        } else {
          n[i] = (b - a + TN - 1) / TN * p.row_tiles;
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
    if (lane == 31) scan_sums[warp] = scan;
    __syncthreads();
    int before = scan - mine;
    for (int w = 0; w < warp; ++w) before += scan_sums[w];
    if (2 * static_cast<int>(threadIdx.x) <= p.E) start[2 * threadIdx.x] = before;
    if (2 * static_cast<int>(threadIdx.x) + 1 <= p.E) start[2 * threadIdx.x + 1] = before + n[0];
    if (threadIdx.x == kTcThreads - 1 && p.E == 2 * kTcThreads) start[p.E] = before + mine;
  }
  __syncthreads();
  const int tiles = start[p.E];
  const int my_tiles = pair < tiles ? (tiles - 1 - pair) / npairs + 1 : 0;

  // Tile i of this pair; e: the expert of an earlier one, or 0.
  auto find_tile = [&](int i, int e) {
    const int t = pair + i * npairs;
    while (start[e + 1] <= t) ++e;
    Tile r;
    r.e = e;
    const int q = t - start[e], part = q / p.row_tiles, rows = place[e + 1] - place[e];
    r.row_tile = q - part * p.row_tiles;
    const int parts = (rows + TN - 1) / TN, each = (rows + parts - 1) / parts;
    r.first = place[e] + part * each;
    r.n = min(each, rows - part * each);
    r.h = (r.n + 31) / 32 * 16;
    return r;
  };
  if (static_cast<int>(threadIdx.x) < min(my_tiles, kTable)) {
    const int i = static_cast<int>(threadIdx.x), at = pair + i * npairs;
    int e = 0;
    for (int end = p.E; end - e > 1;) {  // the last expert whose tiles begin at or before this one
      const int mid = (e + end) / 2;
      if (start[mid] <= at) e = mid;
      else end = mid;
    }
    const Tile t = find_tile(i, e);
    table[i] = make_int4(t.e, t.first, t.n | t.h << 16, t.row_tile);
  }
  auto tile_of = [&](int i, int e) {
    if (i >= kTable) return find_tile(i, e);
    const int4 v = table[i];
    Tile r;
    r.e = v.x, r.first = v.y, r.n = v.z & 0xFFFF, r.h = v.z >> 16, r.row_tile = v.w;
    return r;
  };
  tc_fence_before();
  __syncthreads();
  cluster.sync();  // both CTAs' barriers initialised, tensor memory allocated, lists written
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto aborted = [&]() { return *(volatile unsigned int*)abort_flag != 0u; };
  auto fail = [&]() {
    atomicOr(&g_moe_tc_errors, 1u);
    atomicOr(abort_flag, 1u);
    atomicOr(cluster.map_shared_rank(abort_flag, rank ^ 1u), 1u);
  };
  // Waits for a phase; false where another role gave up, or this wait itself does. A phase that is there costs one try.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
      if (mbar_try_wait(bar, parity)) return true;
      if (aborted()) return false;
      if (globaltimer_ns() - t0 > kTcWaitNs) {
        fail();
        return false;
      }
    }
  };

  // This CTA's first weight row of a tile (of the gate rows and, half further on, of the up rows).
  auto row0_of = [&](const Tile& t) {
    return t.e * (long long)p.N + (p.half ? t.row_tile * TM + static_cast<int>(rank) * (TM / 2) : (2 * t.row_tile + static_cast<int>(rank)) * TM);
  };

  const int wg = warp >> 2;  // each role's register budget is set at the top of its branch
  if (wg == 3) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtlRegs));
    if (warp == kTmaWarp) {
      if (elect_one()) {
        int s = 0, round = 0, e = 0;
        bool ok = true;
        for (int i = 0; i < my_tiles && ok; ++i) {
          const Tile t = tile_of(i, e);
          e = t.e;
          const int r0 = t.first + static_cast<int>(rank) * t.h, boxes = (t.h + kBoxRows - 1) / kBoxRows;
          for (int kt = 0; kt < kt_tile; ++kt) {
            if (round > 0 && !wait(&empty[s], static_cast<uint32_t>(round - 1) & 1u)) { ok = false; break; }
            uint8_t* dst = smem + s * kStageBytes + kWTileBytes;
            const uint32_t fb = cluster_addr(&full[s], 0);
            if (leader) mbar_arrive_expect_tx(&full[s], 2u * boxes * kBoxRows * BK * 2);
            const int col = kt * BK;  // the min-term columns stand behind the K values
            for (int b = 0; b < boxes; ++b) tma_load_2d_pair(dst + b * kBoxRows * BK * 2, &xmap, col, r0 + b * kBoxRows, fb);
            if (++s == STAGES) s = 0, ++round;
          }
        }
      }
    } else if (warp == kMmaWarp) {
      if (leader && elect_one()) {
        int s = 0, grp = 0, e = 0;
        uint32_t par = 0;
        bool ok = true;
        const uint64_t desc0 = smem_desc_sw128(smem_addr(smem));  // addresses count in 16 bytes, and stay below their 14 bits
        for (int i = 0; i < my_tiles && ok; ++i) {
          const Tile t = tile_of(i, e);
          e = t.e;
          const uint32_t idesc = instr_desc(2 * t.h);
          for (int g = 0; g <= nsb && ok; ++g, ++grp) {  // the super-blocks, then the min term
            const int buf = grp & 1;
            if (grp >= 2 && !wait(&acc_empty[buf], static_cast<uint32_t>(grp / 2 - 1) & 1u)) { ok = false; break; }
            tc_fence_after();
            const int n = g == nsb ? p.n_ext : 4;
            for (int kt = 0; kt < n; ++kt) {
              if (!wait(&full[s], par)) { ok = false; break; }
              tc_fence_after();
              const uint64_t wa = desc0 + static_cast<uint32_t>(s * (kStageBytes >> 4)), xa = wa + (kWTileBytes >> 4);
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk)
                umma_pair_f16(tmem + (uint32_t)(buf * TN), wa + 2 * kk, xa + 2 * kk, idesc, (kt != 0 || kk != 0) ? 1u : 0u);
              umma_commit_pair(&empty[s]);
              if (++s == STAGES) s = 0, par ^= 1u;
            }
            if (ok) umma_commit_pair(&acc_full[buf]);
          }
        }
        umma_commit_pair(mma_done);  // the wait point for every MMA this thread issued
        if (!mbar_wait_bounded(mma_done, 0u, kTcWaitNs)) fail();  // whether or not another role gave up
      }
    }
    if (warp == kRawWarp && elect_one()) {
      // raw super-blocks, in the order they are unpacked
      int slot = 0, turn = 0, e = 0;
      bool ok = true;
      for (int i = 0; i < my_tiles && ok; ++i) {
        const Tile t = tile_of(i, e);
        e = t.e;
        const int r0 = static_cast<int>(row0_of(t)), r1 = r0 + (p.half ? p.half : TM / 2);
        for (int g = 0; g < nsb; ++g) {
          if (turn > 0 && !wait(&raw_empty[slot], static_cast<uint32_t>(turn - 1) & 1u)) { ok = false; break; }
          fence_proxy_async_smem();  // the unpacking warps' reads of the slot before the copy's writes
          uint8_t* dst = raw + slot * kRawBytes;
          mbar_arrive_expect_tx(&raw_full[slot], kRawBytes);
          tma_load_2d(dst, &wmap, g * 36, r0, &raw_full[slot]);  // 36 words = 144 bytes; 64 rows a copy
          tma_load_2d(dst + kRawBytes / 2, &wmap, g * 36, r1, &raw_full[slot]);
          if (++slot == RAW_STAGES) slot = 0, ++turn;
        }
      }
    }
    if (!leader && warp == kMmaWarp && elect_one()) {
      // forwarder of rank 1: passes each group's "read out" on to rank 0, one arrival for eight warps
      for (int i = 0; i < my_tiles * (nsb + 1); ++i) {
        if (!wait(&acc_empty[i & 1], static_cast<uint32_t>(i >> 1) & 1u)) break;
        mbar_arrive_remote(cluster_addr(&acc_empty[i & 1], 0));
      }
    }
  } else if (wg == 2) {  // warps 8..11: unpack whole k-tiles (all 128 rows) in turn
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDqRegs));
    const int dw = warp - kEpiWarps;
    int e = 0;
    // Row r of a CTA's tile: with gate | up, 16 gate rows and 16 up rows of every 32.
    auto raw_row = [&](int r) { return p.half ? ((r & 16) ? TM / 2 : 0) + (r >> 5) * 16 + (r & 15) : r; };
    // k-tiles dw, dw + 4, ... of the pair's tiles: stage s in its round-th turn; a main one is chunk km % 4 of the raw super-block in
    // `slot` in that one's `turn`-th turn (a warp has one k-tile of each)
    static_assert(kDqWarps < STAGES, "a step passes one turn of the ring at most");
    int s = dw, round = 0, slot = 0, turn = 0, kt = dw;
    for (int tk = 0; tk < my_tiles; ++tk, kt -= kt_tile) {
      const Tile t = find_tile(tk, e);
      e = t.e;
      // headers of the two super-blocks of min-term tile m, four rows of this lane: asked for long before they are needed (at the
      // start of a tile they cost 2.5 us)
      uint4 head[2][TM / 32];
      auto ask = [&](int m) {
        const long long r0 = row0_of(t), last = static_cast<long long>(p.E) * p.N - 1;
#pragma unroll
        for (int i = 0; i < TM / 32; ++i) {
          const int r = raw_row(32 * i + lane);
          const long long row = min(r0 + (p.half && r >= TM / 2 ? p.half + r - TM / 2 : r), last);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            head[j][i] = 2 * m + j < nsb ? ldg128(p.w + row * p.row_bytes + (2 * m + j) * 144) : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      ask((kt - 4 * nsb) & 3);  // this warp's first one: k-tiles 4 nsb + m = kt modulo 4
      bool ok = true;
      for (; kt < kt_tile; kt += kDqWarps) {
        const bool main = kt < 4 * nsb;
        uint8_t* wt = smem + s * kStageBytes;
        // every lane waits; the outcome is made warp-uniform so that no lane leaves the loop alone
        ok = (!main || wait(&raw_full[slot], static_cast<uint32_t>(turn) & 1u)) && (round == 0 || wait(&empty[s], static_cast<uint32_t>(round - 1) & 1u));
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        if (main) {
          const uint8_t* rs = raw + slot * kRawBytes;
          float* d = dscale + ((tk * (nsb + 1) + (kt >> 2)) % kScaleGroups) * TM + lane;
#pragma unroll 1
          for (int i = 0; i < TM / 32; ++i, d += 32) {
            const uint32_t head0 = unpack_row(rs + raw_row(32 * i + lane) * 144, kt & 3, wt, 32 * i + lane);
            if ((kt & 3) == 0) *d = half_bits_to_float(head0 & 0xFFFFu);
          }
        } else {
          uint32_t big = 0u;
#pragma unroll
          for (int i = 0; i < TM / 32; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) big = max(big, head[j][i].x & 0x7FFF0000u);
          if (big >= 0x4C100000u) {
#pragma unroll
            for (int i = 0; i < TM / 32; ++i)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                if (min_past(head[j][i])) atomicOr(&g_moe_tc_errors, 4u);
          }
#pragma unroll
          for (int i = 0; i < TM / 32; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) min_row(head[j][i], j, wt, 32 * i + lane);
          if (kt + kDqWarps < kt_tile) ask(kt + kDqWarps - 4 * nsb);
        }
        fence_proxy_async_smem();  // generic-proxy writes -> visible to the tensor core
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive_local(&full[s]);
          else mbar_arrive_remote(cluster_addr(&full[s], 0));
          if (main) mbar_arrive_local(&raw_empty[slot]);
        }
        if (main) {
          if (++slot == RAW_STAGES) slot = 0, ++turn;
        }
        s += kDqWarps;
        if (s >= STAGES) s -= STAGES, ++round;
      }
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
    }
  } else {  // warps 0..7: epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int quarter = warp & 3, part = warp >> 2;
    const bool low = lane < 16;
    int grp = 0, e = 0;
    bool stop = false;
    for (int i = 0; i < my_tiles && !stop; ++i) {
      const Tile t = find_tile(i, e);
      e = t.e;
      // this thread's weight row of the expert, and the warp's columns: rows c0 .. c0 + t.h - 1 of the tile
      int n;
      bool nok;
      if (p.half) {
        n = t.row_tile * TM + static_cast<int>(rank) * (TM / 2) + quarter * 16 + (lane & 15);
        nok = n < p.half;
      } else {
        n = (2 * t.row_tile + static_cast<int>(rank)) * TM + quarter * 32 + lane;
        nok = n < p.N;
      }
      const int c0 = part * t.h;
      uint32_t tags[TN / 64];  // of the columns, asked for here: the last sums are not to wait for them
#pragma unroll
      for (int b = 0; b < TN / 64; ++b) {
        const int c = 32 * b + lane;
        tags[b] = c0 + c < t.n && c < t.h ? p.tags[t.first + c0 + c] : kNoPair;
      }
      uint16_t* act = p.act + n;
      float* y = p.y + n;
      float acc[TN / 2];
#pragma unroll
      for (int c = 0; c < TN / 2; ++c) acc[c] = 0.f;
      for (int g = 0; g <= nsb; ++g, ++grp) {
        const int buf = grp & 1;
        const bool ok = wait(&acc_full[buf], static_cast<uint32_t>(grp / 2) & 1u);
        if (!__all_sync(0xFFFFFFFFu, ok)) { stop = true; break; }
        tc_fence_after();
        const float scale = g == nsb ? 1.0f : dscale[grp % kScaleGroups * TM + quarter * 32 + lane];
        const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * TN + c0);
#pragma unroll
        for (int c = 0; c < TN / 2; c += 32) {
          if (c < t.h) {  // up to 16 columns past the part's own are read and never stored
            uint32_t v[32];
            tmem_ld32(base + (uint32_t)c, v);
#pragma unroll
            for (int k = 0; k < 32; ++k) acc[c + k] = __fmaf_rn(scale, __uint_as_float(v[k]), acc[c + k]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_local(&acc_empty[buf]);
      }
      if (stop) break;
      bool bad = false;  // a place of this expert without a pair of this call. Asked here: with the tags it would wait for them (158 -> 161 us)
#pragma unroll
      for (int b = 0; b < TN / 64; ++b) {
        if ((tags[b] & 0x7FFFFFu) >= static_cast<uint32_t>(p.P)) tags[b] = kBadPair;
        bad |= tags[b] > kNoPair;
      }
      if (bad) atomicOr(&g_moe_tc_errors, 2u);
      // results: acc * 2^-e of the column's row, to the row's pair. Nothing branches, so that the columns' chains of shuffles and
      // exponentials run beside each other
#pragma unroll
      for (int b = 0; b < TN / 2; b += 32) {
        if (b < t.h) {
          const uint32_t tag = tags[b / 32];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const uint32_t t0 = __shfl_sync(0xFFFFFFFFu, tag, c), t1 = __shfl_sync(0xFFFFFFFFu, tag, c + 1);
            acc[b + c] *= __uint_as_float(t0 & 0x7F800000u), acc[b + c + 1] *= __uint_as_float(t1 & 0x7F800000u);
            if (!p.half) {
              store_if(nok && t0 < kNoPair, y + (size_t)(t0 & 0x7FFFFFu) * p.N, acc[b + c]);
              store_if(nok && t1 < kNoPair, y + (size_t)(t1 & 0x7FFFFFu) * p.N, acc[b + c + 1]);
            }
          }
          if (p.half) {  // lanes 0..15 hold gate rows and take column c, lanes 16..31 up rows and column c + 1
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const uint32_t q = __shfl_sync(0xFFFFFFFFu, tag, c + (low ? 0 : 1));
              const float o = __shfl_xor_sync(0xFFFFFFFFu, low ? acc[b + c + 1] : acc[b + c], 16);
              const uint16_t v = silu_mul(low ? acc[b + c] : o, low ? o : acc[b + c + 1]);
              store_if(nok && q < kNoPair, act + (size_t)(q & 0x7FFFFFu) * p.half, v);
            }
          }
        }
      }
    }
  }
  // After an abort, copies issued before it may still be landing: give them time before either CTA can exit.
  if (threadIdx.x == 0 && aborted()) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster.sync();  // no remote arrival or MMA operand read is still aimed at either CTA
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// The pre-pass: a warp per row, in the plan's order. x' = fp16(x 2^e), exact for values
// within 2^28 of the row's largest (which lands in [2^14, 2^15)); behind the K values, per super-block, S_hi x 8, S_lo x 8, S_hi x 8,
// zeros x 8, S / 64 = hi + lo of the 32 x' of each sub-block. tags: the bits of 2^-e and the row's pair, below 2^23, in one word, or
// kBadPair: of every place, as the product goes by each expert's own offsets, whatever the last one says.
struct PrepParams {
  const uint16_t* x;
  long long xs;
  int div;  // pairs per row of x
  const int* order;
  int P, K, cols;
  __half* xc;
  uint32_t* tags;
};
constexpr int kPrepWarps = 8, kPrepKeep = 8;

__global__ void __launch_bounds__(kPrepWarps * 32) moe_prep_kernel(const PrepParams p) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, nch = p.K / 8;  // 16-byte parts of a row
  for (int r = blockIdx.x * kPrepWarps + (threadIdx.x >> 5); r < p.P; r += gridDim.x * kPrepWarps) {
    const int pair = p.order[r];
    if (pair < 0 || pair >= p.P) {  // behind the last expert's rows, or a plan out of bounds, which the product tells apart
      if (lane == 0) p.tags[r] = kBadPair;
      continue;
    }
    const uint16_t* src = p.x + (long long)(pair / p.div) * p.xs;
    uint4 keep[kPrepKeep];
    unsigned best = 0u;
    auto most = [&](const uint4& v) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) best = max(best, max((w[i] & 0x7FFFu) << 16, w[i] & 0x7FFF0000u));
    };
#pragma unroll
    for (int i = 0; i < kPrepKeep; ++i) {
      const int c = lane + 32 * i;
      keep[i] = c < nch ? ldg128(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kPrepKeep; ++i) most(keep[i]);
    for (int c = lane + 32 * kPrepKeep; c < nch; c += 32) most(ldg128(src + 8 * c));
    best = __reduce_max_sync(0xFFFFFFFFu, best);
    const int E = static_cast<int>(best >> 23);
    int ex = 0;
    if (best != 0u && E < 255) ex = max(-126, min(126, 14 - (E == 0 ? -126 : E - 127)));
    const float sc = __int_as_float((ex + 127) << 23);
    if (lane == 0) p.tags[r] = __float_as_uint(1.0f / sc) | static_cast<uint32_t>(pair);
    __half* dst = p.xc + (long long)r * p.cols;
    auto put = [&](int c, const uint4& v) {  // all lanes; a sub-block's four parts are in adjacent lanes
      float s = 0.f;
      if (c < nch) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[i] = f2_to_h2(__uint_as_float(w[i] << 16) * sc, __uint_as_float(w[i] & 0xFFFF0000u) * sc);
          s += half_bits_to_float(o[i]);
          s += half_bits_to_float(o[i] >> 16);
        }
        *reinterpret_cast<uint4*>(dst + 8 * c) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
      if (c < nch) {
        const float s64 = s * 0.015625f;
        const __half hi = __float2half_rn(s64), lo = __float2half_rn(s64 - __half2float(hi));
        const int sb = c >> 5, g = (c >> 2) & 7, j = c & 3;  // lane j of the four writes column 8 j + g
        dst[p.K + 32 * sb + 8 * j + g] = j == 3 ? __ushort_as_half(0) : j == 1 ? lo : hi;
      }
    };
#pragma unroll
    for (int i = 0; i < kPrepKeep; ++i)
      if (32 * i < nch) put(lane + 32 * i, keep[i]);
    for (int c = lane + 32 * kPrepKeep; c < nch + lane; c += 32) put(c, c < nch ? ldg128(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u));
    for (int c = p.K / 8 * 9 + lane; c < p.cols; c += 32) dst[c] = __ushort_as_half(0);  // an odd number of super-blocks
  }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                   const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

int columns(int K) { return K + (K / 256 + 1) / 2 * BK; }

}  // namespace

size_t moe_tc_workspace(int P, int K) {
  auto al = [](size_t v) { return (v + 255) & ~size_t(255); };
  return al((size_t)P * columns(K) * 2) + al((size_t)P * 4);
}

int launch_moe_tc(const MoeGemmArgs& a, bool gate_up, float* parts, void* ws, int num_sms, cudaStream_t s, std::string* err) {
  auto al = [](size_t v) { return (v + 255) & ~size_t(255); };
  const int P = a.T * a.k, cols = columns(a.K), N = gate_up ? 2 * a.N : a.N;
  __half* xc = static_cast<__half*>(ws);
  uint32_t* tags = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + al((size_t)P * cols * 2));
  const PrepParams pp = {static_cast<const uint16_t*>(a.x), a.xs, gate_up ? a.k : 1, a.order, P, a.K, cols, xc, tags};
  if (launch_pdl(moe_prep_kernel, dim3(std::min((P + kPrepWarps - 1) / kPrepWarps, 64 * num_sms)), dim3(kPrepWarps * 32), 0, s, pp, "moe pre-pass", err))
    return -1;

  static const EncodeTiledFn enc = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult qr;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &qr) == cudaSuccess &&
                    qr == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<EncodeTiledFn>(f) : nullptr;
  }();
  const long long row_bytes = (long long)kq_row_bytes(a.fmt, a.K);
  CUtensorMap xmap, wmap;
  CUresult cr = CUDA_ERROR_NOT_FOUND;
  if (enc) {
    const cuuint64_t dx[2] = {(cuuint64_t)cols, (cuuint64_t)P}, sx[1] = {(cuuint64_t)cols * 2};
    const cuuint64_t dw[2] = {(cuuint64_t)(row_bytes / 4), (cuuint64_t)a.E * N}, sw[1] = {(cuuint64_t)row_bytes};
    const cuuint32_t bx[2] = {(cuuint32_t)BK, (cuuint32_t)kBoxRows}, bw[2] = {36u, (cuuint32_t)(TM / 2)}, es[2] = {1u, 1u};
    cr = enc(&xmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, xc, dx, sx, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (cr == CUDA_SUCCESS)
      cr = enc(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(a.w), dw, sw, bw, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  if (cr != CUDA_SUCCESS) {
    *err = "cuTensorMapEncodeTiled failed (" + std::to_string((int)cr) + ")";
    return -1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = kTcSmem;
  cfg.stream = s;
  static std::atomic<int> resident[64];  // pairs that fit the device at once
  int dev = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  int n = ce == cudaSuccess && dev < 64 ? resident[dev].load() : 0;
  if (ce == cudaSuccess && n == 0) {
    ce = cudaFuncSetAttribute(moe_q4k_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
    // the warpgroups' shares of registers add up to exactly 512 threads x kLaunchRegs: a build that starts with fewer would
    // leave the epilogue's increase waiting forever
    cudaFuncAttributes fa;
    if (ce == cudaSuccess) ce = cudaFuncGetAttributes(&fa, moe_q4k_tc_kernel);
    if (ce == cudaSuccess && fa.numRegs != kLaunchRegs) {
      *err = "internal: the experts' tensor-core product was built with " + std::to_string(fa.numRegs) + " registers per thread";
      return -1;
    }
    if (ce == cudaSuccess && (cudaOccupancyMaxActiveClusters(&n, moe_q4k_tc_kernel, &cfg) != cudaSuccess || n <= 0)) {
      cudaGetLastError();
      n = num_sms / 2;
    }
    if (ce == cudaSuccess && dev < 64) resident[dev].store(n);
  }
  if (ce != cudaSuccess) {
    *err = std::string("moe tensor-core product: ") + cudaGetErrorString(ce);
    return -1;
  }
  const TcParams p = {static_cast<const uint8_t*>(a.w), tags, a.offsets, a.order, a.E, P, N, a.K, gate_up ? a.N : 0, parts,
                      static_cast<uint16_t*>(a.act), row_bytes, (a.K / 256 + 1) / 2, gate_up ? (a.N + TM - 1) / TM : (a.N + 2 * TM - 1) / (2 * TM)};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(2 * n);
  ce = cudaLaunchKernelEx(&cfg, moe_q4k_tc_kernel, xmap, wmap, p);
  if (ce != cudaSuccess) {
    *err = std::string("moe tensor-core product launch: ") + cudaGetErrorString(ce);
    return -1;
  }
  return 0;
}

unsigned int take_moe_tc_errors() {
  unsigned int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_moe_tc_errors, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  cudaMemcpyToSymbol(g_moe_tc_errors, &z, sizeof(z));
  return v;
}

}  // namespace kq
