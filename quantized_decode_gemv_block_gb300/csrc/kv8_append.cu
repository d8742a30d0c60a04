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
// The tokens of one call that share a page stand next to each other with ascending slots (a run).
// The CTA whose token range holds a run's first token takes the whole run for one head and one of
// k / v: a pass for max|x| (16-byte loads), then a pass that reads the values again (from L1 / L2)
// and writes codes in the cache's order (kv8.cuh), 16 bytes per thread where a group of 16 tokens
// is whole. No CTA waits for another and no atomics meet in memory, so results never vary.
#include <cuda_bf16.h>

#include <cstdint>

#include "kq.h"
#include "kq_device.cuh"
#include "kq_internal.h"
#include "kq_launch.cuh"
#include "kv8.cuh"

namespace kq {
namespace {

constexpr int kThreads = 128;

__device__ unsigned int g_kv8_append_errors = 0;  // bit 1: a slot beyond the cache's pages

struct AppendParams {
  const void* x[2];  // k, v
  long long xs[2];   // elements between tokens
  int8_t* codes[2];
  float* scale[2];
  const int* slot;
  int T, log2p, n_pages, n_kv, D, range;
};

template <typename X>
__device__ __forceinline__ float value(const X* p);
template <>
__device__ __forceinline__ float value<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float value<uint16_t>(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

__device__ __forceinline__ void value4(float (&v)[4], const float* p) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x;
  v[1] = x.y;
  v[2] = x.z;
  v[3] = x.w;
}
__device__ __forceinline__ void value4(float (&v)[4], const uint16_t* p) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(x.x << 16);
  v[1] = __uint_as_float(x.x & 0xFFFF0000u);
  v[2] = __uint_as_float(x.y << 16);
  v[3] = __uint_as_float(x.y & 0xFFFF0000u);
}

// floor(x * inv) as a byte; inv is a power of two (or 0: every code is 0). A negative x whose
// product rounds to zero still has floor -1.
__device__ __forceinline__ uint32_t code(float x, float inv) {
  int c = __float2int_rd(x * inv);
  if (x < 0.f && inv > 0.f) c = min(c, -1);
  return (uint32_t)c & 0xFFu;
}

// Each byte of w shifted right arithmetically by n (0..7).
__device__ __forceinline__ uint32_t shift_bytes(uint32_t w, int n) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) r |= ((uint32_t)((int)(int8_t)(w >> (8 * i)) >> n) & 0xFFu) << (8 * i);
  return r;
}

template <typename X>
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(const AppendParams p) {
  __shared__ int sm_run;
  __shared__ unsigned sm_max[kThreads / 32];
  const int tid = threadIdx.x, h = blockIdx.y, which = blockIdx.z;
  const int P = 1 << p.log2p, D = p.D;
  grid_dependency_wait();
  const int t0 = blockIdx.x * p.range, t1 = min(t0 + p.range, p.T);
  for (int t = t0; t < t1; ++t) {
    const int s0 = p.slot[t];
    if (s0 < 0) continue;
    const int page = s0 >> p.log2p, at = s0 & (P - 1);
    if (page >= p.n_pages) {
      if (tid == 0) atomicOr(&g_kv8_append_errors, 2u);
      continue;
    }
    if (t > 0 && at > 0 && p.slot[t - 1] == s0 - 1) continue;  // inside a run
    // the run's length: up to the page's end
    if (tid == 0) sm_run = min(P - at, p.T - t);
    __syncthreads();
    if (tid < min(P - at, p.T - t) && p.slot[t + tid] != s0 + tid) atomicMin(&sm_run, tid);
    __syncthreads();
    const int n = sm_run;
    const long long xs = which ? p.xs[1] : p.xs[0];
    const X* x = static_cast<const X*>(which ? p.x[1] : p.x[0]) + t * xs + (long long)h * D;
    // largest |x| by its bits: a NaN or infinity is above every finite value
    unsigned top = 0;
    for (int i = tid; i < n * (D / 4); i += kThreads) {
      const int j = i / (D / 4), d = (i - j * (D / 4)) * 4;
      float v[4];
      value4(v, x + j * xs + d);
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    }
    top = __reduce_max_sync(~0u, top);
    if ((tid & 31) == 0) sm_max[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) top = max(top, sm_max[i]);
    float* sp = (which ? p.scale[1] : p.scale[0]) + (long long)page * p.n_kv + h;
    const float old = at ? *sp : 0.f;  // a run from offset 0 starts the page afresh
    const unsigned ex = top >> 23;
    float need = top == 0 ? 0.f : __uint_as_float((ex > 7 ? ex - 6 : 1u) << 23);  // never below 2^-126
    if (ex == 0xFF) need = __uint_as_float(0x7FC00000u);
    const bool broken = old != old || need != need;
    const float now = broken ? __uint_as_float(0x7FC00000u) : fmaxf(old, need);
    const float inv = broken || now == 0.f ? 0.f : __uint_as_float((254u - (__float_as_uint(now) >> 23)) << 23);
    int shift = 0;
    if (!broken && old > 0.f && now > old)
      shift = min((int)(__float_as_uint(now) >> 23) - (int)(__float_as_uint(old) >> 23), 7);
    __syncthreads();  // every thread has read the old scale and the maxima
    if (tid == 0) *sp = now;
    int8_t* codes = (which ? p.codes[1] : p.codes[0]) + ((long long)page * p.n_kv + h) * P * D;
    const int g0 = shift ? 0 : at >> 4, g1 = shift ? P >> 4 : (at + n + 15) >> 4;
    for (int i = tid; i < (g1 - g0) * D; i += kThreads) {
      const int grp = g0 + i / D, ci = i % D, c = ci >> 5, g = (ci >> 2) & 7, q4 = ci & 3;
      uint4* dst = reinterpret_cast<uint4*>(codes + grp * 16 * D + ci * 16);
      const int rel = grp * 16 - at;  // the group's first token in the run
      uint32_t w[4], m[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = m[k] = 0;
      if (which == 0) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int j = rel + 4 * (g >> 1) + 2 * half + (g & 1);
          if (j < 0 || j >= n) continue;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            float v[4];
            value4(v, x + j * xs + 32 * c + 16 * s + 4 * q4);
            w[2 * s + half] = code(v[0], inv) | code(v[1], inv) << 8 | code(v[2], inv) << 16 | code(v[3], inv) << 24;
            m[2 * s + half] = ~0u;
          }
        }
      } else {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int j = rel + 4 * q4 + b;
          if (j < 0 || j >= n) continue;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            w[k] |= code(value<X>(x + j * xs + 32 * c + 8 * k + g), inv) << (8 * b);
            m[k] |= 0xFFu << (8 * b);
          }
        }
      }
      if ((m[0] & m[1] & m[2] & m[3]) == ~0u) {
        *dst = make_uint4(w[0], w[1], w[2], w[3]);
      } else if (shift) {
        const uint4 o = *dst;
        *dst = make_uint4((shift_bytes(o.x, shift) & ~m[0]) | w[0], (shift_bytes(o.y, shift) & ~m[1]) | w[1],
                          (shift_bytes(o.z, shift) & ~m[2]) | w[2], (shift_bytes(o.w, shift) & ~m[3]) | w[3]);
      } else {
        uint32_t* dw = reinterpret_cast<uint32_t*>(dst);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (m[k] == ~0u) dw[k] = w[k];
          else if (m[k]) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
              if (m[k] >> (8 * b) & 1) reinterpret_cast<uint8_t*>(dw + k)[b] = (uint8_t)(w[k] >> (8 * b));
          }
        }
      }
    }
    __syncthreads();  // the shared words are used again by the next run
  }
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
  p.D = c.D;
  // tokens per CTA: one while the grid is small (runs are short: single tokens in parallel), up to a page
  const long long units = (long long)T * c.n_kv * 2;
  long long range = units / ((long long)num_sms * 16);
  p.range = (int)(range < 1 ? 1 : range > (1 << c.log2p) ? (1 << c.log2p) : range);
  const dim3 grid((unsigned)((T + p.range - 1) / p.range), (unsigned)c.n_kv, 2);
  return x_dtype == KQ_F32 ? launch_pdl(kv8_append_kernel<float>, grid, dim3(kThreads), 0, s, p, "kv8_append", err)
                           : launch_pdl(kv8_append_kernel<uint16_t>, grid, dim3(kThreads), 0, s, p, "kv8_append", err);
}

}  // namespace kq
