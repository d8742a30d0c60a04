// Rotary positions with one or more position axes (one for text; time, height and width for
// images and video), on q and k in one launch.
//
// Pair i of a head, (a, b), turns by the angle pos[axis_i][t] * freq_i:
//     a' = a cos - b sin,  b' = b cos + a sin;
// the inverse rotation (the gradient of the forward one) turns by the negative angle.
//
// The angle is formed as a binary fraction of a turn in 64-bit integers, so that positions of any
// size lose nothing: freq = m 2^e (24-bit m) gives F = m C 2^(e-2), C = round(2^64 * 2/pi), the
// turn fraction per position in units of 2^-64 (error below 1 + freq / 8 units); pos * F
// modulo 2^64 is the phase, exact but for pos times that. A frequency that is not finite gives NaN. Its top 32 bits are cut into the nearest
// quarter turn and a rest in [-1/8, 1/8] turn, whose sine and cosine come from sincospif.
//
// Bound by DRAM: q and k are read and written once. A CTA forms the angles of its tokens once, in
// shared memory, and turns up to eight pairs per thread and turn (16-byte accesses for bf16) of all of its
// heads. A prompt of 32768 tokens, 32 + 8 heads of 128 in bf16, takes 110 us, 6.1 TB/s read and written
// (115 us with five CTAs per SM, 123 with eight, whose registers spill). With the angles formed by each
// thread for eight heads, in registers, it took 116.5 us, and 1999 tokens of 20 heads of 64, which leave a
// thread one head, 8.8 us in place of 4.5.
//   Heads or halves that do not divide into 16-byte parts take 4 or 2 pairs at a time: 8192 tokens of 64 heads
// of 80, bf16, 20 dims turned, 59 us by twos and 90 by ones (25 us of DRAM traffic); 4203 tokens of 18 heads of 96,
// 24 dims turned, 11.1 us by fours, 14.8 by twos, 20.3 by ones.
#include <cuda_bf16.h>

#include <cstdint>

#include "kq.h"
#include "kq_device.cuh"
#include "kq_internal.h"
#include "kq_launch.cuh"

namespace kq {
namespace {

constexpr int kThreads = 256;
constexpr int kTable = 2048;  // angles of a CTA at most

struct RopeParams {
  const void *x0, *x1;  // q rows, k rows
  void *y0, *y1;
  long long xs0, xs1, ys0, ys1;  // elements between tokens
  int h0, h1;                    // heads
  int T, D, pairs;
  const float* freq;
  const unsigned char* axis;  // null: axis 0
  const int* pos;             // n_axes rows of T
  int n_axes;
  int inverse;
  int chunks;  // vector chunks of a head: pairs / V turned, then the copied rest
  int tokens;  // tokens of a CTA
  int heads;   // heads of a CTA (its share in blockIdx.y)
};

// Turn fraction per position of `freq` in units of 2^-64 (two's complement for freq < 0).
__device__ __forceinline__ unsigned long long turn_per_position(float freq) {
  const unsigned b = __float_as_uint(freq);
  const int ex = (b >> 23) & 0xFF;
  const unsigned long long m = ex ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu;
  const int sh = (ex ? ex : 1) - 150 - 2;  // freq = m 2^(ex - 150)
  constexpr unsigned long long C = 0xA2F9836E4E44152Aull;  // round(2^64 * 2 / pi)
  const unsigned long long lo = m * C, hi = __umul64hi(m, C);
  unsigned long long f;
  if (sh >= 64) f = 0;
  else if (sh >= 0) f = lo << sh;
  else if (sh > -64) f = (lo >> -sh) | (hi << (64 + sh));
  else if (sh > -128) f = hi >> (-sh - 64);
  else f = 0;
  return b >> 31 ? 0ull - f : f;
}

__device__ __forceinline__ float2 cos_sin_turn(unsigned long long turn, int pos) {
  const int ph = (int)((turn * (unsigned long long)(long long)pos) >> 32);
  const int quarter = (int)((unsigned)ph + 0x20000000u) >> 30;
  const int rest = (int)((unsigned)ph - ((unsigned)quarter << 30));
  float s, c;
  sincospif((float)rest * 4.656612873077393e-10f, &s, &c);  // rest 2^-31 half turns
  const float cc = quarter & 1 ? s : c, ss = quarter & 1 ? c : s;
  return make_float2((quarter + 1) & 2 ? -cc : cc, quarter & 2 ? -ss : ss);
}

// Two fp32 -> packed bf16 (lo = a), round to nearest even, one instruction.
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float a, float b) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
}

template <int V>
__device__ __forceinline__ void load(float (&v)[V], const float* p) {
  if (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 x = reinterpret_cast<const float4*>(p)[i];
      v[4 * i] = x.x;
      v[4 * i + 1] = x.y;
      v[4 * i + 2] = x.z;
      v[4 * i + 3] = x.w;
    }
  } else if (V == 2) {
    const float2 x = *reinterpret_cast<const float2*>(p);
    v[0] = x.x;
    v[V - 1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = p[i];
  }
}
template <int V>
__device__ __forceinline__ void load(float (&v)[V], const uint16_t* p) {
  if (V % 8 == 0) {
#pragma unroll
    for (int i = 0; i < V / 8; ++i) {
      const uint4 x = __ldcs(reinterpret_cast<const uint4*>(p) + i);  // read once
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  } else if (V % 2 == 0) {
    uint32_t w[2];
    if (V == 4) {
      const uint2 x = __ldcs(reinterpret_cast<const uint2*>(p));
      w[0] = x.x;
      w[1] = x.y;
    } else {
      w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
    }
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      v[2 * j] = __uint_as_float(w[j % 2] << 16);
      v[(2 * j + 1) % V] = __uint_as_float(w[j % 2] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = __uint_as_float((uint32_t)p[i] << 16);
  }
}
template <int V>
__device__ __forceinline__ void store(float* p, const float (&v)[V]) {
  if (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else if (V == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[V - 1]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = v[i];
  }
}
template <int V>
__device__ __forceinline__ void store(uint16_t* p, const float (&v)[V]) {
  if (V % 8 == 0) {
#pragma unroll
    for (int i = 0; i < V / 8; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = f32x2_to_bf16x2(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
      reinterpret_cast<uint4*>(p)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else if (V == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(f32x2_to_bf16x2(v[0], v[1 % V]), f32x2_to_bf16x2(v[2 % V], v[3 % V]));
  } else if (V == 2) {
    *reinterpret_cast<uint32_t*>(p) = f32x2_to_bf16x2(v[0], v[V - 1]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = f32_to_bf16_rn(v[i]);
  }
}

// V pairs per thread and turn: 8, 4 or 2 where every row, head and half starts on as many elements, else 1.
template <typename X, typename Y, int V, bool ADJ>
__global__ void __launch_bounds__(kThreads, sizeof(X) == 2 ? 6 : 5) rope_kernel(const RopeParams p) {
  __shared__ __align__(16) float sm_c[kTable], sm_s[kTable];  // [token][pair]
  const int t0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.T - t0), pairs = p.pairs;
  const int h0 = blockIdx.y * p.heads, nh = min(p.heads, p.h0 + p.h1 - h0);
  grid_dependency_wait();
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const int t = i / pairs, pr = i - t * pairs;
    const int ax = p.axis ? p.axis[pr] : 0;
    // an axis beyond the positions' rows turns nothing
    const int pos = ax < p.n_axes ? p.pos[(long long)ax * p.T + t0 + t] : 0;
    const float f = p.freq[pr];
    float2 cs = cos_sin_turn(turn_per_position(f), pos);
    if (ax < p.n_axes && (__float_as_uint(f) & 0x7F800000u) == 0x7F800000u) cs.x = cs.y = __uint_as_float(0x7FC00000u);
    sm_c[i] = cs.x;
    sm_s[i] = p.inverse ? -cs.y : cs.y;
  }
  __syncthreads();
  // (token, head, chunk) of a thread's turns, kThreads apart: chunks fastest
  const int turned = pairs / V, chunks = p.chunks;
  const int d_row = kThreads / chunks, d_ch = kThreads - d_row * chunks, d_t = d_row / nh, d_h = d_row - d_t * nh;
  int row = threadIdx.x / chunks, ch = threadIdx.x - row * chunks, t = row / nh, hh = row - t * nh;
#pragma unroll 1
  for (; t < nt; ch += d_ch, hh += d_h, t += d_t) {
    if (ch >= chunks) {
      ch -= chunks;
      ++hh;
    }
    if (hh >= nh) {
      hh -= nh;
      if (++t >= nt) break;
    }
    const int h = h0 + hh, i0 = ch * V;
    const bool turns = ch < turned, isq = h < p.h0;
    const int d0 = turns ? (ADJ ? 2 * i0 : i0) : 2 * pairs + (ch - turned) * 2 * V;
    const int d1 = turns && !ADJ ? i0 + pairs : d0 + V;
    const bool whole = d1 + V <= p.D;  // the copied rest may be odd: its last chunk is then one value
    const long long token = t0 + t, head = (long long)(isq ? h : h - p.h0) * p.D;
    const X* x = static_cast<const X*>(isq ? p.x0 : p.x1) + token * (isq ? p.xs0 : p.xs1) + head;
    Y* y = static_cast<Y*>(isq ? p.y0 : p.y1) + token * (isq ? p.ys0 : p.ys1) + head;
    float a[V], b[V];
    load<V>(a, x + d0);
    if (whole) load<V>(b, x + d1);
    if (!turns) {
      store<V>(y + d0, a);
      if (whole) store<V>(y + d1, b);
      continue;
    }
    float c[V], s[V], ra[V], rb[V];
    load<V>(c, sm_c + t * pairs + i0);
    load<V>(s, sm_s + t * pairs + i0);
    if (ADJ) {  // a, b hold 2 V adjacent values
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float u = 2 * k < V ? a[(2 * k) % V] : b[(2 * k) % V], w = 2 * k + 1 < V ? a[(2 * k + 1) % V] : b[(2 * k + 1) % V];
        const float nu = u * c[k] - w * s[k], nw = w * c[k] + u * s[k];
        if (2 * k < V) ra[(2 * k) % V] = nu;
        else rb[(2 * k) % V] = nu;
        if (2 * k + 1 < V) ra[(2 * k + 1) % V] = nw;
        else rb[(2 * k + 1) % V] = nw;
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        ra[k] = a[k] * c[k] - b[k] * s[k];
        rb[k] = b[k] * c[k] + a[k] * s[k];
      }
    }
    store<V>(y + d0, ra);
    store<V>(y + d1, rb);
  }
}

template <typename X, typename Y>
int launch_typed(const RopeParams& p, int V, bool adj, dim3 g, cudaStream_t s, std::string* err) {
  const dim3 b(kThreads);
  if (V == 8) return adj ? launch_pdl(rope_kernel<X, Y, 8, true>, g, b, 0, s, p, "rope", err)
                         : launch_pdl(rope_kernel<X, Y, 8, false>, g, b, 0, s, p, "rope", err);
  if (V == 4) return adj ? launch_pdl(rope_kernel<X, Y, 4, true>, g, b, 0, s, p, "rope", err)
                         : launch_pdl(rope_kernel<X, Y, 4, false>, g, b, 0, s, p, "rope", err);
  if (V == 2) return adj ? launch_pdl(rope_kernel<X, Y, 2, true>, g, b, 0, s, p, "rope", err)
                         : launch_pdl(rope_kernel<X, Y, 2, false>, g, b, 0, s, p, "rope", err);
  return adj ? launch_pdl(rope_kernel<X, Y, 1, true>, g, b, 0, s, p, "rope", err)
             : launch_pdl(rope_kernel<X, Y, 1, false>, g, b, 0, s, p, "rope", err);
}

bool starts_on(int bytes, const void* p, long long stride, int elem) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * elem % bytes == 0;
}

}  // namespace

int launch_rope(const RopeArgs& a, int num_sms, cudaStream_t s, std::string* err) {
  const int xe = a.x_dtype == KQ_F32 ? 4 : 2, ye = a.y_dtype == KQ_F32 ? 4 : 2;
  // rows, heads and halves of heads start on V elements, or on 16 bytes
  auto fits_v = [&](int v) {
    auto on = [&](const void* x, long long stride, int e) { return starts_on(e * v < 16 ? e * v : 16, x, stride, e); };
    return a.D % (2 * v) == 0 && a.rot_dim % (2 * v) == 0 && on(a.x0, a.xs0, xe) && on(a.x1, a.xs1, xe) &&
           on(a.y0, a.ys0, ye) && on(a.y1, a.ys1, ye);
  };
  const int V = fits_v(8) ? 8 : fits_v(4) ? 4 : fits_v(2) ? 2 : 1;
  RopeParams p = {a.x0, a.x1, a.y0, a.y1, a.xs0, a.xs1, a.ys0, a.ys1, a.h0, a.h1, a.T, a.D, a.rot_dim / 2,
                  a.freq, a.axis, a.pos, a.n_axes, a.inverse ? 1 : 0, 0, 0};
  p.chunks = p.pairs / V + (a.D - a.rot_dim + 2 * V - 1) / (2 * V);
  // A CTA takes as many tokens as give it four rounds of its threads, and fewer, down to one token and
  // one round of heads, while four CTAs per SM are not reached.
  const int H = a.h0 + a.h1;
  p.heads = H;
  const long long items = (long long)H * p.chunks;
  long long tokens = 4 * kThreads / items;
  const long long fill = a.T / (4LL * num_sms), fits = p.pairs ? kTable / p.pairs : kTable;
  tokens = tokens > fill ? fill : tokens;
  tokens = tokens > fits ? fits : tokens;
  p.tokens = (int)(tokens < 1 ? 1 : tokens);
  if (tokens < 1 && items > kThreads) {
    const long long groups = (items + kThreads - 1) / kThreads, want = (4LL * num_sms + a.T - 1) / a.T;
    p.heads = (int)((H + (groups < want ? groups : want) - 1) / (groups < want ? groups : want));
  }
  const dim3 g((unsigned)((a.T + p.tokens - 1) / p.tokens), (unsigned)((H + p.heads - 1) / p.heads));
  if (g.y > 65535) {
    *err = "rope: too many heads";
    return -1;
  }
  if (a.x_dtype == KQ_F32)
    return a.y_dtype == KQ_F32 ? launch_typed<float, float>(p, V, a.adjacent, g, s, err)
                               : launch_typed<float, uint16_t>(p, V, a.adjacent, g, s, err);
  return a.y_dtype == KQ_F32 ? launch_typed<uint16_t, float>(p, V, a.adjacent, g, s, err)
                             : launch_typed<uint16_t, uint16_t>(p, V, a.adjacent, g, s, err);
}

}  // namespace kq
