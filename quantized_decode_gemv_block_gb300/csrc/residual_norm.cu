// Closing a block: its output's norm, gate and residual scale, the sum with the residual stream, and the norm that the
// next block reads, in one pass.
//
//   z = y, or y / sqrt(mean y^2 + eps) * post      h' = h + scale * gate * z      x = h' / sqrt(mean h'^2 + eps) * pre
//
// Everything between loading and storing is fp32 in registers; h' and x are each rounded once, x from the unrounded h'.
// A row belongs to a group of threads that its length alone sets: thread t takes the parts of eight elements t, t + n,
// ... and sums their squares in order, a butterfly adds the warp's lanes and the warps follow in order. So a row's bits
// depend neither on the other rows nor on whether its address allows wide loads.
//
// Bound by DRAM: each array is read and written once. 8192 rows of 4096 (bf16 y and gate, fp32 residual, bf16 x) take 81 us, 5.8 TB/s.
#include <cuda_bf16.h>

#include <cstdint>

#include "kq.h"
#include "kq_device.cuh"
#include "kq_internal.h"
#include "kq_launch.cuh"

namespace kq {
namespace {

constexpr int kPart = 8;  // elements of a thread's part: 16 bytes of bf16, 32 of fp32

struct NormParams {
  ResidualNormArgs a;
  int group;  // threads of a row, a multiple of 32
  int rows;   // rows of a CTA
};

// Part `c` of a row: elements 8c .. 8c+7, zeros from `H` on.
template <bool VEC>
__device__ __forceinline__ void load_part(float (&v)[kPart], const float* row, int c, int H) {
  if constexpr (VEC) {
    const float4 a = *reinterpret_cast<const float4*>(row + 8 * c), b = *reinterpret_cast<const float4*>(row + 8 * c + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < kPart; ++i) v[i] = 8 * c + i < H ? row[8 * c + i] : 0.f;
  }
}
template <bool VEC>
__device__ __forceinline__ void load_part(float (&v)[kPart], const uint16_t* row, int c, int H) {
  if constexpr (VEC) {
    const uint4 a = *reinterpret_cast<const uint4*>(row + 8 * c);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPart; ++i) v[i] = 8 * c + i < H ? __uint_as_float((uint32_t)row[8 * c + i] << 16) : 0.f;
  }
}
template <bool VEC>
__device__ __forceinline__ void store_part(float* row, const float (&v)[kPart], int c, int H) {
  if constexpr (VEC) {
    *reinterpret_cast<float4*>(row + 8 * c) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(row + 8 * c + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < kPart; ++i)
      if (8 * c + i < H) row[8 * c + i] = v[i];
  }
}
template <bool VEC>
__device__ __forceinline__ void store_part(uint16_t* row, const float (&v)[kPart], int c, int H) {
  if constexpr (VEC) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    *reinterpret_cast<uint4*>(row + 8 * c) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < kPart; ++i)
      if (8 * c + i < H) row[8 * c + i] = f32_to_bf16_rn(v[i]);
  }
}
// The same of either type.
template <bool VEC>
__device__ __forceinline__ void load_any(float (&v)[kPart], const void* row, int dtype, int c, int H) {
  if (dtype == KQ_F32) load_part<VEC>(v, static_cast<const float*>(row), c, H);
  else load_part<VEC>(v, static_cast<const uint16_t*>(row), c, H);
}
// Sum over the row's group of threads, the same in all of them. part: one word per warp of the CTA. The groups of a CTA meet at
// barriers of their own.
__device__ __forceinline__ float group_sum(float s, float* part, int group) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  if (group == 32) return s;
  const int warp = threadIdx.x / 32, row = threadIdx.x / group, first = row * (group / 32);
  if (threadIdx.x % 32 == 0) part[warp] = s;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + row), "r"(group) : "memory");
  s = part[first];
  for (int w = 1; w < group / 32; ++w) s += part[first + w];
  return s;
}

template <typename Y, typename R, int PARTS, bool VEC>
__global__ void __launch_bounds__(PARTS > 2 ? 1024 : 512) residual_norm_kernel(const NormParams p) {
  __shared__ float sums[4][32];
  const ResidualNormArgs& a = p.a;
  grid_launch_dependents();
  grid_dependency_wait();
  const int H = a.H, tid = threadIdx.x % p.group, parts = (H + kPart - 1) / kPart;
  const long long row = (long long)blockIdx.x * p.rows + threadIdx.x / p.group;
  const bool live = row < a.T;  // the last CTA's groups without a row
  const long long t = live ? row : 0;

  float v[PARTS][kPart], h[PARTS][kPart];
  const Y* y = a.y ? static_cast<const Y*>(a.y) + t * a.ys : nullptr;
  const R* r = a.h ? static_cast<const R*>(a.h) + t * a.hs : nullptr;
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const int c = tid + i * p.group;
#pragma unroll
    for (int j = 0; j < kPart; ++j) v[i][j] = 0.f;
    if (PARTS <= 2) {
#pragma unroll
      for (int j = 0; j < kPart; ++j) h[i][j] = 0.f;
    }
    if (c < parts && live) {
      if (y) load_part<VEC>(v[i], y, c, H);
      if (r && PARTS <= 2) load_part<VEC>(h[i], r, c, H);  // four parts of both do not fit 64 registers
    }
  }
  auto norm = [&](float (&u)[PARTS][kPart], const void* w, float (*part)[32]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
#pragma unroll
      for (int j = 0; j < kPart; ++j) s = __fmaf_rn(u[i][j], u[i][j], s);
    s = group_sum(s, part[0], p.group);
    float mean = s / (float)H + a.eps;
    // Squares past fp32: the row again at 2^-96, next to which eps is nothing; below it, under an eps of as good as none: at 2^96
    if (mean < 0x1p-100f || s == INFINITY) {
      const bool large = s == INFINITY;
      const float to = large ? 0x1p-96f : 0x1p96f;
      s = 0.f;
#pragma unroll
      for (int i = 0; i < PARTS; ++i)
#pragma unroll
        for (int j = 0; j < kPart; ++j) {
          u[i][j] *= to;
          s = __fmaf_rn(u[i][j], u[i][j], s);
        }
      s = group_sum(s, part[1], p.group);
      mean = s / (float)H + (large ? 0.f : a.eps * to * to);
    }
    const float f = rsqrtf(mean);
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const int c = tid + i * p.group;
      if (c < parts) {
#pragma unroll
        for (int j = 0; j < kPart; ++j) u[i][j] *= f;
        if (w) {
          float g[kPart];
          load_any<VEC>(g, w, a.w_dtype, c, H);
#pragma unroll
          for (int j = 0; j < kPart; ++j) u[i][j] *= g[j] + a.offset;
        }
      }
    }
  };
  if (a.norm_y) norm(v, a.post, sums);
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const int c = tid + i * p.group;
    if (PARTS > 2) {
#pragma unroll
      for (int j = 0; j < kPart; ++j) h[i][j] = 0.f;
    }
    if (c < parts) {
      if (r && PARTS > 2 && live) load_part<VEC>(h[i], r, c, H);
      if (a.gate) {
        float g[kPart];
        load_part<VEC>(g, static_cast<const Y*>(a.gate) + t * a.gs, c, H);
#pragma unroll
        for (int j = 0; j < kPart; ++j) v[i][j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < kPart; ++j) h[i][j] = __fmaf_rn(a.scale, v[i][j], h[i][j]);
      if (a.h_out && live) store_part<VEC>(static_cast<R*>(a.h_out) + t * a.hos, h[i], c, H);
    }
  }
  if (!a.x) return;
  norm(h, a.pre, sums + 2);
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const int c = tid + i * p.group;
    if (c < parts && live) {
      if (a.x_dtype == KQ_F32) store_part<VEC>(static_cast<float*>(a.x) + t * a.xs, h[i], c, H);
      else store_part<VEC>(static_cast<uint16_t*>(a.x) + t * a.xs, h[i], c, H);
    }
  }
}

template <typename Y, typename R, int PARTS>
int launch_typed(const NormParams& p, bool vec, cudaStream_t s, std::string* err) {
  const dim3 grid((unsigned)((p.a.T + p.rows - 1) / p.rows)), block(p.group * p.rows);
  return vec ? launch_pdl(residual_norm_kernel<Y, R, PARTS, true>, grid, block, 0, s, p, "residual_norm", err)
             : launch_pdl(residual_norm_kernel<Y, R, PARTS, false>, grid, block, 0, s, p, "residual_norm", err);
}
template <typename Y, typename R>
int launch_parts(const NormParams& p, int n, bool vec, cudaStream_t s, std::string* err) {
  return n == 1 ? launch_typed<Y, R, 1>(p, vec, s, err) : n == 2 ? launch_typed<Y, R, 2>(p, vec, s, err) : launch_typed<Y, R, 4>(p, vec, s, err);
}

}  // namespace

int launch_residual_norm(const ResidualNormArgs& a, cudaStream_t s, std::string* err) {
  NormParams p;
  p.a = a;
  const int parts = (a.H + kPart - 1) / kPart;
  // Parts of a thread. What counts is how many rows are in flight: at 4096 four parts in 64 registers (8192 rows with a gate 81 us) beat
  // two with everything asked for at once (90), at 2560 two (54) beat four (57), at 2048 two (39) one (45)
  const int n = parts <= 64 ? 1 : parts <= 400 ? 2 : 4;
  p.group = ((parts + n - 1) / n + 31) / 32 * 32;
  p.rows = p.group >= 256 ? 1 : 256 / p.group;
  // wide loads: every row of every array that is there starts on a part's boundary
  auto wide = [](const void* q, long long stride, int dtype) {
    return !q || (reinterpret_cast<uintptr_t>(q) % 16 == 0 && stride * (dtype == KQ_F32 ? 4 : 2) % 16 == 0);
  };
  const bool vec = a.H % kPart == 0 && wide(a.y, a.ys, a.y_dtype) && wide(a.h, a.hs, a.h_dtype) && wide(a.h_out, a.hos, a.h_dtype) &&
                   wide(a.x, a.xs, a.x_dtype) && wide(a.gate, a.gs, a.y_dtype) && wide(a.post, 0, a.w_dtype) && wide(a.pre, 0, a.w_dtype);
  const bool yf = a.y_dtype == KQ_F32, hf = a.h_dtype == KQ_F32;
  if (yf) return hf ? launch_parts<float, float>(p, n, vec, s, err) : launch_parts<float, uint16_t>(p, n, vec, s, err);
  return hf ? launch_parts<uint16_t, float>(p, n, vec, s, err) : launch_parts<uint16_t, uint16_t>(p, n, vec, s, err);
}

}  // namespace kq
