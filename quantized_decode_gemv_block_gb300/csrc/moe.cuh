// Shared by the experts' products.
#pragma once
#include "kq_device.cuh"

namespace kq {

// bf16(silu(g) u), silu(g) = g / (1 + exp(-g)), by the fast exponential (off by 2 + 1.173 |g| units of 2^-23) and division (2 units):
// within 2^-20 of itself for g >= 0, where the exponential is at most half of the sum, within (5 + 1.2 |g|) 2^-23 for g < 0, which is
// 2^-16 at -80, and 0 from about -87 down; next to the 2^-8 of the rounding. The accurate ones were a tenth of a decoding batch's time.
__device__ __forceinline__ uint16_t silu_mul(float g, float u) { return f32_to_bf16_rn(__fdividef(g, 1.f + __expf(-g)) * u); }

}  // namespace kq
