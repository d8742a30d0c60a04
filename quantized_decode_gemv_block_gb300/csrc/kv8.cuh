// The paged 8-bit KV cache: code order within a (page, kv head), shared by the append and the
// attention kernels.
//
// A page's tokens stand in groups of 16; a group holds 16 * D code bytes. Within a group the codes
// stand in the order of the A operands of mma.sync.m16n8k16, so that a lane (g = lane / 4,
// t = lane % 4) takes the operands of two products with one 16-byte load, 512 consecutive bytes
// per warp and 32 dims:
//   K (rows = tokens, k = dims): byte s*8 + half*4 + b of lane (g, t) is token
//     4 (g / 2) + 2 half + g % 2 at dim 32 c + 16 s + 4 t + b; operand row g + 8 half, and the
//     token order makes the scores of operand rows (2t, 2t+1, 2t+8, 2t+9) those of tokens 4t..4t+3;
//   V (rows = dims, k = tokens): byte s*8 + j*4 + b is token 4 t + b at dim 32 c + 16 s + 8 j + g.
#pragma once
#include <cstdint>

namespace kq {

__host__ __device__ constexpr int kv8_k_offset(int p, int d) {
  return d / 32 * 512 + (p / 4 * 2 + p % 2) * 64 + d / 4 % 4 * 16 + d / 16 % 2 * 8 + p / 2 % 2 * 4 + d % 4;
}
__host__ __device__ constexpr int kv8_v_offset(int p, int d) {
  return d / 32 * 512 + d % 8 * 64 + p / 4 * 16 + d / 16 % 2 * 8 + d / 8 % 2 * 4 + p % 4;
}

}  // namespace kq
