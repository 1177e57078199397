// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC 2011): the counter-based generator of the LoRA dropout.
// Element i of a row-major array uses word i % 4 of the block for counter
// (g mod 2^32, g div 2^32, 0, 0), g = i div 4, under the 64-bit seed as key.
#pragma once
#include "device_common.h"

namespace qlk {

// a ^ b ^ c in one instruction (0x96: the truth table of the three-way xor).
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

// One Philox4x32 block: ten rounds of two 32 x 32 -> 64-bit products with the
// published multipliers, the key bumped by the Weyl constants between rounds.
__device__ __forceinline__ uint4 philox4x32_10(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int rnd = 0; rnd < 10; ++rnd) {
    if (rnd) {
      k0 += 0x9E3779B9u;
      k1 += 0xBB67AE85u;
    }
    const uint64_t p0 = (uint64_t)0xD2511F53u * c.x;
    const uint64_t p1 = (uint64_t)0xCD9E8D57u * c.z;
    c = make_uint4(xor3((uint32_t)(p1 >> 32), c.y, k0), (uint32_t)p1,
                   xor3((uint32_t)(p0 >> 32), c.w, k1), (uint32_t)p0);
  }
  return c;
}

// The dropout of one call: an element is kept when its word is >= threshold.
struct DropKey {
  uint32_t threshold, k0, k1;
};

// Keeps of the 8 consecutive elements i0 .. i0 + 7 (i0 a multiple of 8, below
// 2^34, so that the counter's second word is zero): bit e is element i0 + e.
__device__ __forceinline__ uint32_t philox_keep8(uint64_t i0, const DropKey& d) {
  uint32_t bits = 0;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const uint4 w = philox4x32_10(make_uint4((uint32_t)(i0 >> 2) + b, 0u, 0u, 0u), d.k0, d.k1);
    bits |= (uint32_t)(w.x >= d.threshold) << (4 * b) | (uint32_t)(w.y >= d.threshold) << (4 * b + 1) |
            (uint32_t)(w.z >= d.threshold) << (4 * b + 2) | (uint32_t)(w.w >= d.threshold) << (4 * b + 3);
  }
  return bits;
}

// The 8 bf16 elements i0 .. i0 + 7 with the dropped ones set to +0 (their
// bits are cleared, so an infinity or NaN in a dropped place leaves nothing).
__device__ __forceinline__ uint4 philox_drop8(uint4 v, uint64_t i0, const DropKey& d) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const uint4 p = philox4x32_10(make_uint4((uint32_t)(i0 >> 2) + b, 0u, 0u, 0u), d.k0, d.k1);
    w[2 * b] &= (p.x >= d.threshold ? 0xffffu : 0u) | (p.y >= d.threshold ? 0xffff0000u : 0u);
    w[2 * b + 1] &= (p.z >= d.threshold ? 0xffffu : 0u) | (p.w >= d.threshold ? 0xffff0000u : 0u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace qlk
