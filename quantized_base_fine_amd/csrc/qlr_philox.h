// Dropout masks from a counter: whether an element of an input is kept is a function of its place, a seed and a counter, so that the
// forward and the backward form the same mask each on their own.  Nothing of it is kept between calls.  Within the backward
// three kernels need it: the first to form it (x A^T) leaves its bits in the workspace (an eighth of a byte an element), since the
// rounds cost more than the reading (layer backward of 2048 x 4096 x 11008, formed three times 374 us, so, and with the partial sums of
// t and u added once, 349).
//
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3", SC 2011): ten rounds of
//     (x0, x1, x2, x3) <- (hi(M1 x2) ^ x1 ^ k0, lo(M1 x2), hi(M0 x0) ^ x3 ^ k1, lo(M0 x0)),
// the key raised by (W0, W1) a round.  Counter words: the number g = (m K + k) / 8 of a group of eight neighbouring
// elements of a row (K % 8 == 0), and the mask's 64-bit counter.  The four result words are eight 16-bit numbers, one per
// element: kept iff it is at least thr = round(65536 p).  Eight numbers a call instead of four: the rounds' twenty
// 32 x 32 -> 64 bit products run at a quarter of the vector rate and bound the mask, and 16 bits place p within 2^-17.
#pragma once

#include "qlr_internal.h"

namespace qlr {

namespace {

// The mask's counter: the host's part plus the step that the device holds (a captured call follows it).
__device__ __forceinline__ uint64_t drop_counter(const DropArgs& d, int which) {
  return d.counter + (uint64_t)which + (d.step ? *d.step : 0);
}

__device__ __forceinline__ u32x4_t philox(uint64_t g, uint64_t c, uint64_t seed) {
  uint32_t x0 = (uint32_t)g, x1 = (uint32_t)(g >> 32), x2 = (uint32_t)c, x3 = (uint32_t)(c >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)0xD2511F53u * x0, b = (uint64_t)0xCD9E8D57u * x2;
    x0 = (uint32_t)(b >> 32) ^ x1 ^ k0;
    x1 = (uint32_t)b;
    x2 = (uint32_t)(a >> 32) ^ x3 ^ k1;
    x3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4_t{x0, x1, x2, x3};
}

// Eight bits, element j at bit j, as 16-bit lanes, all ones where the bit is set.
__device__ __forceinline__ u32x4_t bit_lanes(uint32_t b) {
  u32x4_t m;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m[i] = ((uint32_t)__builtin_amdgcn_sbfe((int)b, 2 * i, 1) & 0xFFFFu) | ((uint32_t)__builtin_amdgcn_sbfe((int)b, 2 * i + 1, 1) & 0xFFFF0000u);
  return m;
}

// The group's eight 16-bit lanes, all ones where the element is kept (thr >= 1).
__device__ __forceinline__ u32x4_t drop_lanes(uint64_t g, uint64_t c, const DropArgs& d) {
  typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
  const u32x4_t z = philox(g, c, d.seed);
  const unsigned short t1 = (unsigned short)(d.thr - 1u);
  u32x4_t m;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // number - (thr - 1), saturating at zero, is positive iff number >= thr
    const u16x2_t over = __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2_t, (uint32_t)z[i]), u16x2_t{t1, t1});
    const u16x2_t one = __builtin_elementwise_min(over, u16x2_t{1, 1});
    m[i] = __builtin_bit_cast(uint32_t, (u16x2_t)(u16x2_t{0, 0} - one));
  }
  return m;
}

// The same as eight bits, element j at bit j.
__device__ __forceinline__ uint32_t drop_bits(uint64_t g, uint64_t c, const DropArgs& d) {
  const u32x4_t z = philox(g, c, d.seed);
  uint32_t b = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    b |= (uint32_t)((z[i] & 0xFFFFu) >= d.thr) << (2 * i);
    b |= (uint32_t)((z[i] >> 16) >= d.thr) << (2 * i + 1);
  }
  return b;
}

}  // namespace

}  // namespace qlr
