// What the adapter-gradient kernels share (the expert products' and those of a training step): a step of 32 rows in LDS, Q as
// rows of 128 bf16 and P as rows of 64 in each of three bf16 parts, read with the transpose read.
#pragma once

#include "qlr_tile.h"

namespace qlr {

namespace {

__device__ __forceinline__ s16x4_t train_tr(const char* p) {  // LDS transpose read (see lds_tr16)
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(const_cast<char*>(p)));
}
__device__ __forceinline__ bf16x8_t tr_frag(const char* lo, const char* hi) {
  const s16x4_t l = train_tr(lo), h = train_tr(hi);
  return as_bf16x8(u32x4_t{__builtin_bit_cast(uint2, l).x, __builtin_bit_cast(uint2, l).y, __builtin_bit_cast(uint2, h).x,
                           __builtin_bit_cast(uint2, h).y});
}

// v's three bf16 parts of 8 bits each, the third the whole rest (see split_rest), of two neighbours as one word a part.
__device__ __forceinline__ void three_parts(float a, float b, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
  float a1 = split_rest(a), b1 = split_rest(b), a2 = split_rest(a1), b2 = split_rest(b1);
  p0 = (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xFFFF0000u);
  p1 = (__float_as_uint(a1) >> 16) | (__float_as_uint(b1) & 0xFFFF0000u);
  p2 = (__float_as_uint(a2) >> 16) | (__float_as_uint(b2) & 0xFFFF0000u);
}

constexpr uint32_t kQ = 32 * 256, kP = 32 * 128;  // bytes of a step of Q, and of one part of P
// Row `row`'s 16-byte chunk, XOR-swizzled so that a transpose read's rows lie on different banks.
__device__ __forceinline__ uint32_t q_off(uint32_t row, uint32_t chunk) {
  const uint32_t h = (row & 3u) | (((row >> 3) & 1u) << 2);
  return row * 256u + ((chunk ^ (h << 1)) << 4);
}
__device__ __forceinline__ uint32_t p_off(uint32_t row, uint32_t chunk) {
  const uint32_t h = ((row >> 1) & 1u) | (((row >> 3) & 1u) << 1);
  return row * 128u + ((chunk ^ (h << 1)) << 4);
}

}  // namespace

}  // namespace qlr
