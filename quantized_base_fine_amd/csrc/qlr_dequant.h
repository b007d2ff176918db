// Operand staging helpers shared by the tiled products (prefill GEMM, expert
// products, 8-bit-integer product): LDS accesses by byte address, packed-code
// loads and their dequantization to bf16 pairs, and the LDS swizzles.
#pragma once

#include "qlr_internal.h"
#include "qlr_lut.h"

namespace qlr {

namespace {

// Raw codes of one thread for one block: the 32 codes [32h, 32h+32) of a weight row.
template <int BITS>
struct Codes32 {
  uint32_t w[BITS];  // 32*BITS bits
};

template <int BITS>
__device__ __forceinline__ Codes32<BITS> load_codes32(const uint8_t* p) {
  Codes32<BITS> c;
  if constexpr (BITS == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    c.w[0] = u.x; c.w[1] = u.y;
  } else if constexpr (BITS == 3) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p);  // 12 bytes at a 4-byte boundary
    c.w[0] = q[0]; c.w[1] = q[1]; c.w[2] = q[2];
  } else if constexpr (BITS == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    c.w[0] = u.x; c.w[1] = u.y; c.w[2] = u.z; c.w[3] = u.w;
  } else {
    const uint4 u0 = *reinterpret_cast<const uint4*>(p);
    const uint4 u1 = *reinterpret_cast<const uint4*>(p + 16);
    c.w[0] = u0.x; c.w[1] = u0.y; c.w[2] = u0.z; c.w[3] = u0.w;
    c.w[4] = u1.x; c.w[5] = u1.y; c.w[6] = u1.z; c.w[7] = u1.w;
  }
  return c;
}

// The 16 codes [16 q, 16 q + 16) of a block whose codes start at p (16-byte aligned for 8-bit
// codes, 4-byte for the others), in the low half of the words; of 3-bit codes, 6 bytes at
// 6 q, the two words around them, which place_codes16 shifts into place (apart, so that a
// load well ahead of its use is not waited for by the shift).
template <int BITS>
__device__ __forceinline__ Codes32<BITS> load_codes16(const uint8_t* p, int q) {
  Codes32<BITS> c;
#pragma unroll
  for (int i = 0; i < BITS; ++i) c.w[i] = 0;
  if constexpr (BITS == 2) {
    c.w[0] = *reinterpret_cast<const uint32_t*>(p + 4 * q);
  } else if constexpr (BITS == 3) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p + ((6 * q) & ~3));
    c.w[0] = w[0]; c.w[1] = w[1];
  } else if constexpr (BITS == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p + 8 * q);
    c.w[0] = u.x; c.w[1] = u.y;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p + 16 * q);
    c.w[0] = u.x; c.w[1] = u.y; c.w[2] = u.z; c.w[3] = u.w;
  }
  return c;
}

template <int BITS>
__device__ __forceinline__ void place_codes16(Codes32<BITS>& c, int q) {
  if constexpr (BITS == 3) {
    const uint32_t sh = 16u * (q & 1);
    c.w[0] = __builtin_amdgcn_alignbit(c.w[1], c.w[0], sh);
    c.w[1] = c.w[1] >> sh;
  }
}

// LDS accesses at a byte address of the dynamic LDS block, which starts at LDS
// address 0 (the kernel has no static LDS; the launcher checks this).
typedef float f32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ float2 lds_pair(uint32_t byte_addr) {
  const f32x2_t v = *reinterpret_cast<const __attribute__((address_space(3))) f32x2_t*>((uintptr_t)byte_addr);
  return make_float2(v.x, v.y);
}
__device__ __forceinline__ float lds_f32(uint32_t byte_addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) float*>((uintptr_t)byte_addr);
}
__device__ __forceinline__ u32x4_t lds_u32x4(uint32_t byte_addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) u32x4_t*>((uintptr_t)byte_addr);
}
__device__ __forceinline__ void lds_store_u32x4(uint32_t byte_addr, u32x4_t v) {
  *reinterpret_cast<__attribute__((address_space(3))) u32x4_t*>((uintptr_t)byte_addr) = v;
}
__device__ __forceinline__ void lds_store_f32x4(uint32_t byte_addr, f32x4_t v) {
  *reinterpret_cast<__attribute__((address_space(3))) f32x4_t*>((uintptr_t)byte_addr) = v;
}
__device__ __forceinline__ f32x4_t lds_f32x4(uint32_t byte_addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) f32x4_t*>((uintptr_t)byte_addr);
}
// LDS transpose read of 16-bit elements (ds_read_b64_tr_b16): within each group
// of 16 lanes, lane i receives element i % 4 of the 8-byte reads of lanes
// i / 4, i / 4 + 4, i / 4 + 8 and i / 4 + 12, in that order.
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef s16x4_t u16x4_t;
__device__ __forceinline__ u16x4_t lds_tr16(uint32_t byte_addr) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      reinterpret_cast<__attribute__((address_space(3))) s16x4_t*>((uintptr_t)byte_addr));
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// round-to-nearest-even bf16 pair of (a, b) in one packed conversion
__device__ __forceinline__ uint32_t cvt_pk_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

__device__ __forceinline__ uint32_t perm(uint32_t hi4, uint32_t lo4, uint32_t sel) {
  return __builtin_amdgcn_perm(hi4, lo4, sel);
}

// ---- 4-bit register lookup
// Byte tables of the 8 positive scaled levels P[j] = bf16(L[8 + j] * ap):
// lo = low bytes of P[0..7], hi = high bytes, 8 bytes each (two registers).
struct Lut4 {
  uint32_t lo_a, lo_b, hi_a, hi_b;
};

__device__ __forceinline__ Lut4 make_lut4(const Levels& lv, float ap) {
  const uint32_t p01 = cvt_pk_bf16(lv.v[8] * ap, lv.v[9] * ap);
  const uint32_t p23 = cvt_pk_bf16(lv.v[10] * ap, lv.v[11] * ap);
  const uint32_t p45 = cvt_pk_bf16(lv.v[12] * ap, lv.v[13] * ap);
  const uint32_t p67 = cvt_pk_bf16(lv.v[14] * ap, lv.v[15] * ap);
  return {perm(p23, p01, 0x06040200u), perm(p67, p45, 0x06040200u),
          perm(p23, p01, 0x07050301u), perm(p67, p45, 0x07050301u)};
}

// Eight 4-bit codes (LSB first) -> four bf16 pairs in code order.  Code c maps
// to P[c - 8] for c >= 8 and to -P[7 - c] for c < 8: the index is c ^ 7 when
// bit 3 is clear, and the sign is bit 3 clear, set into bit 15 of the bf16.
__device__ __forceinline__ void lut4_word(uint32_t w, const Lut4& t, uint32_t* o) {
  const uint32_t neg = ~w & 0x88888888u;  // bit 3 of every negative code
  const uint32_t m = neg >> 3;
  const uint32_t idx = w ^ ((m << 3) - m);  // low 3 bits of each nibble: level index
  const uint32_t se = idx & 0x07070707u, so = (idx >> 4) & 0x07070707u;  // even / odd codes
  const uint32_t loe = perm(t.lo_b, t.lo_a, se), loo = perm(t.lo_b, t.lo_a, so);
  const uint32_t hie = perm(t.hi_b, t.hi_a, se) | ((neg << 4) & 0x80808080u);
  const uint32_t hio = perm(t.hi_b, t.hi_a, so) | (neg & 0x80808080u);
  const uint32_t l03 = perm(loo, loe, 0x05010400u), h03 = perm(hio, hie, 0x05010400u);
  const uint32_t l47 = perm(loo, loe, 0x07030602u), h47 = perm(hio, hie, 0x07030602u);
  o[0] = perm(h03, l03, 0x05010400u);
  o[1] = perm(h03, l03, 0x07030602u);
  o[2] = perm(h47, l47, 0x05010400u);
  o[3] = perm(h47, l47, 0x07030602u);
}

// A lane's copy of the level table: at an LDS byte address, or behind a pointer.
struct TabAt {
  uint32_t tp;
  __device__ __forceinline__ float one(uint32_t off) const { return lds_f32(tp + off); }
  __device__ __forceinline__ float2 pair(uint32_t off) const { return lds_pair(tp + off); }
};
struct TabPtr {
  const char* p;
  __device__ __forceinline__ float one(uint32_t off) const { return *reinterpret_cast<const float*>(p + off); }
  __device__ __forceinline__ float2 pair(uint32_t off) const { return *reinterpret_cast<const float2*>(p + off); }
};

// Float32 levels of codes 2 j, 2 j + 1 of one thread's 32 codes, for widths other
// than 4.
template <int BITS, typename Tab>
__device__ __forceinline__ float2 level_pair(const Codes32<BITS>& c, int j, const Tab& tab) {
  if constexpr (BITS == 8) {
    // one float32 level per code; 16 lane copies, entry e of copy l at e*64 + 4l
    const uint32_t w = c.w[j >> 1] >> (16 * (j & 1));
    return make_float2(tab.one((w & 255u) << 6), tab.one(((w >> 8) & 255u) << 6));
  } else {
    // float32 level pairs of two neighbouring codes; 32 lane copies, entry e at e*256 + 8l
    uint32_t e;
    if constexpr (BITS == 2) {
      e = (c.w[j >> 3] >> (4 * (j & 7))) & 15u;
    } else {
      const int bit = 6 * j, wd = bit >> 5, sh = bit & 31;
      uint32_t v = c.w[wd] >> sh;
      if (sh + 6 > 32) v |= c.w[wd + 1] << (32 - sh);
      e = v & 63u;
    }
    return tab.pair(e << 8);
  }
}

// Pairs [J0, J1) of the 16 bf16 pairs of one thread's 32 codes, for widths
// other than 4: o[j] = bf16 pair of codes 2j, 2j+1, scaled by ap.
template <int BITS, int J0, int J1>
__device__ __forceinline__ void dequant_pairs(const Codes32<BITS>& c, float ap, uint32_t tp, uint32_t (&o)[16]) {
#pragma unroll
  for (int j = J0; j < J1; ++j) {
    const float2 p = level_pair<BITS>(c, j, TabAt{tp});
    o[j] = cvt_pk_bf16(p.x * ap, p.y * ap);
  }
}

// XOR swizzle of the 16-byte chunks of LDS tile row r (see the header).
__device__ __forceinline__ uint32_t swz(uint32_t r) {
  return (r ^ ((r >> 2) & 1u) ^ ((r >> 3) & 1u)) & 7u;
}
// Physical 16-byte chunk of logical chunk c (0..15) of row R of the transposed
// GEMM's weight tile: c ^ (0, 6, 10, 12)[R mod 4] ^ bit 3 of c.
__device__ __forceinline__ uint32_t tr_chunk(uint32_t c, uint32_t R) {
  return c ^ ((0xCA60u >> (4u * (R & 3u))) & 15u) ^ ((c >> 3) & 1u);
}

}  // namespace

}  // namespace qlr
