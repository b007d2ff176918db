// What the kernels of a few rows on the coded base share (the expert products' and the gated block's): the level table in
// LDS, the lookup of a lane's codes in it, and a wave's slice for its rows of x.
#pragma once

#include "qlr_tile.h"

namespace qlr {

namespace {

constexpr uint32_t kXRow = 256 + 16, kXSlice = 16 * kXRow;  // a wave's slice: two blocks of 16 rows, padded

template <int BITS>
struct FewTab {
  static constexpr int kEntries = BITS == 8 ? 256 : 1 << (2 * BITS);
  static constexpr uint32_t kBytes = kEntries * 128;
};

// Words of a lane's 16 codes.
template <int BITS>
constexpr int kFewWords = BITS == 8 ? 4 : BITS == 2 ? 1 : 2;

// bf16 levels of the lane's 16 codes, pairs in code order; tl = 4 (lane % 32).
template <int BITS>
__device__ __forceinline__ void few_levels(const uint32_t (&w)[kFewWords<BITS>], uint32_t tl, uint32_t (&o)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (BITS == 8) {
      const uint32_t v = w[j >> 1] >> (16 * (j & 1));
      o[j] = __builtin_amdgcn_perm(lds_word(((v >> 8) & 255u) << 7 | tl), lds_word((v & 255u) << 7 | tl), 0x05040100u);
    } else if constexpr (BITS == 3) {
      const int bit = 6 * j, wd = bit >> 5, sh = bit & 31;
      const uint32_t v = sh + 6 > 32 ? __builtin_amdgcn_alignbit(w[wd < 1 ? wd + 1 : wd], w[wd], sh) : w[wd] >> sh;
      o[j] = lds_word((v & 63u) << 7 | tl);
    } else {
      constexpr uint32_t mask = (1u << (2 * BITS)) - 1;
      o[j] = lds_word(((w[(2 * BITS * j) >> 5] >> ((2 * BITS * j) & 31)) & mask) << 7 | tl);
    }
  }
}

// Before a launch.  The level table is read at LDS addresses from 0, so the kernel must not have static LDS; `checked` is the
// kernel's own flag (host threads may come here at once: each sets the same).
inline hipError_t few_prepare(const void* kern, size_t shmem, std::atomic<bool>& checked) {
  if (!checked) {
    hipFuncAttributes fa;
    const hipError_t e = hipFuncGetAttributes(&fa, kern);
    if (e != hipSuccess) return e;
    if (fa.sharedSizeBytes != 0) return hipErrorInvalidKernelFile;
    checked = true;
  }
  return hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)shmem);
}

}  // namespace

}  // namespace qlr
