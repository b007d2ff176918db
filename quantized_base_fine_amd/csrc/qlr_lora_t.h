// The adapter product t = x A^T of a few rows (device body, shared by the kernels
// that run it alone and beside other work).
#pragma once

#include "qlr_internal.h"

namespace qlr {

namespace {

// bf16 x and A, M <= 16 (one 16-row MFMA tile): K-split partial sums
// p[s][m][j] of t = x A^T.  Workgroup (16 adapter rows j0 .. j0 + 15, split s)
// of 16 waves: wave w takes the 32-column steps c0 + w, c0 + w + 16, ... of the
// split, issues the loads of up to kLtSteps of them before any product (the
// split count keeps a split within one such round for the decode shapes), and
// multiplies on 16x16x32 bf16 MFMA (x rows as the A operand, adapter rows as
// B).  A step's loads give each quad of lanes one row's 64 bytes (lane l: row
// l / 4, 8 columns from 8 (l % 4)), the rate the address unit sustains, and a
// lane permute per word puts row n's piece g in lane 16 g + n, the fragment
// layout.  The 16 waves' sums are added through LDS in wave order.
constexpr int kLtWaves = 16, kLtSteps = 8;
__device__ __forceinline__ void lora_t_small_body(const uint16_t* __restrict__ x, int64_t M, int64_t K,
                                                  const uint16_t* __restrict__ A, int r, float* __restrict__ p,
                                                  int j0, int S, int sidx, float (*red)[256]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = lane >> 2, g = lane & 3;  // the lane's loads
  const bool xv = row < M, av = j0 + row < r;
  const uint16_t* xp = x + (int64_t)(xv ? row : 0) * K + g * 8;
  const uint16_t* ap = A + (int64_t)(av ? j0 + row : 0) * K + g * 8;
  const int src = (4 * (lane & 15) + (lane >> 4)) << 2;  // lane 16 g + n <- lane 4 n + g
  const int64_t nsteps = K / 32;
  const int64_t c0 = nsteps * sidx / S, c1 = nsteps * (sidx + 1) / S;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  for (int64_t base = c0 + wave; base < c1; base += kLtWaves * kLtSteps) {
    u32x4_t xa[kLtSteps], ab[kLtSteps];
#pragma unroll
    for (int i = 0; i < kLtSteps; ++i) {
      const int64_t st = base + (int64_t)i * kLtWaves;
      const bool sv = st < c1;
      const int64_t k = (sv ? st : c0) * 32;
      xa[i] = (xv && sv) ? *reinterpret_cast<const u32x4_t*>(xp + k) : zero;
      ab[i] = (av && sv) ? *reinterpret_cast<const u32x4_t*>(ap + k) : zero;
    }
#pragma unroll
    for (int i = 0; i < kLtSteps; ++i) {
      if (base + (int64_t)i * kLtWaves >= c1) break;  // uniform: the split's last steps
      u32x4_t xf, af;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        xf[j] = (uint32_t)__builtin_amdgcn_ds_bpermute(src, (int)xa[i][j]);
        af[j] = (uint32_t)__builtin_amdgcn_ds_bpermute(src, (int)ab[i][j]);
      }
      acc = mfma16x16x32(as_bf16x8(xf), as_bf16x8(af), acc);
    }
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) red[wave][lane * 4 + v] = acc[v];
  __syncthreads();
  if (threadIdx.x < 256) {
    const int e = threadIdx.x;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kLtWaves; ++w) sum += red[w][e];
    const int l = e >> 2, v = e & 3;
    const int m = 4 * (l >> 4) + v;  // MFMA output row (x row)
    const int j = j0 + (l & 15);     // MFMA output column (adapter row)
    if (m < M && j < r) p[((int64_t)sidx * M + m) * r + j] = sum;
  }
}

}  // namespace

}  // namespace qlr
