// Expert-grouped products of a mixture-of-experts layer on the coded base: rows
// sorted by expert, device offsets, one stacked weight, one adapter per expert.
// This file holds the forward for experts with few rows and the adapter
// products; the tiled products are instantiated per code width elsewhere.
#include "qlr_tile.h"

namespace qlr {

namespace {

// ---------------------------------------------------------------- experts of 1 .. 16 rows
//
// Bound by the stream of the experts' codes.  A workgroup of 8 waves takes 16 G
// weight rows of one expert; the waves share K in pairs of 64-element blocks
// (wave w the pairs w, w + 8, ...).  A lane holds 32 consecutive codes of one
// weight row (row lane % 16, codes 32 (lane / 16) .. + 32 of the pair: one load),
// dequantizes them to bf16 (scaled levels) straight into four MFMA A fragments
// and multiplies them with the expert's rows as B (16x16x32, token lanes past
// the expert's rows hold zeros).  The waves' sums are added through LDS in wave
// order, then scale t B^T.
constexpr int kFewWaves = 8;

template <int BITS>
struct FewTab {
  static constexpr uint32_t kBytes = BITS == 4 ? 0 : BITS == 8 ? 256 * 16 * 4 : PairTableF32<BITS>::kBytes;
  // the waves' sums (the staging of the levels shares the area)
  __host__ __device__ static constexpr uint32_t kRedBytes(int G) { return kFewWaves * 16 * 16 * 4 * G; }
};

template <int BITS, int G>
__global__ __launch_bounds__(512) void k_grouped_few(TileArgs P, Levels lv) {
  constexpr uint32_t kTab = 0, kRed = FewTab<BITS>::kBytes;
  extern __shared__ uint32_t smem[];
  int a, b;
  const int e = blockIdx.y;
  expert_range(P.offsets, e, (int)P.M, a, b);
  const int rows = b - a;
  if (rows < 1 || rows > kFewRows) return;  // the whole workgroup
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if constexpr (BITS != 4) {
    float* sL = reinterpret_cast<float*>(smem) + kRed / 4;
    stage_levels<1 << BITS>(lv, sL);
    __syncthreads();
    float* tab = reinterpret_cast<float*>(smem);
    if constexpr (BITS == 8) {
      for (int i = tid; i < 256 * 16; i += 512) tab[i] = sL[i >> 4];
    } else {
      constexpr int NL = 1 << BITS;
      for (int i = tid; i < PairTableF32<BITS>::kEntries * 32; i += 512) {
        tab[2 * i] = sL[(i >> 5) & (NL - 1)];
        tab[2 * i + 1] = sL[(i >> 5) >> BITS];
      }
    }
    __syncthreads();
  }
  const int64_t N = P.N, K = P.K, nb = K >> 6;
  const int np = (int)((nb + 1) / 2);
  const int n0 = blockIdx.x * 16 * G;
  const int row = lane & 15, g = lane >> 4;
  const uint32_t tp = kTab + (BITS == 8 ? 4u * (lane & 15) : 8u * (lane & 31));
  const uint16_t* xp = reinterpret_cast<const uint16_t*>(P.x) + (int64_t)(a + min(row, rows - 1)) * K;
  int64_t wblk[G];
#pragma unroll
  for (int i = 0; i < G; ++i) wblk[i] = ((int64_t)e * N + min<int64_t>(n0 + 16 * i + row, N - 1)) * nb;
  FewAdapter<16 * G> ad;
  ad.load(P.t, 1, P.M, a, rows, P.ab + (int64_t)e * N * P.r, n0, (int)min<int64_t>(16 * G, N - n0), P.r);
  f32x4_t acc[G];
#pragma unroll
  for (int i = 0; i < G; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const u32x4_t zero4 = {0u, 0u, 0u, 0u};
  struct Ld {
    u32x4_t x[4];
    Codes32<BITS> c[G];
    uint32_t q8[G];
    float sc[G];
  };
  auto load = [&](int p, Ld& d) {
    const int64_t blk = 2 * (int64_t)p + (g >> 1);
    const bool ok = p < np && blk < nb;
    const int64_t bl = ok ? blk : 0;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      d.c[i] = load_codes32<BITS>(P.w + (wblk[i] + bl) * (8 * BITS) + (g & 1) * (4 * BITS));
      d.q8[i] = ok ? P.q8[wblk[i] + bl] : 0u;
      d.sc[i] = P.cst[(wblk[i] + bl) >> 8];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      d.x[i] = ok && row < rows ? *reinterpret_cast<const u32x4_t*>(xp + bl * 64 + 32 * (g & 1) + 8 * i) : zero4;
  };
  auto compute = [&](const Ld& d) {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const float ap = (float)d.q8[i] * d.sc[i];
      uint32_t o[16];
      if constexpr (BITS == 4) {
        const Lut4 lut = make_lut4(lv, ap);
#pragma unroll
        for (int j = 0; j < 4; ++j) lut4_word(d.c[i].w[j], lut, o + 4 * j);
      } else {
        dequant_pairs<BITS, 0, 16>(d.c[i], ap, tp, o);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i] = mfma16x16x32(as_bf16x8(u32x4_t{o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]}), as_bf16x8(d.x[j]),
                              acc[i]);
    }
  };
  Ld d0, d1;
  load(wave, d0);
  for (int p = wave; p < np; p += 2 * kFewWaves) {
    load(p + kFewWaves, d1);
    compute(d0);
    load(p + 2 * kFewWaves, d0);
    if (p + kFewWaves < np) compute(d1);
  }
  // [wave][token][weight row] sums
  float* red = reinterpret_cast<float*>(smem) + kRed / 4;
  if constexpr (BITS != 4) __syncthreads();  // the level staging above shared this area
#pragma unroll
  for (int i = 0; i < G; ++i)
    *reinterpret_cast<f32x4_t*>(red + (wave * 16 + row) * (16 * G) + 16 * i + 4 * g) = acc[i];
  char* ad_lds = reinterpret_cast<char*>(smem) + kRed + FewTab<BITS>::kRedBytes(G);
  ad.stage(ad_lds, 1, rows, P.r);
  __syncthreads();
  for (int idx = tid; idx < rows * 16 * G; idx += 512) {
    const int m = idx / (16 * G), c = idx % (16 * G);
    const int n = n0 + c;
    if (n >= N) continue;
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) y += red[(w * 16 + m) * (16 * G) + c];
    if (P.r > 0)
      y = fmaf(P.scale, ad.dot(ad_lds, P.t, 1, P.M, a, m, P.ab + (int64_t)e * N * P.r, n0, c, P.r), y);
    const int64_t o = (int64_t)(a + m) * N + n;
    if (P.ydt == DT_F32) reinterpret_cast<float*>(P.y)[o] = y;
    else reinterpret_cast<uint16_t*>(P.y)[o] = (uint16_t)f32_to_bf16_bits(y);
  }
}

template <int BITS, int G>
hipError_t launch_few_g(const TileArgs& a, const Levels& lv, hipStream_t s) {
  auto kern = k_grouped_few<BITS, G>;
  const size_t shmem = FewTab<BITS>::kBytes + FewTab<BITS>::kRedBytes(G) + (a.r > 0 ? FewAdapter<16 * G>::kBytes : 0);
  const hipError_t e =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, (int)shmem);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)((a.N + 16 * G - 1) / (16 * G)), (unsigned)a.experts), dim3(512), shmem, s, a,
                     lv);
  return hipGetLastError();
}

template <int BITS>
hipError_t launch_few_b(const TileArgs& a, const Levels& lv, hipStream_t s) {
  // workgroups of the experts that can have rows; 16 rows each until they fill the GPU
  const int64_t wgs = std::min<int64_t>(a.experts, a.M) * ((a.N + 15) / 16);
  if (wgs >= 4096) return launch_few_g<BITS, 4>(a, lv, s);
  if (wgs >= 2048) return launch_few_g<BITS, 2>(a, lv, s);
  return launch_few_g<BITS, 1>(a, lv, s);
}

// ---------------------------------------------------------------- t = x A_e^T
//
// A workgroup of 8 waves takes 16 RT rows of one expert x 64 adapter rows; the
// waves split K in 32-element steps and multiply on 16x16x32 bf16 MFMA (x rows
// as A, adapter rows as B); their sums are added through LDS in wave order.
template <int RT>
__global__ __launch_bounds__(512) void k_grouped_t(const uint16_t* __restrict__ x, int64_t M, int64_t K,
                                                   const uint16_t* __restrict__ A, int r, const int32_t* offsets,
                                                   int experts, float* __restrict__ t) {
  __shared__ float red[kFewWaves][RT * 16 * 64];
  int e = 0, row0 = 0, row_end = 0;
  const int total = tile_scan(offsets, experts, (int)M, 0, 16 * RT, -1, e, row0, row_end);
  if ((int)blockIdx.x >= total) return;  // the whole workgroup
  tile_scan(offsets, experts, (int)M, 0, 16 * RT, blockIdx.x, e, row0, row_end);
  e = __builtin_amdgcn_readfirstlane(e);
  row0 = __builtin_amdgcn_readfirstlane(row0);
  row_end = __builtin_amdgcn_readfirstlane(row_end);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int rows = min(16 * RT, row_end - row0), j0 = blockIdx.y * 64;
  const int row = lane & 15, g = lane >> 4;
  const uint16_t* xp[RT];
  const uint16_t* ap[4];
#pragma unroll
  for (int i = 0; i < RT; ++i) xp[i] = x + (int64_t)(row0 + min(16 * i + row, rows - 1)) * K + 8 * g;
#pragma unroll
  for (int c = 0; c < 4; ++c) ap[c] = A + ((int64_t)e * r + min(j0 + 16 * c + row, r - 1)) * K + 8 * g;
  const int jt = min(4, (r - j0 + 15) / 16);
  f32x4_t acc[RT][4];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[i][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int nst = (int)((K + 31) / 32);
  const int s0 = (int)((int64_t)nst * wave / kFewWaves), s1 = (int)((int64_t)nst * (wave + 1) / kFewWaves);
  const u32x4_t zero4 = {0u, 0u, 0u, 0u};
  struct Ld { u32x4_t x[RT], a[4]; };
  auto load = [&](int st, Ld& d) {
    const int64_t k = (int64_t)st * 32;
    const bool ok = st < s1 && k + 8 * g < K;  // past the range or the row's end: zeros
#pragma unroll
    for (int i = 0; i < RT; ++i) d.x[i] = ok ? *reinterpret_cast<const u32x4_t*>(xp[i] + k) : zero4;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      d.a[c] = ok && c < jt ? *reinterpret_cast<const u32x4_t*>(ap[c] + k) : zero4;
  };
  auto compute = [&](const Ld& d) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][c] = mfma16x16x32(as_bf16x8(d.x[i]), as_bf16x8(d.a[c]), acc[i][c]);
  };
  Ld d0, d1;
  load(s0, d0);
  for (int st = s0; st < s1; st += 2) {
    load(st + 1, d1);
    compute(d0);
    load(st + 2, d0);
    compute(d1);
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[wave][(16 * i + 4 * g + v) * 64 + 16 * c + row] = acc[i][c][v];
  __syncthreads();
  for (int idx = tid; idx < rows * 64; idx += 512) {
    const int m = idx >> 6, j = j0 + (idx & 63);
    if (j >= r) continue;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) sum += red[w][idx];
    t[(int64_t)(row0 + m) * r + j] = sum;
  }
}

// Bt[e][j][n] = B[e][n][j]
__global__ __launch_bounds__(256) void k_grouped_transpose(const uint16_t* __restrict__ B, int64_t N, int r,
                                                           uint16_t* __restrict__ Bt) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= N * r) return;
  const int64_t j = i / N, n = i % N, base = (int64_t)blockIdx.y * N * r;
  Bt[base + i] = B[base + n * r + j];
}

}  // namespace

hipError_t launch_grouped_few(const TileArgs& a, const Levels& lv, hipStream_t s) {
  switch (a.bits) {
    case 2: return launch_few_b<2>(a, lv, s);
    case 3: return launch_few_b<3>(a, lv, s);
    case 4: return launch_few_b<4>(a, lv, s);
    default: return launch_few_b<8>(a, lv, s);
  }
}

hipError_t launch_grouped_t(const uint16_t* x, int64_t M, int64_t K, const uint16_t* A, int r, const int32_t* offsets,
                            int experts, float* t, hipStream_t s) {
  const unsigned jg = (unsigned)((r + 63) / 64);
  const unsigned tiles = (unsigned)tile_bound(M, experts, 16);
  hipLaunchKernelGGL(k_grouped_t<1>, dim3(tiles, jg), dim3(512), 0, s, x, M, K, A, r, offsets, experts, t);
  return hipGetLastError();
}

hipError_t launch_grouped_transpose(const uint16_t* B, int experts, int64_t N, int r, uint16_t* Bt, hipStream_t s) {
  hipLaunchKernelGGL(k_grouped_transpose, dim3((unsigned)((N * r + 255) / 256), (unsigned)experts), dim3(256), 0, s, B, N,
                     r, Bt);
  return hipGetLastError();
}

}  // namespace qlr
