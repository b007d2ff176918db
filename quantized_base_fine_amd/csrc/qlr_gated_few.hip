// Gated block of up to 16 rows (decoding): bound by the stream of both projections' codes.
#include "qlr_few.h"

namespace qlr {

namespace {

// As the few-rows kernel of the expert products: levels from a table in LDS (pairs of codes as bf16, 32 copies), the
// block's scale on its products, a wave's rows of x through a slice of LDS of its own.  A level is held as one bf16 (off by half a
// step, 2^-8 of it, at most; see kLevelUnit; the scale stays float32): two parts would double the lookups and products that bound the kernel beside the stream.
// A workgroup of 8 waves takes 8 NS output columns as NS sets of 16 weight rows, 8 of the gate and the up rows of the same columns; each
// wave multiplies all sets over an eighth of K, so that a block of x is read once for NS sets.  Four blocks of 64 columns a
// step (of 4-bit codes, one line of 128 bytes a row), the next step's codes in flight.  The waves' sums are added through LDS
// in wave order, then each thread forms one output: both adapters' terms, the activation and the product.
//
// 16 rows of 2 x 22016 x 8192, 4-bit: 75 us (181 MB of codes, 2.4 TB/s) with two sets, one 92 (each set's own x), four 88 (one
// workgroup to a CU).  Without x's loads and writes it ran in 52, without the lookups in 66, without the codes' loads in 62: no
// one of them bounds it.  One row of 2 x 11008 x 4096: 20 us of the call's 24; two sets of 8 columns each, one 27; with
// r = 64 25. 16 rows of it, r = 16: 28, r = 64: 33 (the products before it write as many partial sums as the kernel stages, see FewAd;
// read from memory by every output they took 94 and 122).
//
// The table holds the levels times a unit f 2^-7, the results are divided by it once they are added up.  2^-7: 64 of bf16's largest
// values times levels of at most 1 stay inside float32 before the scale, and a scale times 2^7 is never formed.  f: of the bf16
// numbers in [1, 2) (so that a level of 1 stays exact) one at which bf16(f level) is close to f level.  What the rounding costs a
// product with normally distributed weights and rows, in relative 2-norm: 2 bits 4.0e-6 (at f = 1 7.9e-4), 3 bits 1.8e-4 (4.0e-4), 4 bits
// 7.0e-4 (1.18e-3), 8 bits 1.30e-3 (1.61e-3).
template <int BITS>
constexpr float kLevelUnit = (BITS == 2 ? 1.6640625f : BITS == 3 ? 1.1953125f : BITS == 4 ? 1.6015625f : 1.59375f) / 128.0f;
constexpr int kWaves = 8;
template <int BITS>
constexpr int kFewChunk = BITS == 8 ? 2 : 4;  // (four of 8 bits spill)
template <int NS>
constexpr uint32_t kRedBytes = kWaves * 16 * 16 * NS * 4;   // the waves' sums, over the slices

// The adapters' operands of 8 NS columns, and all of the kernel's dynamic LDS.
template <int NS>
using FewAd = FewAdapter<8 * NS, kGatedFewT>;
template <int BITS, int NS>
constexpr uint32_t kFewBytes = FewTab<BITS>::kBytes + (kWaves * kXSlice > kRedBytes<NS> + 2 * FewAd<NS>::kBytes ? kWaves * kXSlice : kRedBytes<NS> + 2 * FewAd<NS>::kBytes);

// P.t: the gate's t_splits x M x r partial sums, then the up projection's.
template <int BITS, int NS>
__global__ __launch_bounds__(512, 4) void k_gated_few(TrainArgs P, Levels lv) {
  constexpr int NR = 16 * NS, NO = NR / 2, NW = kFewWords<BITS>, kChunk = kFewChunk<BITS>;
  typedef FewAd<NS> Adapter;
  constexpr uint32_t kRed = FewTab<BITS>::kBytes;
  extern __shared__ uint32_t smem[];
  const int rows = (int)P.M;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t N = P.N, K = P.K, nb = K >> 6, n0 = (int64_t)blockIdx.x * NO;
  const int row = lane >> 2, g = lane & 3, src = (4 * (lane & 15) + (lane >> 4)) << 2;  // of the loads; the permute's source
  const int frow = lane & 15, fg = lane >> 4;                                           // of the fragments
  const int b0 = (int)(nb * wave / kWaves), b1 = (int)(nb * (wave + 1) / kWaves);
  // the lane's codes, scales (of block g of a step's four) and constants of each set's row
  const uint8_t *cp[NS], *qp[NS];
  const float* sp[NS];
  uint32_t srel[NS];
#pragma unroll
  for (int q = 0; q < NS; ++q) {
    const int64_t blk = ((int64_t)(row >> 3) * N + min<int64_t>(n0 + 8 * q + (row & 7), N - 1)) * nb;
    cp[q] = P.w + blk * (8 * BITS);
    qp[q] = P.q8 + blk;
    sp[q] = P.cst + (blk >> 8);
    srel[q] = (uint32_t)(blk & 255);
  }
  // x loads: piece lane % 16 of rows lane / 16 + 4 i of the two blocks
  const int xr = lane >> 4, xc = lane & 15;
  // (rows past M repeat the last, columns past K the last piece: they only reach results that are dropped, and blocks not used)
  const uint16_t* xp = reinterpret_cast<const uint16_t*>(P.x);
  struct Ld {
    Codes32<BITS> c[NS][kChunk];
    uint32_t q8[NS];
    float sc[NS];
  };
  auto load = [&](int bl, Ld& d) {
    if (bl >= b1) return;  // (the same for the whole wave)
    const uint32_t bs = (uint32_t)min(bl + (g & (kChunk - 1)), b1 - 1);
#pragma unroll
    for (int q = 0; q < NS; ++q) {
#pragma unroll
      for (int i = 0; i < kChunk; ++i)  // (a block past the range repeats the last one and is not used)
        d.c[q][i] = load_codes16<BITS>(cp[q] + (int64_t)min(bl + i, b1 - 1) * (8 * BITS), g);
      d.q8[q] = qp[q][bs];
      d.sc[q] = sp[q][(srel[q] + bs) >> 8];
    }
  };
  u32x4_t xv[4];
  auto load_x = [&](int bl) {
    const int64_t k = min<int64_t>((int64_t)bl * 64 + 8 * xc, K - 8);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * i < rows)  // (the same for the whole workgroup)
        xv[i] = *reinterpret_cast<const u32x4_t*>(xp + (int64_t)min(4 * i + xr, rows - 1) * K + k);
  };
  Ld d0, d1;
  load(b0, d0);
  load_x(b0);
  // the level table, while the first loads are on their way
  {
    float* sL = reinterpret_cast<float*>(smem) + kRed / 4;
    stage_levels<1 << BITS>(lv, sL);
    __syncthreads();
    constexpr int NL = 1 << BITS;
    for (int i = tid; i < FewTab<BITS>::kEntries * 8; i += 512) {  // four copies each
      const int en = i >> 3;
      const uint32_t v = BITS == 8 ? f32_to_bf16_bits(kLevelUnit<BITS> * sL[en])
                                   : pack_bf16x2(kLevelUnit<BITS> * sL[en & (NL - 1)], kLevelUnit<BITS> * sL[en >> BITS]);
      reinterpret_cast<u32x4_t*>(smem)[i] = u32x4_t{v, v, v, v};
    }
    __syncthreads();
  }
  const uint32_t tl = 4u * (lane & 31);
  f32x4_t acc[NS];
  char* const xs = reinterpret_cast<char*>(smem) + kRed + wave * kXSlice;
  auto compute = [&](int bl, const Ld& d) {
    float ap[NS];
#pragma unroll
    for (int q = 0; q < NS; ++q) ap[q] = (float)d.q8[q] * d.sc[q];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      if (bl + i >= b1) return;  // (the same for the whole wave)
      if (i % 2 == 0) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (4 * t < rows) *reinterpret_cast<u32x4_t*>(xs + (4 * t + xr) * kXRow + 16 * xc) = xv[t];
        load_x(bl + i + 2);
      }
      const char* xf = xs + frow * kXRow + 128 * (i % 2) + 32 * fg;
      // (rows past M hold anything: they only reach results that are dropped)
      const bf16x8_t x0 = as_bf16x8(*reinterpret_cast<const u32x4_t*>(xf)), x1 = as_bf16x8(*reinterpret_cast<const u32x4_t*>(xf + 16));
#pragma unroll
      for (int q = 0; q < NS; ++q) {
        Codes32<BITS> c = d.c[q][i];
        place_codes16<BITS>(c, g);
        uint32_t w[NW], o[8];
#pragma unroll
        for (int j = 0; j < NW; ++j) w[j] = (uint32_t)__builtin_amdgcn_ds_bpermute(src, (int)c.w[j]);
        const float a = __int_as_float(__builtin_amdgcn_ds_bpermute(16 * frow + 4 * i, __float_as_int(ap[q])));
        few_levels<BITS>(w, tl, o);
        f32x4_t s = {0.f, 0.f, 0.f, 0.f};
        s = mfma16x16x32(x0, as_bf16x8(u32x4_t{o[0], o[1], o[2], o[3]}), s);
        s = mfma16x16x32(x1, as_bf16x8(u32x4_t{o[4], o[5], o[6], o[7]}), s);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[q][v] = fmaf(a, s[v], acc[q][v]);
      }
    }
  };
  float* const red = reinterpret_cast<float*>(smem) + kRed / 4;
  char* const ad_lds = reinterpret_cast<char*>(smem) + kRed + kRedBytes<NS>;
  const int64_t tside = (int64_t)P.t_splits * rows * P.r;
#pragma unroll
  for (int q = 0; q < NS; ++q) acc[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int bl = b0; bl < b1; bl += 2 * kChunk) {
    load(bl + kChunk, d1);
    compute(bl, d0);
    if (bl + kChunk >= b1) break;
    load(bl + 2 * kChunk, d0);
    compute(bl + kChunk, d1);
  }
  const int live = (int)min<int64_t>(NO, N - n0);
  Adapter ad[2];
#pragma unroll
  for (int sd = 0; sd < 2; ++sd)
    ad[sd].load(P.t + sd * tside, P.t_splits, P.M, 0, rows, P.ab + (int64_t)sd * N * P.r, n0, live, P.r);
  __syncthreads();  // (the sums and the adapters' operands overlay the waves' slices)
  // [K range][token][weight row]: the lane's tokens 4 fg + v of weight row frow
#pragma unroll
  for (int q = 0; q < NS; ++q)
#pragma unroll
    for (int v = 0; v < 4; ++v) red[(wave * 16 + 4 * fg + v) * NR + 16 * q + frow] = acc[q][v];
#pragma unroll
  for (int sd = 0; sd < 2; ++sd) ad[sd].stage(ad_lds + sd * Adapter::kBytes, P.t_splits, rows, P.r);
  __syncthreads();
  const int m = tid / NO, c = tid % NO;  // (16 rows x 32 columns at most: one output a thread)
  if (m < rows && c < live) {
    float gv[2];
#pragma unroll
    for (int sd = 0; sd < 2; ++sd) {
      float y = 0.0f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) y += red[(k * 16 + m) * NR + 16 * (c >> 3) + 8 * sd + (c & 7)];
      y *= 1.0f / kLevelUnit<BITS>;
      if (P.r > 0)
        y = fmaf(P.scale, ad[sd].dot(ad_lds + sd * Adapter::kBytes, P.t + sd * tside, P.t_splits, P.M, 0, m,
                                     P.ab + (int64_t)sd * N * P.r, n0, c, P.r), y);
      gv[sd] = y;
      if (P.gu) P.gu[(int64_t)m * 2 * N + sd * N + n0 + c] = (uint16_t)f32_to_bf16_bits(y);
    }
    const float a = P.act == ACT_SILU ? act_f<ACT_SILU>(gv[0]) : P.act == ACT_GELU ? act_f<ACT_GELU>(gv[0]) : act_f<ACT_GELU_TANH>(gv[0]);
    const int64_t o = (int64_t)m * N + n0 + c;
    if (P.ydt == DT_F32) reinterpret_cast<float*>(P.y)[o] = a * gv[1];
    else reinterpret_cast<uint16_t*>(P.y)[o] = (uint16_t)f32_to_bf16_bits(a * gv[1]);
  }
}

template <int BITS, int NS>
hipError_t launch_few_r(const TrainArgs& a, const Levels& lv, hipStream_t s) {
  auto kern = k_gated_few<BITS, NS>;
  static std::atomic<bool> checked{false};
  constexpr size_t shmem = kFewBytes<BITS, NS>;
  const hipError_t e = few_prepare(reinterpret_cast<const void*>(kern), shmem, checked);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(a.N + 8 * NS - 1) / (8 * NS)), dim3(512), shmem, s, a, lv);
  return hipGetLastError();
}

template <int BITS>
hipError_t launch_few_b(const TrainArgs& a, const Levels& lv, hipStream_t s) {
  // two sets where that leaves 512 workgroups, two to a CU
  const int64_t sets = (a.N + 7) / 8;
  if (sets >= 2 * 512) return launch_few_r<BITS, 2>(a, lv, s);
  return launch_few_r<BITS, 1>(a, lv, s);
}

}  // namespace

hipError_t launch_gated_few(const TrainArgs& a, const Levels& lv, hipStream_t s) {
  if (a.M > kFewRows) return hipErrorInvalidValue;
  switch (a.bits) {
    case 2: return launch_few_b<2>(a, lv, s);
    case 3: return launch_few_b<3>(a, lv, s);
    case 4: return launch_few_b<4>(a, lv, s);
    default: return launch_few_b<8>(a, lv, s);
  }
}

}  // namespace qlr
