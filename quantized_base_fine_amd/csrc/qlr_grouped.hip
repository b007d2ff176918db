// Expert-grouped products of a mixture-of-experts layer on the coded base: rows
// sorted by expert, device offsets, one stacked weight, one adapter per expert.
// This file holds the forward for experts with few rows and the adapter
// products; the tiled products are instantiated per code width elsewhere.
#include "qlr_few.h"

namespace qlr {

namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
// LDS transpose read of 16-bit elements (see lds_tr16) by pointer
__device__ __forceinline__ s16x4_t lds_tr16p(const char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(const_cast<char*>(p)));
}

// ---------------------------------------------------------------- experts of 1 .. 16 rows
//
// Bound by the stream of the experts' codes, so the dequantization has to stay
// off its way: levels come from a table in LDS (pairs of codes, bf16, 32 copies
// that keep a wave's lookups on different banks: about 50 vector instructions per KB of
// 4-bit codes, where forming scaled levels in registers took 144 and bound the kernel), and
// the block's scale multiplies its products.  A level is held as one bf16 (half a step, 2^-8 of it; the scale stays float32):
// two parts would double the lookups and products of a kernel that these bound.  Against 64 bits a bf16 result is off by
// 2.0e-3 in relative 2-norm, its own rounding being 1.7e-3.
//   y[m][n] = sum over blocks of scale[n][block] (sum_k x[m][k] level[n][k])
// A workgroup of 8 waves takes 16 RS weight rows of one expert: RS sets of 16
// rows, the 8 / RS waves of a set sharing K in ranges of 64-element blocks.  Per
// block a lane loads 16 codes of one row, each quad of lanes a row's whole
// block (8-byte pieces in MFMA fragment order read at 4.0 TB/s, quads on one row's bytes at 5.5),
// lane permutes bring them to fragment order, and two 16x16x32 MFMAs (the expert's rows
// as A) start from zero.  Codes are loaded kFewChunk to 2 kFewChunk blocks ahead; the rows' elements two
// blocks ahead, four rows to a load, and go through a slice of LDS of the wave's
// own (a wave's LDS accesses run in order).  The waves' sums are added through LDS
// in wave order, then scale t B^T.
//
// 32 rows of 8 experts of 11008 x 4096, 4-bit: 48 us for 180 MB of codes that the last cache holds in part (3.8 TB/s), 56
// for codes from memory.  What bounds it: the vector units are busy 42 % of the cycles and each KB of codes takes 26 LDS
// accesses of a wave (levels, permutes, x), which the loads cover only in part.  Whole 128-byte lines through a wave's slice of LDS instead of 32-byte
// pieces of 16 rows took 57 us from memory and 55 from cache, and 2-bit codes 11 % longer: not kept.
constexpr int kFewWaves = 8, kFewChunk = 2;

template <int BITS, int RS>
__global__ __launch_bounds__(512, 4) void k_grouped_few(TileArgs P, Levels lv) {
  constexpr int NR = 16 * RS, KS = kFewWaves / RS, NW = kFewWords<BITS>;
  typedef FewAdapter<NR, 1024> Adapter;
  constexpr uint32_t kRed = FewTab<BITS>::kBytes;
  extern __shared__ uint32_t smem[];
  int a, b;
  const int e = blockIdx.y;
  expert_range(P.offsets, e, (int)P.M, a, b);
  const int rows = b - a;
  if (rows < 1 || rows > kFewRows) return;  // the whole workgroup
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t N = P.N, K = P.K, nb = K >> 6;
  const int n0 = blockIdx.x * NR, rs = wave / KS, ks = wave % KS;
  const int row = lane >> 2, g = lane & 3, src = (4 * (lane & 15) + (lane >> 4)) << 2;  // of the loads; the permute's source
  const int frow = lane & 15, fg = lane >> 4;                                           // of the fragments
  const int b0 = (int)(nb * ks / KS), b1 = (int)(nb * (ks + 1) / KS);
  const int64_t wblk = ((int64_t)e * N + min<int64_t>(n0 + 16 * rs + row, N - 1)) * nb;
  // x loads: piece lane % 16 of rows lane / 16 + 4 i of the two blocks
  const int xr = lane >> 4, xc = lane & 15;
  const uint16_t* xp = reinterpret_cast<const uint16_t*>(P.x) + (int64_t)a * K + 8 * xc;
  struct Ld {
    uint32_t c[kFewChunk][NW];
    uint32_t q8[kFewChunk];
    float sc[kFewChunk];
  };
  const u32x4_t zero4 = {0u, 0u, 0u, 0u};
  auto load = [&](int bl, Ld& d) {  // (blocks past the wave's range repeat its last one and are not used)
#pragma unroll
    for (int i = 0; i < kFewChunk; ++i) {
      const int64_t blk = wblk + max(min(bl + i, b1 - 1), 0);
      Codes32<BITS> c = load_codes16<BITS>(P.w + blk * (8 * BITS), g);
      place_codes16<BITS>(c, g);
#pragma unroll
      for (int j = 0; j < NW; ++j) d.c[i][j] = c.w[j];
      d.q8[i] = P.q8[blk];
      d.sc[i] = P.cst[blk >> 8];
    }
  };
  u32x4_t xv[4];
  auto load_x = [&](int bl) {
    const int64_t k = (int64_t)bl * 64;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * i < rows)  // (the same for the whole workgroup)
        xv[i] = 4 * i + xr < rows && k + 8 * xc < K && bl < b1
                    ? *reinterpret_cast<const u32x4_t*>(xp + (int64_t)(4 * i + xr) * K + k) : zero4;
  };
  Ld d0, d1;
  load(b0, d0);
  load_x(b0);
  Adapter ad;
  ad.load(P.t, 1, P.M, a, rows, P.ab + (int64_t)e * N * P.r, n0, (int)min<int64_t>(NR, N - n0), P.r);
  // the level table, while the first loads are on their way
  {
    float* sL = reinterpret_cast<float*>(smem) + kRed / 4;
    stage_levels<1 << BITS>(lv, sL);
    __syncthreads();
    constexpr int NL = 1 << BITS;
    for (int i = tid; i < FewTab<BITS>::kEntries * 32; i += 512) {
      const int en = i >> 5;
      smem[i] = BITS == 8 ? f32_to_bf16_bits(sL[en]) : pack_bf16x2(sL[en & (NL - 1)], sL[en >> BITS]);
    }
    __syncthreads();
  }
  const uint32_t tl = 4u * (lane & 31);
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  char* const xs = reinterpret_cast<char*>(smem) + kRed + wave * kXSlice;
  auto compute = [&](int bl, const Ld& d) {
#pragma unroll
    for (int i = 0; i < kFewChunk; ++i) {
      if (bl + i >= b1) return;  // (the same for the whole wave)
      if (i % 2 == 0) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (4 * t < rows) *reinterpret_cast<u32x4_t*>(xs + (4 * t + xr) * kXRow + 16 * xc) = xv[t];
        load_x(bl + i + 2);
      }
      uint32_t w[NW], o[8];
#pragma unroll
      for (int j = 0; j < NW; ++j) w[j] = (uint32_t)__builtin_amdgcn_ds_bpermute(src, (int)d.c[i][j]);
      const float ap = __int_as_float(__builtin_amdgcn_ds_bpermute(src, __float_as_int((float)d.q8[i] * d.sc[i])));
      few_levels<BITS>(w, tl, o);
      const char* xf = xs + frow * kXRow + 128 * (i % 2) + 32 * fg;
      // (rows past the expert's hold anything: they only reach results that are dropped)
      f32x4_t s = {0.f, 0.f, 0.f, 0.f};
      s = mfma16x16x32(as_bf16x8(*reinterpret_cast<const u32x4_t*>(xf)), as_bf16x8(u32x4_t{o[0], o[1], o[2], o[3]}), s);
      s = mfma16x16x32(as_bf16x8(*reinterpret_cast<const u32x4_t*>(xf + 16)), as_bf16x8(u32x4_t{o[4], o[5], o[6], o[7]}), s);
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[v] = fmaf(ap, s[v], acc[v]);
    }
  };
  for (int bl = b0; bl < b1; bl += 2 * kFewChunk) {
    load(bl + kFewChunk, d1);
    compute(bl, d0);
    if (bl + kFewChunk >= b1) break;
    load(bl + 2 * kFewChunk, d0);
    compute(bl + kFewChunk, d1);
  }
  __syncthreads();  // (the sums overlay the waves' slices)
  // [K range][token][weight row]: the lane's tokens 4 fg + v of weight row frow
  float* red = reinterpret_cast<float*>(smem) + kRed / 4;
#pragma unroll
  for (int v = 0; v < 4; ++v) red[(ks * 16 + 4 * fg + v) * NR + 16 * rs + frow] = acc[v];
  char* ad_lds = reinterpret_cast<char*>(smem) + kRed + kFewWaves * kXSlice;
  ad.stage(ad_lds, 1, rows, P.r);
  __syncthreads();
  for (int idx = tid; idx < rows * NR; idx += 512) {
    const int m = idx / NR, c = idx % NR;
    const int n = n0 + c;
    if (n >= N) continue;
    float y = 0.0f;
#pragma unroll
    for (int k = 0; k < KS; ++k) y += red[(k * 16 + m) * NR + c];
    if (P.r > 0)
      y = fmaf(P.scale, ad.dot(ad_lds, P.t, 1, P.M, a, m, P.ab + (int64_t)e * N * P.r, n0, c, P.r), y);
    const int64_t o = (int64_t)(a + m) * N + n;
    if (P.ydt == DT_F32) reinterpret_cast<float*>(P.y)[o] = y;
    else reinterpret_cast<uint16_t*>(P.y)[o] = (uint16_t)f32_to_bf16_bits(y);
  }
}

template <int BITS, int RS>
hipError_t launch_few_r(const TileArgs& a, const Levels& lv, hipStream_t s) {
  auto kern = k_grouped_few<BITS, RS>;
  static std::atomic<bool> checked{false};
  const size_t shmem = FewTab<BITS>::kBytes + kFewWaves * kXSlice + (a.r > 0 ? FewAdapter<16 * RS, 1024>::kBytes : 0);
  const hipError_t e = few_prepare(reinterpret_cast<const void*>(kern), shmem, checked);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)((a.N + 16 * RS - 1) / (16 * RS)), (unsigned)a.experts), dim3(512), shmem, s, a, lv);
  return hipGetLastError();
}

template <int BITS>
hipError_t launch_few_b(const TileArgs& a, const Levels& lv, hipStream_t s) {
  // as many rows to a workgroup (one level table) as still gives the experts that can have rows 512 of them
  const int64_t rows16 = std::min<int64_t>(a.experts, a.M) * ((a.N + 15) / 16);
  if (rows16 >= 4 * 512) return launch_few_r<BITS, 4>(a, lv, s);
  if (rows16 >= 2 * 512) return launch_few_r<BITS, 2>(a, lv, s);
  return launch_few_r<BITS, 1>(a, lv, s);
}

// ---------------------------------------------------------------- t = x A_e^T, u = dy B_e
//
// A workgroup of W waves takes 16 RT rows of one expert x 16 JT adapter columns of
// one product (the backward's two run in one launch); the waves split K in 32-element steps and multiply on 16x16x32 bf16
// MFMA (x rows as A, the adapter as B).  Loads give each quad of lanes one row's
// 64 bytes; a slice of LDS of the wave's own brings them to the fragment layout
// (80-byte rows, free of bank conflicts).  An adapter given as K x r (the
// backward's B) is staged row-major, 32 rows of K, and read with the LDS transpose
// read.  NB steps of loads are in flight while the NB before them are
// multiplied.  The waves' sums are added through LDS in wave order.  Bound by reading x:
// 4096 rows of x and dy of 4096, r = 16: 67 MB in 19 us (3.5 TB/s); 8192 rows, r = 64: 67 MB in 28.
constexpr uint32_t kTRowB = 80;

struct TJob {
  const uint16_t* x;  // M x K
  const uint16_t* A;  // experts x r x K, or (BT) experts x K x r
  int64_t K;
  float* t;           // M x r
};
struct TJobs {
  TJob j[2];
  int64_t M;
  int r, experts;
  const int32_t* offsets;
};

// Bytes of row k of a staged K x r step (16 JT columns): rows 8 .. 15 of every 16 swap halves of a
// 128-byte window where rows are 32 bytes, so that the transpose reads of rows {q .. q + 3} and {q + 8 .. q + 11} by
// one half-wave hit distinct banks; longer rows are padded by 16 bytes.
template <int JT>
__device__ __forceinline__ uint32_t bt_off(uint32_t k) {
  return JT == 1 ? (k * 32u) ^ (((k >> 3) & 1u) << 7) : k * (32u * JT + 16u);
}

template <int RT, int JT, int W, int NB, bool BT>
__device__ __forceinline__ void t_tile(const TJob& job, int64_t M, int r, int e, int row0, int rows, int j0, char* lds) {
  constexpr uint32_t kASlice = BT ? (JT == 1 ? 1024u : 32u * (32u * JT + 16u)) : 16u * JT * kTRowB;
  constexpr uint32_t kSlice = 16 * RT * kTRowB + kASlice;
  const int64_t K = job.K;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = lane >> 2, g = lane & 3;     // of the loads
  const int frow = lane & 15, fg = lane >> 4;  // of the fragments
  const uint16_t* xp[RT];
  const uint16_t* ap[JT];
#pragma unroll
  for (int i = 0; i < RT; ++i) xp[i] = job.x + (int64_t)(row0 + min(16 * i + row, rows - 1)) * K + 8 * g;
  // BT: load c of a step holds 16-byte pieces 64 c + lane of the 32 rows' 2 JT pieces each
  int brow[JT], bcol[JT];
#pragma unroll
  for (int c = 0; c < JT; ++c) {
    brow[c] = (64 * c + lane) / (2 * JT);
    bcol[c] = 8 * ((64 * c + lane) % (2 * JT));
    if constexpr (BT) ap[c] = job.A + ((int64_t)e * K + brow[c]) * r + min(j0 + bcol[c], r - 8);
    else ap[c] = job.A + ((int64_t)e * r + min(j0 + 16 * c + row, r - 1)) * K + 8 * g;
  }
  f32x4_t acc[RT][JT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int c = 0; c < JT; ++c) acc[i][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int nst = (int)((K + 31) / 32);
  const int s0 = (int)((int64_t)nst * wave / W), s1 = (int)((int64_t)nst * (wave + 1) / W);
  const u32x4_t zero4 = {0u, 0u, 0u, 0u};
  struct Ld { u32x4_t x[NB][RT], a[NB][JT]; };
  // rows past the range or the adapter's rank repeat the last one: their results are dropped
  auto load = [&](int st, Ld& d) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int64_t k = (int64_t)(st + b) * 32;
      const bool ok = st + b < s1 && k + 8 * g < K;  // past the range or the row's end: zeros
#pragma unroll
      for (int i = 0; i < RT; ++i) d.x[b][i] = ok ? *reinterpret_cast<const u32x4_t*>(xp[i] + k) : zero4;
#pragma unroll
      for (int c = 0; c < JT; ++c) {
        if constexpr (BT) d.a[b][c] = st + b < s1 && k + brow[c] < K ? *reinterpret_cast<const u32x4_t*>(ap[c] + k * r) : zero4;
        else d.a[b][c] = ok ? *reinterpret_cast<const u32x4_t*>(ap[c] + k) : zero4;
      }
    }
  };
  char* const sl = lds + wave * kSlice;
  char* const sa = sl + 16 * RT * kTRowB;
  auto compute = [&](const Ld& d) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int i = 0; i < RT; ++i) *reinterpret_cast<u32x4_t*>(sl + (16 * i + row) * kTRowB + 16 * g) = d.x[b][i];
#pragma unroll
      for (int c = 0; c < JT; ++c) {
        if constexpr (BT) *reinterpret_cast<u32x4_t*>(sa + bt_off<JT>(brow[c]) + 2 * bcol[c]) = d.a[b][c];
        else *reinterpret_cast<u32x4_t*>(sa + (16 * c + row) * kTRowB + 16 * g) = d.a[b][c];
      }
      bf16x8_t xf[RT], af[JT];
#pragma unroll
      for (int i = 0; i < RT; ++i) xf[i] = as_bf16x8(*reinterpret_cast<const u32x4_t*>(sl + (16 * i + frow) * kTRowB + 16 * fg));
#pragma unroll
      for (int c = 0; c < JT; ++c) {
        if constexpr (BT) {
          // rows 8 fg + {0 .. 3} and {4 .. 7} of adapter column 16 c + lane % 16
          const uint32_t kr = 8u * fg + (frow >> 2), co = 32u * c + 8u * (frow & 3);
          const s16x4_t lo = lds_tr16p(sa + bt_off<JT>(kr) + co), hi = lds_tr16p(sa + bt_off<JT>(kr + 4) + co);
          af[c] = as_bf16x8(u32x4_t{__builtin_bit_cast(uint2, lo).x, __builtin_bit_cast(uint2, lo).y,
                                    __builtin_bit_cast(uint2, hi).x, __builtin_bit_cast(uint2, hi).y});
        } else {
          af[c] = as_bf16x8(*reinterpret_cast<const u32x4_t*>(sa + (16 * c + frow) * kTRowB + 16 * fg));
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < JT; ++c) acc[i][c] = mfma16x16x32(xf[i], af[c], acc[i][c]);
    }
  };
  Ld d0, d1;
  load(s0, d0);
  for (int st = s0; st < s1; st += 2 * NB) {
    load(st + NB, d1);
    compute(d0);
    if (st + NB >= s1) break;
    load(st + 2 * NB, d0);
    compute(d1);
  }
  __syncthreads();
  float* red = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int c = 0; c < JT; ++c)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        red[wave * (RT * 16 * JT * 16) + (16 * i + 4 * fg + v) * (16 * JT) + 16 * c + frow] = acc[i][c][v];
  __syncthreads();
  for (int idx = tid; idx < rows * 16 * JT; idx += 64 * W) {
    const int m = idx / (16 * JT), j = j0 + idx % (16 * JT);
    if (j >= r) continue;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += red[w * (RT * 16 * JT * 16) + idx];
    job.t[(int64_t)(row0 + m) * r + j] = sum;
  }
}

// blockIdx.z = 0: job 0 (adapter r x K); 1: job 1 (the backward's, adapter K x r, r % 8 == 0)
template <int RT, int JT, int W, int NB>
__global__ __launch_bounds__(64 * W) void k_grouped_t(TJobs J) {
  constexpr uint32_t kA = 16u * JT * kTRowB, kB = JT == 1 ? 1024u : 32u * (32u * JT + 16u);
  constexpr uint32_t kSlice = 16 * RT * kTRowB + (kA > kB ? kA : kB), kSum = RT * 16 * JT * 16 * 4;
  __shared__ __attribute__((aligned(16))) char lds[W * (kSlice > kSum ? kSlice : kSum)];
  int e = 0, row0 = 0, row_end = 0;
  ScanChunk c0;
  const int total = tile_count(J.offsets, J.experts, (int)J.M, 0, 16 * RT, c0);
  // each XCD a contiguous range of row tiles (the grid's rows are a multiple of 8): an expert's adapter in few L2s
  const int per = (total + 7) / 8, loc = (int)(blockIdx.x >> 3), tile = (int)(blockIdx.x & 7) * per + loc;
  if (loc >= per || tile >= total) return;  // the whole workgroup
  tile_find(J.offsets, J.experts, (int)J.M, 0, 16 * RT, c0, tile, e, row0, row_end);
  e = __builtin_amdgcn_readfirstlane(e);
  row0 = __builtin_amdgcn_readfirstlane(row0);
  row_end = __builtin_amdgcn_readfirstlane(row_end);
  const int rows = min(16 * RT, row_end - row0), j0 = blockIdx.y * 16 * JT;
  if (blockIdx.z == 0) t_tile<RT, JT, W, NB, false>(J.j[0], J.M, J.r, e, row0, rows, j0, lds);
  else t_tile<RT, JT, W, NB, true>(J.j[1], J.M, J.r, e, row0, rows, j0, lds);
}

template <int RT, int JT, int W, int NB>
hipError_t launch_t(const TJobs& J, int jobs, hipStream_t s) {
  hipLaunchKernelGGL((k_grouped_t<RT, JT, W, NB>),
                     dim3((unsigned)((tile_bound(J.M, J.experts, 16 * RT) + 7) / 8 * 8), (unsigned)((J.r + 16 * JT - 1) / (16 * JT)), (unsigned)jobs),
                     dim3(64 * W), 0, s, J);
  return hipGetLastError();
}

hipError_t launch_t_jobs(const TJobs& J, int jobs, hipStream_t s) {
  // Few row tiles: 16 waves, 8 steps of loads in flight each (a decode call waits for one round trip).  Many: 32 rows
  // against up to 64 adapter columns, which halves the reads of A; 64 rows where the ranges fill them and A is wide (8192
  // rows of 4096, r = 64: 37 us with 32 rows, 30 with 64, of 13 for reading x).  Narrow A: 8 waves with 2 steps in flight
  // (4096 rows of x and dy, r = 16: 19.0 us, 4 waves with 4 steps 19.4; 4096 rows of 2048: 7.0 and 7.8).
  const bool few = tile_bound(J.M, J.experts, 16) * ((J.r + 15) / 16) <= 256;
  if (few) return launch_t<1, 1, 16, 4>(J, jobs, s);
  if (J.r <= 16) return launch_t<2, 1, 8, 2>(J, jobs, s);
  if (J.r <= 32) return launch_t<2, 2, 4, 2>(J, jobs, s);
  if (J.M < (int64_t)J.experts * 128) return launch_t<2, 4, 4, 2>(J, jobs, s);
  return launch_t<4, 4, 8, 1>(J, jobs, s);
}

// Bt[e][j][n] = B[e][n][j]
__global__ __launch_bounds__(256) void k_grouped_transpose(const uint16_t* __restrict__ B, int64_t N, int r,
                                                           uint16_t* __restrict__ Bt) {
  const int64_t base = (int64_t)blockIdx.y * N * r;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < N * r; i += (int64_t)gridDim.x * 256) {
    const int64_t j = i / N, n = i % N;
    Bt[base + i] = B[base + n * r + j];
  }
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
  TJobs J{};
  J.j[0] = TJob{x, A, K, t};
  J.M = M;
  J.r = r;
  J.experts = experts;
  J.offsets = offsets;
  return launch_t_jobs(J, 1, s);
}

hipError_t launch_grouped_tu(const uint16_t* x, const uint16_t* dy, int64_t M, int64_t N, int64_t K, const uint16_t* A,
                             const uint16_t* B, int r, const int32_t* offsets, int experts, float* t, float* u,
                             hipStream_t s) {
  if (r % 8 != 0) return hipErrorInvalidValue;
  TJobs J{};
  J.j[0] = TJob{x, A, K, t};
  J.j[1] = TJob{dy, B, N, u};
  J.M = M;
  J.r = r;
  J.experts = experts;
  J.offsets = offsets;
  return launch_t_jobs(J, 2, s);
}

hipError_t launch_grouped_transpose(const uint16_t* B, int experts, int64_t N, int r, uint16_t* Bt, hipStream_t s) {
  hipLaunchKernelGGL(k_grouped_transpose, dim3((unsigned)std::min((N * r + 255) / 256, kLaunchBlocks), (unsigned)experts), dim3(256),
                     0, s, B, N, r, Bt);
  return hipGetLastError();
}

}  // namespace qlr
