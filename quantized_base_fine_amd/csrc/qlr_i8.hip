// The linear layer in 8-bit integers: y = (sum_k xq wq) sx[m] sw[n] with one
// scale per token and one per output channel, plus the unmerged adapter branch
// of the frozen base (LoRDBA page, "adapter mode").
//
// Row quantization (tokens and weight channels alike): s = fl32(max|x| fl32(1 / 127)),
// q = the integer nearest x / s, ties to even, in [-127, 127].  (The product, not
// the quotient, which can be a last place away and then takes exact ties to the other
// side: amax() / 127 on the GPU in PyTorch is this product, so rows quantized by
// either agree bit for bit.)
#include "qlr_lora_t.h"
#include "qlr_tile.h"

namespace qlr {

namespace {

// ---------------------------------------------------------------- row quantization
//
// One workgroup per row.  Pieces of 8 elements stay in registers (as loaded)
// between the maximum and the rounding, NP per thread; longer rows read the rest
// again, from cache.  The quotient is decided exactly: q0 = rint(x * fl(1/s)) is
// within one of x / s, the residual x - q0 s is exact in float32 (a multiple of
// s's last place, below s), and comparing twice the residual with s settles the
// nearest integer and ties.
__device__ __forceinline__ int quantize_exact(float w, float s, float inv) {
  const float q0 = __builtin_rintf(inv > 0.0f ? w * inv : w / s);
  const float d = fmaf(-q0, s, w);
  const float d2 = 2.0f * fabsf(d);
  int q = (int)q0;
  if (d2 > s || (d2 == s && (q & 1))) q += d > 0.0f ? 1 : -1;
  return min(max(q, -127), 127);
}

// Eight elements as loaded.
template <int DT>
struct Raw8 { u32x4_t v[DT == DT_F32 ? 2 : 1]; };
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const void* p, int64_t i) {
  Raw8<DT> r;
  const u32x4_t* q = reinterpret_cast<const u32x4_t*>(reinterpret_cast<const char*>(p) + i * (DT == DT_F32 ? 4 : 2));
  r.v[0] = q[0];
  if constexpr (DT == DT_F32) r.v[1] = q[1];
  return r;
}
template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT>& r, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = r.v[0][e];
    if constexpr (DT == DT_F32) {
      const uint32_t w2 = r.v[1][e];
      v[e] = __uint_as_float(w);
      v[4 + e] = __uint_as_float(w2);
    } else if constexpr (DT == DT_BF16) {
      v[2 * e] = __uint_as_float(w << 16);
      v[2 * e + 1] = __uint_as_float(w & 0xFFFF0000u);
    } else {
      v[2 * e] = f16_bits_to_f32((uint16_t)w);
      v[2 * e + 1] = f16_bits_to_f32((uint16_t)(w >> 16));
    }
  }
}

// VEC: cols % 8 == 0 (16-byte loads, 8-byte stores); otherwise element by element.
// Called by a whole workgroup of NTH threads; red: NTH / 64 words of LDS.
template <int DT, bool VEC, int NP, int NTH>
__device__ __forceinline__ void quantize_row(const void* __restrict__ X, int64_t row, int64_t cols,
                                             int8_t* __restrict__ q, float* __restrict__ scale, uint32_t* red) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t base = row * cols;
  // |x| as bits: ordered like the magnitudes, Inf and NaN above every finite value
  uint32_t am = 0;
  Raw8<DT> v[NP];
  auto amax8 = [&](const Raw8<DT>& r) {
    float w[8];
    widen8<DT>(r, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) am = max(am, __float_as_uint(fabsf(w[e])));
  };
  if constexpr (VEC) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int64_t c = 8 * ((int64_t)p * NTH + tid);
      if (c < cols) v[p] = load8<DT>(X, base + c);
    }
#pragma unroll
    for (int p = 0; p < NP; ++p)
      if (8 * ((int64_t)p * NTH + tid) < cols) amax8(v[p]);
    for (int64_t c = 8 * ((int64_t)NP * NTH + tid); c < cols; c += 8 * NTH) amax8(load8<DT>(X, base + c));
  } else {
    for (int64_t c = tid; c < cols; c += NTH) am = max(am, __float_as_uint(fabsf(load_elem<DT>(X, base + c))));
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) am = max(am, (uint32_t)__shfl_xor((int)am, off, 64));
  if (lane == 0) red[wave] = am;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NTH / 64; ++w) am = max(am, red[w]);
  const bool finite = am < 0x7F800000u;
  const float s = finite ? __uint_as_float(am) * (1.0f / 127.0f) : __uint_as_float(0x7FC00000u);
  if (tid == 0) scale[row] = s;
  const bool live = finite && s > 0.0f;
  // below 2^-125 the reciprocal could overflow: divide instead
  const float inv = s >= 2.350988701644575e-38f ? 1.0f / s : 0.0f;
  auto q1 = [&](float w) { return live ? quantize_exact(w, s, inv) : 0; };
  auto put8 = [&](int64_t c, const Raw8<DT>& r) {
    float w[8];
    widen8<DT>(r, w);
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo |= ((uint32_t)q1(w[e]) & 255u) << (8 * e);
      hi |= ((uint32_t)q1(w[4 + e]) & 255u) << (8 * e);
    }
    *reinterpret_cast<uint2*>(q + base + c) = uint2{lo, hi};
  };
  if constexpr (VEC) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int64_t c = 8 * ((int64_t)p * NTH + tid);
      if (c < cols) put8(c, v[p]);
    }
    for (int64_t c = 8 * ((int64_t)NP * NTH + tid); c < cols; c += 8 * NTH) put8(c, load8<DT>(X, base + c));
  } else {
    for (int64_t c = tid; c < cols; c += NTH) q[base + c] = (int8_t)q1(load_elem<DT>(X, base + c));
  }
}

template <int DT, bool VEC, int NP, int NTH>
__global__ __launch_bounds__(NTH) void k_quantize_i8(const void* __restrict__ X, int64_t cols, int8_t* __restrict__ q,
                                                     float* __restrict__ scale) {
  __shared__ uint32_t red[NTH / 64];
  quantize_row<DT, VEC, NP, NTH>(X, blockIdx.x, cols, q, scale, red);
}

// A decode call's tokens: the first M workgroups quantize a row each, the others
// compute the partial sums of t = x A^T (both read x only), in one launch.
__global__ __launch_bounds__(kLtWaves * 64) void k_i8_prep(const uint16_t* __restrict__ x, int64_t M, int64_t K,
                                                           int8_t* __restrict__ q, float* __restrict__ scale,
                                                           const uint16_t* __restrict__ A, int r, int jtiles, int splits,
                                                           float* __restrict__ t) {
  __shared__ float red[kLtWaves][256];
  const int b = (int)blockIdx.x - (int)M;
  if (b < 0) quantize_row<DT_BF16, true, 2, kLtWaves * 64>(x, blockIdx.x, K, q, scale, reinterpret_cast<uint32_t*>(&red[0][0]));
  else lora_t_small_body(x, M, K, A, r, t, (b % jtiles) * 16, splits, b / jtiles, red);
}

// Long rows: 1024 threads a row while there is at most a row per CU (16 rows of 8192: 5.1 us, with 256 threads 7.7),
// 256 threads for more (4096 rows of 11008: 38 us, with 1024 threads 42).  2048 rows of 4096 take 10.5 us (2.4 TB/s; a copy of as
// many bytes takes 4.9): of the 20 thousand cycles beyond an empty launch's, the vector units are busy 14 with widening, the
// maximum and the exact rounding, about 15 instructions an element.
template <int DT>
hipError_t launch_quantize_dt(const void* X, int64_t rows, int64_t cols, int8_t* q, float* scale, hipStream_t s) {
  for (int64_t r0 = 0; r0 < rows; r0 += 1 << 23) {  // (a launch holds fewer than 2^32 threads)
    const dim3 n((unsigned)std::min<int64_t>(rows - r0, 1 << 23));
    const char* x0 = reinterpret_cast<const char*>(X) + r0 * cols * (DT == DT_F32 ? 4 : 2);
    int8_t* q0 = q + r0 * cols;
    if (cols % 8 != 0) hipLaunchKernelGGL((k_quantize_i8<DT, false, 1, 256>), n, dim3(256), 0, s, x0, cols, q0, scale + r0);
    else if (cols <= 2 * 2048) hipLaunchKernelGGL((k_quantize_i8<DT, true, 2, 256>), n, dim3(256), 0, s, x0, cols, q0, scale + r0);
    else if (rows <= 256) hipLaunchKernelGGL((k_quantize_i8<DT, true, 2, 1024>), n, dim3(1024), 0, s, x0, cols, q0, scale + r0);
    else hipLaunchKernelGGL((k_quantize_i8<DT, true, 8, 256>), n, dim3(256), 0, s, x0, cols, q0, scale + r0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---------------------------------------------------------------- M <= 16
//
// The weight's stream: a workgroup of 8 waves takes 16 weight rows, wave w the
// w-th eighth of K in 128-element steps, multiplied on 16x16x64 int8 MFMA (the
// tokens as A, weight rows as B; token lanes past M hold zeros).  A load of the weight
// covers whole 128-byte lines, 8 lanes to each of 8 rows: the memory behind the
// caches is asked for full lines (22016 x 8192 from there: 64-byte pieces of
// 16 rows 55.6 us a call, full lines 50.8, and read past the caches'
// allocation, which a weight used once a token cannot profit from, 46).
// Lane permutes bring both loads' rows to fragment order.  The tokens, which stay in L2, come in quads
// of lanes on one row's 64 bytes.  NB steps are in flight while the NB before them are
// multiplied.  The waves' integer sums are added
// through LDS; the adapter's t B^T is added in float32 before the store.
constexpr int kFewWaves = 8;

template <int NB>
__global__ __launch_bounds__(512) void k_i8_few(TileArgs P, int block0) {
  typedef FewAdapter<16, 4096> Adapter;
  __shared__ __attribute__((aligned(16))) char ad_lds[Adapter::kBytes];
  __shared__ int red[kFewWaves][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n0 = (block0 + (int)blockIdx.x) * 16;
  const int M = (int)P.M;
  const int64_t K = P.K, N = P.N;
  // weight: load 2 s + i of a step, rows n0 + 8 i + lane / 8, bytes 16 (lane % 8) of the step's 128
  const int wr = lane >> 3, wc = lane & 7;
  const int8_t* wp[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    wp[i] = reinterpret_cast<const int8_t*>(P.w) + std::min<int64_t>(n0 + 8 * i + wr, N - 1) * K + 16 * wc;
  const int wsrc = (8 * (lane & 7) + (lane >> 4)) << 2;  // lane 16 g + n <- lane 8 (n % 8) + 4 half + g of load n / 8
  const bool low = (lane & 15) < 8;
  // tokens: quads, lane 16 g + n <- lane 4 n + g
  const int row = lane >> 2, g = lane & 3, xsrc = (4 * (lane & 15) + (lane >> 4)) << 2;
  const int8_t* xp = reinterpret_cast<const int8_t*>(P.x) + (int64_t)std::min(row, M - 1) * K + 16 * g;
  const int nst = (int)((K + 127) / 128);
  const int s0 = (int)((int64_t)nst * wave / kFewWaves), s1 = (int)((int64_t)nst * (wave + 1) / kFewWaves);
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  i32x4_t acc = {0, 0, 0, 0};
  struct Ld { u32x4_t w[NB][2], x[NB][2]; };
  auto load = [&](int b, Ld& d) {
#pragma unroll
    for (int s = 0; s < NB; ++s) {
      const int64_t k = (int64_t)(b + s) * 128;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        d.w[s][i] = b + s < s1 && k + 16 * wc < K ? __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(wp[i] + k)) : zero;
        const int64_t kx = k + 64 * i;
        d.x[s][i] = b + s < s1 && kx + 16 * g < K && row < M ? *reinterpret_cast<const u32x4_t*>(xp + kx) : zero;
      }
    }
  };
  auto compute = [&](const Ld& d) {
#pragma unroll
    for (int s = 0; s < NB; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // elements 64 i .. + 63 of the step
        i32x4_t xf, wf;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          xf[j] = __builtin_amdgcn_ds_bpermute(xsrc, (int)d.x[s][i][j]);
          const int w0 = __builtin_amdgcn_ds_bpermute(wsrc + 16 * i, (int)d.w[s][0][j]);
          const int w1 = __builtin_amdgcn_ds_bpermute(wsrc + 16 * i, (int)d.w[s][1][j]);
          wf[j] = low ? w0 : w1;
        }
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(xf, wf, acc, 0, 0, 0);
      }
  };
  Ld d0, d1;
  load(s0, d0);
  Adapter ad;
  ad.load(P.t, P.t_splits, M, 0, M, P.ab, n0, (int)std::min<int64_t>(16, N - n0), P.r);
  for (int b = s0; b < s1; b += 2 * NB) {
    load(b + NB, d1);
    compute(d0);
    if (b + NB >= s1) break;
    load(b + 2 * NB, d0);
    compute(d1);
  }
  // [token][weight row]: the lane's tokens 4 (lane / 16) + v of weight row lane % 16
#pragma unroll
  for (int v = 0; v < 4; ++v) red[wave][(4 * (lane >> 4) + v) * 16 + (lane & 15)] = acc[v];
  ad.stage(ad_lds, P.t_splits, M, P.r);
  __syncthreads();
  const int m = tid >> 4, c = tid & 15, n = n0 + c;
  if (m >= M || n >= N) return;
  int sum = 0;
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w) sum += red[w][tid];
  float y = (float)sum * P.sx[m] * P.sw[n];
  if (P.r > 0) y = fmaf(P.scale, ad.dot(ad_lds, P.t, P.t_splits, M, 0, m, P.ab, n0, c, P.r), y);
  if (P.ydt == DT_F32) reinterpret_cast<float*>(P.y)[m * N + n] = y;
  else reinterpret_cast<uint16_t*>(P.y)[m * N + n] = (uint16_t)f32_to_bf16_bits(y);
}

}  // namespace

hipError_t launch_quantize_i8(const void* X, int dt, int64_t rows, int64_t cols, int8_t* q, float* scale, hipStream_t s) {
  switch (dt) {
    case DT_F32: return launch_quantize_dt<DT_F32>(X, rows, cols, q, scale, s);
    case DT_F16: return launch_quantize_dt<DT_F16>(X, rows, cols, q, scale, s);
    default: return launch_quantize_dt<DT_BF16>(X, rows, cols, q, scale, s);
  }
}

hipError_t launch_i8_prep(const void* x, int64_t M, int64_t K, int8_t* q, float* scale, const void* A, int r, int splits,
                          float* t, hipStream_t s) {
  if (M < 1 || M > 16 || K % 64 != 0 || r < 1 || splits < 1) return hipErrorInvalidValue;
  const int jt = (r + 15) / 16;
  hipLaunchKernelGGL(k_i8_prep, dim3((unsigned)(M + (int64_t)jt * splits)), dim3(kLtWaves * 64), 0, s,
                     reinterpret_cast<const uint16_t*>(x), M, K, q, scale, reinterpret_cast<const uint16_t*>(A), r, jt, splits, t);
  return hipGetLastError();
}

hipError_t launch_i8_few(const TileArgs& a, hipStream_t s) {
  if (a.M < 1 || a.M > kFewRows || a.K % 16 != 0) return hipErrorInvalidValue;
  return launch_blocks((a.N + 15) / 16,
                       [&](unsigned n, int b0) { hipLaunchKernelGGL((k_i8_few<1>), dim3(n), dim3(512), 0, s, a, b0); });
}

hipError_t launch_i8_gemm(const TileArgs& a, hipStream_t s) {
  static const Levels none{};
  return launch_tile<TILE_I8, 4>(a, none, s);
}

}  // namespace qlr
