// Adapter products and gradients of a training step: under dropout masks formed on the way (qlr_philox.h), and of the gated
// block's backward, whose dg = dh up act'(gate) and dv = dh act(gate) are formed on the way too.
#include "qlr_grad_tile.h"

namespace qlr {

namespace {

__device__ __forceinline__ u32x4_t ld16g(const void* p) { return *reinterpret_cast<const u32x4_t*>(p); }

// Eight (dg, dv) from dh, g and v, as bf16 pieces: rounded to nearest (gn, vn), and as three parts (8 bits each, the third the whole
// rest: see split_rest) for the products whose results are float32.
struct Dgu {
  u32x4_t gn, vn, g[3], v[3];
};
template <int ACT, bool NEAREST, bool G, bool V>
__device__ __forceinline__ void form_dgu(u32x4_t dh, u32x4_t gate, u32x4_t up, Dgu& o) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float dg[2], dv[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float d = k ? __uint_as_float(dh[i] & 0xFFFF0000u) : __uint_as_float(dh[i] << 16);
      const float g = k ? __uint_as_float(gate[i] & 0xFFFF0000u) : __uint_as_float(gate[i] << 16);
      const float u = k ? __uint_as_float(up[i] & 0xFFFF0000u) : __uint_as_float(up[i] << 16);
      float slope = 0.0f;
      const float q = act_gate<ACT, G>(g, slope);
      dg[k] = d * u * slope;
      dv[k] = d * (g * q);
    }
    if constexpr (NEAREST) {
      o.gn[i] = pack_bf16x2(dg[0], dg[1]);
      o.vn[i] = pack_bf16x2(dv[0], dv[1]);
    }
    uint32_t p0, p1, p2;
    if constexpr (G) {
      three_parts(dg[0], dg[1], p0, p1, p2);
      o.g[0][i] = p0, o.g[1][i] = p1, o.g[2][i] = p2;
    }
    if constexpr (V) {
      three_parts(dv[0], dv[1], p0, p1, p2);
      o.v[0][i] = p0, o.v[1][i] = p1, o.v[2][i] = p2;
    }
  }
}

// ---------------------------------------------------------------- t = x A^T
//
// A workgroup of W waves takes 16 RT rows x 16 JT adapter columns of one product and one range of K; the waves split that range
// in 32-column steps and multiply on 16x16x32 bf16 MFMA (x rows as A, the adapter as B).  Loads give each quad of lanes one
// row's 64 bytes, whose 16-byte pieces are each one group of the mask; a slice of LDS of the wave's own brings them to the
// fragment layout (80-byte rows, free of bank conflicts).  An adapter given as K x r is staged row-major and read with the
// LDS transpose read.  One step's loads are in flight while the step before is multiplied; the waves' sums are added
// through LDS in wave order.
constexpr uint32_t kRowB = 80;  // bytes of a staged row of 32 columns
template <int JT>
constexpr uint32_t kBtRow = 32u * JT + 16u;  // bytes of a staged row of 16 JT adapter columns

struct TrainProds {
  TrainProd j[4];
  int64_t M;
  int splits;
  int block0;  // the launch's first row tile
  DropArgs drop;
};

// A launch of 2^32 threads or more runs the excess only (see launch_blocks): row tiles in launches of at most kLaunchBlocks workgroups.
template <typename F>
hipError_t launch_rows(int64_t tiles, int64_t others, F launch) {
  const int64_t per = std::max<int64_t>(1, kLaunchBlocks / others);
  for (int64_t b0 = 0; b0 < tiles; b0 += per) {
    launch((unsigned)std::min(per, tiles - b0), (int)b0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// A piece of 8 adapter columns of row k of a K x r adapter, zeros past r.
__device__ __forceinline__ u32x4_t ld_cols(const uint16_t* A, int64_t k, int r, int j, bool r8) {
  u32x4_t v = {0u, 0u, 0u, 0u};
  const uint16_t* p = A + k * r + j;
  if (r8) {
    if (j < r) v = ld16g(p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j + i < r) v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  }
  return v;
}

template <int RT, int JT, int W, bool BT>
__device__ __forceinline__ void prod_tile(const TrainProd& job, const TrainProds& J, int split, int64_t row0, int j0, char* lds) {
  constexpr uint32_t kA = BT ? 32u * kBtRow<JT> : 16u * JT * kRowB, kSlice = 16u * RT * kRowB + kA;
  const int64_t K = job.K, M = J.M;
  const int r = job.r, rows = (int)min<int64_t>(16 * RT, M - row0);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = lane >> 2, g = lane & 3;     // of the loads
  const int frow = lane & 15, fg = lane >> 4;  // of the fragments
  const bool r8 = (r & 7) == 0;
  const bool masked = job.mask >= 0 && J.drop.thr > 0;
  const uint64_t ctr = masked ? drop_counter(J.drop, job.mask) : 0;
  // (the workgroups of the first adapter columns leave the mask's bits for the kernels behind)
  uint8_t* const keep = masked && J.drop.bits && j0 == 0 ? J.drop.bits + (int64_t)job.mask * M * (K >> 3) : nullptr;
  const int64_t nst = (K + 31) / 32;
  const int64_t a0 = nst * split / J.splits, a1 = nst * (split + 1) / J.splits;
  const int64_t s0 = a0 + (a1 - a0) * wave / W, s1 = a0 + (a1 - a0) * (wave + 1) / W;
  const u32x4_t zero4 = {0u, 0u, 0u, 0u};
  int64_t xrow[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) xrow[i] = row0 + min(16 * i + row, rows - 1);
  struct Ld { u32x4_t x[RT], a[JT]; };
  // (rows past the range and adapter rows past r repeat the last one: their results are dropped)
  auto load = [&](int64_t st, Ld& d) {
    const int64_t k = 32 * st + 8 * g;
    const bool ok = st < s1 && k < K;
#pragma unroll
    for (int i = 0; i < RT; ++i) d.x[i] = ok ? ld16g(job.x + xrow[i] * K + k) : zero4;
#pragma unroll
    for (int c = 0; c < JT; ++c) {
      if constexpr (BT) {
        const int p = 64 * c + lane;
        const int64_t kr = 32 * st + p / (2 * JT);
        d.a[c] = st < s1 && kr < K ? ld_cols(job.A, kr, r, j0 + 8 * (p % (2 * JT)), r8) : zero4;
      } else {
        d.a[c] = ok ? ld16g(job.A + (int64_t)min(j0 + 16 * c + row, r - 1) * K + k) : zero4;
      }
    }
  };
  f32x4_t acc[RT][JT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int c = 0; c < JT; ++c) acc[i][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  char* const sl = lds + wave * kSlice;
  char* const sa = sl + 16 * RT * kRowB;
  auto compute = [&](int64_t st, const Ld& d) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      u32x4_t v = d.x[i];
      if (masked) {
        const int64_t group = xrow[i] * (K >> 3) + 4 * st + g;
        if (keep) {
          const uint32_t b = drop_bits((uint64_t)group, ctr, J.drop);
          if (16 * i + row < rows && 32 * st + 8 * g < K) keep[group] = (uint8_t)b;
          v &= bit_lanes(b);
        } else {
          v &= drop_lanes((uint64_t)group, ctr, J.drop);
        }
      }
      *reinterpret_cast<u32x4_t*>(sl + (16 * i + row) * kRowB + 16 * g) = v;
    }
#pragma unroll
    for (int c = 0; c < JT; ++c) {
      const int p = 64 * c + lane;
      if constexpr (BT) *reinterpret_cast<u32x4_t*>(sa + (p / (2 * JT)) * kBtRow<JT> + 16 * (p % (2 * JT))) = d.a[c];
      else *reinterpret_cast<u32x4_t*>(sa + (16 * c + row) * kRowB + 16 * g) = d.a[c];
    }
    bf16x8_t xf[RT], af[JT];
#pragma unroll
    for (int i = 0; i < RT; ++i) xf[i] = as_bf16x8(*reinterpret_cast<const u32x4_t*>(sl + (16 * i + frow) * kRowB + 16 * fg));
#pragma unroll
    for (int c = 0; c < JT; ++c) {
      if constexpr (BT) {
        const char* p = sa + (8u * fg + (frow >> 2)) * kBtRow<JT> + 32u * c + 8u * (frow & 3);
        af[c] = tr_frag(p, p + 4 * kBtRow<JT>);
      } else {
        af[c] = as_bf16x8(*reinterpret_cast<const u32x4_t*>(sa + (16 * c + frow) * kRowB + 16 * fg));
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < JT; ++c) acc[i][c] = mfma16x16x32(xf[i], af[c], acc[i][c]);
  };
  Ld d0, d1;
  load(s0, d0);
  for (int64_t st = s0; st < s1; st += 2) {
    load(st + 1, d1);
    compute(st, d0);
    if (st + 1 >= s1) break;
    load(st + 2, d0);
    compute(st + 1, d1);
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
    job.t[((int64_t)split * M + row0 + m) * job.ldt + job.col0 + j] = sum;
  }
}

// blockIdx: row tile, group of 16 JT adapter columns, product and split
template <int RT, int JT, int W>
__global__ __launch_bounds__(64 * W) void k_train_t(TrainProds J) {
  constexpr uint32_t kA = 16u * JT * kRowB, kB = 32u * kBtRow<JT>;
  constexpr uint32_t kSlice = 16 * RT * kRowB + (kA > kB ? kA : kB), kSum = RT * 16 * JT * 16 * 4;
  __shared__ __attribute__((aligned(16))) char lds[W * (kSlice > kSum ? kSlice : kSum)];
  const int ji = (int)blockIdx.z / J.splits, split = (int)blockIdx.z % J.splits;
  const int64_t row0 = (int64_t)(J.block0 + (int)blockIdx.x) * 16 * RT;
  const TrainProd& job = J.j[ji];
  if (job.bt) prod_tile<RT, JT, W, true>(job, J, split, row0, blockIdx.y * 16 * JT, lds);
  else prod_tile<RT, JT, W, false>(job, J, split, row0, blockIdx.y * 16 * JT, lds);
}

template <int RT, int JT, int W>
hipError_t launch_t(TrainProds J, int n, int r, hipStream_t s) {
  const unsigned cols = (unsigned)((r + 16 * JT - 1) / (16 * JT)), each = (unsigned)(n * J.splits);
  return launch_rows((J.M + 16 * RT - 1) / (16 * RT), (int64_t)cols * each, [&](unsigned tiles, int b0) {
    J.block0 = b0;
    hipLaunchKernelGGL((k_train_t<RT, JT, W>), dim3(tiles, cols, each), dim3(64 * W), 0, s, J);
  });
}

constexpr int kMaxSplits = 8;
// Ranges of the contraction so that about `target` workgroups run, each wave with two steps at least.
int range_splits(int64_t wgs, int64_t steps, int waves, int target = 512) {
  const int64_t want = (target + wgs - 1) / wgs, most = steps / (2 * waves);
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, most), kMaxSplits));
}

// ---------------------------------------------------------------- dgu and u = [dg Bg | dv Bu]
//
// As the product above with dg and dv formed between the loads and the fragments; both products of a row tile run in one
// workgroup, so that dh, g and v are read once.  The workgroups of the first 16 JT adapter columns write dgu.
// JT = 0: dgu alone.
struct GatedU {
  const uint16_t *dh, *gu, *B;
  uint16_t* dgu;
  float* u;
  int64_t M, N;
  int r, splits;
  int block0;  // the launch's first row tile
};

template <int ACT, int RT, int JT, int W>
__global__ __launch_bounds__(64 * W) void k_gated_u(GatedU G) {
  constexpr uint32_t kXs = 16u * RT * kRowB, kBs = 32u * kBtRow<JT>, kSlice = JT ? 6u * kXs + 2u * kBs : 16u;
  constexpr uint32_t kSum = RT * 16 * JT * 16 * 4 * 2;
  __shared__ __attribute__((aligned(16))) char lds[W * (kSlice > kSum ? kSlice : kSum)];
  const int64_t N = G.N, M = G.M, row0 = (int64_t)(G.block0 + (int)blockIdx.x) * 16 * RT;
  const int r = G.r, rows = (int)min<int64_t>(16 * RT, M - row0), j0 = blockIdx.y * 16 * JT, split = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = lane >> 2, g = lane & 3, frow = lane & 15, fg = lane >> 4;
  const bool r8 = (r & 7) == 0, first = blockIdx.y == 0;
  const int64_t nst = (N + 31) / 32;
  const int64_t a0 = nst * split / G.splits, a1 = nst * (split + 1) / G.splits;
  const int64_t s0 = a0 + (a1 - a0) * wave / W, s1 = a0 + (a1 - a0) * (wave + 1) / W;
  const u32x4_t zero4 = {0u, 0u, 0u, 0u};
  int64_t xrow[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) xrow[i] = row0 + min(16 * i + row, rows - 1);
  constexpr int JA = JT ? JT : 1;
  struct Ld { u32x4_t dh[RT], g[RT], v[RT], b[2][JA]; };
  auto load = [&](int64_t st, Ld& d) {
    const int64_t k = 32 * st + 8 * g;
    const bool ok = st < s1 && k < N;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      d.dh[i] = ok ? ld16g(G.dh + xrow[i] * N + k) : zero4;
      d.g[i] = ok ? ld16g(G.gu + xrow[i] * 2 * N + k) : zero4;
      d.v[i] = ok ? ld16g(G.gu + xrow[i] * 2 * N + N + k) : zero4;
    }
    if constexpr (JT > 0) {
#pragma unroll
      for (int c = 0; c < JT; ++c) {
        const int p = 64 * c + lane;
        const int64_t kr = 32 * st + p / (2 * JA);
#pragma unroll
        for (int sd = 0; sd < 2; ++sd)
          d.b[sd][c] = st < s1 && kr < N ? ld_cols(G.B, sd * N + kr, r, j0 + 8 * (p % (2 * JA)), r8) : zero4;
      }
    }
  };
  f32x4_t acc[2][RT][JA];
#pragma unroll
  for (int sd = 0; sd < 2; ++sd)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < JA; ++c) acc[sd][i][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  char* const sl = lds + wave * kSlice;
  char* const sb = sl + 6 * kXs;
  auto compute = [&](int64_t st, const Ld& d) {
    const int64_t k = 32 * st + 8 * g;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      Dgu o;
      form_dgu<ACT, true, true, true>(d.dh[i], d.g[i], d.v[i], o);
      if (first && k < N && 16 * i + row < rows) {
        *reinterpret_cast<u32x4_t*>(G.dgu + xrow[i] * 2 * N + k) = o.gn;
        *reinterpret_cast<u32x4_t*>(G.dgu + xrow[i] * 2 * N + N + k) = o.vn;
      }
      if constexpr (JT > 0) {
        char* const p = sl + (16 * i + row) * kRowB + 16 * g;
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          *reinterpret_cast<u32x4_t*>(p + q * kXs) = o.g[q];
          *reinterpret_cast<u32x4_t*>(p + (3 + q) * kXs) = o.v[q];
        }
      }
    }
    if constexpr (JT > 0) {
#pragma unroll
      for (int c = 0; c < JT; ++c) {
        const int p = 64 * c + lane;
#pragma unroll
        for (int sd = 0; sd < 2; ++sd)
          *reinterpret_cast<u32x4_t*>(sb + sd * kBs + (p / (2 * JA)) * kBtRow<JT> + 16 * (p % (2 * JA))) = d.b[sd][c];
      }
#pragma unroll
      for (int sd = 0; sd < 2; ++sd) {
        bf16x8_t xf[RT][3], bf[JA];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int q = 0; q < 3; ++q)
            xf[i][q] = as_bf16x8(*reinterpret_cast<const u32x4_t*>(sl + (3 * sd + q) * kXs + (16 * i + frow) * kRowB + 16 * fg));
#pragma unroll
        for (int c = 0; c < JT; ++c) {
          const char* p = sb + sd * kBs + (8u * fg + (frow >> 2)) * kBtRow<JT> + 32u * c + 8u * (frow & 3);
          bf[c] = tr_frag(p, p + 4 * kBtRow<JT>);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int c = 0; c < JT; ++c)
#pragma unroll
            for (int q = 2; q >= 0; --q) acc[sd][i][c] = mfma16x16x32(xf[i][q], bf[c], acc[sd][i][c]);
      }
    }
  };
  Ld d0, d1;
  load(s0, d0);
  for (int64_t st = s0; st < s1; st += 2) {
    load(st + 1, d1);
    compute(st, d0);
    if (st + 1 >= s1) break;
    load(st + 2, d0);
    compute(st + 1, d1);
  }
  if constexpr (JT > 0) {
    __syncthreads();
    // [wave][side][row][column]
    float* red = reinterpret_cast<float*>(lds);
    constexpr int kOne = RT * 16 * JT * 16;
#pragma unroll
    for (int sd = 0; sd < 2; ++sd)
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < JT; ++c)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            red[(2 * wave + sd) * kOne + (16 * i + 4 * fg + v) * (16 * JT) + 16 * c + frow] = acc[sd][i][c][v];
    __syncthreads();
    for (int idx = tid; idx < 2 * rows * 16 * JT; idx += 64 * W) {
      const int sd = idx / (rows * 16 * JT), at = idx % (rows * 16 * JT), m = at / (16 * JA), j = j0 + at % (16 * JA);
      if (j >= r) continue;
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) sum += red[(2 * w + sd) * kOne + at];
      G.u[((int64_t)split * M + row0 + m) * 2 * r + sd * r + j] = sum;
    }
  }
}

template <int ACT, int RT, int JT, int W>
hipError_t launch_u(GatedU G, hipStream_t s) {
  const unsigned cols = JT ? (unsigned)((G.r + 16 * JT - 1) / (16 * (JT ? JT : 1))) : 1u, each = (unsigned)G.splits;
  return launch_rows((G.M + 16 * RT - 1) / (16 * RT), (int64_t)cols * each, [&](unsigned tiles, int b0) {
    G.block0 = b0;
    hipLaunchKernelGGL((k_gated_u<ACT, RT, JT, W>), dim3(tiles, cols, each), dim3(64 * W), 0, s, G);
  });
}
// More than 16 adapter columns: a workgroup of 8 waves takes 64 rows x 64 columns of both sides, 64 columns of dh a step; wave w
// takes rows 16 (w % 4) .. and half w / 4 of the step.  B's rows are staged once for the workgroup and read with the transpose
// read; dh, g and v are loaded in the fragments' layout (16 bytes of each of 16 rows a quarter wave) and their parts stay in
// registers.  The kernel above with four times the columns holds both sides' B per wave: 256 registers, one wave a SIMD, 103 us at
// 2048 x 11008, r = 64, where this one takes 77 (the arrays' 225 MB: 44).
template <int ACT>
__global__ __launch_bounds__(512, 2) void k_gated_u_wide(GatedU G) {
  constexpr uint32_t kRow = kBtRow<4>, kSide = 64u * kRow, kBuf = 2u * kSide;
  __shared__ __attribute__((aligned(16))) char lds[2 * kBuf];
  static_assert(2 * kBuf >= 4 * 32 * 64 * 4, "the second half's sums overlay the buffers");
  const int64_t N = G.N, M = G.M, row0 = (int64_t)(G.block0 + (int)blockIdx.x) * 64;
  const int r = G.r, j0 = blockIdx.y * 64, split = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave & 3, ws = wave >> 2, frow = lane & 15, fg = lane >> 4;
  const bool r8 = (r & 7) == 0, first = blockIdx.y == 0;
  const int64_t nst = (N + 63) / 64;
  const int64_t a0 = nst * split / G.splits, a1 = nst * (split + 1) / G.splits;
  const u32x4_t zero4 = {0u, 0u, 0u, 0u};
  const int64_t row = min<int64_t>(row0 + 16 * wr + frow, M - 1);
  const bool live = row0 + 16 * wr + frow < M;
  struct Ld { u32x4_t dh, g, v, b[2]; };
  auto load = [&](int64_t st, Ld& d) {
    const int64_t k = 64 * st + 32 * ws + 8 * fg, n = 64 * st + (tid >> 3);
    const bool ok = st < a1 && k < N;
    d.dh = ok ? ld16g(G.dh + row * N + k) : zero4;
    d.g = ok ? ld16g(G.gu + row * 2 * N + k) : zero4;
    d.v = ok ? ld16g(G.gu + row * 2 * N + N + k) : zero4;
#pragma unroll
    for (int sd = 0; sd < 2; ++sd) d.b[sd] = st < a1 && n < N ? ld_cols(G.B, sd * N + n, r, j0 + 8 * (tid & 7), r8) : zero4;
  };
  f32x4_t acc[2][4];
#pragma unroll
  for (int sd = 0; sd < 2; ++sd)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[sd][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](int64_t st, const Ld& d, char* buf) {
#pragma unroll
    for (int sd = 0; sd < 2; ++sd) *reinterpret_cast<u32x4_t*>(buf + sd * kSide + (tid >> 3) * kRow + 16 * (tid & 7)) = d.b[sd];
    Dgu o;
    form_dgu<ACT, true, true, true>(d.dh, d.g, d.v, o);
    const int64_t k = 64 * st + 32 * ws + 8 * fg;
    if (first && live && k < N) {
      *reinterpret_cast<u32x4_t*>(G.dgu + row * 2 * N + k) = o.gn;
      *reinterpret_cast<u32x4_t*>(G.dgu + row * 2 * N + N + k) = o.vn;
    }
    __syncthreads();
    const char* const p = buf + (32u * ws + 8u * fg + (frow >> 2)) * kRow + 8u * (frow & 3);
#pragma unroll
    for (int sd = 0; sd < 2; ++sd)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bf16x8_t b = tr_frag(p + sd * kSide + 32 * c, p + sd * kSide + 32 * c + 4 * kRow);
#pragma unroll
        for (int q = 2; q >= 0; --q) acc[sd][c] = mfma16x16x32(as_bf16x8(sd ? o.v[q] : o.g[q]), b, acc[sd][c]);
      }
  };
  // (a buffer is written again two steps later, behind the barrier that every wave passes past its reads)
  Ld d0, d1;
  load(a0, d0);
  for (int64_t st = a0; st < a1; st += 2) {
    load(st + 1, d1);
    compute(st, d0, lds);
    if (st + 1 >= a1) break;
    load(st + 2, d0);
    compute(st + 1, d1, lds + kBuf);
  }
  __syncthreads();
  f32x4_t* const red = reinterpret_cast<f32x4_t*>(lds) + wr * 8 * 64 + lane;
  if (ws == 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) red[i * 64] = acc[i >> 2][i & 3];
  __syncthreads();
  if (ws == 1) return;
#pragma unroll
  for (int sd = 0; sd < 2; ++sd)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const f32x4_t other = red[(4 * sd + c) * 64];
      const int j = j0 + 16 * c + frow;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t m = row0 + 16 * wr + 4 * fg + v;
        if (m < M && j < r) G.u[((int64_t)split * M + m) * 2 * r + sd * r + j] = acc[sd][c][v] + other[v];
      }
    }
}

// rows of a workgroup, as gated_u_splits counts them
int u_rows(int64_t M, int r) { return r > 16 ? 64 : M >= 512 ? 32 : 16; }
template <int ACT>
hipError_t launch_u_act(GatedU G, hipStream_t s) {
  if (G.r > 16) {
    const unsigned cols = (unsigned)((G.r + 63) / 64), each = (unsigned)G.splits;
    return launch_rows((G.M + 63) / 64, (int64_t)cols * each, [&](unsigned tiles, int b0) {
      G.block0 = b0;
      hipLaunchKernelGGL(k_gated_u_wide<ACT>, dim3(tiles, cols, each), dim3(512), 0, s, G);
    });
  }
  const bool two = u_rows(G.M, G.r) == 32;
  if (!G.u) return two ? launch_u<ACT, 2, 0, 4>(G, s) : launch_u<ACT, 1, 0, 4>(G, s);
  return two ? launch_u<ACT, 2, 1, 4>(G, s) : launch_u<ACT, 1, 1, 4>(G, s);
}

// ---------------------------------------------------------------- adapter gradients
//
// out[j][c] = s sum_m P[m][j] Q[m][c], computed as out^T[c][j] on 16x16x32 bf16 MFMA: Q^T as the A operand and P^T as B, both
// read from row-major LDS tiles with the transpose read.  P (float32) enters as three bf16 parts (24 bits); Q is bf16, under
// its mask where it has one, or dg or dv formed from dh, g and v, in three parts too (the three smallest products of parts, 2^-24 and
// less, are left out).  A workgroup of 4 waves takes 128 columns x 64 adapter rows x one chunk of rows, 32 rows per step in one of two
// LDS buffers, the next two steps' loads in registers.  The first chunk goes to the output itself, the others to float32 partials
// in the outputs' order that a second kernel adds in chunk order: results do not depend on timing.
//
// Chunk: as many as give about 256 workgroups, of at most 512 rows.
int64_t grad_chunk(int64_t M, int64_t CC) {
  const int64_t tiles = (CC + 127) / 128, chunks = std::max<int64_t>(1, (256 + tiles - 1) / tiles);
  return std::max<int64_t>(64, std::min<int64_t>(512, ((M + chunks - 1) / chunks + 31) / 32 * 32));
}

struct TrainGrads {
  TrainGrad j[4];
  int64_t at[4];  // first column of the job's part among the columns of all
  int tile0[5];   // first column tile of each job
  const uint16_t* gu;
  int64_t M, N, CC;
  int n, r, block0, chunk;
  float scale;
  DropArgs drop;
  float* part;    // extra chunks x (the jobs' outputs)
};

// SRC 0: Q as it is or masked; 1: dg; 2: dv
template <int SRC, int ACT>
__device__ __forceinline__ void grad_tile(const TrainGrads& G, const TrainGrad& job, int ji, int64_t mb, int chunk, int cb, int j0,
                                          char* lds) {
  constexpr int QP = SRC == 0 ? 1 : 3;  // parts of Q
  constexpr uint32_t kBuf = QP * kQ + 3 * kP;
  const int r = G.r;
  const int64_t C = job.C, M = G.M;
  const int rows = (int)min<int64_t>(G.chunk, M - mb);
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int jt = min(4, (r - j0 + 15) / 16);
  const bool r4 = (r & 3) == 0;
  const bool masked = SRC == 0 && job.mask >= 0 && G.drop.thr > 0;
  const uint8_t* const keep = masked ? G.drop.bits + ((int64_t)job.mask * M + mb) * (C >> 3) : nullptr;
  const __amdgpu_buffer_rsrc_t qr = tile_rsrc(job.Q + mb * C, (uint32_t)(rows * C * 2));
  const __amdgpu_buffer_rsrc_t gr = tile_rsrc(SRC ? G.gu + mb * 2 * C : nullptr, SRC ? (uint32_t)(rows * C * 4) : 0u);
  const uint32_t qrow = (uint32_t)tid >> 4, qch = (uint32_t)tid & 15u;
  const int64_t qcol = min<int64_t>(cb + 8 * qch, C - 8);  // clamped: outputs past C are dropped
  struct Stage { u32x4_t q[2], g[2], v[2]; f32x4_t p[2]; uint32_t keep[2]; };
  auto ld = [](__amdgpu_buffer_rsrc_t rs, int64_t elem) {
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, (uint32_t)(elem * 2), 0, 0));
  };
  auto load = [&](int m0, Stage& s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t row = m0 + (int)qrow + 16 * i;  // rows past the chunk read zero
      s.q[i] = ld(qr, row * C + qcol);
      if constexpr (SRC > 0) s.g[i] = ld(gr, row * 2 * C + qcol);
      if constexpr (SRC == 1) s.v[i] = ld(gr, row * 2 * C + C + qcol);
      if constexpr (SRC == 0) s.keep[i] = masked && row < rows ? keep[row * (C >> 3) + (qcol >> 3)] : 255u;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = m0 + (int)qrow + 16 * i, jb = j0 + 4 * (int)qch;
      f32x4_t v = {0.f, 0.f, 0.f, 0.f};
      if (m < rows && jb < r) {
#pragma unroll 4
        for (int sp = 0; sp < job.p_splits; ++sp) {
          const float* p = job.P + ((int64_t)sp * M + mb + m) * job.ldp + job.col0 + jb;
          if (r4) {
            const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p);
#pragma unroll
            for (int t = 0; t < 4; ++t) v[t] += a[t];
          } else {
#pragma unroll
            for (int t = 0; t < 4; ++t)
              if (jb + t < r) v[t] += p[t];
          }
        }
      }
      s.p[i] = v;
    }
  };
  auto store = [&](int m0, const Stage& s, char* buf) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t row = qrow + 16u * i;
      char* const at = buf + q_off(row, qch);
      if constexpr (SRC == 0) {
        u32x4_t q = s.q[i];
        if (masked) q &= bit_lanes(s.keep[i]);
        *reinterpret_cast<u32x4_t*>(at) = q;
      } else {
        Dgu o;
        form_dgu<ACT, false, SRC == 1, SRC == 2>(s.q[i], s.g[i], SRC == 1 ? s.v[i] : s.g[i], o);
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<u32x4_t*>(at + k * kQ) = SRC == 1 ? o.g[k] : o.v[k];
      }
      uint32_t part[3][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) three_parts(s.p[i][2 * t], s.p[i][2 * t + 1], part[0][t], part[1][t], part[2][t]);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        *reinterpret_cast<uint2*>(buf + QP * kQ + k * kP + p_off(row, qch >> 1) + 8u * (qch & 1u)) = uint2{part[k][0], part[k][1]};
    }
  };
  // transpose-read addresses: lane group g takes rows 8 g .. 8 g + 7 (two reads), lane sp the four elements from column
  // 4 (sp % 4) of row sp / 4
  const uint32_t g = (uint32_t)lane >> 4, sp = (uint32_t)lane & 15u;
  uint32_t qa[2][2], pa[4][2];
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    const uint32_t row = 8u * g + 4u * hf + (sp >> 2);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t col = 32u * w + 16u * c + 4u * (sp & 3u);
      qa[c][hf] = q_off(row, col >> 3) + 2u * (col & 7u);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t col = 16u * t + 4u * (sp & 3u);
      pa[t][hf] = QP * kQ + p_off(row, col >> 3) + 2u * (col & 7u);
    }
  }
  f32x4_t acc[2][4];
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[c][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  Stage s0, s1;
  load(0, s0);
  load(32, s1);
  auto step = [&](int m0, Stage& s, char* buf) {
    store(m0, s, buf);
    load(m0 + 64, s);
    __syncthreads();
    bf16x8_t q[QP][2];
#pragma unroll
    for (int k = 0; k < QP; ++k)
#pragma unroll
      for (int c = 0; c < 2; ++c) q[k][c] = tr_frag(buf + k * kQ + qa[c][0], buf + k * kQ + qa[c][1]);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t >= jt) break;
#pragma unroll
      for (int k = 2; k >= 0; --k) {  // smallest parts first
        const bf16x8_t p = tr_frag(buf + k * kP + pa[t][0], buf + k * kP + pa[t][1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int l = QP - 1; l >= 0; --l)
            if (k + l < 3) acc[c][t] = mfma16x16x32(q[l][c], p, acc[c][t]);
        }
      }
    }
  };
  // buffer i is written again two steps later, after the barrier that every wave passes past its reads
  for (int m0 = 0; m0 < rows; m0 += 64) {
    step(m0, s0, lds);
    if (m0 + 32 < rows) step(m0 + 32, s1, lds + kBuf);
  }
  // D[c][j]: lane holds columns 4 g .. + 3 of adapter row sp
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int j = j0 + 16 * t + (int)sp;
    if (t >= jt || j >= r) continue;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int64_t c0 = cb + 32 * w + 16 * c + 4 * (int64_t)g;
      if (c0 >= C) continue;  // C % 4 == 0: whole pieces
      const f32x4_t v = acc[c][t];
      float* const out = chunk > 0 ? G.part + ((int64_t)(chunk - 1) * G.CC + G.at[ji]) * r : job.out;
      const float f = chunk > 0 ? 1.0f : G.scale;
      if (!job.cols_major) {
        *reinterpret_cast<f32x4_t*>(out + (int64_t)j * C + c0) = f32x4_t{f * v[0], f * v[1], f * v[2], f * v[3]};
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) out[(c0 + i) * r + j] = f * v[i];
      }
    }
  }
}

// ACT < 0: no job forms dg or dv
template <int ACT>
__global__ __launch_bounds__(256) void k_train_grad(TrainGrads G) {
  __shared__ __attribute__((aligned(16))) char lds[2 * ((ACT < 0 ? 1 : 3) * kQ + 3 * kP)];
  const int ct = G.tile0[G.n];
  const int block = G.block0 + (int)blockIdx.x, chunk = block / ct, bx = block % ct;
  int ji = 0;
  while (ji + 1 < G.n && bx >= G.tile0[ji + 1]) ++ji;
  const TrainGrad& job = G.j[ji];
  const int64_t mb = (int64_t)chunk * G.chunk;
  const int cb = (bx - G.tile0[ji]) * 128, j0 = blockIdx.y * 64;
  if constexpr (ACT >= 0) {
    if (job.kind == 1) return grad_tile<1, ACT>(G, job, ji, mb, chunk, cb, j0, lds);
    if (job.kind == 2) return grad_tile<2, ACT>(G, job, ji, mb, chunk, cb, j0, lds);
  }
  grad_tile<0, ACT>(G, job, ji, mb, chunk, cb, j0, lds);
}

// out += scale * (the further chunks, in order)
__global__ __launch_bounds__(256) void k_train_grad_add(TrainGrads G, int chunks) {
  const int64_t n = G.CC * G.r / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int c = 0; c < chunks; ++c) {
      const f32x4_t p = reinterpret_cast<const f32x4_t*>(G.part)[(int64_t)c * n + i];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += p[k];
    }
    int ji = 0;
    while (ji + 1 < G.n && 4 * i >= G.at[ji + 1] * G.r) ++ji;
    f32x4_t* const o = reinterpret_cast<f32x4_t*>(G.j[ji].out + 4 * i - G.at[ji] * G.r);
    f32x4_t w = *o;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] += G.scale * v[k];
    *o = w;
  }
}

struct TrainSums {
  TrainSum j[2];
};
__global__ __launch_bounds__(256) void k_train_sum(TrainSums S, int64_t M) {
  const TrainSum& job = S.j[blockIdx.y];
  const int64_t n = M * job.ld;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * 1024) {
    if (n % 4 == 0) {
      f32x4_t v = *reinterpret_cast<const f32x4_t*>(job.t + i);
#pragma unroll 4
      for (int c = 1; c < job.splits; ++c) {
        const f32x4_t p = *reinterpret_cast<const f32x4_t*>(job.t + c * n + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] += p[k];
      }
      *reinterpret_cast<f32x4_t*>(job.t + i) = v;
    } else {
      for (int k = 0; k < 4 && i + k < n; ++k) {
        float v = job.t[i + k];
        for (int c = 1; c < job.splits; ++c) v += job.t[c * n + i + k];
        job.t[i + k] = v;
      }
    }
  }
}

}  // namespace

int train_t_splits(int64_t M, int64_t K, int r, int jobs) {
  if (M <= 0 || r <= 0) return 1;
  // (one product's sums are added by every tile of the kernel behind: half as many)
  return range_splits((M + 15) / 16 * jobs * ((r + 63) / 64), (K + 31) / 32, 8, jobs > 1 ? 1024 : 512);
}

hipError_t launch_train_t(const TrainProd* jobs, int n, int64_t M, int splits, const DropArgs& drop, hipStream_t s) {
  if (M == 0 || n == 0 || jobs[0].r == 0) return hipSuccess;
  if (n > 4) return hipErrorInvalidValue;
  TrainProds J{};
  for (int i = 0; i < n; ++i) {
    if (jobs[i].r != jobs[0].r || jobs[i].K % 8 != 0) return hipErrorInvalidValue;
    J.j[i] = jobs[i];
  }
  J.M = M;
  J.splits = splits;
  J.drop = drop;
  const int r = jobs[0].r;
  const bool two = M >= 512;
  if (r <= 16) return two ? launch_t<2, 1, 8>(J, n, r, s) : launch_t<1, 1, 8>(J, n, r, s);
  // (32 rows: 2048 x 11008 under a mask and x 4096, r = 64: 36 us, four waves and 512 workgroups 57, 16 rows 42)
  return two ? launch_t<2, 4, 8>(J, n, r, s) : launch_t<1, 4, 8>(J, n, r, s);
}

int gated_u_splits(int64_t M, int64_t N, int r) {
  if (M <= 0) return 1;
  const int rows = u_rows(M, r);
  if (rows == 64) return range_splits((M + 63) / 64 * ((r + 63) / 64), (N + 63) / 64, 1);
  return range_splits((M + rows - 1) / rows, (N + 31) / 32, 4);
}

hipError_t launch_gated_u(const uint16_t* dh, const uint16_t* gu, int act, int64_t M, int64_t N, const uint16_t* B, int r,
                          uint16_t* dgu, float* u, int splits, hipStream_t s) {
  if (M == 0) return hipSuccess;
  if (N % 8 != 0) return hipErrorInvalidValue;
  const GatedU G{dh, gu, B, dgu, u, M, N, r, splits, 0};
  switch (act) {
    case ACT_SILU: return launch_u_act<ACT_SILU>(G, s);
    case ACT_GELU: return launch_u_act<ACT_GELU>(G, s);
    default: return launch_u_act<ACT_GELU_TANH>(G, s);
  }
}

hipError_t launch_train_sum(const TrainSum* jobs, int n, int64_t M, hipStream_t s) {
  TrainSums S{};
  int live = 0, ld = 0;
  for (int i = 0; i < n; ++i) {
    if (jobs[i].splits < 2 || live == 2) continue;
    S.j[live++] = jobs[i];
    ld = std::max(ld, jobs[i].ld);
  }
  if (live == 0 || M == 0) return hipSuccess;
  hipLaunchKernelGGL(k_train_sum, dim3((unsigned)std::min<int64_t>((M * ld + 1023) / 1024, 2048), (unsigned)live), dim3(256), 0, s, S, M);
  return hipGetLastError();
}

size_t train_grad_floats(int64_t M, int64_t C_total, int r) {
  return M > 0 ? (size_t)((M - 1) / grad_chunk(M, C_total)) * (size_t)r * (size_t)C_total : 0;
}

hipError_t launch_train_grads(const TrainGrad* jobs, int n, int64_t M, int r, const uint16_t* gu, int64_t N, int act, float scale,
                              const DropArgs& drop, float* part, hipStream_t s) {
  if (r == 0 || n == 0) return hipSuccess;
  if (n > 4) return hipErrorInvalidValue;
  TrainGrads G{};
  bool gated = false;
  for (int i = 0; i < n; ++i) {
    if (jobs[i].C % 8 != 0) return hipErrorInvalidValue;
    G.j[i] = jobs[i];
    G.at[i] = G.CC;
    G.CC += jobs[i].C;
    G.tile0[i + 1] = G.tile0[i] + (int)((jobs[i].C + 127) / 128);
    gated = gated || jobs[i].kind != 0;
  }
  G.gu = gu;
  G.M = M;
  G.N = N;
  G.n = n;
  G.r = r;
  G.scale = scale;
  G.drop = drop;
  G.part = part;
  G.chunk = (int)grad_chunk(M, G.CC);
  const int64_t chunks = std::max<int64_t>(1, (M + G.chunk - 1) / G.chunk), wgs = chunks * G.tile0[n];
  if (wgs > INT_MAX) return hipErrorInvalidValue;
  const int64_t jt = (r + 63) / 64;
  const hipError_t e = launch_rows(wgs, jt, [&](unsigned blocks, int b0) {
    const dim3 grid(blocks, (unsigned)jt);
    G.block0 = b0;
    if (!gated) hipLaunchKernelGGL(k_train_grad<-1>, grid, dim3(256), 0, s, G);
    else if (act == ACT_SILU) hipLaunchKernelGGL(k_train_grad<ACT_SILU>, grid, dim3(256), 0, s, G);
    else if (act == ACT_GELU) hipLaunchKernelGGL(k_train_grad<ACT_GELU>, grid, dim3(256), 0, s, G);
    else hipLaunchKernelGGL(k_train_grad<ACT_GELU_TANH>, grid, dim3(256), 0, s, G);
  });
  if (e != hipSuccess || chunks == 1) return e;
  hipLaunchKernelGGL(k_train_grad_add, dim3((unsigned)std::min<int64_t>((G.CC * r + 1023) / 1024, 2048)), dim3(256), 0, s, G,
                     (int)(chunks - 1));
  return hipGetLastError();
}

}  // namespace qlr
