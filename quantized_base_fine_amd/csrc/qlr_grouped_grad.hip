// Adapter gradients of the expert products: with e's rows R_e,
//     dA_e = s u_e^T x_e   (r x K),   dB_e = s dy_e^T t_e   (N x r),
// u = dy B_e and t = x A_e^T in float32.
#include "qlr_tile.h"

namespace qlr {

namespace {

// Both are out[j][c] = s sum_m P[m][j] Q[m][c] with (P, Q, C) = (u, x, K) and
// (t, dy, N), computed as out^T[c][j] on 16x16x32 bf16 MFMA: Q^T as the A
// operand and P^T as B, both read from row-major LDS tiles with the transpose
// read.  P enters as three bf16 parts (hi, mid, lo: 24 significant bits, see split_rest), so the
// products are those of float32 P; the extra products are cheap beside the reads
// of Q, which bound the kernel.
//
// A workgroup of 4 waves takes 128 columns x 64 adapter rows x up to
// kGradChunk rows of one expert, 32 rows per step: 32 x 128 of Q and 32 x 64 of
// P in one of two LDS buffers, the next two steps' loads in registers.  An
// expert's first chunk goes to the output itself (zeros for an expert without
// rows); the chunks of longer experts go to float32 partials that a second
// kernel adds in chunk order, so results do not depend on timing.
// 4096 rows in 8 ranges of 4096 x 4096, r = 16: 15 us for the 67 MB of x and dy (4.5 TB/s; a device copy moves 5.1)
// and 5.5 us for the sums of 6 longer ranges' chunks.
constexpr int kGradChunk = 512;
constexpr uint32_t kGQ = 32 * 256, kGP = 32 * 128, kGBuf = kGQ + 3 * kGP;

struct GroupGrads {
  const float* P[2];
  const uint16_t* Q[2];
  float* out[2];
  int64_t C[2];
  int ct0, ct;  // column tiles of job 0 and of both
  int extra;    // slots of extra chunks in part
  int block0;   // the launch's first workgroup among the call's
  int64_t M;
  int r, experts;
  const int32_t* offsets;
  float scale;
  float* part;  // extra chunks x r x (C[0] + C[1])
};

// Extra chunks (beyond the first) of an expert's rows.
__device__ __forceinline__ int extra_chunks(int rows) { return rows > kGradChunk ? (rows - 1) / kGradChunk : 0; }

// Extra chunks of the experts before e (want < 0), or the expert that holds
// extra chunk `want` (returned in e, -1 if there is none) and its number among
// that expert's chunks (1 ..).  Called by whole waves.
__device__ __forceinline__ int extra_scan(const int32_t* offsets, int E, int M, int want, int& e) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    int a = 0, b = 0;
    if (e0 + lane < E) expert_range(offsets, e0 + lane, M, a, b);
    const int nx = extra_chunks(b - a);
    int inc = nx;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(inc, d, 64);
      if (lane >= d) inc += up;
    }
    if (want < 0) {
      if (e < e0 + 64) return before + __shfl(inc - nx, e - e0, 64);
    } else if (want < before + __shfl(inc, 63, 64)) {
      const int src = __ffsll((unsigned long long)__ballot(before + inc > want)) - 1;
      e = e0 + src;
      return want - (before + __shfl(inc - nx, src, 64)) + 1;
    }
    before += __shfl(inc, 63, 64);
  }
  e = -1;
  return before;
}

__device__ __forceinline__ uint32_t gq_off(uint32_t row, uint32_t chunk) {
  const uint32_t h = (row & 3u) | (((row >> 3) & 1u) << 2);
  return row * 256u + ((chunk ^ (h << 1)) << 4);
}
__device__ __forceinline__ uint32_t gp_off(uint32_t row, uint32_t chunk) {
  const uint32_t h = ((row >> 1) & 1u) | (((row >> 3) & 1u) << 1);
  return row * 128u + ((chunk ^ (h << 1)) << 4);
}
__device__ __forceinline__ s16x4_t grad_tr(const char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(const_cast<char*>(p)));
}

// R4: r % 4 == 0 (16-byte loads of P)
template <bool R4>
__global__ __launch_bounds__(256) void k_grouped_grad(GroupGrads G) {
  __shared__ __attribute__((aligned(16))) char lds[2 * kGBuf];
  const int M = (int)G.M, r = G.r;
  // workgroups: per expert (its first chunk), then per extra chunk, the column tiles of both jobs
  const int block = G.block0 + (int)blockIdx.x, by = block / G.ct, bx = block % G.ct;
  int e = by, chunk = 0;
  if (e >= G.experts) {
    const int want = e - G.experts;
    chunk = extra_scan(G.offsets, G.experts, M, want, e);
    if (e < 0) return;  // the whole workgroup
    e = __builtin_amdgcn_readfirstlane(e);
    chunk = __builtin_amdgcn_readfirstlane(chunk);
  }
  int a, b;
  expert_range(G.offsets, e, M, a, b);
  const int mb = a + chunk * kGradChunk, me = min(b, mb + kGradChunk);
  const int job = bx >= G.ct0;
  const float* __restrict__ P = G.P[job];
  const uint16_t* __restrict__ Q = G.Q[job];
  const int64_t C = G.C[job];
  const int cb = (bx - (job ? G.ct0 : 0)) * 128, j0 = blockIdx.y * 64;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int jt = min(4, (r - j0 + 15) / 16);

  const __amdgpu_buffer_rsrc_t qr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(Q + (int64_t)mb * C), (short)0, (int)(max(me - mb, 0) * C * 2), 0x00020000);
  const uint32_t qrow = (uint32_t)tid >> 4, qch = (uint32_t)tid & 15u;
  const int64_t qcol = min<int64_t>(cb + 8 * qch, C - 8);  // clamped: outputs past C are dropped
  struct Stage { u32x4_t q[2]; f32x4_t p[2]; };
  auto load = [&](int m0, Stage& s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t row = (uint32_t)(m0 - mb) + qrow + 16u * i;  // rows past me read zero
      s.q[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(qr, (uint32_t)((row * C + qcol) * 2), 0, 0));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = m0 + (int)qrow + 16 * i, jb = j0 + 4 * (int)qch;
      f32x4_t v = {0.f, 0.f, 0.f, 0.f};
      if (m < me && jb < r) {
        const float* p = P + (int64_t)m * r + jb;
        if constexpr (R4) {
          v = *reinterpret_cast<const f32x4_t*>(p);
        } else {
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (jb + t < r) v[t] = p[t];
        }
      }
      s.p[i] = v;
    }
  };
  auto store = [&](const Stage& s, uint32_t buf) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t row = qrow + 16u * i;
      *reinterpret_cast<u32x4_t*>(lds + buf + gq_off(row, qch)) = s.q[i];
      uint32_t part[3][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float v0 = s.p[i][2 * t], v1 = s.p[i][2 * t + 1];
#pragma unroll
        for (int k = 0; k < 3; ++k) {  // (the third part is the whole rest: at most 8 bits)
          const float r0 = k < 2 ? split_rest(v0) : 0.0f, r1 = k < 2 ? split_rest(v1) : 0.0f;
          part[k][t] = (__float_as_uint(v0) >> 16) | (__float_as_uint(v1) & 0xFFFF0000u);
          v0 = r0;
          v1 = r1;
        }
      }
#pragma unroll
      for (int k = 0; k < 3; ++k)
        *reinterpret_cast<uint2*>(lds + buf + kGQ + k * kGP + gp_off(row, qch >> 1) + 8u * (qch & 1u)) =
            uint2{part[k][0], part[k][1]};
    }
  };
  // transpose-read addresses: lane group g takes rows 8 g .. 8 g + 7 (two reads), lane sp the
  // four elements from column 4 (sp % 4) of row sp / 4
  const uint32_t g = (uint32_t)lane >> 4, sp = (uint32_t)lane & 15u;
  uint32_t qa[2][2], pa[4][2];
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    const uint32_t row = 8u * g + 4u * hf + (sp >> 2);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t col = 32u * w + 16u * c + 4u * (sp & 3u);
      qa[c][hf] = gq_off(row, col >> 3) + 2u * (col & 7u);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t col = 16u * t + 4u * (sp & 3u);
      pa[t][hf] = kGQ + gp_off(row, col >> 3) + 2u * (col & 7u);
    }
  }
  auto frag = [&](uint32_t lo, uint32_t hi) {
    const s16x4_t l = grad_tr(lds + lo), h = grad_tr(lds + hi);
    return as_bf16x8(u32x4_t{__builtin_bit_cast(uint2, l).x, __builtin_bit_cast(uint2, l).y,
                             __builtin_bit_cast(uint2, h).x, __builtin_bit_cast(uint2, h).y});
  };
  f32x4_t acc[2][4];
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[c][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  Stage s0, s1;
  load(mb, s0);
  load(mb + 32, s1);
  auto step = [&](int m0, Stage& s, uint32_t buf) {
    store(s, buf);
    load(m0 + 64, s);
    __syncthreads();
    bf16x8_t q[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) q[c] = frag(buf + qa[c][0], buf + qa[c][1]);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t >= jt) break;
#pragma unroll
      for (int k = 2; k >= 0; --k) {  // smallest part first
        const bf16x8_t p = frag(buf + k * kGP + pa[t][0], buf + k * kGP + pa[t][1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) acc[c][t] = mfma16x16x32(q[c], p, acc[c][t]);
      }
    }
  };
  // buffer i is written again two steps later, after the barrier that every wave passes past its reads
  for (int m0 = mb; m0 < me; m0 += 64) {
    step(m0, s0, 0);
    if (m0 + 32 < me) step(m0 + 32, s1, kGBuf);
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
      if (chunk > 0) {
        const int64_t slot = by - G.experts;
        *reinterpret_cast<f32x4_t*>(G.part + (slot * r + j) * (G.C[0] + G.C[1]) + (job ? G.C[0] : 0) + c0) = v;
      } else if (job == 0) {
        *reinterpret_cast<f32x4_t*>(G.out[0] + ((int64_t)e * r + j) * C + c0) =
            f32x4_t{G.scale * v[0], G.scale * v[1], G.scale * v[2], G.scale * v[3]};
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) G.out[1][((int64_t)e * C + c0 + i) * r + j] = G.scale * v[i];
      }
    }
  }
}

// out += scale * (the expert's further chunks, in order)
__global__ __launch_bounds__(256) void k_grouped_grad_add(GroupGrads G) {
  const int e = blockIdx.y;
  int a, b;
  expert_range(G.offsets, e, (int)G.M, a, b);
  int ee = e, nx = extra_chunks(b - a);
  if (nx == 0) return;
  const int slot0 = extra_scan(G.offsets, G.experts, (int)G.M, -1, ee);
  nx = min(nx, G.extra - slot0);  // (overlapping ranges of malformed offsets could count more chunks than there are)
  const int64_t CC = G.C[0] + G.C[1], n = CC * G.r;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    float v = 0.0f;
    for (int s = 0; s < nx; ++s) v += G.part[(int64_t)(slot0 + s) * n + i];
    const int64_t j = i / CC, c = i % CC;
    float* o = c < G.C[0] ? G.out[0] + ((int64_t)e * G.r + j) * G.C[0] + c
                          : G.out[1] + ((int64_t)e * G.C[1] + c - G.C[0]) * G.r + j;
    *o += G.scale * v;
  }
}

}  // namespace

size_t grouped_grad_floats(int64_t M, int64_t N, int64_t K, int r, int experts) {
  (void)experts;
  return (size_t)(M / kGradChunk) * (size_t)r * (size_t)(N + K);
}

hipError_t launch_grouped_grads(const float* u, const float* t, const uint16_t* x, const uint16_t* dy, int64_t M,
                                int64_t N, int64_t K, int r, const int32_t* offsets, int experts, float scale, float* dA,
                                float* dB, float* part, hipStream_t s) {
  GroupGrads G;
  G.P[0] = u;
  G.P[1] = t;
  G.Q[0] = x;
  G.Q[1] = dy;
  G.out[0] = dA;
  G.out[1] = dB;
  G.C[0] = K;
  G.C[1] = N;
  G.ct0 = (int)((K + 127) / 128);
  G.M = M;
  G.r = r;
  G.experts = experts;
  G.offsets = offsets;
  G.scale = scale;
  G.part = part;
  const unsigned extra = (unsigned)(M / kGradChunk);  // at most: every extra chunk follows a full one
  G.ct = G.ct0 + (int)((N + 127) / 128);
  G.extra = (int)extra;
  const int64_t wgs = (int64_t)G.ct * (experts + (int64_t)extra);
  if (wgs > INT_MAX) return hipErrorInvalidValue;
  const hipError_t e = launch_blocks(wgs, [&](unsigned n, int b0) {
    const dim3 grid(n, (unsigned)((r + 63) / 64));
    G.block0 = b0;
    if (r % 4 == 0) hipLaunchKernelGGL(k_grouped_grad<true>, grid, dim3(256), 0, s, G);
    else hipLaunchKernelGGL(k_grouped_grad<false>, grid, dim3(256), 0, s, G);
  });
  if (e != hipSuccess || extra == 0) return e;
  const int64_t n = (N + K) * r;
  hipLaunchKernelGGL(k_grouped_grad_add, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 256), (unsigned)experts),
                     dim3(256), 0, s, G);
  return hipGetLastError();
}

}  // namespace qlr
