// Products of many rows: the coded weight is dequantized once into the workspace (bf16), and a product of two bf16 matrices
// runs on it.  The tiled product of qlr_tile.h dequantizes a weight once per row tile, between the products; here every weight
// is dequantized once, 2 bytes written and read, and the product's loop has nothing but loads and matrix instructions.
//
// Loop.  A workgroup of 8 waves owns 256 x 256 results, as four quadrants of two pieces of 128 rows of x and two of 128 rows
// of the weight; wave (wm, wn) takes 64 x 32 of each quadrant in 16 x 16 MFMA tiles.  A step contracts 64 elements: rows of 128
// bytes in LDS, 16-byte chunks XOR-swizzled by row (swz), all loaded straight into LDS.  Two buffers of the four pieces.  In the
// order (t, l) (t, r) (b, r) (b, l) a step's pieces t and l are in registers when it begins, r is read during its first
// quarter and b during its second, so that after the first half the whole buffer is free: the loads of the step after the next
// go into t and l during the first half (free since the half before) and into r and b during the second, each a
// step and a half ahead of its first read.  One barrier per half.  Each half's wait leaves the 8 newest loads open.
//
// What bounds it (2048 x 22016 x 4096, 688 tiles, the product alone): 298 us (1.24 PFLOP/s), on zeros 271 (the clock falls with the power).  32 x 32
// MFMA tiles took 310 and 254: they are the faster ones but draw more.  Half steps of 32 elements in a ring of five buffers, rows
// of 64 bytes, took 352: the loads of half lines bound that loop (without them it ran as fast as without the LDS reads).
// 128 x 128 results a wave, which would read a third less of LDS, spill.
//
// Adapter.  t = x A^T enters as extra steps of 32 adapter columns: x side [hi(s t) | lo(s t)], weight side [B | B], both laid out
// beforehand (k_dense_xt, k_dense_wt).  Of the gated block's two adapters each enters its own side only (a zero block on the
// other side would carry an infinity over).  Under a mask the products are formed apart, a quadrant at a time behind the loop.
//
// Results go through LDS in one short loop.  Written out over the registers, with the adapter's steps behind the loop too,
// the code of a tile's end ran to 100 KB, and fetching it cost 15 to 30 us a tile (2048 x 22016 x 4096 with saved pre-activations:
// 465 us the call, so 392).
//
// Rest.  A last partial round of R tiles, R <= 128, would leave half of the CUs idle: its tiles are split along the
// contraction into 256 / R parts (at most 4), whose sums go to the workspace and are added in order by a second kernel.
#include "qlr_tile.h"

namespace qlr {

namespace {

enum { DENSE_PLAIN = 0, DENSE_GATED = 1, DENSE_DROP = 2 };

constexpr uint32_t kPiece = 128 * 128;  // bytes: 128 rows of 64 bf16
constexpr int kTileFloats = 256 * 256;
// Of a split contraction of the tiled product: steps of 64 in a range at least, and ranges at most.
constexpr int64_t kSplitSteps = 4, kMaxSplits = 8;

struct FragX { u32x4_t f[4][2]; };
struct FragW { u32x4_t f[2][2]; };
typedef f32x4_t Quad[4][2];  // a wave's 64 x 32 results of a quadrant

__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <int KIND>
struct Dense {
  static constexpr int kCols = KIND == DENSE_GATED ? 128 : 256;  // output columns of a tile
  int lane, wave, wm, wn;
  int64_t row0, n0, NO;
  uint32_t xa[2], wa[2];  // fragment addresses within a piece

  __device__ __forceinline__ Dense(const DenseArgs& P, int tile, int tid) {
    NO = P.NO;
    lane = tid & 63;
    wave = scalar(tid >> 6);
    wm = wave >> 2;
    wn = wave & 3;
    // tiles in blocks of kGroupM row tiles, their column tiles one after the other, row tiles innermost (scalar: a buffer
    // resource needs scalar words)
    const int mt = (int)((P.M + 255) / 256), grp = tile / (kGroupM * P.ntiles), in = tile - grp * kGroupM * P.ntiles;
    const int gm = min(kGroupM, mt - grp * kGroupM);
    row0 = (int64_t)scalar(grp * kGroupM + in % gm) * 256;
    n0 = (int64_t)scalar(in / gm) * kCols;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t r = lane & 15, c = 4u * s + (lane >> 4);
      xa[s] = (64u * wm + r) * 128u + 16u * (c ^ swz(r));
      wa[s] = (32u * wn + r) * 128u + 16u * (c ^ swz(r));
    }
  }
  __device__ __forceinline__ void read(const char* p, FragX& f) const {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) f.f[i][s] = *reinterpret_cast<const u32x4_t*>(p + xa[s] + 2048u * i);
  }
  __device__ __forceinline__ void read(const char* p, FragW& f) const {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int c = 0; c < 2; ++c) f.f[c][s] = *reinterpret_cast<const u32x4_t*>(p + wa[s] + 2048u * c);
  }
  static __device__ __forceinline__ void mul(Quad& a, const FragX& x, const FragW& w) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) a[i][c] = mfma16x16x32(as_bf16x8(w.f[c][s]), as_bf16x8(x.f[i][s]), a[i][c]);
  }
  // first row of the weight's pieces l and r, and how many of its rows exist
  __device__ __forceinline__ int64_t wrow(int b) const { return KIND == DENSE_GATED ? b * NO + n0 : n0 + 128 * b; }
  __device__ __forceinline__ int64_t wlive(int b) const {
    const int64_t left = NO - (KIND == DENSE_GATED ? n0 : n0 + 128 * b);
    return max<int64_t>(0, min<int64_t>(128, left));
  }
};

// Direct loads of a piece: load j (0, 1) of wave w fills rows 16 w + 8 j .. + 7, lane l at byte 16 l: row l / 8, slot l % 8, which
// holds the chunk that the swizzle puts there.
// (The whole offset goes into the vector register: a scalar offset is taken from the resource's size, which may be smaller.)
__device__ __forceinline__ void piece_load(__amdgpu_buffer_rsrc_t r, char* dst, int wave, const uint32_t (&off)[2], uint32_t o) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (void __attribute__((address_space(3)))*)(dst + (2 * wave + j) * 1024), 16, off[j] + o,
                                             0, 0, 0);
}
__device__ __forceinline__ uint32_t piece_chunk(int lane, uint32_t r) { return 16u * (((uint32_t)lane & 7u) ^ swz(r & 15u)); }

// The LDS row r of a weight piece holds the piece's row w_row(r): of a wave's 32, MFMA tile c's row 4 q + v is the strip's column
// 8 q + 4 c + v, so that a lane ends up with 8 neighbouring columns.
__device__ __forceinline__ uint32_t w_row(uint32_t r) { return (r & ~31u) | (8u * ((r & 15u) >> 2) + 4u * ((r >> 4) & 1u) + (r & 3u)); }

// The eight pieces of LDS, by their addresses.  (Opaque ones where one is chosen: the compiler makes a choice among known ones a
// table in memory, which it then cannot emit, and one among members an indexed load.)
typedef __attribute__((address_space(3))) char lds_t;
struct Pieces {
  lds_t *p0, *p1, *p2, *p3, *p4, *p5, *p6, *p7;
  __device__ __forceinline__ Pieces(char* a, char* b, char* c, char* d, char* e, char* f, char* g, char* h)
      : p0((lds_t*)a), p1((lds_t*)b), p2((lds_t*)c), p3((lds_t*)d), p4((lds_t*)e), p5((lds_t*)f), p6((lds_t*)g), p7((lds_t*)h) {}
  static __device__ __forceinline__ uint32_t opaque(lds_t* p) {
    uint32_t o = (uint32_t)(uintptr_t)p;
    asm("" : "+s"(o));
    return o;
  }
  __device__ __forceinline__ lds_t* at(int k) const {  // (k scalar)
    const uint32_t a = opaque(p0), b = opaque(p1), c = opaque(p2), d = opaque(p3), e = opaque(p4), f = opaque(p5), g = opaque(p6), h = opaque(p7);
    uint32_t r = a;
    r = k == 1 ? b : r;
    r = k == 2 ? c : r;
    r = k == 3 ? d : r;
    r = k == 4 ? e : r;
    r = k == 5 ? f : r;
    r = k == 6 ? g : r;
    r = k == 7 ? h : r;
    return (lds_t*)(uintptr_t)r;
  }
  static __device__ __forceinline__ lds_t* of(bool second, lds_t* a, lds_t* b) {
    const uint32_t u = opaque(a), v = opaque(b);
    return (lds_t*)(uintptr_t)(second ? v : u);
  }
};
typedef __attribute__((address_space(3))) f32x4_t lds4_t;

// 8 neighbouring results, those of columns col .. NO - 1, to out[at ..] (bf16 or float32), in 16-byte stores where they may be.
__device__ __forceinline__ void put8(void* out, int dt, int64_t ld, int64_t row, int64_t col, int64_t NO, const f32x4_t& a, const f32x4_t& b) {
  const int es = dt == DT_F32 ? 4 : 2;
  char* const o = reinterpret_cast<char*>(out) + (row * ld + col) * es;
  const bool vec = (ld * es) % 16 == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0 && col + 8 <= NO;
  if (dt == DT_F32) {
    if (vec) {
      reinterpret_cast<f32x4_t*>(o)[0] = a;
      reinterpret_cast<f32x4_t*>(o)[1] = b;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col + e < NO) reinterpret_cast<float*>(o)[e] = e < 4 ? a[e & 3] : b[e & 3];
    }
  } else {
    const u32x4_t v = {pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
    if (vec) {
      *reinterpret_cast<u32x4_t*>(o) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col + e < NO) reinterpret_cast<uint16_t*>(o)[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
  }
}
template <int A>
__device__ __forceinline__ f32x4_t gate4(const f32x4_t& g, const f32x4_t& v) {
  return f32x4_t{act_f<A>(g[0]) * v[0], act_f<A>(g[1]) * v[1], act_f<A>(g[2]) * v[2], act_f<A>(g[3]) * v[3]};
}
// The outputs of 8 neighbouring columns of a row: of their sums, y; of the gate's (a) and the up projection's (v), gu and h.
template <int KIND>
__device__ __forceinline__ void result8(const DenseArgs& P, int64_t row, int64_t col, f32x4_t a0, f32x4_t a1, const f32x4_t& v0, const f32x4_t& v1) {
  if constexpr (KIND == DENSE_GATED) {
    if (P.gu) {
      put8(P.gu, DT_BF16, 2 * P.NO, row, col, P.NO, a0, a1);
      put8(P.gu + P.NO, DT_BF16, 2 * P.NO, row, col, P.NO, v0, v1);
    }
    if (P.act == ACT_SILU) a0 = gate4<ACT_SILU>(a0, v0), a1 = gate4<ACT_SILU>(a1, v1);
    else if (P.act == ACT_GELU) a0 = gate4<ACT_GELU>(a0, v0), a1 = gate4<ACT_GELU>(a1, v1);
    else a0 = gate4<ACT_GELU_TANH>(a0, v0), a1 = gate4<ACT_GELU_TANH>(a1, v1);
  }
  put8(P.y, P.ydt, P.NO, row, col, P.NO, a0, a1);
}

// Results of a tile, 128 rows at a time through all of LDS: 16 rows of 256 float32 a piece, 16-byte chunks XOR-swizzled by the row.
// (One short loop: unrolled over the registers the code ran to 100 KB, and fetching it took 15 to 30 us a tile.)
template <int KIND>
__device__ __forceinline__ void dense_results(const DenseArgs& P, const Dense<KIND>& D, const Quad (&acc)[2][2], Pieces L) {
  const int q = D.lane >> 4;
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    auto put = [&](int i, lds_t* piece) __attribute__((always_inline)) {
      const uint32_t r = D.lane & 15;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          *(lds4_t*)(piece + r * 1024u + 16u * ((32u * b + 8u * D.wn + 2u * q + c) ^ r)) = acc[a][b][i][c];
    };
    put(0, Pieces::of(D.wm, L.p0, L.p4));
    put(1, Pieces::of(D.wm, L.p1, L.p5));
    put(2, Pieces::of(D.wm, L.p2, L.p6));
    put(3, Pieces::of(D.wm, L.p3, L.p7));
    __syncthreads();
    const int64_t rows = P.M - D.row0 - 128 * a;
    const int tid = 64 * D.wave + D.lane;
#pragma unroll 1
    for (int it = 0; it < (KIND == DENSE_GATED ? 4 : 8); ++it) {
      int row, c;  // of the 128; 8 columns c of the tile's output columns
      lds_t* p;
      if constexpr (KIND == DENSE_GATED) {
        row = 32 * it + (tid >> 4), c = tid & 15;
        p = L.at(2 * it + (D.wave >> 2));
      } else {
        row = 16 * it + (tid >> 5), c = tid & 31;
        p = L.at(it);
      }
      const uint32_t r = row & 15;
      const int64_t col = D.n0 + 8 * c;
      p += r * 1024u;
      auto get = [&](uint32_t ch) __attribute__((always_inline)) { return *(lds4_t*)(p + 16u * (ch ^ r)); };
      const f32x4_t a0 = get(2 * c), a1 = get(2 * c + 1);
      f32x4_t v0 = a0, v1 = a1;
      if constexpr (KIND == DENSE_GATED) v0 = get(32 + 2 * c), v1 = get(32 + 2 * c + 1);
      if (row < rows && col < D.NO) result8<KIND>(P, D.row0 + 128 * a + row, col, a0, a1, v0, v1);
    }
    __syncthreads();
  }
}

// Results under a mask, a quadrant at a time: y = sums + sum over the halves of mask (x side)(weight side), the adapter's products from
// fragments read straight from memory (the next product's behind the one before).  stage(ab) puts the quadrant's sums into the first
// four pieces, 32 rows of 128 float32 a piece, the products go to the others; a thread takes 8 neighbouring columns, one byte of the
// mask, of four rows.
__device__ __forceinline__ lds4_t* drop_at(lds_t* piece, uint32_t row, uint32_t ch) {
  return (lds4_t*)(piece + (row & 31u) * 512u + 16u * (ch ^ (row & 15u)));
}
template <typename S>
__device__ __forceinline__ void dense_drop(const DenseArgs& P, const Dense<DENSE_DROP>& D, int ab0, int ab1, Pieces L, S stage) {
  const int q = D.lane >> 4, l = D.lane & 15, tid = 64 * D.wave + D.lane;
  const int64_t kb = P.NO >> 3;
  FragX x;
  FragW w;
  auto fetch = [&](int ab, int e) __attribute__((always_inline)) {
    const int64_t row0 = D.row0 + 128 * (ab >> 1) + 64 * D.wm, n0 = D.n0 + 128 * (ab & 1) + 32 * D.wn;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < 4; ++i)  // (rows and columns past the end repeat the last: their results are dropped)
        x.f[i][s] = *reinterpret_cast<const u32x4_t*>(P.xt + ((int64_t)e * P.M + min<int64_t>(row0 + 16 * i + l, P.M - 1)) * 64 + 32 * s + 8 * q);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        w.f[c][s] = *reinterpret_cast<const u32x4_t*>(P.wt + ((int64_t)e * P.NO + min<int64_t>(n0 + (int)w_row(16u * c + l), P.NO - 1)) * 64 + 32 * s + 8 * q);
    }
  };
  fetch(ab0, 0);
#pragma unroll 1
  for (int ab = ab0; ab < ab1; ++ab) {
    const int64_t row0 = D.row0 + 128 * (ab >> 1), n0 = D.n0 + 128 * (ab & 1), col = n0 + 8 * (tid & 15);
#pragma unroll 1
    for (int hf = 0; hf < P.halves; ++hf) {
      uint32_t keep = 0;
#pragma unroll
      for (int it = 0; it < 4; ++it)
        keep |= (uint32_t)P.drop.bits[((int64_t)hf * P.M + min<int64_t>(row0 + 32 * it + (tid >> 4), P.M - 1)) * kb + min<int64_t>(col, P.NO - 8) / 8] << (8 * it);
      Quad part;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) part[i][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int j = 0; j < P.nb; ++j) {
        const int e = hf * P.nb + j;
        Dense<DENSE_DROP>::mul(part, x, w);
        const bool last = e + 1 == P.halves * P.nb;
        if (!last || ab + 1 < ab1) fetch(last ? ab + 1 : ab, last ? 0 : e + 1);
      }
      if (hf == 0) stage(ab);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t row = 64u * D.wm + 16u * i + l;
        lds_t* const piece = i < 2 ? Pieces::of(D.wm, L.p4, L.p6) : Pieces::of(D.wm, L.p5, L.p7);
#pragma unroll
        for (int c = 0; c < 2; ++c) *drop_at(piece, row, 8u * D.wn + 2u * q + c) = part[i][c];
      }
      __syncthreads();
#pragma unroll 1
      for (int it = 0; it < 4; ++it, keep >>= 8) {
        const uint32_t r = 32u * it + (tid >> 4), c = tid & 15;
        const int64_t row = row0 + r;
        lds_t *const b = L.at(it), *const a = L.at(4 + it);
        f32x4_t s0 = *drop_at(b, r, 2 * c), s1 = *drop_at(b, r, 2 * c + 1);
        const f32x4_t p0 = *drop_at(a, r, 2 * c), p1 = *drop_at(a, r, 2 * c + 1);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          s0[v] += (keep >> v) & 1u ? p0[v] : 0.0f;
          s1[v] += (keep >> (4 + v)) & 1u ? p1[v] : 0.0f;
        }
        if (hf + 1 < P.halves) {
          *drop_at(b, r, 2 * c) = s0;
          *drop_at(b, r, 2 * c + 1) = s1;
        } else if (row < P.M && col < P.NO) {
          put8(P.y, P.ydt, P.NO, row, col, P.NO, s0, s1);
        }
      }
      __syncthreads();
    }
  }
}

template <int KIND>
__global__ __launch_bounds__(512, 1) void k_dense(DenseArgs P) {
  __shared__ __attribute__((aligned(16))) char X0t[kPiece], X0b[kPiece], W0l[kPiece], W0r[kPiece];
  __shared__ __attribute__((aligned(16))) char X1t[kPiece], X1b[kPiece], W1l[kPiece], W1r[kPiece];
  // which tile, or which part of one: each XCD (workgroup b runs on XCD b % 8) takes a contiguous range of either
  int tile, unit = -1;
  {
    const int b = P.block0 + (int)blockIdx.x, per = (P.whole + 7) / 8;
    if (b < 8 * per) {
      tile = (b & 7) * per + (b >> 3);
      if (tile >= P.whole) return;
    } else {
      const int u = b - 8 * per, n = P.rest * P.splits, peru = (n + 7) / 8;
      unit = (u & 7) * peru + (u >> 3);
      if ((u >> 3) >= peru || unit >= n) return;
      tile = P.whole + unit / P.splits;
    }
  }
  const Dense<KIND> D(P, tile, threadIdx.x);
  const int lane = D.lane, wave = D.wave;
  const uint32_t kb = (uint32_t)P.KC * 2u;  // bytes of a row
  const int all = (int)((kb + 127) / 128), total = all + (KIND == DENSE_DROP ? 0 : P.halves * P.nb);  // steps, with the adapter's
  const int sp = unit >= 0 ? unit % P.splits : 0, parts = unit >= 0 ? P.splits : 1;
  const int k0 = scalar(all * sp / parts), k1 = scalar(sp + 1 < parts ? all * (sp + 1) / parts : total);
  const __amdgpu_buffer_rsrc_t xr = tile_rsrc(P.x + D.row0 * P.KC, (uint32_t)min<int64_t>(256, P.M - D.row0) * kb);
  const __amdgpu_buffer_rsrc_t wl = tile_rsrc(P.w + D.wrow(0) * P.KC, (uint32_t)D.wlive(0) * kb);
  const __amdgpu_buffer_rsrc_t wr = tile_rsrc(P.w + D.wrow(1) * P.KC, (uint32_t)D.wlive(1) * kb);
  uint32_t off[2], woff[2];  // of the next step to be loaded
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t r = 16u * wave + 8u * j + (lane >> 3);
    off[j] = r * kb + piece_chunk(lane, r) + (uint32_t)k0 * 128u;
    woff[j] = w_row(r) * kb + piece_chunk(lane, r) + (uint32_t)k0 * 128u;
  }
  const uint32_t half = 128u * kb;
  // A piece of a step of the weight's, and of an adapter step e = (half, block): x side M x 64, weight side rows x 64.
  enum { XT, XB, WL, WR };
  auto load = [&](auto which, char* dst) __attribute__((always_inline)) {
    constexpr int W = decltype(which)::value;
    if constexpr (W == XT || W == XB) piece_load(xr, dst, wave, off, W == XB ? half : 0);
    else piece_load(W == WL ? wl : wr, dst, wave, woff, 0);
  };
  auto adapter = [&](int e, auto which, char* dst) __attribute__((always_inline)) {
    constexpr int W = decltype(which)::value;
    uint32_t o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t r = 16u * wave + 8u * j + (lane >> 3);
      o[j] = (W == XT || W == XB ? r : w_row(r)) * 128u + piece_chunk(lane, r);
    }
    if constexpr (W == XT || W == XB) {
      const uint32_t live = (uint32_t)min<int64_t>(256, P.M - D.row0) * 128u;
      piece_load(tile_rsrc(P.xt + ((int64_t)e * P.M + D.row0) * 64, live), dst, wave, o, W == XB ? 128u * 128u : 0);
    } else {
      const uint16_t* const w = P.wt + (KIND == DENSE_GATED ? (int64_t)(e % P.nb) * 2 * P.NO : (int64_t)e * P.NO) * 64;
      piece_load(tile_rsrc(w + D.wrow(W - WL) * 64, (uint32_t)D.wlive(W - WL) * 128u), dst, wave, o, 0);
    }
  };
  // ... of either.  (Steps past the last are loaded and not used.)
  auto fetch = [&](int k, auto which, char* dst) __attribute__((always_inline)) {
    if (KIND == DENSE_DROP || k < all || k >= total) load(which, dst);
    else adapter(k - all, which, dst);
  };
  constexpr std::integral_constant<int, XT> xt_{};
  constexpr std::integral_constant<int, XB> xb_{};
  constexpr std::integral_constant<int, WL> wl_{};
  constexpr std::integral_constant<int, WR> wr_{};
  auto advance = [&] {
#pragma unroll
    for (int j = 0; j < 2; ++j) off[j] += 128u, woff[j] += 128u;
  };
  // Before the loads of a last step that the contraction fills in part: its chunks past the end of the rows read zero, at an
  // offset past every range.
  auto clip = [&](int k) __attribute__((always_inline)) {
    if (k == all - 1 && (kb & 127u) != 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (piece_chunk(lane, 16u * wave + 8u * j + (lane >> 3)) >= (kb & 127u)) off[j] = woff[j] = 0x80000000u;
    }
  };
  Quad acc[2][2];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) acc[a][b][i][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  FragX xt, xb;
  FragW wp, wq;
  // Every wave's reads of the half are done, and all loads but the 8 newest have arrived.
  auto barrier = [&] {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0078);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  clip(k0);
  fetch(k0, xt_, X0t);
  fetch(k0, wl_, W0l);
  fetch(k0, wr_, W0r);
  fetch(k0, xb_, X0b);
  advance();
  clip(k0 + 1);
  fetch(k0 + 1, xt_, X1t);
  fetch(k0 + 1, wl_, W1l);
  fetch(k0 + 1, wr_, W1r);
  fetch(k0 + 1, xb_, X1b);
  advance();
  barrier();
  D.read(X0t, xt);
  D.read(W0l, wp);
  barrier();  // (t and l of the first buffer are loaded again in the first half)
  // One step.  edge: it, or the step that it loads, may be an adapter's; of the gated block's adapters each enters its own side only.
  auto step = [&](int k, auto edge, char* T, char* B, char* L, char* R, const char* nT, const char* nL, FragW& l, FragW& r)
      __attribute__((always_inline)) {
    constexpr bool E = decltype(edge)::value && KIND != DENSE_DROP;
    const bool left = !E || KIND != DENSE_GATED || k < all + P.nb, right = !E || KIND != DENSE_GATED || k < all || k >= all + P.nb;
    auto next = [&](auto which, char* dst) __attribute__((always_inline)) {
      if constexpr (E) fetch(k + 2, which, dst);
      else load(which, dst);
    };
    __builtin_amdgcn_sched_barrier(0);
    D.read(R, r);
    clip(k + 2);
    next(xt_, T);
    next(wl_, L);
    __builtin_amdgcn_sched_barrier(0);
    if (left) Dense<KIND>::mul(acc[0][0], xt, l);
    __builtin_amdgcn_sched_barrier(0);
    D.read(B, xb);
    __builtin_amdgcn_sched_barrier(0);
    if (right) Dense<KIND>::mul(acc[0][1], xt, r);
    barrier();
    D.read(nT, xt);
    next(wr_, R);
    next(xb_, B);
    advance();
    __builtin_amdgcn_sched_barrier(0);
    if (right) Dense<KIND>::mul(acc[1][1], xb, r);
    __builtin_amdgcn_sched_barrier(0);
    D.read(nL, r);
    __builtin_amdgcn_sched_barrier(0);
    if (left) Dense<KIND>::mul(acc[1][0], xb, l);
    barrier();
  };
  int k = k0;
  {
    constexpr std::false_type inner{};
    for (; k + 2 <= k1 && (KIND == DENSE_DROP || k + 3 < all); k += 2) {
      step(k, inner, X0t, X0b, W0l, W0r, X1t, W1l, wp, wq);
      step(k + 1, inner, X1t, X1b, W1l, W1r, X0t, W0l, wq, wp);
    }
    constexpr std::true_type edge{};
    for (; k < k1; k += 2) {
      step(k, edge, X0t, X0b, W0l, W0r, X1t, W1l, wp, wq);
      if (k + 1 < k1) step(k + 1, edge, X1t, X1b, W1l, W1r, X0t, W0l, wq, wp);
    }
  }
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));  // (nothing of what follows is formed before the loop and kept)
  const Dense<KIND> E(P, tile, tid);
  const int q = E.lane >> 4;
  if (unit >= 0) {  // sums, 256 x 256 row-major
    float* const p = P.part + (int64_t)unit * kTileFloats + (64 * E.wm + (E.lane & 15)) * 256 + 32 * E.wn + 8 * q;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) *reinterpret_cast<f32x4_t*>(p + (128 * a + 16 * i) * 256 + 128 * b + 4 * c) = acc[a][b][i][c];
    return;
  }
  __builtin_amdgcn_s_waitcnt(0x0070);  // the loads past the last step too, before the buffers are used again
  __syncthreads();
  const Pieces L{X0t, X0b, W0l, W0r, X1t, X1b, W1l, W1r};
  if constexpr (KIND == DENSE_DROP) {
    dense_drop(P, E, 0, 4, L, [&](int ab) __attribute__((always_inline)) {
      auto put = [&](const Quad& sum) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t row = 64u * E.wm + 16u * i + (E.lane & 15);
          lds_t* const piece = i < 2 ? (Pieces::of(E.wm, L.p0, L.p2)) : (Pieces::of(E.wm, L.p1, L.p3));
#pragma unroll
          for (int c = 0; c < 2; ++c) *drop_at(piece, row, 8u * E.wn + 2u * q + c) = sum[i][c];
        }
      };
      if (ab == 0) put(acc[0][0]);
      else if (ab == 1) put(acc[0][1]);
      else if (ab == 2) put(acc[1][0]);
      else put(acc[1][1]);
    });
  } else {
    dense_results<KIND>(P, E, acc, L);
  }
}

// The tiles of the rest: their parts' sums added in order, 8 output columns of a row to a thread.
template <int KIND>
__global__ __launch_bounds__(256) void k_dense_rest(DenseArgs P) {
  constexpr int kItems = KIND == DENSE_GATED ? 16 : 32;  // of a tile's row
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int rest = scalar((int)(id / (256 * kItems)));
  const int row = (int)(id / kItems) & 255, c = (int)(id % kItems);
  const Dense<KIND> D(P, P.whole + rest, 0);
  const int64_t col = D.n0 + 8 * c;
  if (D.row0 + row >= P.M || col >= D.NO) return;
  const float* p = P.part + (int64_t)rest * P.splits * kTileFloats + row * 256 + 8 * c;
  f32x4_t s[4] = {};
  for (int k = 0; k < P.splits; ++k, p += kTileFloats) {
#pragma unroll
    for (int h = 0; h < (KIND == DENSE_GATED ? 4 : 2); ++h) {
      const f32x4_t u = *reinterpret_cast<const f32x4_t*>(p + (h >> 1) * 128 + 4 * (h & 1));
#pragma unroll
      for (int j = 0; j < 4; ++j) s[h][j] += u[j];
    }
  }
  result8<KIND>(P, D.row0 + row, col, s[0], s[1], s[2], s[3]);
}

// The same under a mask: quadrant blockIdx.x % 4 of tile whole + blockIdx.x / 4.
__global__ __launch_bounds__(512) void k_dense_rest_drop(DenseArgs P) {
  __shared__ __attribute__((aligned(16))) char b[8][kPiece];
  const int rest = (int)blockIdx.x >> 2, quad = (int)blockIdx.x & 3;
  const Dense<DENSE_DROP> D(P, P.whole + rest, threadIdx.x);
  const Pieces L{b[0], b[1], b[2], b[3], b[4], b[5], b[6], b[7]};
  dense_drop(P, D, quad, quad + 1, L, [&](int) __attribute__((always_inline)) {
    const float* const p = P.part + (int64_t)rest * P.splits * kTileFloats + (quad >> 1) * 128 * 256 + (quad & 1) * 128;
#pragma unroll 1
    for (int it = 0; it < 8; ++it) {
      const uint32_t row = 16u * it + (threadIdx.x >> 5), ch = threadIdx.x & 31;
      const float* e = p + row * 256 + 4 * ch;
      f32x4_t s = *reinterpret_cast<const f32x4_t*>(e);
      for (int k = 1; k < P.splits; ++k) {
        e += kTileFloats;
        const f32x4_t u = *reinterpret_cast<const f32x4_t*>(e);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] += u[j];
      }
      *drop_at(L.at(it >> 1), row, ch) = s;
    }
  });
}

// The sums of a tiled product's ranges (64 x 128 and 128 x 128 tiles, qlr_tile.h) added in order, 8 output columns of a row to a thread.
template <int KIND>
__global__ __launch_bounds__(256) void k_tile_sum(DenseArgs P, int64_t ld) {
  const int64_t items = (P.NO + 7) / 8, id = (int64_t)blockIdx.x * 256 + threadIdx.x, row = id / items, col = id % items * 8;
  if (row >= P.M) return;
  const float* p = P.part + row * ld + col;
  const bool two = col + 4 < P.NO;  // (the columns' second four are there, a row's end rounded up to four)
  f32x4_t s[4] = {};
#pragma unroll 4
  for (int k = 0; k < P.splits; ++k, p += P.M * ld) {
#pragma unroll
    for (int h = 0; h < (KIND == DENSE_GATED ? 4 : 2); ++h) {
      f32x4_t u = {0.f, 0.f, 0.f, 0.f};
      if ((h & 1) == 0 || two) u = *reinterpret_cast<const f32x4_t*>(p + (h >> 1) * (ld / 2) + 4 * (h & 1));
#pragma unroll
      for (int j = 0; j < 4; ++j) s[h][j] += u[j];
    }
  }
  result8<KIND>(P, row, col, s[0], s[1], s[2], s[3]);
}

// ---------------------------------------------------------------- the weight
//
// Wd = bf16(level scale), row by row (rows x K), or transposed (K x rows); each weight rounded once to nearest.
// A thread takes 8 codes of one block.  Bound by the 2 bytes written a weight.
template <int BITS>
struct Deq {
  // 8 codes from bit 8 BITS i of a block's codes
  static __device__ __forceinline__ u32x4_t eight(const uint8_t* blk, int i, float ap, const float* sL, const Levels& lv) {
    u32x4_t o;
    if constexpr (BITS == 4) {
      uint32_t w[4];
      lut4_word(*reinterpret_cast<const uint32_t*>(blk + 4 * i), make_lut4(lv, ap), w);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = w[j];
    } else {
      uint32_t c[8];
      if constexpr (BITS == 8) {
        const uint2 u = *reinterpret_cast<const uint2*>(blk + 8 * i);
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = ((j < 4 ? u.x : u.y) >> (8 * (j & 3))) & 255u;
      } else {
        uint32_t u = 0;
#pragma unroll
        for (int j = 0; j < BITS; ++j) u |= (uint32_t)blk[BITS * i + j] << (8 * j);
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = (u >> (BITS * j)) & ((1u << BITS) - 1);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = cvt_pk_bf16(sL[c[2 * j]] * ap, sL[c[2 * j + 1]] * ap);
    }
    return o;
  }
};

template <int BITS>
__global__ __launch_bounds__(256) void k_dense_weight(DenseWeight G, Levels lv) {
  __shared__ float sL[1 << BITS];
  if constexpr (BITS != 4) {
    stage_levels<1 << BITS>(lv, sL);
    __syncthreads();
  }
  const int64_t n = G.rows * G.K / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t blk = i >> 3;
    const float ap = (float)G.q8[blk] * G.cst[blk >> 8];
    reinterpret_cast<u32x4_t*>(G.out)[i] = Deq<BITS>::eight(G.codes + blk * (8 * BITS), (int)(i & 7), ap, sL, lv);
  }
}

// A workgroup transposes 128 weight rows x 64 columns (one block of each row) through LDS: rows of 64 bf16 written as they are
// dequantized, 8 rows of one column read back with the transpose read.
template <int BITS>
__global__ __launch_bounds__(256) void k_dense_weight_tr(DenseWeight G, Levels lv) {
  __shared__ float sL[1 << BITS];
  __shared__ __attribute__((aligned(16))) char lds[128 * 144];
  if constexpr (BITS != 4) {
    stage_levels<1 << BITS>(lv, sL);
    __syncthreads();
  }
  const int64_t nb = G.K >> 6, r0 = (int64_t)blockIdx.x * 128;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int64_t kb = blockIdx.y; kb < nb; kb += gridDim.y) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int row = 32 * p + (tid >> 3), i = tid & 7;
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (r0 + row < G.rows) {
        const int64_t blk = (r0 + row) * nb + kb;
        v = Deq<BITS>::eight(G.codes + blk * (8 * BITS), i, (float)G.q8[blk] * G.cst[blk >> 8], sL, lv);
      }
      *reinterpret_cast<u32x4_t*>(lds + row * 144 + 16 * i) = v;
    }
    __syncthreads();
    // each 16 lanes: 8 rows (two reads of 4) of 16 columns; a wave's four groups take 32 rows, its passes the 64 columns
    const int g = lane >> 4, s = lane & 15;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int row = 32 * wave + 8 * g, col = 16 * c;
      const char* p = lds + (row + (s >> 2)) * 144 + 2 * col + 8 * (s & 3);
      const u16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)const_cast<char*>(p));
      const u16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)const_cast<char*>(p + 4 * 144));
      if (r0 + row < G.rows)  // (rows % 8 == 0)
        *reinterpret_cast<u32x4_t*>(G.out + (kb * 64 + col + s) * G.rows + r0 + row) =
            u32x4_t{__builtin_bit_cast(uint2, lo).x, __builtin_bit_cast(uint2, lo).y, __builtin_bit_cast(uint2, hi).x,
                    __builtin_bit_cast(uint2, hi).y};
    }
    __syncthreads();
  }
}

// The adapters' steps: xt[e][m] = [hi(s t) | lo(s t)] of 32 columns of half e / nb, and wt[e][n] = [B | B] (SIDE 0: B is
// rows x r, given as halves of rows / 2 rows for the gated block) or of A^T (A: halves x r x rows).
__global__ __launch_bounds__(256) void k_dense_xt(DenseAdapter G) {
  const int64_t n = (int64_t)G.halves * G.nb * G.M * 4;  // pieces of 8 columns
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int c = (int)(i & 3);
    const int64_t m = (i >> 2) % G.M, e = (i >> 2) / G.M;
    const int hf = (int)(e / G.nb), j0 = 32 * (int)(e % G.nb) + 8 * c;
    u32x4_t hi, lo;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float u[2] = {0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (j0 + 2 * k + j < G.r) {
          for (int s = 0; s < G.t_splits; ++s) u[j] += G.t[((int64_t)s * G.M + m) * G.ldt + hf * G.r + j0 + 2 * k + j];
          u[j] *= G.scale;
        }
      const float l0 = split_rest(u[0]), l1 = split_rest(u[1]);
      hi[k] = (__float_as_uint(u[0]) >> 16) | (__float_as_uint(u[1]) & 0xFFFF0000u);
      lo[k] = pack_bf16x2(l0, l1);
    }
    uint16_t* const o = G.xt + (e * G.M + m) * 64 + 8 * c;
    *reinterpret_cast<u32x4_t*>(o) = hi;
    *reinterpret_cast<u32x4_t*>(o + 32) = lo;
  }
}
__global__ __launch_bounds__(256) void k_dense_wt(DenseAdapter G) {
  const int64_t n = (int64_t)(G.tr ? G.halves : 1) * G.nb * G.rows * 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int c = (int)(i & 3);
    const int64_t row = (i >> 2) % G.rows, e = (i >> 2) / G.rows;
    const int hf = (int)(e / G.nb), j0 = 32 * (int)(e % G.nb) + 8 * c;
    u32x4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (j0 + k < G.r)
        v[k >> 1] |= (uint32_t)(G.tr ? G.ab[((int64_t)hf * G.r + j0 + k) * G.rows + row] : G.ab[row * G.r + j0 + k]) << (16 * (k & 1));
    uint16_t* const o = G.wt + (e * G.rows + row) * 64 + 8 * c;
    *reinterpret_cast<u32x4_t*>(o) = v;
    *reinterpret_cast<u32x4_t*>(o + 32) = v;
  }
}

template <int KIND>
hipError_t launch_dense_k(DenseArgs a, hipStream_t s) {
  const int64_t blocks = 8 * (((int64_t)a.whole + 7) / 8) + 8 * (((int64_t)a.rest * a.splits + 7) / 8);
  hipError_t e = launch_blocks(blocks, [&](unsigned n, int b0) {
    a.block0 = b0;
    hipLaunchKernelGGL(k_dense<KIND>, dim3(n), dim3(512), 0, s, a);
  });
  if (e != hipSuccess || a.rest == 0) return e;
  if constexpr (KIND == DENSE_DROP) hipLaunchKernelGGL(k_dense_rest_drop, dim3((unsigned)(4 * a.rest)), dim3(512), 0, s, a);
  else hipLaunchKernelGGL(k_dense_rest<KIND>, dim3((unsigned)(a.rest * (KIND == DENSE_GATED ? 16 : 32))), dim3(256), 0, s, a);
  return hipGetLastError();
}

unsigned grid_of(int64_t items) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>((items + 255) / 256, 256 * 16)); }

}  // namespace

// A step of a tile is bound by its workgroup's LDS traffic (dequantized weights in and fragments out), so more rows a tile and all
// CUs at work are what counts: up to 64 rows 64 x 128 tiles, from there on 128 x 128 ones, in ranges that make about 512
// workgroups, two to a CU.  Input gradient of 777 rows, 2048 columns over 5632 (2-bit): 40 us and 6.5 for the sums, as 64 x 128 tiles
// 55, in two ranges of those 47 and 5; of 333, 4096 over 4096 (8-bit): 37 and 6.6, 57, 50 and 5; of 64, 1024 over 2048: 11 and 4,
// unsplit 24.  Up to 40 steps, 128 tiles of 64 x 128 and more run unsplit (the sums' kernel and the ranges' ends cost 6 to 10 us).  Gated
// forward, r = 8, 4-bit, whole call, unsplit and in the 2 to 8 ranges that 512 workgroups would make, 32, 40 and 64 steps: 333 rows x 1403 (132
// tiles) 29 and 37, 33 and 32, 47 and 37; 333 x 2048 (192) 27 and 32, 31 and 35, 44 and 40; 600 x 1024 (160) 27 and 32, 31 and 33,
// 45 and 38; 130 x 4096 (192) 26 and 31, 31 and 34, 43 and 41; 64 x 11008 (172) 27 and 32, 32 and 36, 44 and 45.  With 66 tiles (333 x
// 700) 28 and 27, 32 and 28, 44 and 32.  Layer's backward, 333 rows, 4096 columns (192 tiles) 38 and 45, 44 and 46, 58 and 52.
// The layer's forward under dropout (r = 16, 4-bit), whole call, ranges and the prefill
// kernel without them: 64 rows of 1024 x 1024 15 and 25 us, of 4096 x 4096 21 and 64; 333 rows 18 and 25, 37 and 64; 777 rows
// 21 and 27, 60 and 67.
int train_tile_splits(int64_t M, int64_t cols, int64_t KC) {
  // (256 x 256 tiles: see launch_tile)
  if ((M + 255) / 256 * ((cols + 255) / 256) >= 192) return 1;
  const int64_t nt = (cols + 127) / 128, steps = (KC + 63) / 64;
  if (steps <= 40 && (M + 63) / 64 * nt >= 128) return 1;
  const int64_t bm = M <= 64 ? 64 : 128, tiles = (M + bm - 1) / bm * nt;
  return (int)std::max<int64_t>(1, std::min({(int64_t)512 / tiles, steps / kSplitSteps, (int64_t)kMaxSplits}));
}

hipError_t launch_tile_sum(const TrainArgs& a, int64_t NO, bool gated, hipStream_t s) {
  DenseArgs d{};
  d.M = a.M;
  d.NO = NO;
  d.y = a.y;
  d.ydt = a.ydt;
  d.act = a.act;
  d.gu = a.gu;
  d.splits = a.splits;
  d.part = a.part;
  const dim3 grid((unsigned)((a.M * ((NO + 7) / 8) + 255) / 256));
  if (gated) hipLaunchKernelGGL(k_tile_sum<DENSE_GATED>, grid, dim3(256), 0, s, d, train_part_cols(NO, true));
  else hipLaunchKernelGGL(k_tile_sum<DENSE_PLAIN>, grid, dim3(256), 0, s, d, train_part_cols(NO, false));
  return hipGetLastError();
}

// When.  The copy costs a fixed time for the weight, 0.5 ns per 1000 weights and two to four launches, and saves the tiled product's own
// dequantization, whose part grows with the rows; its tiles take longer to begin and to end.  The call through the copy and on
// the tiled product, 4-bit, r = 16, us.
// Gated forward, two rounds of its tiles at least.  2048 rows, N = 11008, K = 64, 512, 2048, 8192: 59 and 62, 98 and 103, 213 and 228, 725 and
// 749; 4096 rows 102 and 115, 175 and 198, 397 and 450, 1315 and 1490; 4096 rows, N = 4096: 46 and 46, 73 and 74, 148 and 164, 479 and 537.
// At the border, 1536 rows, N = 11008 (two rounds and four tiles), K = 512, 1024, 2048, 4096, 8192: 95 and 88, 129 and 120, 188 and 189, 297 and
// 306, 574 and 615.  Less than two rounds: 2048 rows, N = 4096, K = 512, 1024, 2048, 4096, 8192 45 and 39, 57 and 53, 83 and 84, 136 and 135,
// 257 and 270; 1024 rows, N = 11008, K = 4096 224 and 213.
// Backward, a contraction of 8192 at least, under a mask and without one.  Gated, K = 4096, rows 1536, 2048, 4096: N = 4096 242 and 251, 272 and
// 277, 438 and 424 (214 and 244, 248 and 269, 396 and 403); N = 5632 350 and 370 at 2048, 568 and 567 at 4096; N = 11008 511 and 565 at 1536,
// 959 and 997 at 4096.  Layer, 2048 rows, N x K: 8192 x 4096 208 and 230, 11008 x 4096 265 and 293; 4096 x 4096 157 and 136, 4096 x 11008 333
// and 303, 1024 x 1024 80 and 38.
// Not where the input gradient's tiles fill most of one round and no second one: there the tiled product has 256 x 256 tiles on every CU
// too, and the copy saves it little up to 2048 rows.  Layer, 8192 x 8192, 1536, 1800 and 2048 rows (192 and 256 tiles): 292 and 262, 327 and 304, 330 and
// 310 (264 and 256, 307 and 297, 311 and 303); gated N = 4096, K = 8192 379 and 333, 417 and 379, 422 and 388.  But 2048 rows of 8192 x 5632 (176
// tiles) 263 and 312, of 8192 x 11008 (344) 474 and 479, 3500 rows of 8192 x 4096 403 and 424, 4096 rows of it (256) 305 and 314.
constexpr int64_t kDenseRows = 1536;

DensePlan dense_plan(int64_t M, int64_t NO, int64_t KC, bool gated) {
  DensePlan p{};
  p.ntiles = (int)((NO + (gated ? 127 : 255)) / (gated ? 128 : 256));
  const int64_t total = (M + 255) / 256 * p.ntiles, rest = total % kCus;
  // (32-bit offsets: 256 rows of x or of the weight stay below 2^31 bytes)
  const bool round = M <= 2048 && total >= 192 && total <= kCus;
  p.ok = M >= kDenseRows && (gated ? total >= 512 : KC >= 8192 && total >= 96 && !round) && KC < (int64_t)1 << 21 && total < INT_MAX - 256;
  p.whole = (int)total;
  p.splits = 1;
  const int64_t steps = (KC + 63) / 64, sp = rest > 0 ? std::min({(int64_t)4, kCus / rest, steps / 16}) : 1;
  if (sp >= 2) {
    p.whole = (int)(total - rest);
    p.rest = (int)rest;
    p.splits = (int)sp;
  }
  return p;
}

hipError_t launch_dense_weight(const DenseWeight& w, bool tr, const Levels& lv, hipStream_t s) {
  if (w.K % 64 != 0 || (tr && w.rows % 8 != 0)) return hipErrorInvalidValue;
  if (tr) {
    const int64_t tiles = (w.rows + 127) / 128;
    const dim3 grid((unsigned)tiles, (unsigned)std::max<int64_t>(1, std::min<int64_t>(w.K / 64, kLaunchBlocks / tiles)));
    switch (w.bits) {
      case 2: hipLaunchKernelGGL(k_dense_weight_tr<2>, grid, dim3(256), 0, s, w, lv); break;
      case 3: hipLaunchKernelGGL(k_dense_weight_tr<3>, grid, dim3(256), 0, s, w, lv); break;
      case 4: hipLaunchKernelGGL(k_dense_weight_tr<4>, grid, dim3(256), 0, s, w, lv); break;
      default: hipLaunchKernelGGL(k_dense_weight_tr<8>, grid, dim3(256), 0, s, w, lv); break;
    }
  } else {
    const dim3 grid(grid_of(w.rows * w.K / 8));
    switch (w.bits) {
      case 2: hipLaunchKernelGGL(k_dense_weight<2>, grid, dim3(256), 0, s, w, lv); break;
      case 3: hipLaunchKernelGGL(k_dense_weight<3>, grid, dim3(256), 0, s, w, lv); break;
      case 4: hipLaunchKernelGGL(k_dense_weight<4>, grid, dim3(256), 0, s, w, lv); break;
      default: hipLaunchKernelGGL(k_dense_weight<8>, grid, dim3(256), 0, s, w, lv); break;
    }
  }
  return hipGetLastError();
}

hipError_t launch_dense_adapter(const DenseAdapter& a, hipStream_t s) {
  hipLaunchKernelGGL(k_dense_xt, dim3(grid_of((int64_t)a.halves * a.nb * a.M * 4)), dim3(256), 0, s, a);
  hipLaunchKernelGGL(k_dense_wt, dim3(grid_of((int64_t)a.halves * a.nb * a.rows * 4)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_dense(const DenseArgs& a, bool gated, hipStream_t s) {
  if (a.KC % 8 != 0 || (!gated && a.drop.thr > 0 && a.NO % 8 != 0)) return hipErrorInvalidValue;
  if (gated) return launch_dense_k<DENSE_GATED>(a, s);
  if (a.drop.thr > 0 && a.nb > 0) return launch_dense_k<DENSE_DROP>(a, s);
  return launch_dense_k<DENSE_PLAIN>(a, s);
}

}  // namespace qlr
