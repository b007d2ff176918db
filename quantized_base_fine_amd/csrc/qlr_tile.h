// Tiled matrix product over ranges of rows: the core of the expert products
// (rows grouped by expert, one stacked coded weight) and of the 8-bit-integer
// product (one range, both operands int8).
//
//   KIND TILE_I8    y = (sum_k xq wq) sx[m] sw[n]          (+ adapter)
//   KIND TILE_CODED y[m] = x[m] W'_e^T, e the row's expert  (+ adapter)
//   KIND TILE_TR    y[m] = x[m] W'_e (x = dy, y = dx)       (+ adapter)
//
// Tiling.  A workgroup of 8 waves owns BM rows x BN columns (256 x 256 down to 64
// x 128), divided among WM x WN waves in 32 x 32 MFMA tiles.  A step contracts 128 bytes of each row of x: 64 bf16 or 128
// int8 elements.  MFMA operands: A = weight rows, B = x rows (32x32x16 bf16 or
// 32x32x32 int8), so a lane's results are 4 neighbouring columns of one output
// row and the epilogue stages whole 8- or 16-byte pieces.
//
// Pipeline.  LDS buffers of BM + BN rows of 128 bytes, 16-byte chunks
// XOR-swizzled by row (swz) so that fragment reads and tile writes are free of
// bank conflicts.  While step k is multiplied, x (and int8 weights) of a later step come
// into another buffer by direct loads, and the codes of step k + 1, loaded into registers
// before, are dequantized to bf16 between the products (32 or 16 codes per thread and
// step); one barrier ends the step.  Each weight is dequantized once per tile.  The
// first products of a step wait for their fragments only: with addresses and the level
// table before them, mid-size products took 3 to 7 % longer.
//
// What bounds it (counters at the sizes named): the 256 x 256 tiles keep the matrix pipes busy
// 53 % of the cycles of 8192 x 4096 x 4096 in 8 ranges with 4-bit codes (1.03 PFLOP/s over the 512 tiles; the same loop on
// zeros runs a step in 1.3 us, on random values in 1.8: the clock falls with the
// power) and 50 % of those of the transposed product; the vector units are busy 37 % with the codes.
// The smaller tiles spend more on the codes than on the products: 128 x 128 ones on the last 64 tiles of
// that call keep the vector units busy 41 % and the matrix pipes 25 %, 64 x 128 ones on 777 rows in 64 ranges of
// 1408 x 2048 (3-bit, transposed) 50 and 19 %; the rest is waiting at the barriers.
//
// Rounding.  A coded weight enters rounded to bf16 (half a step, 2^-8 of it), as in the prefill GEMM: a second bf16 part would
// double the matrix work and the weight's LDS, the tiles' two busiest parts.  Against 64 bits a bf16 result is off by 2.3e-3 in
// relative 2-norm, of which its own rounding is 1.7e-3; a float32 weight gives 1.7e-3.
//
// Adapter.  t = x A_e^T (float32 partial sums) enters after the last step as
// blocks of 32 adapter columns: the x side holds [hi(s t) | lo(s t)] (two bf16
// parts, about 16 significant bits of s t, see split_rest), the weight side [B | B].
//
// Ranges.  Expert e's rows are [offsets[e], offsets[e + 1]); every offset is
// clamped into [0, M] and to its predecessor, so no offset can lead out of
// bounds.  Each workgroup finds its tile by a wave scan over the experts' tile
// counts; workgroups past the last tile exit before any barrier.
#pragma once

#include <algorithm>
#include <climits>
#include <type_traits>

#include "qlr_dequant.h"
#include "qlr_internal.h"

namespace qlr {

enum { TILE_I8 = 0, TILE_CODED = 1, TILE_TR = 2 };

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

// Rows [a, b) of expert e, clamped.
__device__ __forceinline__ void expert_range(const int32_t* offsets, int e, int M, int& a, int& b) {
  a = min(max(offsets[e], 0), M);
  b = max(a, min(max(offsets[e + 1], 0), M));
}

// 256 x 256 tiles run one to a CU.  A last round of at most kRestMax of them would
// leave most of the 256 CUs idle for a whole tile's time: those tiles are
// run as 128 x 128 ones (two to a CU) instead: the last 80 of 336 tiles of a 4096 x 4096 transposed product take 58 us so, as
// long as a round of 256 x 256 ones takes 122; at 144 tiles, 576 quarters on the 512 places, the two meet.  Returns the
// tiles that stay.
constexpr int kCus = 256, kRestMax = 144;
// Tile order.  The 32 tiles that an XCD works on at a time cover kGroupM row
// tiles x 32 / kGroupM column tiles, which share its L2: row by row (1 x 32), the int8
// product of 2048 x 11008 x 4096 read 293 MB through the fabric (4.3 TB/s, its
// bound) and took 149 us with its other launches; in blocks of 8 x 4 it read 193 MB and took 135.
constexpr int kGroupM = 8;
__host__ __device__ __forceinline__ int tile_split(int total) {
  const int rest = total % kCus;
  return total > kCus && rest <= kRestMax ? total - rest : total;
}

// Sum over the lanes up to this one.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // rows of 16 lanes: shifts by 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lane 15 of rows 0 and 2 to rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31 to rows 2 and 3
  return v;
}

// 64 ranges of a scan, one to a lane: first and end row, tiles of BM rows (0 of a range of at most min_rows rows), and the
// tiles up to it.
struct ScanChunk { int a, b, nt, inc; };
__device__ __forceinline__ ScanChunk scan_chunk(const int32_t* offsets, int E, int M, int min_rows, int BM, int e) {
  ScanChunk c{0, 0, 0, 0};
  if (e < E) {
    if (offsets) expert_range(offsets, e, M, c.a, c.b);
    else c.b = M;
  }
  c.nt = c.b - c.a > min_rows ? (c.b - c.a + BM - 1) / BM : 0;
  c.inc = wave_scan(c.nt);
  return c;
}

// Tiles of BM rows over the ranges holding more than min_rows rows: tile_count
// returns their number and the first chunk of the scan, tile_find the expert of tile `want` and its
// first and end row (as they are given if there is none).  Called by whole waves.
__device__ __forceinline__ int tile_count(const int32_t* offsets, int E, int M, int min_rows, int BM, ScanChunk& c0) {
  const int lane = threadIdx.x & 63;
  c0 = scan_chunk(offsets, E, M, min_rows, BM, lane);
  int total = __builtin_amdgcn_readlane(c0.inc, 63);
  for (int e0 = 64; e0 < E; e0 += 64)
    total += __builtin_amdgcn_readlane(scan_chunk(offsets, E, M, min_rows, BM, e0 + lane).inc, 63);
  return total;
}
__device__ __forceinline__ void tile_find(const int32_t* offsets, int E, int M, int min_rows, int BM, const ScanChunk& c0,
                                          int want, int& e_out, int& row0, int& row_end) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  ScanChunk c = c0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    if (e0 > 0) c = scan_chunk(offsets, E, M, min_rows, BM, e0 + lane);
    const int last = __builtin_amdgcn_readlane(c.inc, 63);
    if (want < before + last) {
      const uint64_t hit = __ballot(before + c.inc > want);
      const int src = __ffsll((unsigned long long)hit) - 1;  // the first expert whose tiles reach past `want`
      e_out = e0 + src;
      row0 = __builtin_amdgcn_readlane(c.a, src) + (want - before - __builtin_amdgcn_readlane(c.inc - c.nt, src)) * BM;
      row_end = __builtin_amdgcn_readlane(c.b, src);
      return;
    }
    before += last;
  }
}

// A workgroup's part of the rest: the 128 x 128 quarters of the 256 x 256 tiles split .. total - 1
// that hold a row and a column, counted through (workgroups that find nothing to do must come last: among the
// others they would leave some CUs two workgroups and others none, 80 us instead of 64 for a 4096 x 4096 backward of 8
// ragged ranges).  ntiles: column tiles of 256; ncols: of 128; half: kRestRows words of LDS for each wave.  Returns the
// tile, or -1.  c: the first chunk of the scan of tiles of 256 rows.  Called by whole waves.
constexpr int kRestRows = kRestMax + kGroupM;  // at most that many row tiles have tiles in the rest
__device__ __forceinline__ int rest_tile(const int32_t* offsets, int E, int M, int min_rows, ScanChunk c, int split, int total,
                                         int ntiles, int ncols, uint32_t* half, int& row_half, int& col_half) {
  const int lane = threadIdx.x & 63;
  const int lo = split / (kGroupM * ntiles) * kGroupM, mt_total = total / ntiles;
  for (int i = lane; i < kRestRows; i += 64) half[i] = 2;
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    if (e0 > 0) c = scan_chunk(offsets, E, M, min_rows, 256, e0 + lane);
    const int at = before + c.inc - 1 - lo;  // the range's last row tile
    if (c.nt > 0 && c.b - c.a - (c.nt - 1) * 256 <= 128 && at >= 0 && at < kRestRows) half[at] = 1;
    before += __builtin_amdgcn_readlane(c.inc, 63);
  }
  __builtin_amdgcn_wave_barrier();
  // quarters of a lane's tiles, the tile's row and column halves
  constexpr int kPer = (kRestMax + 63) / 64;
  int cnt[kPer], rows[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int big = split + kPer * lane + i;
    cnt[i] = rows[i] = 0;
    if (big < total) {
      int row = 0, in = big - lo * ntiles;  // the group's first row tile, from lo, and the place in the group
      for (; in >= kGroupM * ntiles; in -= kGroupM * ntiles) row += kGroupM;
      const uint32_t gm = (uint32_t)min(kGroupM, mt_total - lo - row), col = (uint32_t)in / gm;
      rows[i] = (int)half[row + in - (int)(col * gm)];
      cnt[i] = rows[i] * (2 * (int)col + 1 < ncols ? 2 : 1);
    }
    sum += cnt[i];
  }
  const int inc = wave_scan(sum), all = __builtin_amdgcn_readlane(inc, 63), per = (all + 7) / 8, loc = (int)(blockIdx.x >> 3);
  const int want = (int)(blockIdx.x & 7) * per + loc;  // each XCD a contiguous range
  if (loc >= per || want >= all) return -1;
  int first = inc - sum, tile = -1, q = 0, nr = 1;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (want >= first && want < first + cnt[i]) {
      tile = split + kPer * lane + i;
      q = want - first;
      nr = rows[i];
    }
    first += cnt[i];
  }
  const int src = __ffsll((unsigned long long)__ballot(tile >= 0)) - 1;
  q = __builtin_amdgcn_readlane(q, src);  // 0 .. 3
  row_half = __builtin_amdgcn_readlane(nr, src) == 2 ? q & 1 : 0;
  col_half = __builtin_amdgcn_readlane(nr, src) == 2 ? q >> 1 : q;
  return __builtin_amdgcn_readlane(tile, src);
}

template <int KIND, int BITS, int BM, int BN>
struct TileLds {
  static constexpr uint32_t kX = BM * 128, kW = BN * 128;
  static constexpr uint32_t kTabBytes = (KIND == TILE_I8 || BITS == 4) ? 0
                                        : BITS == 8                    ? 256 * 16 * 4
                                                                       : PairTableF32<BITS>::kBytes;
  // Buffers.  Two; the 64 x 128 tiles, which run few to a CU and have little work to hide a load behind, have more: the
  // integer one three of each operand (333 x 5003 x 4096: 23.1 us, with two 28.9), the coded ones four of x (input
  // gradient of 777 rows in 64 ranges, 3-bit: 50 us, with two 57).  A third for the 128 x 128 tiles gained nothing.
  static constexpr int kXBufs = BM > 64 ? 2 : KIND == TILE_I8 ? 3 : 4, kWBufs = KIND == TILE_I8 ? kXBufs : 2;
  static_assert(BM != 128 || kW >= 8 * kRestRows * 4, "rest_tile's words overlay a buffer");
  static_assert(kXBufs * kX + kWBufs * kW + kTabBytes <= 160 * 1024, "LDS budget");
};

// v as a sum of bf16 parts for products on bf16 MFMA: v becomes the next part (its low 16 bits zero), the result the rest
// (16 of float32's 24 significant bits at most).  The part is the largest one below v in magnitude, so the parts have v's sign and
// none but a zero's is zero: their products add up to v's own with an infinity on either side too (Inf B = hi B + Inf B, v Inf =
// hi Inf + lo Inf).  The nearest part would leave a rest of either sign or none, whose products with an infinity, and an
// infinite v's rest Inf - Inf, are NaN; and it rounds the largest values to infinity.  The rest is that of the rounded v, not
// contracted with a product that formed v.
__device__ __forceinline__ float split_rest(float& v) {
#pragma clang fp contract(off)
  const float hi = __uint_as_float((__float_as_uint(v) - (v != 0.0f ? 1u : 0u)) & 0xFFFF0000u), rest = v - hi;
  v = hi;
  return rest;
}

__device__ __forceinline__ f32x16_t tile_mfma(u32x4_t a, u32x4_t b, f32x16_t c) {
  return mfma32x32x16(as_bf16x8(a), as_bf16x8(b), c);
}
__device__ __forceinline__ f32x16_t tile_mfma_i8(u32x4_t a, u32x4_t b, f32x16_t c) {
  return __builtin_bit_cast(
      f32x16_t, __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b),
                                                      __builtin_bit_cast(i32x16_t, c), 0, 0, 0));
}

// Buffer resource over n bytes from p, its words made scalar (a resource in vector
// registers would turn every load into a loop over the lanes' values).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rsrc(const void* p, uint32_t n) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a), hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uint64_t)lo | ((uint64_t)hi << 32)), (short)0,
                                           (int)__builtin_amdgcn_readfirstlane(n), 0x00020000);
}

// block0: the launch's first workgroup among the call's (a multiple of 8); before the levels, whose kilobyte lies
// in cache lines of its own (behind them, its load took 0.3 us of 333 x 5003 x 4096)
template <int KIND, int BITS, int BM, int BN>
__global__ __launch_bounds__(512, BM * BN <= 128 * 128 ? 4 : 1) void k_tile(TileArgs P, int block0, Levels lv) {
  using L = TileLds<KIND, BITS, BM, BN>;
  constexpr int WM = (BN == 256 || BM == 64) ? 2 : 4, WN = 8 / WM;
  constexpr int MT = BM / WM / 32, NT = BN / WN / 32;  // MFMA tiles of a wave
  constexpr int XL = BM / 64;  // direct loads of x per wave and step
  constexpr int WL = BN / 64;  // the same of an int8 weight; 8-code parts of a coded one per thread
  constexpr int CPT = BN / 8;  // codes per thread and step
  // x and int8 weights are loaded straight into LDS.  The buffers are separate LDS variables, so that the compiler knows
  // that the fragment reads of one do not touch the loads in flight into the other and does not wait for them.
  __shared__ __attribute__((aligned(16))) char sX0[L::kX], sX1[L::kX], sW0[L::kW], sW1[L::kW];
  __shared__ __attribute__((aligned(16))) char sX2[L::kXBufs > 2 ? L::kX : 16], sX3[L::kXBufs > 3 ? L::kX : 16];
  __shared__ __attribute__((aligned(16))) char sW2[L::kWBufs > 2 ? L::kW : 16];
  __shared__ __attribute__((aligned(16))) char sT[L::kTabBytes ? L::kTabBytes : 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 31, h = lane >> 5;
  auto st16 = [](char* p, u32x4_t v) { *reinterpret_cast<u32x4_t*>(p) = v; };
  auto ld16 = [](const char* p) { return *reinterpret_cast<const u32x4_t*>(p); };
  auto ld_tr = [](char* p) -> u16x4_t {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)p);
  };

  // ---- which tile.  Workgroup b runs on XCD b % 8; each XCD takes a contiguous range of tiles.
  // With P.rest the tiles are counted in 256 x 256 ones and those of a last partial
  // round are left to the 128 x 128 kernel (tile_split): this kernel takes either part.
  int e = 0, row0 = 0, row_end = (int)P.M, tile_n;
  {
    constexpr int kBig = 256;
    const bool sub = BM == 128 && P.rest;  // the 128 x 128 kernel on the rest of the 256 x 256 tiles
    const int step_m = sub ? kBig : BM, ntiles = sub ? (P.ntiles + kBig / BN - 1) / (kBig / BN) : P.ntiles;
    const int ranges = P.offsets ? P.experts : 1;
    ScanChunk c0;
    const int mt_total = tile_count(P.offsets, ranges, (int)P.M, P.min_rows, step_m, c0);
    const int total = mt_total * ntiles;
    const int split = P.rest ? tile_split(total) : total;
    int big, row_half = 0, col_half = 0;
    if (sub) {
      // (its words lie in a buffer that no wave writes before the first barrier, which every wave reaches after reading them)
      big = rest_tile(P.offsets, ranges, (int)P.M, P.min_rows, c0, split, total, ntiles, P.ntiles,
                      reinterpret_cast<uint32_t*>(sW1) + wave * kRestRows, row_half, col_half);
      if (big < 0) return;  // (as below)
    } else {
      const int per = (split + 7) / 8, loc = (block0 + (int)blockIdx.x) >> 3;
      big = (int)(blockIdx.x & 7) * per + loc;
      if (loc >= per || big >= split) return;  // the whole workgroup, before any barrier
    }
    // order: blocks of kGroupM row tiles, their column tiles one after the other, row tiles innermost
    const int grp = big / (kGroupM * ntiles), in = big - grp * kGroupM * ntiles;
    const int gm = min(kGroupM, mt_total - grp * kGroupM);
    const int mi = grp * kGroupM + in % gm;
    tile_n = in / gm;
    row_end = 0;
    tile_find(P.offsets, ranges, (int)P.M, P.min_rows, step_m, c0, mi, e, row0, row_end);
    if (sub) {
      row0 += row_half * BM;
      tile_n = tile_n * (kBig / BN) + col_half;
      if (row0 >= row_end || tile_n >= P.ntiles) return;
    }
    // (scalar: a buffer resource needs scalar words)
    e = __builtin_amdgcn_readfirstlane(e);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    row_end = __builtin_amdgcn_readfirstlane(row_end);
    tile_n = __builtin_amdgcn_readfirstlane(tile_n);
  }
  const int mrows = min(BM, row_end - row0);
  const int64_t N = P.N, K = P.K;
  const int64_t NO = KIND == TILE_TR ? K : N;            // output columns
  const int n0 = tile_n * BN;
  const uint32_t kbytes = (uint32_t)(KIND == TILE_I8 ? K : KIND == TILE_TR ? 2 * N : 2 * K);  // bytes of one x row
  const int nsteps = (int)((kbytes + 127) / 128);

  if constexpr (L::kTabBytes > 0) {
    float* sL = reinterpret_cast<float*>(sX0);
    stage_levels<1 << BITS>(lv, sL);
    __syncthreads();
    float* tab = reinterpret_cast<float*>(sT);
    if constexpr (BITS == 8) {
      for (int i = tid; i < 256 * 16; i += 512) tab[i] = sL[i >> 4];
    } else {
      constexpr int NL = 1 << BITS;
      for (int i = tid; i < PairTableF32<BITS>::kEntries * 32; i += 512) {
        const int en = i >> 5;
        tab[2 * i] = sL[en & (NL - 1)];
        tab[2 * i + 1] = sL[en >> BITS];
      }
    }
    __syncthreads();
  }

  // ---- x, and int8 weights: direct loads.  Load j of the J of wave w fills tile rows 8 (J w + j) .. + 7 (1 KB, lane l at
  // byte 16 l: row l / 8, slot l % 8), so lane l reads the chunk that the swizzle puts at its slot; that depends on the load
  // through (J w + j) % 2 only.  Rows past the range and chunks past the row's end read zero.
  const char* xbase = reinterpret_cast<const char*>(P.x) + (int64_t)row0 * kbytes;
  const __amdgpu_buffer_rsrc_t xr = tile_rsrc(xbase, (uint32_t)mrows * kbytes);
  const uint32_t t8 = (uint32_t)lane >> 3;
  const uint32_t dch0 = 16u * (((uint32_t)lane & 7u) ^ swz(t8)), dch1 = 16u * (((uint32_t)lane & 7u) ^ swz(t8 + 8u));
  const uint32_t dchw = (wave & 1) ? dch1 : dch0;
  auto direct = [&](__amdgpu_buffer_rsrc_t rsrc, char* dst, int k, auto loads) {
    constexpr int J = decltype(loads)::value;
    const uint32_t kb = (uint32_t)k * 128u;
    uint32_t off[2];
#pragma unroll
    for (int p = 0; p < (J < 2 ? J : 2); ++p) {
      const uint32_t chb = J == 1 ? dchw : p ? dch1 : dch0;
      uint32_t o = ((uint32_t)(8 * J * wave) + t8) * kbytes + kb + chb;
      asm volatile("" : "+v"(o));  // keep the select a select (no branch around the loads)
      // (a chunk past the row's end: an offset past every range, rows of at most 2^21 bytes added)
      off[p] = kb + chb < kbytes ? o : 0x80000000u;
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (void __attribute__((address_space(3)))*)(dst + (J * wave + j) * 1024), 16,
                                               off[j & 1] + (uint32_t)j * 8u * kbytes, 0, 0, 0);
  };
  constexpr std::integral_constant<int, XL> xloads{};
  constexpr std::integral_constant<int, WL> wloads{};

  // ---- weight loads
  // I8: as x, the rows from n0 (rows past N zero).
  // CODED: thread = row tid / TPB, codes [CPT dh, + CPT) of the step's block (TPB threads share a block).
  // TR: thread = weight row 64 k + tid / 8, codes [CPT dh, + CPT) of block column n0 / 64 + bq.
  struct Ws {
    Codes32<BITS> c;
    uint8_t q8;
    float sc;
  };
  const int wrows = (int)min<int64_t>(BN, N - n0);
  const char* wbase = reinterpret_cast<const char*>(P.w) + (int64_t)n0 * K;
  const __amdgpu_buffer_rsrc_t wr = tile_rsrc(KIND == TILE_I8 ? wbase : nullptr, KIND == TILE_I8 ? (uint32_t)wrows * kbytes : 0u);
  constexpr int TPB = 64 / CPT;
  const int rr = KIND == TILE_TR ? (tid >> 3) : tid / TPB, dh = tid % TPB, bq = KIND == TILE_TR ? (tid & 7) / TPB : 0;
  // Addresses of a coded weight's blocks: a scalar part (the tile's first block and the step) plus a 32-bit part
  // per lane, fixed for all steps but TR's last, whose rows past N read row N - 1 with scale 0.
  const int64_t nbK = K >> 6;
  const int64_t gb = KIND == TILE_TR ? (int64_t)e * N * nbK + (n0 >> 6) : ((int64_t)e * N + n0) * nbK;
  bool wv = true, wv_last = true;
  uint32_t lb = 0, lb_last = 0;  // the lane's block, relative
  if constexpr (KIND == TILE_CODED) {
    wv = wv_last = n0 + rr < N;
    lb = lb_last = (uint32_t)(min<int64_t>(rr, N - 1 - n0) * nbK);
  } else if constexpr (KIND == TILE_TR) {
    wv = (n0 >> 6) + bq < nbK;
    const uint32_t col = (uint32_t)min<int64_t>(bq, nbK - 1 - (n0 >> 6));
    const int64_t nl = N - 64 * (int64_t)(nsteps - 1);  // rows of the last step
    wv_last = wv && rr < nl;
    lb = (uint32_t)((int64_t)rr * nbK) + col;
    lb_last = (uint32_t)(min<int64_t>(rr, nl - 1) * nbK) + col;
  }
  const uint8_t* const wb8 = P.w + (KIND == TILE_I8 ? 0 : gb * (8 * BITS));
  const uint8_t* const qb8 = KIND == TILE_I8 ? nullptr : P.q8 + gb;
  const float* const cb = KIND == TILE_I8 ? nullptr : P.cst + (gb >> 8);
  const uint32_t gl = (uint32_t)(gb & 255);
  uint32_t wst[WL];
#pragma unroll
  for (int q = 0; q < WL; ++q) {
    if constexpr (KIND == TILE_TR)
      wst[q] = (uint32_t)(bq >> 1) * 16384u + (uint32_t)rr * 256u +
               (tr_chunk((uint32_t)(8 * (bq & 1) + WL * dh + q), (uint32_t)rr) << 4);
    else
      wst[q] = (uint32_t)rr * 128u + ((((uint32_t)(WL * dh + q)) ^ swz((uint32_t)rr & 15u)) << 4);
  }
  const uint32_t tl = BITS == 8 ? 4u * (lane & 15) : 8u * fr;  // the lane's copy of the level table
  const TabPtr tab{sT + tl};
  auto load_w = [&](int k, Ws& s) {
    if constexpr (KIND != TILE_I8) {
      const int kk = min(k, nsteps - 1);
      const bool last = kk == nsteps - 1;  // (scalar)
      const int64_t ks = KIND == TILE_TR ? 64 * (int64_t)kk * nbK : kk;  // the step's first block
      const uint32_t l = last ? lb_last : lb;
      const uint8_t* const wk = wb8 + ks * (8 * BITS);
      if constexpr (CPT == 32) s.c = load_codes32<BITS>(wk + l * (uint32_t)(8 * BITS) + dh * (4 * BITS));
      else s.c = load_codes16<BITS>(wk + l * (uint32_t)(8 * BITS), dh);
      s.q8 = (qb8 + ks)[l];
      s.sc = (cb + (ks >> 8))[(gl + (uint32_t)(ks & 255) + l) >> 8];
    }
  };
  // The scale of step k's weights, 0 outside the weight.  (Selected here, where it is used: a select next to the loads
  // would wait for them.)
  auto scale_of = [&](const Ws& s, int k) {
    return KIND != TILE_I8 && (k < nsteps - 1 ? wv : wv_last) ? (float)s.q8 * s.sc : 0.0f;
  };
  // part I (0 .. WL - 1) of the thread's coded weights, dequantized, into buffer buf
  auto store_w = [&](const Ws& s, const Lut4& lut, float ap, auto part, char* buf) {
    constexpr int I = decltype(part)::value;
    if constexpr (KIND != TILE_I8) {
      uint32_t o[4];
      if constexpr (BITS == 4) {
        lut4_word(s.c.w[I], lut, o);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 p = level_pair<BITS>(s.c, 4 * I + j, tab);
          o[j] = cvt_pk_bf16(p.x * ap, p.y * ap);
        }
      }
      st16(buf + wst[I], u32x4_t{o[0], o[1], o[2], o[3]});
    }
  };
  // the same in two halves, for the widths whose levels come from LDS: the lookups before a run of products, the rest after
  constexpr bool kLook = KIND != TILE_I8 && BITS != 4;
  float2 look[4];
  auto lookup_w = [&](const Ws& s, auto part) {
    if constexpr (kLook) {
#pragma unroll
      for (int j = 0; j < 4; ++j) look[j] = level_pair<BITS>(s.c, 4 * decltype(part)::value + j, tab);
    }
  };
  auto finish_w = [&](float ap, auto part, char* buf) {
    if constexpr (kLook) {
      u32x4_t o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = cvt_pk_bf16(look[j].x * ap, look[j].y * ap);
      st16(buf + wst[decltype(part)::value], o);
    }
  };
  // ---- fragments: MFMA step s (0..3) of a buffer, row fr (+ 32 per tile), chunk 2 s + h
  const int mh = wave / WN, nh = wave % WN;
  uint32_t xb[4], wb[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const uint32_t fo = (uint32_t)(fr * 128) + ((((uint32_t)(2 * s + h)) ^ swz((uint32_t)fr & 15u)) << 4);
    xb[s] = (uint32_t)(mh * (BM / WM) * 128) + fo;
    wb[s] = (uint32_t)(nh * (BN / WN) * 128) + fo;
  }
  uint32_t tbo[NT];
  {
    const uint32_t g = (uint32_t)lane >> 4, sp = (uint32_t)lane & 15u;
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      const uint32_t col = (uint32_t)(nh * (BN / WN) + 32 * c);
      const uint32_t chunk = ((col & 127u) >> 3) + 2u * (g & 1u) + ((sp >> 1) & 1u);
      tbo[c] = (col >> 7) * 16384u + (8u * h + (sp >> 2)) * 256u + (tr_chunk(chunk, sp >> 2) << 4) +
               8u * (sp & 1u);
    }
  }
  u32x4_t fx[2][MT], fw[2][NT];
  auto read_frags = [&](const char* bx, char* bw, int s, int slot) {
#pragma unroll
    for (int i = 0; i < MT; ++i) fx[slot][i] = ld16(bx + xb[s] + 4096u * i);
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      if constexpr (KIND == TILE_TR) {
        char* const ad = bw + tbo[c] + 4096u * s;
        const u16x4_t lo = ld_tr(ad), hi = ld_tr(ad + 1024u);
        fw[slot][c] = u32x4_t{__builtin_bit_cast(uint2, lo).x, __builtin_bit_cast(uint2, lo).y,
                              __builtin_bit_cast(uint2, hi).x, __builtin_bit_cast(uint2, hi).y};
      } else {
        fw[slot][c] = ld16(bw + wb[s] + 4096u * c);
      }
    }
  };
  f32x16_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][c][v] = 0.0f;  // also the integer zero
  auto mfmas = [&](int slot) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        if constexpr (KIND == TILE_I8) acc[i][c] = tile_mfma_i8(fw[slot][c], fx[slot][i], acc[i][c]);
        else acc[i][c] = tile_mfma(fw[slot][c], fx[slot][i], acc[i][c]);
      }
  };

  // ---- the steps
  // x (and int8 weights) of step k are loaded kAhead steps before, codes kSets steps before.
  constexpr int kAhead = L::kXBufs - 1, kSets = L::kXBufs == 4 ? 4 : 2;
  Ws wa, wb_, wc, wd;
  direct(xr, sX0, 0, xloads);
  if constexpr (KIND == TILE_I8) direct(wr, sW0, 0, wloads);
  if constexpr (kAhead > 1) {
    direct(xr, sX1, 1, xloads);
    if constexpr (KIND == TILE_I8) direct(wr, sW1, 1, wloads);
  }
  if constexpr (kAhead > 2) direct(xr, sX2, 2, xloads);
  if constexpr (KIND != TILE_I8) {
    load_w(0, wa);
    // (loads in the steps' order.  The loop's head waits for all loads, or all but one to three, all the same: in one of four
    // steps of the coded 64 x 128 tiles what was loaded ahead has to have arrived)
    __builtin_amdgcn_sched_barrier(0);
    load_w(1, wb_);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kSets == 4) {
      load_w(2, wc);
      __builtin_amdgcn_sched_barrier(0);
      load_w(3, wd);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (CPT == 16) place_codes16<BITS>(wa.c, dh);
    Lut4 lut{};
    const float ap = scale_of(wa, 0);
    if constexpr (BITS == 4) lut = make_lut4(lv, ap);
    store_w(wa, lut, ap, std::integral_constant<int, 0>{}, sW0);
    store_w(wa, lut, ap, std::integral_constant<int, 1>{}, sW0);
    if constexpr (WL == 4) {
      store_w(wa, lut, ap, std::integral_constant<int, 2>{}, sW0);
      store_w(wa, lut, ap, std::integral_constant<int, 3>{}, sW0);
    }
  }
  __syncthreads();
  // The end of a step: every wave's share of the next one is in LDS.  Behind the loads that must have arrived there are those
  // of the kAhead - 1 steps after the next: XL (+ WL) direct loads each and, from the next step's on, at least three of codes,
  // scale and constant (loads return in order).  That count holds while each step issues its loads within the step: keep
  // stops the compiler from moving a memory access past it (the three loads come from three arrays, so they cannot be
  // one), and tests/test_host_tile_waits.py counts the loads in the compiled loops.
  auto keep = [] {
    if constexpr (kAhead > 1) asm volatile("" ::: "memory");
  };
  auto step_barrier = [&] {
    if constexpr (kAhead > 1) {
      constexpr int kOpen = (kAhead - 1) * (XL + (KIND == TILE_I8 ? WL : 0)) + (KIND == TILE_I8 ? 0 : 3 * kAhead);
      static_assert(kOpen < 16, "wait count");
      keep();
      __builtin_amdgcn_s_waitcnt(0x0070 | kOpen);  // and no LDS access open
      __builtin_amdgcn_s_barrier();
      keep();
    } else {
      __syncthreads();
    }
  };
  // Step k multiplies buffers bx, bw while step k + kAhead comes into ox (and ow) by direct loads issued first; the codes of
  // step k + 1, in cur, are dequantized between the products (into ow), and those of step k + kSets loaded into nxt.
  // The first products wait for nothing but their fragments; addresses, the level table and the next codes' loads go between
  // the products.
  auto step = [&](int k, char* bx, char* bw, char* ox, char* ow, Ws& cur, Ws& nxt) {
    __builtin_amdgcn_sched_barrier(0);
    read_frags(bx, bw, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    keep();
    direct(xr, ox, k + kAhead, xloads);
    if constexpr (KIND == TILE_I8) direct(wr, ow, k + kAhead, wloads);
    keep();
    __builtin_amdgcn_sched_barrier(0);
    Lut4 lut{};
    float ap = 0.0f;
    // (opaque from here: the compiler would otherwise start the codes' arithmetic right after their load, a
    // step early, and wait for them there)
    auto pin = [&] {
      if constexpr (KIND != TILE_I8) {
#pragma unroll
        for (int i = 0; i < BITS; ++i) asm volatile("" : "+v"(cur.c.w[i]));
        asm volatile("" : "+v"(cur.sc));
        if constexpr (CPT == 16) place_codes16<BITS>(cur.c, dh);
      }
    };
    if constexpr (kLook) pin();
    auto sub = [&](auto spos) {
      constexpr int S = decltype(spos)::value;
      if constexpr (S < 3) read_frags(bx, bw, S + 1, (S + 1) & 1);
      constexpr bool kPart = WL == 4 || S % 2 == 0;
      constexpr std::integral_constant<int, WL == 4 ? S : S / 2> wpart{};
      if constexpr (kLook && kPart) lookup_w(cur, wpart);
      __builtin_amdgcn_sched_barrier(0);
      mfmas(S & 1);
      if constexpr (S == 0 && KIND != TILE_I8) {
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!kLook) pin();
        ap = scale_of(cur, k + 1);
        if constexpr (BITS == 4) lut = make_lut4(lv, ap);
      }
      if constexpr (kLook && kPart) {
        __builtin_amdgcn_sched_barrier(0);
        finish_w(ap, wpart, ow);
      } else if constexpr (kPart) {
        store_w(cur, lut, ap, wpart, ow);
      }
      if constexpr (S == 1 && KIND != TILE_I8) {
        __builtin_amdgcn_sched_barrier(0);
        keep();
        load_w(k + kSets, nxt);
        keep();
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    sub(std::integral_constant<int, 0>{});
    sub(std::integral_constant<int, 1>{});
    sub(std::integral_constant<int, 2>{});
    sub(std::integral_constant<int, 3>{});
    step_barrier();
  };
  int k = 0;
  if constexpr (kAhead == 2) {
    for (;;) {
      step(k, sX0, sW0, sX2, sW2, wa, wa);
      if (++k >= nsteps) break;
      step(k, sX1, sW1, sX0, sW0, wa, wa);
      if (++k >= nsteps) break;
      step(k, sX2, sW2, sX1, sW1, wa, wa);
      if (++k >= nsteps) break;
    }
  } else if constexpr (kAhead == 3) {
    for (;;) {
      step(k, sX0, sW0, sX3, sW1, wb_, wa);
      if (++k >= nsteps) break;
      step(k, sX1, sW1, sX0, sW0, wc, wb_);
      if (++k >= nsteps) break;
      step(k, sX2, sW0, sX1, sW1, wd, wc);
      if (++k >= nsteps) break;
      step(k, sX3, sW1, sX2, sW0, wa, wd);
      if (++k >= nsteps) break;
    }
  } else {
    for (; k + 1 < nsteps; k += 2) {
      step(k, sX0, sW0, sX1, sW1, wb_, wa);
      step(k + 1, sX1, sW1, sX0, sW0, wa, wb_);
    }
    if (k < nsteps) step(k, sX0, sW0, sX1, sW1, wb_, wa);
  }
  if constexpr (kAhead > 1) {
    __builtin_amdgcn_s_waitcnt(0x0070);  // the loads past the last step too, before the buffers are used again
    __syncthreads();
  }

  // ---- row and column scales of the integer product
  if constexpr (KIND == TILE_I8) {
    float sx[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int m = mh * (BM / WM) + 32 * i + fr;
      sx[i] = P.sx[row0 + min(m, mrows - 1)];
    }
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int n = n0 + nh * (BN / WN) + 32 * c + 8 * (v >> 2) + 4 * h + (v & 3);
        const float sw = P.sw[min<int64_t>(n, N - 1)];
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i][c][v] = (float)__float_as_int(acc[i][c][v]) * sx[i] * sw;
      }
  }

  // ---- adapter blocks (buffer 0 is free: the last barrier has passed)
  if (P.r > 0) {
    const int r = P.r;
    const bool r8 = (r & 7) == 0;
    const u32x4_t zero4 = {0u, 0u, 0u, 0u};
    for (int j0 = 0; j0 < r; j0 += 32) {
      // the weight side's pieces first, so that both sides' loads are on their way together
      constexpr int kAP = BN / 128;
      u32x4_t av[kAP];
#pragma unroll
      for (int u = 0; u < kAP; ++u) {
        const int idx = tid + 512 * u;
        av[u] = zero4;
        if constexpr (KIND == TILE_TR) {  // A[j0 + row][n0 + 8 c ..]
          const int row = idx / (BN / 8);
          const int64_t col = n0 + 8 * (idx % (BN / 8));
          if (j0 + row < r && col < K) av[u] = *reinterpret_cast<const u32x4_t*>(P.ab + ((int64_t)e * r + j0 + row) * K + col);
        } else {  // B[n0 + row][j0 + 8 c ..]
          const int row = idx >> 2, jb = j0 + 8 * (idx & 3);
          if (n0 + row < N && jb < r) {
            const uint16_t* bp = P.ab + ((int64_t)e * N + n0 + row) * r + jb;
            if (r8) {
              av[u] = *reinterpret_cast<const u32x4_t*>(bp);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t lo = jb + 2 * i < r ? bp[2 * i] : 0u, hi = jb + 2 * i + 1 < r ? bp[2 * i + 1] : 0u;
                av[u][i] = lo | (hi << 16);
              }
            }
          }
        }
      }
      // x side: row (idx / 4), adapter columns j0 + 8 (idx % 4) .. + 8
      for (int idx = tid; idx < BM * 4; idx += 512) {
        const int row = idx >> 2, c = idx & 3, jb = j0 + 8 * c;
        float tv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) tv[i] = 0.0f;
        if (row < mrows && jb < r) {
          for (int sp = 0; sp < P.t_splits; ++sp) {
            const float* tq = P.t + ((int64_t)sp * P.M + row0 + row) * r + jb;
            if (r8) {
              const f32x4_t v0 = *reinterpret_cast<const f32x4_t*>(tq), v1 = *reinterpret_cast<const f32x4_t*>(tq + 4);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                tv[i] += v0[i];
                tv[4 + i] += v1[i];
              }
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (jb + i < r) tv[i] += tq[i];
            }
          }
        }
        u32x4_t hv, lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float u0 = P.scale * tv[2 * i], u1 = P.scale * tv[2 * i + 1];
          const float l0 = split_rest(u0), l1 = split_rest(u1);
          hv[i] = (__float_as_uint(u0) >> 16) | (__float_as_uint(u1) & 0xFFFF0000u);
          lo[i] = pack_bf16x2(l0, l1);
        }
        const uint32_t xrow = (uint32_t)row * 128u;
        st16(sX0 + xrow + ((((uint32_t)c) ^ swz((uint32_t)row & 15u)) << 4), hv);
        st16(sX0 + xrow + ((((uint32_t)(4 + c)) ^ swz((uint32_t)row & 15u)) << 4), lo);
      }
      // weight side, twice: [B | B], for A the rows 0..31 and 32..63
#pragma unroll
      for (int u = 0; u < kAP; ++u) {
        const int idx = tid + 512 * u;
        if constexpr (KIND == TILE_TR) {
          const int row = idx / (BN / 8), c = idx % (BN / 8);
          const uint32_t base = (uint32_t)(c >> 4) * 16384u;
          st16(sW0 + base + (uint32_t)row * 256u + (tr_chunk((uint32_t)(c & 15), (uint32_t)row) << 4), av[u]);
          st16(sW0 + base + (uint32_t)(row + 32) * 256u + (tr_chunk((uint32_t)(c & 15), (uint32_t)row) << 4), av[u]);
        } else {
          const int row = idx >> 2, c = idx & 3;
          const uint32_t wrow = (uint32_t)row * 128u;
          st16(sW0 + wrow + ((((uint32_t)c) ^ swz((uint32_t)row & 15u)) << 4), av[u]);
          st16(sW0 + wrow + ((((uint32_t)(4 + c)) ^ swz((uint32_t)row & 15u)) << 4), av[u]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        read_frags(sX0, sW0, s, 0);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int c = 0; c < NT; ++c) acc[i][c] = tile_mfma(fw[0][c], fx[0][i], acc[i][c]);
      }
      __syncthreads();
    }
  }

  // ---- output: staged row-major in LDS, stored in 16-byte pieces
  const int es = P.ydt == DT_F32 ? 4 : 2;
  const bool vec = (NO * es) % 16 == 0;
  const int cpr = BN * es / 16;  // 16-byte pieces of a staged row (a power of two)
  auto put = [&](int row, int c, u32x4_t v) {  // piece c of tile row `row`
    const int64_t col = n0 + c * (16 / es);
    if (col >= NO) return;
    char* dst = reinterpret_cast<char*>(P.y) + ((int64_t)(row0 + row) * NO + col) * es;
    if (vec) {
      *reinterpret_cast<u32x4_t*>(dst) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = v[i];
        if (es == 4) {
          if (col + i < NO) reinterpret_cast<uint32_t*>(dst)[i] = w;
        } else {
          if (col + 2 * i < NO) reinterpret_cast<uint16_t*>(dst)[2 * i] = (uint16_t)w;
          if (col + 2 * i + 1 < NO) reinterpret_cast<uint16_t*>(dst)[2 * i + 1] = (uint16_t)(w >> 16);
        }
      }
    }
  };
  // Each buffer holds rpb rows (of the 64-row tile only the weight's buffers, the others are half as large), their 16-byte
  // pieces XOR-swizzled by the row.  All bf16 rows go at once, the float32 rows of a 256 x 256 tile in two passes.
  constexpr int kBufs = BM == 64 ? 2 : 4;
  auto sbuf = [&](int b) { return kBufs == 2 ? (b ? sW1 : sW0) : b < 2 ? (b ? sX1 : sX0) : (b == 3 ? sW1 : sW0); };
  const int rpb = es == 4 ? 32 : 64;
  const uint32_t rowb = (uint32_t)(BN * es), mask = min(31, cpr - 1);
  for (int first = 0; first < mrows; first += kBufs * rpb) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int tr = mh * (BM / WM) + 32 * i - first;  // the MFMA tile's first row in this pass
      if (tr >= 0 && tr < kBufs * rpb) {
        const uint32_t lr = (uint32_t)((es == 4 ? 0 : tr & 32) + fr);
        char* const st = sbuf(tr / rpb) + lr * rowb;
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t col = (uint32_t)(nh * (BN / WN) + 32 * c + 8 * q);
            const float v0 = acc[i][c][4 * q], v1 = acc[i][c][4 * q + 1], v2 = acc[i][c][4 * q + 2], v3 = acc[i][c][4 * q + 3];
            if (es == 4)
              *reinterpret_cast<f32x4_t*>(st + 16u * ((col / 4 + h) ^ (lr & mask))) = f32x4_t{v0, v1, v2, v3};
            else
              *reinterpret_cast<u32x2v_t*>(st + 16u * ((col / 8) ^ (lr & mask)) + 8u * h) =
                  u32x2v_t{pack_bf16x2(v0, v1), pack_bf16x2(v2, v3)};
          }
      }
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < kBufs; ++b) {
      const int r0 = first + b * rpb, rows = min(rpb, mrows - r0);
      for (int idx = tid; idx < rows * cpr; idx += 512) {
        const int lr = es == 4 ? idx / (BN / 4) : idx / (BN / 8), c = idx & (cpr - 1);
        put(r0 + lr, c, ld16(sbuf(b) + lr * rowb + 16u * ((uint32_t)c ^ ((uint32_t)lr & mask))));
      }
    }
    __syncthreads();
  }
}

// The adapter branch of a few-rows kernel (rows <= 32 of x against
// NR weight rows, NTH threads): the operands are loaded into registers before the weight
// stream and staged in LDS after it, so their latency hides behind it.
//   t: splits x M x r partials in global memory (rows row0 ..), B: rows x r bf16.
// st tells whether the sizes fit (r % 8 == 0 and the pieces a thread can hold);
// otherwise the dot product reads global memory.
template <int NR, int KT, int NTH = 512>
struct FewAdapter {
  static constexpr int kT = KT;  // floats of t staged at most
  static constexpr int kTPieces = (KT / 4 + NTH - 1) / NTH, kBPieces = (NR * 8 + NTH - 1) / NTH;
  static constexpr uint32_t kBytes = kT * 4 + NR * 64 * 2;
  f32x4_t tv[kTPieces];
  u32x4_t bv[kBPieces];
  bool st;

  __device__ __forceinline__ void load(const float* t, int splits, int64_t M, int row0, int rows, const uint16_t* B,
                                       int64_t brow0, int brows, int r) {
    const int tid = threadIdx.x;
    st = r > 0 && r <= 64 && (r & 7) == 0 && splits * rows * r <= kT;
    if (!st) return;
    const int per = rows * r / 4;  // pieces of one split's rows
#pragma unroll
    for (int i = 0; i < kTPieces; ++i) {
      const int p = tid + NTH * i;
      if (p < splits * per)
        tv[i] = *reinterpret_cast<const f32x4_t*>(t + ((int64_t)(p / per) * M + row0) * r + 4 * (p % per));
    }
    const int rp = r >> 3;
#pragma unroll
    for (int i = 0; i < kBPieces; ++i) {
      const int p = tid + NTH * i;
      if (p < NR * rp)
        bv[i] = *reinterpret_cast<const u32x4_t*>(B + (brow0 + min(p / rp, brows - 1)) * r + 8 * (p % rp));
    }
  }
  // called by the whole workgroup; lds: kBytes of it, free after the barrier that the caller has passed
  __device__ __forceinline__ void stage(char* lds, int splits, int rows, int r) {
    if (!st) return;
    const int tid = threadIdx.x;
    float* ts = reinterpret_cast<float*>(lds);
    const int per = rows * r / 4;
#pragma unroll
    for (int i = 0; i < kTPieces; ++i) {
      const int p = tid + NTH * i;
      if (p < splits * per) *reinterpret_cast<f32x4_t*>(ts + 4 * p) = tv[i];
    }
    const int rp = r >> 3;
#pragma unroll
    for (int i = 0; i < kBPieces; ++i) {
      const int p = tid + NTH * i;
      if (p < NR * rp) *reinterpret_cast<u32x4_t*>(lds + kT * 4 + 16 * p) = bv[i];
    }
    __syncthreads();
    if (splits > 1) {  // the split sums, in split order
      for (int i = tid; i < rows * r; i += NTH) {
        float v = 0.0f;
        for (int sp = 0; sp < splits; ++sp) v += ts[sp * rows * r + i];
        ts[i] = v;
      }
      __syncthreads();
    }
  }
  // sum_j t[m][j] B[n][j], m and n relative to the staged rows
  __device__ __forceinline__ float dot(const char* lds, const float* t, int splits, int64_t M, int row0, int m,
                                       const uint16_t* B, int64_t brow0, int n, int r) const {
    float lo = 0.0f;
    if (st) {
      const float* ts = reinterpret_cast<const float*>(lds) + m * r;
      const uint16_t* bs = reinterpret_cast<const uint16_t*>(lds + kT * 4) + n * r;
      for (int j = 0; j < r; j += 8) {
        const u32x4_t b = *reinterpret_cast<const u32x4_t*>(bs + j);
        const f32x4_t t0 = *reinterpret_cast<const f32x4_t*>(ts + j), t1 = *reinterpret_cast<const f32x4_t*>(ts + j + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = b[i];
          const float ta = i < 2 ? t0[2 * i] : t1[2 * i - 4], tb = i < 2 ? t0[2 * i + 1] : t1[2 * i - 3];
          lo = fmaf(ta, __uint_as_float(w << 16), lo);
          lo = fmaf(tb, __uint_as_float(w & 0xFFFF0000u), lo);
        }
      }
      return lo;
    }
    for (int j = 0; j < r; ++j) {
      float tj = 0.0f;
      for (int sp = 0; sp < splits; ++sp) tj += t[((int64_t)sp * M + row0 + m) * r + j];
      lo = fmaf(tj, bf16_bits_to_f32(B[(brow0 + n) * r + j]), lo);
    }
    return lo;
  }
};

// A launch of 2^32 threads or more runs the excess only, without an error: grids whose sizes allow that are launched in parts
// of at most kLaunchBlocks workgroups (of up to 512 threads), launch(n, b0) workgroups b0 .. b0 + n - 1.
constexpr int64_t kLaunchBlocks = 1 << 22;
template <typename F>
hipError_t launch_blocks(int64_t blocks, F launch) {
  for (int64_t b0 = 0; b0 < blocks; b0 += kLaunchBlocks) {
    launch((unsigned)std::min(kLaunchBlocks, blocks - b0), (int)b0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Upper bound of the row tiles of any `experts` ranges over M rows.
inline int64_t tile_bound(int64_t M, int experts, int BM) { return M / BM + std::min<int64_t>(experts, M); }

template <int KIND, int BITS, int BM, int BN>
hipError_t launch_tile_t(TileArgs a, const Levels& lv, hipStream_t s) {
  auto kern = k_tile<KIND, BITS, BM, BN>;
  const int64_t no = KIND == TILE_TR ? a.K : a.N;
  a.ntiles = (int)((no + BN - 1) / BN);
  // (only so many ranges can hold more than min_rows rows)
  const int ranges = (int)std::min<int64_t>(a.experts, a.M / (a.min_rows + 1));
  int64_t tiles = (a.offsets ? tile_bound(a.M, ranges, BM) : (a.M + BM - 1) / BM) * a.ntiles;
  if (a.rest && BM < 256) tiles = kRestMax * (256 / BM) * (256 / BN);
  if (tiles <= 0) return hipSuccess;
  if (tiles > INT32_MAX - 8) return hipErrorInvalidValue;
  return launch_blocks(8 * ((tiles + 7) / 8), [&](unsigned n, int b0) { hipLaunchKernelGGL(kern, dim3(n), dim3(512), 0, s, a, b0, lv); });
}

// The tile shape, from the sizes the host knows (the rows of an expert only by their
// mean).  256 x 256 tiles multiply most per byte moved and watt, but need a
// round of them to fill the 256 CUs and ranges of a few hundred rows to be
// full: at 8192 x 4096 x 4096 in 8 ranges with 4-bit codes (all tiles written from registers then) they took 359 us, 128 x
// 128 ones 434 and 64 x 128 ones 629; at 777 rows in 64 ranges of 1408 x 2048 (2-bit) 55, 27 and 23 us.
// Between 256 x 256 and 128 x 128 tiles of expert ranges the estimated times decide, in rounds of the former: a rest of at most
// kRestMax takes half a round, 512 of the latter (two to a CU) 0.79.  3000 rows in 8 ranges of 4096 x 4096: 129
// us and 168 (the rule 1.0 and 1.33), 5000 in 16 of 2816 x 2048 105 and 114 (1.5 and 1.6), 4096 in 16 of 2816 x 2048 116
// and 111 (1.5 and 1.36).
template <int KIND, int BITS>
hipError_t launch_tile(TileArgs a, const Levels& lv, hipStream_t s) {
  const int64_t no = KIND == TILE_TR ? a.K : a.N;
  // tiles of b x c: whole ones, and half a partial one per range
  auto count = [&](int64_t b, int64_t c) {
    const int64_t nt = (no + c - 1) / c;
    return a.offsets ? (a.M / b + (std::min<int64_t>(a.experts, a.M) + 1) / 2) * nt : (a.M + b - 1) / b * nt;
  };
  const bool short_ranges = a.offsets && a.M < (int64_t)a.experts * 96;
  const int64_t n256 = count(256, 256), over = n256 % kCus;
  const double t256 = (double)(n256 / kCus) + (over == 0 ? 0.0 : n256 > kCus && over <= kRestMax ? 0.5 : 1.0);
  const double t128 = 0.79 / 512 * (double)count(128, 128);
  if (!short_ranges && (a.offsets ? t256 < t128 : n256 >= 192)) {
    a.rest = 1;
    const hipError_t e = launch_tile_t<KIND, BITS, 256, 256>(a, lv, s);
    if (e != hipSuccess) return e;
    // the rest kernel: known not to be needed only without offsets
    if (!a.offsets && tile_split((int)n256) == (int)n256) return hipSuccess;
    return launch_tile_t<KIND, BITS, 128, 128>(a, lv, s);
  }
  a.rest = 0;
  if (a.M < (a.offsets ? (int64_t)a.experts * 64 : 65) || count(128, 128) < 256) return launch_tile_t<KIND, BITS, 64, 128>(a, lv, s);
  return launch_tile_t<KIND, BITS, 128, 128>(a, lv, s);
}

}  // namespace

}  // namespace qlr
