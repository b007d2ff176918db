// Internal launch interface between the host library (qlr_host.cpp) and the
// kernel translation units.  Arguments are validated by the host library
// before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "qlr_device.h"

namespace qlr {

hipError_t launch_fill_u32(uint32_t* p, uint32_t value, int64_t n, hipStream_t s);

// Quantize numel elements of W (dtype wdt) into codes / absmax_q8 / absmax_c;
// sets *flag nonzero if W holds a non-finite value (flag must be zero before).
hipError_t launch_quantize(const void* W, int wdt, int64_t numel, int bits, const Levels& lv,
                           uint8_t* codes, uint8_t* q8, float* cst, uint32_t* flag,
                           hipStream_t s);

hipError_t launch_dequantize(const uint8_t* codes, const uint8_t* q8, const float* cst,
                             int64_t numel, int bits, const Levels& lv, void* out, int odt,
                             hipStream_t s);

// Number of K-splits of the adapter product t = x A^T for M rows, K columns and
// rank r: the product is written as `splits` partial sums p[s][M][r] (float32)
// that the consumers add in split order; splits * M * r <= kTPartsMax (the
// decode kernel prefetches them all at once).  K need not be a multiple of 64
// (the backward's u = dy B contracts over the weight's rows); such products run
// one split on the float32 kernel.
constexpr int kTPartsMax = 4096;
int lora_t_splits(int64_t M, int64_t K, int r, int xdt, int abdt);

// p[s][m][j] = sum over split s's K range of x[m,k] A[j,k]  (float32 partials).
hipError_t launch_lora_t(const void* x, int xdt, int64_t M, int64_t K, const void* A, int abdt,
                         int r, float* t, int splits, hipStream_t s);

// bf16 products of several linears with one M > 16 (a mixed stack's adapters):
// up to lora_t_group_max() per launch, each written in one K pass (splits 1).
struct LoraTItem {
  const void* x;   // M x K bf16
  const void* A;   // r x K bf16, or K x r when bt (then r % 8 == 0)
  float* t;        // M x r float32
  int64_t K;
  int r;
  bool bt;
  int splits;      // M <= 16: partial sums, or 0 (lora_t_splits)
};
int lora_t_group_max();
hipError_t launch_lora_t_group(const LoraTItem* items, int n, int64_t M, hipStream_t s);
// The same for M <= 16 (bf16, K % 64 == 0, not bt): each item written as
// its number of partial sums (lora_t_splits(M, K, r), as launch_lora_t would, where it names none); up to
// lora_t_small_group_max() items per launch.
int lora_t_small_group_max();
hipError_t launch_lora_t_small_group(const LoraTItem* items, int n, int64_t M, hipStream_t s);

struct LinearArgs {
  const void* x;
  int xdt;
  int64_t M, N, K;
  int bits;
  const uint8_t* codes;
  const uint8_t* q8;
  const float* cst;
  const float* t;  // splits x M x r float32 partials of x A^T (NULL if r == 0)
  int t_splits;
  const void* A;   // r x K
  const void* B;   // N x r
  int abdt;
  int r;
  float scale;
  void* y;
  int ydt;
  // optional float32 M x N term added to every output before rounding (the
  // sparse side channel's x S^T); null when absent
  const float* addend = nullptr;
  // optional CSR side channel (N rows) summed inside the single-row decode
  // kernel (see gemv_fuses_sparse); null when absent
  const int32_t* sp_row_ptr = nullptr;
  const int32_t* sp_col = nullptr;
  const float* sp_val = nullptr;
  int64_t sp_nnz = 0;
  // >= 0: the side channel multiplies the Walsh-Hadamard transform of x over
  // blocks of 2^sp_wht_lp columns, scaled by 2^-sp_wht_lp, instead of x
  int sp_wht_lp = -1;
  // prefill GEMM (forward): the CSR side channel's entries are added to the
  // dequantized weights of every 128-row tile whose entries number at most
  // gemm_sparse_cap(bits); the other tiles add `addend`, which then holds
  // their rows (launch_sparse_addend with that cap)
  bool sp_gemm = false;
  // optional double-binary branch (l = 1, r = its rank <= 16) summed inside the
  // single-row decode kernel in place of A and B (see gemv_fuses_dba)
  const uint32_t* dba_b1 = nullptr;
  const uint32_t* dba_b2 = nullptr;
  const uint16_t* dba_alpha = nullptr;
  const uint16_t* dba_beta = nullptr;
  const uint16_t* dba_gamma = nullptr;
};

// float32 path: any dtypes, any M.
hipError_t launch_linear_f32(const LinearArgs& a, const Levels& lv, hipStream_t s);
// bf16 decode path, M <= 16.
hipError_t launch_gemv(const LinearArgs& a, const Levels& lv, hipStream_t s);
// True when launch_gemv computes t = x A^T itself for this call (a single x
// row and a small rank): the adapter-product kernel is then not launched and
// a.t is not read.
bool gemv_fuses_adapter(const LinearArgs& a);
// True when launch_gemv can add a CSR side channel (a.sp_*) itself for this
// call: the single-row path with a short chunk stream.
bool gemv_fuses_sparse(const LinearArgs& a);
// True when launch_gemv can form the double-binary branch itself (a.dba_*, one
// envelope term, a.r = its rank <= 16, a single x row).
bool gemv_fuses_dba(const LinearArgs& a);
// Grouped single-row decode: up to gemv_group_max() linears of one code width
// and output dtype at M = 1 in one launch (a mixed stack's decode), each
// accepted by gemv_groupable (bits 2/4/8, bf16, x in LDS, adapter partials in t
// from the small-M adapter product, no side channel or addend).
int gemv_group_max();
bool gemv_groupable(const LinearArgs& a);
hipError_t launch_gemv_group(const LinearArgs* ls, int n, const Levels& lv, hipStream_t s);
// bf16 tiled GEMM path.
hipError_t launch_gemm(const LinearArgs& a, const Levels& lv, hipStream_t s);
// Weight rows per tile of the prefill GEMM, and the most side-channel entries a
// tile adds to its weights itself (0: none; widths whose level table fills LDS).
constexpr int64_t kGemmTileRows = 128;
int64_t gemm_sparse_cap(int bits);
// Up to gemm_group_max() independent linears of one code width, one M and one
// output dtype in one launch (mixed stacks); lv holds that width's levels.
int gemm_group_max();
hipError_t launch_gemm_group(const LinearArgs* ls, int n, const Levels& lv, hipStream_t s);

// ---- double-binary adapter branch
struct DbaArgs {
  int R, ell;
  const uint32_t* b1;     // N x ceil(R/32) words
  const uint32_t* b2;     // R x ceil(K/32) words
  const uint16_t* alpha;  // fp16, ell x N
  const uint16_t* beta;   // fp16, ell x R
  const uint16_t* gamma;  // fp16, ell x K
};
// K splits of the branch's first stage (float32 partials that the forward
// kernels add, like the adapter product's).
int dba_t_splits(int64_t M, int64_t K, int xdt, int R, int ell);
// t2 (splits x M x 2 ell R float32) = [t' | t'] and beff (N x 2 ell R bf16): the
// branch as an exact rank-2 ell R adapter with scale 1.
hipError_t launch_dba_prep(const DbaArgs& d, const void* x, int xdt, int64_t M, int64_t N, int64_t K, float* t2,
                           int splits, uint16_t* beff, hipStream_t s);

// ---- hybrid outlier split
size_t outlier_ws_bytes(int64_t numel, int64_t k);
// Select the k largest |w| (ties to the lower index), compact their flat
// indices (ascending) and values, and write W with them zeroed (same dtype) into
// the workspace; *flag (device) becomes nonzero if W holds NaN or Inf.
hipError_t launch_outlier_split(const void* W, int wdt, int64_t numel, int64_t k, void* ws, void** dense,
                                uint32_t** flag, int32_t** oidx, float** oval, hipStream_t s);
// After the dense part is quantized: row_ptr, columns, and residuals w - w'.
hipError_t launch_outlier_finish(int64_t rows, int64_t cols, int64_t k, int bits, const Levels& lv,
                                 const uint8_t* codes, const uint8_t* q8, const float* cst, const int32_t* oidx,
                                 const float* oval, int32_t* row_ptr, int32_t* col, float* val, hipStream_t s);
// *out = the largest entry count over the row groups [128 g, 128 g + 128) of a CSR
// with `rows` rows and k entries (one workgroup).
hipError_t launch_group_max(int64_t rows, int64_t k, const int32_t* row_ptr, uint32_t* out, hipStream_t s);
// C (M x N float32) = x S^T for S in CSR (N rows, K columns).  cap >= 0: only
// the rows of aligned kGemmTileRows-row groups holding more than cap entries
// are computed (the others are left as they are).
hipError_t launch_sparse_addend(const void* x, int xdt, int64_t M, int64_t K, int64_t N, const int32_t* row_ptr,
                                const int32_t* col, const float* val, int64_t nnz, float* C, hipStream_t s,
                                int64_t cap = -1);

// C (M x N float32) = z F^T, z = x blockdiag(H_P) / P (P = 2^lp), F in CSR (N rows, K columns);
// K % 8 == 0 and K <= wha_max_cols(); nnz >= 1.
hipError_t launch_wha_addend(const void* x, int xdt, int64_t M, int64_t K, int64_t N, int lp, const int32_t* row_ptr,
                             const int32_t* col, const float* val, int64_t nnz, float* C, hipStream_t s);
int64_t wha_max_cols();
// The branch merged into the weight for the prefill GEMM: Wd (N x K bf16) =
// bf16(W' + F blockdiag(H_P) / P), P = 2^lp, F in CSR (N rows, K columns);
// K % 64 == 0 and K <= wha_max_cols().
hipError_t launch_wha_merge(const uint8_t* codes, const uint8_t* q8, const float* cst, int bits, const Levels& lv,
                            int64_t N, int64_t K, int lp, const int32_t* row_ptr, const int32_t* col, const float* val,
                            int64_t nnz, uint16_t* out, hipStream_t s);
// Prefill GEMM on a dense bf16 weight held in a.codes (N x K row-major,
// N K 2 <= INT_MAX bytes): y = x Wd^T (+ a.addend); no adapter.
hipError_t launch_gemm_dense(const LinearArgs& a, hipStream_t s);

// ---- backward (adapter training)
// Input gradient dx = dy W' + scale u A on the transposed bf16 GEMM: a.x = dy
// (M x N bf16), a.y = dx (M x K), a.t = u partials (t_splits x M x r float32),
// a.B = A (r x K bf16), a.N / a.K the weight's rows / columns (both multiples
// of 64).
hipError_t launch_gemm_dx(const LinearArgs& a, const Levels& lv, hipStream_t s);
// Rows of x per GEMM launch for a contraction length KC (0: KC too large).
int64_t gemm_max_rows_of(int64_t KC);
// The same on the float32 path (any dtypes, any N).
hipError_t launch_dx_f32(const LinearArgs& a, const Levels& lv, hipStream_t s);
// Bt (r x N) = B^T for B (N x r) of dtype dt.
hipError_t launch_transpose_nr(const void* B, int dt, int64_t N, int r, void* Bt, hipStream_t s);
// dA = scale u^T x (r x K) and dB = scale dy^T t (N x r), float32, from the
// float32 partials of u (M x r) and t (M x r); x and dy share dtype qdt.
// mfma: bf16 MFMA kernel (qdt bf16, K and N multiples of 8), else float32 FMA.
// part: grad_partial_floats(M, N, K, r) floats of scratch.
size_t grad_partial_floats(int64_t M, int64_t N, int64_t K, int r);
hipError_t launch_lora_grads(const float* u, int u_splits, const float* t, int t_splits, const void* x,
                             const void* dy, int qdt, bool mfma, int64_t M, int64_t N, int64_t K, int r,
                             float scale, float* dA, float* dB, float* part, hipStream_t s);

// ---- products over ranges of rows: expert-grouped linears and the 8-bit-integer linear
struct TileArgs {
  const void* x;           // M x K bf16 (TR: dy, M x N; the 8-bit product: int8 M x K)
  int64_t M;               // rows of x, y and t
  const int32_t* offsets;  // experts + 1 device offsets, or null: one range of M rows
  int experts;
  int64_t N, K;            // one expert's weight
  int bits;
  const uint8_t* w;        // packed codes of the stacked weight, or int8 values
  const uint8_t* q8;
  const float* cst;
  const float* sx;         // 8-bit product: scale per token and per output channel
  const float* sw;
  const float* t;          // t_splits x M x r float32 partials of the adapter product (TR: of u)
  int t_splits;
  const uint16_t* ab;      // bf16 adapter operand: B (experts x N x r); TR: A (experts x r x K)
  int r;
  float scale;
  void* y;
  int ydt;
  int min_rows;            // experts with at most this many rows are left out (the few-rows kernel takes them)
  int ntiles, rest;        // set by the launcher: column tiles; whether a last partial round is split finer
};
// Dropout of an adapter's input (see qlr_philox.h); thr = 0: none.
struct DropArgs {
  uint64_t seed, counter;
  const uint64_t* step;  // device, added to counter when a kernel runs, or null
  uint32_t thr;          // an element is kept iff its 16-bit number is at least thr
  uint8_t* bits;         // backward: the masks (which x rows x K / 8 bytes, bit j of a byte its element j), formed once (launch_train_t)
};
enum { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2 };
// The products of a training step and of the gated block.  Gated: N is one projection's rows, w the two stacked (gate, up),
// t and u hold 2 r columns (gate's, up's), ab is B as 2 x N x r.
struct TrainArgs : TileArgs {
  DropArgs drop;
  int halves;  // transposed with dropout: adapters side by side, each with r columns of t, rows of ab and a mask of its own
  int act;
  uint16_t* gu;  // gated: M x 2N bf16 pre-activations, or null
  int splits;    // ranges of the contraction whose sums go to part (splits x M x train_part_cols floats), or 1
  float* part;
};
// Ranges of the contraction (KC) for the calls that run as 64 x 128 or 128 x 128 tiles of `cols` columns (gated: both sides'): see launch_tile.
int train_tile_splits(int64_t M, int64_t cols, int64_t KC);
constexpr int64_t train_part_cols(int64_t NO, bool gated) { return (gated ? 2 : 1) * ((NO + 3) / 4 * 4); }
// y (and gu) from the ranges' sums.
hipError_t launch_tile_sum(const TrainArgs& a, int64_t NO, bool gated, hipStream_t s);
// Rows up to which the few-rows kernels take an expert, or a call of the 8-bit product.
constexpr int kFewRows = 16;

// q (rows x cols) and scale (rows) of rows of dtype dt.
hipError_t launch_quantize_i8(const void* X, int dt, int64_t rows, int64_t cols, int8_t* q, float* scale, hipStream_t s);
// The same for a few bf16 rows (M <= 16, K % 64 == 0), with t = x A^T as `splits` partial sums (lora_t_splits), in one launch.
hipError_t launch_i8_prep(const void* x, int64_t M, int64_t K, int8_t* q, float* scale, const void* A, int r, int splits,
                          float* t, hipStream_t s);
// y = (x w^T) sx sw + scale t B^T with int8 x, w (K % 16 == 0).
hipError_t launch_i8_gemm(const TileArgs& a, hipStream_t s);
hipError_t launch_i8_few(const TileArgs& a, hipStream_t s);  // M <= kFewRows

// Expert products of the coded weight: every expert of more than a.min_rows rows ...
hipError_t launch_grouped_gemm(const TileArgs& a, const Levels& lv, hipStream_t s);
// ... and those of 1 .. kFewRows rows.
hipError_t launch_grouped_few(const TileArgs& a, const Levels& lv, hipStream_t s);
// dx = dy W'_e + scale u A_e (N % 8 == 0, K % 64 == 0).
hipError_t launch_grouped_dx(const TileArgs& a, const Levels& lv, hipStream_t s);
// t (M x r float32) = x A_e^T over each expert's rows, A experts x r x K bf16, K % 8 == 0.
hipError_t launch_grouped_t(const uint16_t* x, int64_t M, int64_t K, const uint16_t* A, int r, const int32_t* offsets,
                            int experts, float* t, hipStream_t s);
// That and u (M x r) = dy B_e, B experts x N x r, in one launch; r, N and K multiples of 8.
hipError_t launch_grouped_tu(const uint16_t* x, const uint16_t* dy, int64_t M, int64_t N, int64_t K, const uint16_t* A,
                             const uint16_t* B, int r, const int32_t* offsets, int experts, float* t, float* u,
                             hipStream_t s);
// Bt (experts x r x N) = B^T per expert, B experts x N x r bf16.
hipError_t launch_grouped_transpose(const uint16_t* B, int experts, int64_t N, int r, uint16_t* Bt, hipStream_t s);
// ---- adapter dropout and the gated block (no offsets: one range of M rows)
// Floats of a side's partial sums of t that the gated block's decode kernel stages.
constexpr int kGatedFewT = 2048;
// Ranks at which up to kFewRows rows run on the decode kernel.  It stages ranks of 8, 16 .. 64; at any other each output reads its t and
// B from memory one by one, and the tiles are faster from rank 3 on.  Decode kernel and tiles, 4-bit, us, one row of 2 x 11008 x 4096: r = 1
// 29 and 42, r = 2 37 and 43, r = 3 45 and 44, r = 12 115 and 47, r = 16 24 and 41, r = 128 540 and 55; 16 rows: 41 and 42, 56 and 44, 57 and 44,
// 59 and 48, 28 and 41, 162 and 57; one row of 2 x 1024 x 1024: r = 2 10 and 15, r = 3 11 and 15, r = 12 21 and 17, r = 128 156 and 23.
constexpr bool gated_few_takes(int r) { return r <= 2 || (r <= 64 && r % 8 == 0); }
// h = act(gate) up, M x N (and gu): rows of x from 17 on, and up to kFewRows rows.
hipError_t launch_gated_gemm(const TrainArgs& a, const Levels& lv, hipStream_t s);
hipError_t launch_gated_few(const TrainArgs& a, const Levels& lv, hipStream_t s);
// y = x W'^T + scale t B^T in a.splits ranges of the contraction.
hipError_t launch_drop_fwd(const TrainArgs& a, const Levels& lv, hipStream_t s);
// dx = dy W' + sum over the halves of mask (scale u A), of everything without a mask: K % 64 == 0, N % 8 == 0.
hipError_t launch_drop_dx(const TrainArgs& a, const Levels& lv, hipStream_t s);

// The same products of many rows through a dense bf16 copy of the weight in the workspace (qlr_dense.hip).
struct DensePlan {
  int ntiles, whole, rest, splits;  // column tiles; tiles computed whole; tiles split along the contraction, into how many parts
  bool ok;
};
DensePlan dense_plan(int64_t M, int64_t NO, int64_t KC, bool gated);
constexpr int64_t kDensePartFloats = 256 * 256;  // of each of the rest x splits sums
struct DenseWeight {
  const uint8_t* codes;
  const uint8_t* q8;
  const float* cst;
  int64_t rows, K;
  int bits;
  uint16_t* out;  // rows x K, or (tr) K x rows
};
hipError_t launch_dense_weight(const DenseWeight& w, bool tr, const Levels& lv, hipStream_t s);
struct DenseAdapter {
  const float* t;      // t_splits x M x ldt, half h in columns h r ..
  int t_splits, ldt;
  const uint16_t* ab;  // rows x r, or (tr) halves x r x rows
  bool tr;
  int64_t M, rows;
  int r, nb, halves;   // nb = ceil(r / 32)
  float scale;
  uint16_t* xt;        // halves nb x M x 64
  uint16_t* wt;        // (tr ? halves : 1) nb x rows x 64
};
hipError_t launch_dense_adapter(const DenseAdapter& a, hipStream_t s);
struct DenseArgs {
  const uint16_t* x;   // M x KC
  const uint16_t* w;   // output columns x KC (gated: 2 NO rows)
  int64_t M, KC, NO;
  int ntiles, whole, rest, splits, block0;
  const uint16_t *xt, *wt;
  int nb, halves;      // nb = 0: no adapter
  void* y;
  int ydt, act;
  uint16_t* gu;        // gated: M x 2 NO, or null
  DropArgs drop;
  float* part;
};
hipError_t launch_dense(const DenseArgs& a, bool gated, hipStream_t s);

// One product t = src A^T over K columns, as `splits` float32 partial sums of M x ldt floats each, columns col0 .. col0 + r - 1.
struct TrainProd {
  const uint16_t* x;   // M x K bf16
  const uint16_t* A;   // r x K, or K x r (bt)
  int64_t K;
  float* t;
  int r, ldt, col0;
  int mask;            // >= 0: x under mask number `mask`
  bool bt;
};
// Up to four products of one M, rank and number of partial sums, in one launch; K % 8 == 0.
int train_t_splits(int64_t M, int64_t K, int r, int jobs);
hipError_t launch_train_t(const TrainProd* jobs, int n, int64_t M, int splits, const DropArgs& drop, hipStream_t s);
// The gated block's backward up to the products: from dh (M x N) and gu (M x 2N) dgu = [dg | dv] (M x 2N bf16, rounded to
// nearest) and, where u is given, u (splits x M x 2r) = [dg Bg | dv Bu] from unrounded dg and dv.
int gated_u_splits(int64_t M, int64_t N, int r);
hipError_t launch_gated_u(const uint16_t* dh, const uint16_t* gu, int act, int64_t M, int64_t N, const uint16_t* B, int r,
                          uint16_t* dgu, float* u, int splits, hipStream_t s);
// Adapter gradients: out = scale P^T Q (r x C), or its transpose, for up to four jobs of one M and rank.
struct TrainGrad {
  const float* P;      // p_splits x M x ldp, columns col0 .. col0 + r - 1
  int p_splits, ldp, col0;
  const uint16_t* Q;   // M x C (kinds 1 and 2: dh, with gu)
  int64_t C;
  float* out;
  int kind;            // 0: Q; 1, 2: dg, dv formed from dh and gu
  int mask;            // >= 0: Q under mask number `mask` (kind 0)
  bool cols_major;     // out is C x r
};
// Partial sums t (splits x M x ld) added into the first, for up to two buffers.
struct TrainSum {
  float* t;
  int splits, ld;
};
hipError_t launch_train_sum(const TrainSum* jobs, int n, int64_t M, hipStream_t s);
size_t train_grad_floats(int64_t M, int64_t C_total, int r);
hipError_t launch_train_grads(const TrainGrad* jobs, int n, int64_t M, int r, const uint16_t* gu, int64_t N, int act, float scale,
                              const DropArgs& drop, float* part, hipStream_t s);

// dA (experts x r x K) = scale u^T x and dB (experts x N x r) = scale dy^T t, float32, zero for experts
// without rows; K % 8 == 0 and N % 8 == 0.  part: grouped_grad_floats() floats of scratch.
size_t grouped_grad_floats(int64_t M, int64_t N, int64_t K, int r, int experts);
hipError_t launch_grouped_grads(const float* u, const float* t, const uint16_t* x, const uint16_t* dy, int64_t M,
                                int64_t N, int64_t K, int r, const int32_t* offsets, int experts, float scale, float* dA,
                                float* dB, float* part, hipStream_t s);

}  // namespace qlr
