// launch.h - internal launch interface between the C ABI (api.cpp) and the
// device code (kernels.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm.h"

namespace lora {

// rows per tile of the rank-r panel kernel (the split choice in api.cpp uses it)
constexpr int PANEL_BM = 128;
// The bf16 panel (G_BF16_PANEL_SPLIT_NT) runs panel_dma_kernel, which alone
// takes Bop rows from several sources (GemmArgs::n_src), for these shapes.
bool panel_dma_fits(int64_t n_store, int64_t lda, int64_t ldb);
// The whole-tile kernels' buffer offsets stay in range for operands with row
// strides up to ld (elements).
bool whole_ld_fits(int64_t ld);

// GEMM instances.  Suffixes: NT/NN = layout of the second operand, then the
// epilogue.  "BIG" = 256x256 tiles, "MED" = 128x128 (4 waves), "PANEL" =
// 64x64 rank-r panels, "SPLIT" = 64x256 split-contraction partials,
// "PANEL_SPLIT" = 256x64 split-contraction partials of a rank-r panel,
// "MED_*_PARTIAL" = 128x128 split-contraction partials of the layer's own
// GEMMs when their tiles alone cannot fill the chip (few tokens), "ADD" =
// the product plus an addend (the merge of the adapter into W).
enum GemmKind : int {
  G_BF16_BIG_NT_STORE,
  G_BF16_BIG_NT_ROPE,
  G_BF16_MED_NT_STORE,
  G_BF16_MED_NT_ROPE,
  G_BF16_BIG_NN_STORE,
  G_BF16_MED_NN_STORE,
  G_NF4_BIG_NT_STORE,
  G_NF4_MED_NT_STORE,
  G_NF4_BIG_NN_STORE,
  G_NF4_MED_NN_STORE,
  G_BF16_SPLIT_NN_PARTIAL,
  G_F32_NT_STORE,
  G_F32_NT_ROPE,
  G_F32_NN_STORE,
  G_F32_PANEL_NT_STORE,
  G_F32_PANEL_NT_STORE_T,
  G_F32_PANEL_NN_BOTH,
  G_F32_SPLIT_NN_PARTIAL,
  G_BF16_PANEL_SPLIT_NT,
  G_BF16_MED_NT_PARTIAL,
  G_BF16_MED_NN_PARTIAL,
  G_NF4_MED_NT_PARTIAL,
  G_NF4_MED_NN_PARTIAL,
  G_BF16_MED_NN_ADD,
  G_F32_NN_ADD,
  G_BF16_WHOLE_SWIGLU,
  G_BF16_MED_NN_ADD_MASKED,
  G_F32_NN_ADD_MASKED,
  G_BF16_WHOLE_GROUP,  // several projections' forward GEMMs in one whole-tile launch (GemmArgs::n_mem)
  G_NF4_WHOLE_NT_STORE,  // whole-tile forward GEMM, NF4 W expanded in the load stage (gemm_w4_nf4_kernel)
  // forwards with the bias / activation / residual epilogue (GemmArgs::ep)
  G_BF16_BIG_NT_EPI,
  G_BF16_MED_NT_EPI,
  G_NF4_BIG_NT_EPI,
  G_NF4_MED_NT_EPI,
  G_NF4_WHOLE_NT_EPI,
  G_F32_NT_EPI,
  G_BF16_HALF_EPI,    // 128 x 256 tiles, up to one a CU (gemm_w4_half_kernel)
  G_BF16_STREAM_EPI,  // 256 x 256 tiles, ragged and split over the CUs (gemm_w4_stream_kernel)
  // fp32 partials over splits of the contraction (an epilogue layer's few tiles)
  G_F32_NT_PARTIAL,
  G_F32_NN_PARTIAL,
  G_F32_PANEL_NT_PARTIAL,
  G_F32_PANEL_NN_PARTIAL,
  G_KIND_COUNT
};

struct TileShape {
  int bm, bn;
};
TileShape gemm_tile(GemmKind k);

// Sets a.tiles_m from a.m_store and launches over (tiles_m * tiles_n, 1, splits).
hipError_t launch_gemm(GemmKind k, GemmArgs a, int splits, hipStream_t st);
// Two G_BF16_PANEL_SPLIT_NT (of the same panel size) or two
// G_BF16_SPLIT_NN_PARTIAL (of as many rows) with sa and sb splits in one
// launch, bit for bit what each alone gives; where gemm_pair_fits.
bool gemm_pair_fits(GemmKind k, const GemmArgs& a, const GemmArgs& b);
hipError_t launch_gemm_pair(GemmKind k, const GemmArgs& a, int sa, const GemmArgs& b, int sb, hipStream_t st);

// Bt[q, i] = q < r ? B[i, q] : 0, bf16 [rows, r] -> [r_pad, rows].
hipError_t launch_transpose_pad(const uint16_t* src, uint16_t* dst, int64_t rows, int64_t r, int64_t r_pad,
                                hipStream_t st);

// dst[c, q] = q < R ? src[q, c] : 0 (c < C, q < Rpad; row strides lds, ldd):
// src [R, C] bf16 transposed to [C, Rpad] with zero columns R..Rpad.
hipError_t launch_transpose_tile(const uint16_t* src, int64_t lds, int64_t R, int64_t C, uint16_t* dst, int64_t ldd,
                                 int64_t Rpad, hipStream_t st);

// dst[i, j] = j < r ? src[i, j] : 0 for a [rows, r] matrix widened to [rows, r_pad].
hipError_t launch_pad_cols(int elem_bytes, const void* src, void* dst, int64_t rows, int64_t r,
                           int64_t r_pad, hipStream_t st);

// G = R(-angle) dY for rotate-half pairs of 128-wide heads.
hipError_t launch_rope_inverse(int elem_bytes, const void* dY, void* G, int64_t M, int64_t d_out,
                               const int32_t* pos, const float* cosc, const float* sinc, int64_t max_pos,
                               hipStream_t st);

hipError_t launch_rope_cache(int64_t max_pos, int head_dim, double theta, float* cosc, float* sinc,
                             hipStream_t st);

// out = sum over z < splits of part[z] (fixed order).  part[z] is [rows_pad, N]
// fp32.  transpose = false: out[q * N + n]; true: out[n * rows + q]; q < rows.
hipError_t launch_reduce_splits(const float* part, int splits, int64_t rows, int64_t N,
                                int64_t part_stride, bool transpose, float* out, hipStream_t st);

// Several independent launch_reduce_splits / launch_transpose_tile jobs in ONE
// launch (a layer's dA and dB sums, a group's A^T and B^T): the blocks are
// dealt to the jobs in order.  add() checks each job as the single launch
// would and returns hipErrorInvalidValue (job not added) otherwise.
constexpr int kBatchJobsMax = 16;
struct ReduceJob {
  const float* part;
  float* out;
  int64_t rows, N, part_stride;
  int splits, transpose, block0, tiles_n;
};
struct ReduceBatch {
  int n = 0, blocks = 0;
  bool low = false;  // the outputs are bf16 arrays
  ReduceJob j[kBatchJobsMax];
  hipError_t add(const float* part, int splits, int64_t rows, int64_t N, int64_t part_stride, bool transpose,
                 float* out);
};
hipError_t launch_reduce_batch(const ReduceBatch& b, hipStream_t st);

struct TransposeJob {
  const uint16_t* src;
  uint16_t* dst;
  int64_t lds, R, C, ldd, Rpad;
  int block0, tiles_c;
};
struct TransposeBatch {
  int n = 0, blocks = 0;
  TransposeJob j[kBatchJobsMax];
  hipError_t add(const uint16_t* src, int64_t lds, int64_t R, int64_t C, uint16_t* dst, int64_t ldd, int64_t Rpad);
};
hipError_t launch_transpose_batch(const TransposeBatch& b, hipStream_t st);

// Per-column scale of a panel: column c takes s[i] for the first i < n with
// c < end[i] (one entry per projection of a group; n = 1 for one projection).
constexpr int kColScaleMax = 8;
struct ColScale {
  int n;
  int64_t end[kColScaleMax];
  float s[kColScaleMax];
};
inline ColScale col_scale(float s) {
  ColScale c{};
  c.n = 1;
  c.end[0] = INT64_MAX;
  c.s[0] = s;
  return c;
}

// Rank-r panel from split partials: v = scale(c) * sum over z < splits of
// part[z][q, c] (fixed order) for q < rows, c < n; written as bf16 to
// out[q * ldo + c] and/or outt[c * ldot + q] (either may be null).
// Also clears zero[0 .. nzero) (a later launch's counters).
hipError_t launch_panel_reduce(const float* part, int splits, int64_t part_stride, int64_t ldp, int64_t rows,
                               int64_t n, const ColScale& scale, uint16_t* out, int64_t ldo, uint16_t* outt,
                               int64_t ldot, hipStream_t st, int* zero = nullptr, int nzero = 0);
// The same of two panels of `rows` rows and n columns (row-major outputs n
// wide, transposed ones `rows` wide).
struct PanelSum {
  const float* part;
  int splits;
  uint16_t* out;
  uint16_t* outt;
  const float* tscale = nullptr;  // outt's values times their row's power of two (rows [0, tn), 0 past them)
  int64_t tn = 0;
  bool rest = false;  // outt has n rows more: what the rounding of the first n left, rounded
};
hipError_t launch_panel_reduce_pair(const PanelSum& a, const PanelSum& b, int64_t rows, int64_t n,
                                    const ColScale& scale, hipStream_t st, int* zero, int nzero);

// out [M, N] bf16 (row stride ldo) = fixed-order sum of split partials
// (part[z * part_stride + m * N + n]); with pos != NULL also the RoPE rotation
// of the pairs (n, n + 64) of each 128-wide head (N a multiple of 128; a
// position outside [0, max_pos) gives zeros).
hipError_t launch_split_finish(const float* part, int splits, int64_t part_stride, int64_t M, int64_t N,
                               uint16_t* out, int64_t ldo, const int32_t* pos, const float* cosc, const float* sinc,
                               int64_t max_pos, hipStream_t st);

// The same sums with an epilogue: out [M, N] (bf16 or fp32, by elem_bytes) =
// act(sum + bias) + residual.
hipError_t launch_split_finish_epi(int elem_bytes, const float* part, int splits, int64_t part_stride, int64_t M,
                                   int64_t N, void* out, const EpiArgs& ep, hipStream_t st);
// fp32 panel: out [rows, n] and / or outt [n, rows] = scale * the sum over splits
// of part [splits][rows, n].
hipError_t launch_panel_sum_f32(const float* part, int splits, int64_t rows, int64_t n, float scale, float* out,
                                float* outt, hipStream_t st);

// Backward of the epilogue over [M, N]: dZ = dY act'(Z) (neither is touched
// without an activation) and, with part, the column sums of dZ over `chunks`
// (1 .. 64) ranges of the tokens, fp32 [chunks][N].
hipError_t launch_epi_grad(int elem_bytes, const void* dY, const void* Z, void* dZ, float* part, int chunks, int64_t M,
                           int64_t N, int act, hipStream_t st);
// dbias [N] = the sum over chunks (1 .. 64) of part [chunks][N].
hipError_t launch_bias_grad(const float* part, int chunks, int64_t N, float* dbias, hipStream_t st);

hipError_t launch_fill_zero(float* p, int64_t n, hipStream_t st);

// SwiGLU elementwise passes over n elements of bf16 (elem_bytes 2) or fp32:
// H = silu(G) U; dG = dH U silu'(G), dU = dH silu(G); dst += src.
hipError_t launch_swiglu_apply(int elem_bytes, const void* G, const void* U, void* H, int64_t n, hipStream_t st);
hipError_t launch_swiglu_grad(int elem_bytes, const void* dH, const void* G, const void* U, void* dG, void* dU,
                              int64_t n, hipStream_t st);
hipError_t launch_add_into(int elem_bytes, void* dst, const void* src, int64_t n, hipStream_t st);

// out = X with the elements whose keep bit is clear set to 0 (n elements,
// n % 8 == 0, bit b of keep[e] is element 8 e + b).
hipError_t launch_mask_copy(int elem_bytes, const void* X, const uint8_t* keep, void* out, int64_t n,
                            hipStream_t st);
// Philox4x32-10 keep mask of n elements (8 | n): packed bits into keep and/or
// the masked copy of X into out (either may be null; out needs X).
hipError_t launch_dropout_philox(int elem_bytes, const void* X, void* out, uint8_t* keep, int64_t n, uint32_t thr,
                                 uint64_t seed, uint64_t offset, hipStream_t st);

// blocks x 256 threads of the MFMA-rate kernel (iters rounds of 8 MFMAs per
// wave); out [blocks * 256] receives one float per thread.
hipError_t launch_mfma_rate(int iters, int blocks, float* out, hipStream_t st);

// Tiny fp32 problems (tiny.h): forward (bwd false) Y = X W^T + s (X A^T) B^T
// in one launch; backward dX (nullable), dA, dB of it for G in two launches,
// the rank rows s X A^T and s G B going through Ps and Qs (M r floats each).
// Only where tiny_fits holds (else hipErrorInvalidValue).
bool tiny_fits(int64_t M, int64_t K, int64_t N, int64_t r);
hipError_t launch_tiny(bool bwd, const float* X, const float* W, const float* A, const float* B, const float* G,
                       float* Y, float* dX, float* dA, float* dB, float* Ps, float* Qs, int64_t M, int64_t K,
                       int64_t N, int64_t r, float s, hipStream_t st, const EpiArgs* ep = nullptr);

// Few-token forward in one launch (skinny.h): Y = X W^T + bf16(s X A^T) B^T,
// mode 0 plain, 1 RoPE (pos / cosc / sinc, N % 128 == 0), bf16 W.  Requires
// 1 <= M <= 64, r % 8 == 0, r <= 64 (skinny_fits).
struct SkinnyArgs;
bool skinny_fits(int64_t M, int64_t K, int64_t N, int64_t r, int mode);
hipError_t launch_skinny_fwd(const SkinnyArgs& a, int mode, hipStream_t st);

// W^T [cols, rows] bf16 from the NF4 codes of W [rows, cols] (cols % 64 == 0,
// rows % 8 == 0), the same values as launch_nf4_dequant.
hipError_t launch_nf4_dequant_t(const uint8_t* codes, const float* absmax, int64_t rows, int64_t cols,
                                const float* table16, uint16_t* out, hipStream_t st);

hipError_t launch_nf4_dequant(const uint8_t* codes, const float* absmax, int64_t n,
                              const float* table16, uint16_t* out, hipStream_t st);

// Few-token path (few.h), MB = 16-row blocks of tokens (1, 2, 4 or 8): the
// panel partials (Sp + Sq blocks); the backward's panel sums when the stream
// does not fold them; the W stream of the forward (NF4 or bf16 W) or of the
// backward (nblk <= 256 blocks, each a contiguous range of the tiles' stages).
struct FewArgs;
hipError_t launch_few_panel(const FewArgs& a, int MB, hipStream_t st);
hipError_t launch_few_reduce(const FewArgs& a, hipStream_t st);  // backward: P_s, Q_s between the launches
hipError_t launch_few_fwd(const FewArgs& a, int MB, bool nf4, bool epil, hipStream_t st);
hipError_t launch_few_multi(const FewArgs& a, int MB, hipStream_t st);  // bf16 W, strips of FewArgs::ad
hipError_t launch_few_bwd(const FewArgs& a, int MB, bool nf4, hipStream_t st);

// Token log-probabilities (loss.hip): logp [rows] and stats [rows, 2] (row
// maximum, log of the row's sum) from logits z [rows, V] (row stride ld, bf16
// or fp32), and dz (row stride ldd) from dlogp [rows].  V < 2^31; a target
// outside [0, V) gives logp 0 and a zero gradient row.
hipError_t launch_token_logp(int elem_bytes, const void* z, int64_t ld, int64_t rows, int64_t V, const int64_t* target,
                             float tau, float* logp, float* stats, hipStream_t st);
hipError_t launch_token_logp_grad(int elem_bytes, const void* z, int64_t ld, int64_t rows, int64_t V,
                                  const int64_t* target, float tau, const float* stats, const float* dlogp, void* dz,
                                  int64_t ldd, hipStream_t st);

// Losses over S packed sequences of N tokens (loss.hip): cu int64 [S + 1],
// mask [N] or NULL.  The forward's workspace is loss_workspace(S, N, nv) bytes
// (nv: 2 preference, 4 policy), 16-byte aligned.
constexpr int64_t SEQ_SMALL = 8192;  // tokens up to which one block runs the whole forward,
constexpr int SEQ_LDS = 1024;        // and sequences whose sums it holds in LDS
struct LossSeqs {
  const int64_t* cu;
  const uint8_t* mask;
  int64_t S, N;
};
struct PrefLossArgs {
  const float* logp;
  const float* ref;
  int kind, average;
  double beta, eps;
  float* loss;
  float* pair_loss;
  float* rewards;
  float* coef;
};
struct PolicyLossArgs {
  const float* logp;
  const float* old;
  const float* ref;
  const float* adv;
  int adv_per_token, reduction;
  double eps_low, eps_high, beta, norm;
  float* loss;
  float* stats;
  float* weight;
};
int loss_chunk_log2(int64_t N);
size_t loss_workspace(int64_t S, int64_t N, int nv);
hipError_t launch_pref_loss(const LossSeqs& q, const PrefLossArgs& l, void* ws, hipStream_t st);
hipError_t launch_pref_grad(const LossSeqs& q, const float* coef, const float* dloss, float* dlogp, hipStream_t st);
hipError_t launch_policy_loss(const LossSeqs& q, const PolicyLossArgs& l, void* ws, hipStream_t st);
hipError_t launch_policy_grad(const LossSeqs& q, const PolicyLossArgs& l, const float* dloss, float* dlogp,
                              hipStream_t st);

// Root-mean-square norm (norm.hip) of M rows of d (1 .. kNormMaxDim) elements:
// h = X + residual (NULL: X), H = h, Y = h rstd weight, codes / scale8 = Y in 8
// bits; H, Y, codes (with scale8) and rstd may each be NULL.  X and residual
// have row strides, the others d.  H may be X or the residual, Y too.
constexpr int64_t kNormMaxDim = 32768;
struct RmsNormArgs {
  const void* X;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  const void* weight;
  void* H;
  void* Y;
  uint8_t* codes;
  float* scale8;
  float* rstd;
  int64_t M;
  int d;
  float eps;
};
hipError_t launch_rmsnorm(int elem_bytes, const RmsNormArgs& a, hipStream_t st);
// dX = rstd (dY w - xh mean(dY w xh)) + dH (dX and dH may be NULL, dX may be dY
// or dH) and, with part (fp32 [rmsnorm_grad_blocks][d]), dw [d] (2 or 4 bytes
// an element) = the sum over rows of dY xh.  M = 0 gives zeros.
struct RmsNormGradArgs {
  const void* H;
  const void* weight;
  const float* rstd;
  const void* dY;
  const void* dH;
  void* dX;
  float* part;
  int64_t M;
  int d;
};
int rmsnorm_grad_blocks(int64_t M, int d);
hipError_t launch_rmsnorm_grad(int elem_bytes, const RmsNormGradArgs& a, void* dw, int dw_bytes, hipStream_t st);

// Rows kept in 8 bits (norm.hip): e4m3 codes [M, d] and a power of two a row.
hipError_t launch_act8_pack(int elem_bytes, const void* X, int64_t ldx, int64_t M, int d, uint8_t* codes, float* scale8,
                            hipStream_t st);
// out = in in bf16, two arrays (either may be empty).
hipError_t launch_to_bf16(const float* a, int64_t na, uint16_t* oa, const float* b, int64_t nb, uint16_t* ob, hipStream_t st);
hipError_t launch_act8_unpack(int elem_bytes, const uint8_t* codes, const float* scale8, int64_t M, int64_t d, void* X,
                              hipStream_t st);

// Stacks transposed: dst [n][C, R] = src [n][R, C], bf16.
struct MultiTranspose {
  const void* src;  // NULL: none
  void* dst;
  int64_t R, C;
};

// Rows with an adapter of their own (multi.hip).  index int [M]: a row's adapter,
// none outside [0, n).  Lists: per 128- and per 256-row tile its adapters
// (rows of min(rows, n) entries and counts), per group of `per` adapters
// (ceil(n / per) = groups) the 64-token tiles they occur in (rows of
// ceil(M / 64)); counts of 0 blocks leave that list out.  Transposes in the same launch.
constexpr int kMultiMaxRank = 128;
struct MultiLists {
  const int* index;
  int64_t M;
  int n, per;
  int t128, t256, groups;
  int* list128;
  int* cnt128;
  int* list256;
  int* cnt256;
  int* glist;
  int* gcnt;
  int* zero;  // nzero ints cleared
  int nzero;
  // whether an adapter of a row holds infinities or NaNs in `scan` (bf16,
  // scan16 16-byte pieces an adapter): bad [n][chunks], a chunk `pieces` pieces
  const void* scan;
  int64_t scan16;
  int chunks, pieces;
  int* bad;
  MultiTranspose tr[2];
  int64_t tr0;  // (set by the launch)
  __host__ __device__ int cap(int rows) const { return n < rows ? n : rows; }
};
hipError_t launch_multi_lists(MultiLists q, hipStream_t st);
// bf16 strip partials: GemmArgs with ad_of, ad_list (128-row tiles), ad_cnt,
// ad_cap, ad_r; C = fp32 [splits][M, ad_r].  b (may be NULL): another in the same launch.
hipError_t launch_multi_panel(const GemmArgs& a, int sa, const GemmArgs* b, int sb, hipStream_t st);
struct MultiStrip {
  int ops;               // strips of one operand or of two
  const float* part[2];  // [splits][M, r]
  int splits[2];
  uint16_t* P[2];        // [M, r], or NULL
  uint16_t* Pt[2];       // [n r, ceil8(M)] in the groups' tiles, or NULL (both)
  int* mask;             // with Pt: 64 bits a 64-token tile
  int* gbad;             // with Pt: [n], cleared before
  const int* index;
  const float* scales;
  int64_t M;
  int n, r, per;
  const int* bad;        // [n][chunks] of the lists (chunks 0: none)
  int chunks;
  int* list128;          // the product's lists, marked (one of the two, or none)
  const int* cnt128;
  int* list256;
  const int* cnt256;
};
hipError_t launch_multi_strip(const MultiStrip& s, hipStream_t st);
// The product with its rows' adapters (ad_list of 128-row tiles where low, else of 256-row ones).
hipError_t launch_multi_gemm(GemmArgs a, bool low, hipStream_t st);
// The simple kernels (few rows, fp32).  fp32 strips P = s_a X A_a^T and, with Q, Q =
// s_a dY B_a (also clears zero[0 .. nzero)); out = P B_a^T with B [n][N, r], P fp32 (P32) or
// bf16; out = Q A_a with A [n][r, K].
struct MultiDot {
  const void* X;  // [M, K]
  const void* A;  // [n][r, K]
  float* P;
  const void* dY;  // [M, N]
  const void* B;   // [n][N, r]
  float* Q;        // or NULL
  const float* scales;
  const int* index;
  int64_t M, K, N;
  int n, r;
  int* zero;
  int nzero;
};
hipError_t launch_multi_dot(int elem_bytes, const MultiDot& d, hipStream_t st);
hipError_t launch_multi_update(int elem_bytes, const void* P, bool P32, const void* B, const int* index, int64_t M, int64_t N, int n, int r,
                               void* out, hipStream_t st);
hipError_t launch_multi_update_rows(int elem_bytes, const float* Q, const void* A, const int* index, int64_t M, int64_t K, int n, int r,
                                    void* out, hipStream_t st);
// Gradient partials [splits][total, N] of two products Pt X (ad_list: the groups'
// token tiles), `rows` rows of Pt a group; their sums.
hipError_t launch_multi_grad(const GemmArgs& a, int sa, const GemmArgs& b, int sb, int rows, int total, hipStream_t st);
struct MultiGradSum {
  const float* part;
  int splits;
  int64_t N;
  int tr;
  void* out;
};
hipError_t launch_multi_grad_sum(int out_bytes, const MultiGradSum& a, const MultiGradSum& b, const int* gbad, int n, int r,
                                 hipStream_t st);
// gbad may be NULL.  The simple gradients: two sums over tokens of P[t, q] X[t, j],
// with partials for multi_grad_sum where splits > 1.
struct MultiOuter {
  const float* P;  // [M, r]
  const void* X;   // [M, N]
  int64_t N;
  int tr;
  void* out;
  float* part;
};
hipError_t launch_multi_outer(int elem_bytes, const MultiOuter& a, const MultiOuter& b, const int* index, int64_t M, int n, int r, int splits,
                              int out_bytes, hipStream_t st);

// The panel s X A^T and the adapter's gradient from X in 8 bits (act8.hip): fp32
// partials of codes A^T times the rows' scales, [splits][rows, r8] (zeros from row
// M and column r on), and of Qt codes over ranges of tokens, [gsplits][r8, d].
struct Act8Args {
  const uint8_t* codes;  // [M, d], 16-byte aligned, d a multiple of 16
  const float* scale8;   // [M]
  int64_t M, d;
  const uint16_t* A;     // [r, d]
  int64_t rows, r, r8;   // r8 <= 128
  int splits;
  int64_t ksplit;        // a multiple of 128
  float* part;
  const uint16_t* Qt;    // [qr, rows], its rows' values times the tokens' scales
  int64_t qr;            // r8, or 2 r8: the values in two parts
  int gsplits;
  int64_t gksplit;       // a multiple of 64
  float* gpart;
};
// Such a backward's own scratch: both strips transposed and the gradients' partials.
struct Act8Call {
  Act8Args k;  // (Qt, gpart)
  uint16_t* Pt;
  float* partb;
};
bool act8_fits(int64_t d, int64_t r8);
// Beside a bf16 panel (its splits sb) and beside a bf16 gradient, as launch_gemm_pair.
hipError_t launch_act8_panel_pair(const Act8Args& a, const GemmArgs& b, int sb, hipStream_t st);
hipError_t launch_act8_grad_pair(const Act8Args& a, const GemmArgs& b, int sb, hipStream_t st);

}  // namespace lora
