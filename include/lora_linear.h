/*
 * lora_linear.h - C ABI of the MI355X (gfx950) fused LoRA linear layer.
 *
 * The layer (page "UnSloth加速微调体验：在LoRA基础上再提速3倍的秘密", section
 * 算子融合, equation y = Wx + ΔWx = Wx + BAx, with B in R^{d x r} and
 * A in R^{r x k}) computes, for every token x (one row of X):
 *
 *     y = W x + s * B (A x),        s = alpha / r (the caller passes s)
 *
 * with the base weight W frozen.  Row-major, one token per row:
 *
 *     X  [M, d_in]     W  [d_out, d_in]     A [r, d_in]     B [d_out, r]
 *     Y  [M, d_out]    dY [M, d_out]        dX [M, d_in]
 *     dA [r, d_in] fp32                     dB [d_out, r] fp32
 *
 * Backward (section 反向传播优化 of the same page; its printed gradient formulas
 * are garbled, these follow the chain rule):
 *
 *     dX = dY W + s (dY B) A,   dB = s dY^T (X A^T),   dA = s (dY B)^T X
 *
 * X A^T is recomputed, never stored by the forward.  No dW is ever formed:
 * only the adapters train (page "Unsloth教程：本地微调大模型速度提升数倍，显存
 * 节省60%", section 显存优化策略, 4-bit QLoRA paragraph).
 *
 * Conventions shared by every entry point
 *  - Pointers are DEVICE pointers (caller-owned, e.g. torch allocations) unless
 *    an argument says "host".  The library never allocates or frees device
 *    memory; scratch space comes from the caller's workspace `ws` of
 *    `ws_bytes` bytes, sized by lora_workspace_bytes().  The workspace holds
 *    nothing between calls.
 *  - bf16 tensors are passed as their 16-bit patterns.  Accumulation is fp32.
 *    dA and dB are always fp32 and are OVERWRITTEN (not accumulated into).
 *  - `stream` is a hipStream_t (NULL = default stream).  Calls only enqueue
 *    work on it and never synchronise.  The library is re-entrant; calls that
 *    share a workspace must be ordered by the caller.
 *  - Every pointer must be 16-byte aligned; d_in and d_out must be multiples
 *    of 8; 1 <= r <= 256; M >= 0 (M = 0 gives empty Y/dX and zero dA, dB; the
 *    pointers to the M-row tensors X, Y, dY, dX and positions may then be NULL).
 *  - Validation happens before any HIP call: on error nothing is launched and
 *    no output is touched.  A failed launch returns LORA_ERR_DEVICE.  No
 *    exception crosses the ABI and nothing is printed.
 *  - A shape the kernels do not support returns LORA_ERR_SHAPE; there is no
 *    slower fallback path.
 */
#ifndef LORA_LINEAR_H
#define LORA_LINEAR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_ABI_VERSION 1

/* Largest RoPE cache (rows) the q/k projections accept: 2^23 - 1, so that a
 * row's byte offset (256 bytes a row) stays below 2^31. */
#define LORA_ROPE_MAX_POS ((1 << 23) - 1)

/* element types of X, W, A, B, Y, dY, dX */
enum { LORA_F32 = 0, LORA_BF16 = 1 };

/* return codes */
enum {
  LORA_OK = 0,
  LORA_ERR_NULL = -1,      /* a required pointer is NULL */
  LORA_ERR_SHAPE = -2,     /* a size is out of range or breaks a divisibility rule */
  LORA_ERR_ALIGN = -3,     /* a pointer is not 16-byte aligned */
  LORA_ERR_DTYPE = -4,     /* unknown dtype, or a dtype the entry point does not take */
  LORA_ERR_WORKSPACE = -5, /* ws_bytes < lora_workspace_bytes(...) or ws NULL when needed */
  LORA_ERR_DEVICE = -6,    /* current device is not gfx950, or a launch failed */
  LORA_ERR_SCRATCH = -7    /* lora_linear_fwd_noalloc: the problem needs more than the static scratch */
};

/* operation ids for lora_workspace_bytes */
enum {
  LORA_OP_FWD = 0,
  LORA_OP_BWD = 1,
  LORA_OP_ROPE_FWD = 2,
  LORA_OP_ROPE_BWD = 3,
  LORA_OP_NF4_FWD = 4,
  LORA_OP_NF4_BWD = 5,
  LORA_OP_MERGE = 6,
  LORA_OP_DROPOUT_FWD = 7,
  LORA_OP_DROPOUT_BWD = 8
};

/* Library version; equals LORA_ABI_VERSION of the header it was built from. */
int lora_abi_version(void);

/* Static description of a return code ("ok", "null pointer", ...). */
const char* lora_strerror(int code);

/*
 * Bytes of workspace that entry point `op` needs for these sizes (0 if none).
 * Pure host arithmetic; no device query.  Returns 0 for invalid arguments
 * (the entry point itself then reports the error).
 */
size_t lora_workspace_bytes(int op, int dtype, int64_t M, int64_t d_in, int64_t d_out, int64_t r);

/*
 * Forward: Y = X W^T + s (X A^T) B^T.
 * Page "UnSloth加速微调体验…", section 算子融合: W x and the low-rank update are
 * produced by one fused pass; the rank-r panel s X A^T is added into the same
 * fp32 accumulator as X W^T, so no intermediate of size [M, d_out] exists.
 * dtype: LORA_F32 or LORA_BF16 (X, W, A, B, Y all of that type).
 */
int lora_linear_fwd(int dtype, int64_t M, int64_t d_in, int64_t d_out, int64_t r, float scale,
                    const void* X, const void* W, const void* A, const void* B, void* Y,
                    void* ws, size_t ws_bytes, void* stream);

/*
 * lora_linear_fwd for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same result as lora_linear_fwd, bit for bit, with no workspace
 * argument.  Its scratch is a static device array inside the library,
 * LORA_STATIC_SCRATCH_BYTES (32 MiB) per GPU, held by every GPU the library
 * runs on until the process ends; the call itself never allocates or frees
 * memory.  The caller still passes X, W, A, B and Y.  Problems whose
 * workspace (lora_workspace_bytes(LORA_OP_FWD, ...)) exceeds that size
 * return LORA_ERR_SCRATCH before any launch (bf16 at r = 64 fits up to about
 * 87000 tokens at the large-weight shapes).  All calls on one GPU share its array, which keeps the last
 * call's contents: calls that overlap on one GPU (different streams, or
 * threads without ordering) race and must be serialised by the caller.
 */
#define LORA_STATIC_SCRATCH_BYTES (32u << 20)
int lora_linear_fwd_noalloc(int dtype, int64_t M, int64_t d_in, int64_t d_out, int64_t r, float scale,
                            const void* X, const void* W, const void* A, const void* B, void* Y,
                            void* stream);

/*
 * Backward: dX = dY W + s (dY B) A (skipped when dX is NULL),
 *           dB = s dY^T (X A^T),  dA = s (dY B)^T X  (fp32, overwritten).
 * Page "UnSloth加速微调体验…", section 反向传播优化: X A^T is recomputed here
 * instead of being kept from the forward.  No dW.
 */
int lora_linear_bwd(int dtype, int64_t M, int64_t d_in, int64_t d_out, int64_t r, float scale,
                    const void* X, const void* W, const void* A, const void* B, const void* dY,
                    void* dX, float* dA, float* dB, void* ws, size_t ws_bytes, void* stream);

/*
 * Fill the RoPE cache: cos_cache[p * head_dim/2 + i] = cos(p * theta^(-2i/head_dim)),
 * sin_cache likewise, for p < max_pos and i < head_dim/2, computed in fp64 and
 * rounded to fp32.  Page "UnSloth加速微调体验…", section RoPE缓存集成: the cos/sin
 * values live in one contiguous block and a position selects a row by a
 * pointer offset.  Both arrays are device fp32 [max_pos, head_dim/2].
 */
int lora_rope_cache(int64_t max_pos, int head_dim, double theta, float* cos_cache,
                    float* sin_cache, void* stream);

/*
 * q/k projection with the RoPE rotation as the forward epilogue
 * (section RoPE缓存集成: the rotation is applied while q_proj(x) + lora_q(x) is
 * produced).  Within every head of width head_dim (must be 128, and d_out a
 * multiple of it), element i pairs with i + 64 and rotates by the angle whose
 * cos/sin sit in row positions[t] of the caches (rotate-half pairing):
 *     y_i = z_i cos - z_{i+64} sin,   y_{i+64} = z_{i+64} cos + z_i sin,
 * where z is the fused LoRA output.  1 <= max_pos <= LORA_ROPE_MAX_POS
 * (2^23 - 1; else LORA_ERR_SHAPE).  positions: device int32 [M], each meant to lie in
 * [0, max_pos).  The host cannot read them before the launch;
 * the kernels check each one against max_pos and read no cache row for a
 * position outside that range: such a row of y comes out as zeros (and in
 * the backward its gradient is taken as zero), so a bad position never reads
 * outside the caches.
 */
int lora_qk_rope_fwd(int dtype, int64_t M, int64_t d_in, int64_t d_out, int64_t r, float scale,
                     const void* X, const void* W, const void* A, const void* B, int head_dim,
                     const int32_t* positions, const float* cos_cache, const float* sin_cache,
                     int64_t max_pos, void* Y, void* ws, size_t ws_bytes, void* stream);

/*
 * Backward of lora_qk_rope_fwd: the inverse rotation (the transpose, angle
 * negated) is applied to dY, then the LoRA backward runs on the result.
 * Outputs as lora_linear_bwd.
 */
int lora_qk_rope_bwd(int dtype, int64_t M, int64_t d_in, int64_t d_out, int64_t r, float scale,
                     const void* X, const void* W, const void* A, const void* B, int head_dim,
                     const int32_t* positions, const float* cos_cache, const float* sin_cache,
                     int64_t max_pos, const void* dY, void* dX, float* dA, float* dB, void* ws,
                     size_t ws_bytes, void* stream);

/*
 * Forward with an NF4 base weight (QLoRA; page "Unsloth教程…", section 显存优化策略;
 * page "Unsloth自动化优化：无需手动调参的实现原理", section 5: NF4 is the default).
 * W_nf4: device uint8 [d_out * d_in / 2], element e = i*d_in + j of W in byte
 * e/2, high nibble for even e.  absmax: device fp32 [d_out * d_in / blocksize],
 * one per block of `blocksize` consecutive elements.  table16: HOST pointer to
 * the 16 fp32 code values (copied into the launch).  The weight used is
 *     W[e] = bf16_rne(fp32_rne(table16[code_e] * absmax[e / blocksize])).
 * Below LORA_NF4_DEQUANT_MIN_TOKENS tokens (M) it is formed inside the GEMM's
 * load stage and never written to memory: there the GEMM is bound by reading
 * W, and the codes are a quarter of its bf16 bytes.  From that M on, either
 * the whole-tile GEMM expands W in its load stage (M and d_out multiples of
 * 256), or the same routine writes W once per call into the workspace
 * (2 * d_out * d_in bytes, included in lora_workspace_bytes) and the bf16
 * GEMMs read it; lora_set_nf4_fwd_path picks between them.  Every path gives
 * the same W bit for bit.
 * blocksize must be 64 and d_in a multiple of 64.  X, A, B, Y are bf16.
 */
#define LORA_NF4_DEQUANT_MIN_TOKENS 512

/*
 * Which NF4 forward path runs from LORA_NF4_DEQUANT_MIN_TOKENS tokens on, for
 * every later call in the process (a measurement and test control):
 *   LORA_NF4_PATH_AUTO        the library's choice by shape (the default);
 *   LORA_NF4_PATH_DEQUANT     W dequantised once per call, then the bf16 GEMM;
 *   LORA_NF4_PATH_LOAD_STAGE  the whole-tile GEMM expanding W in its load
 *                             stage wherever M and d_out are multiples of 256.
 * lora_workspace_bytes depends on it: size the workspace after setting it,
 * and do not change it while a call that was sized under another mode is
 * pending.  Returns the previous mode, or LORA_ERR_SHAPE for another value
 * (no change).  No HIP call.
 */
#define LORA_NF4_PATH_AUTO 0
#define LORA_NF4_PATH_DEQUANT 1
#define LORA_NF4_PATH_LOAD_STAGE 2
int lora_set_nf4_fwd_path(int mode);
int nf4_lora_linear_fwd(int64_t M, int64_t d_in, int64_t d_out, int64_t r, float scale,
                        const void* X, const uint8_t* W_nf4, const float* absmax, int blocksize,
                        const float* table16, const void* A, const void* B, void* Y, void* ws,
                        size_t ws_bytes, void* stream);

/* Backward with the NF4 base weight; outputs as lora_linear_bwd.  Never forms dW. */
int nf4_lora_linear_bwd(int64_t M, int64_t d_in, int64_t d_out, int64_t r, float scale,
                        const void* X, const uint8_t* W_nf4, const float* absmax, int blocksize,
                        const float* table16, const void* A, const void* B, const void* dY,
                        void* dX, float* dA, float* dB, void* ws, size_t ws_bytes, void* stream);

/*
 * Dequantise n NF4 elements to bf16 bit patterns with the same device routine
 * the NF4 GEMMs use in their load stage (exposed so it can be checked bit for
 * bit).  n must be a multiple of blocksize (64).  table16 is a HOST pointer.
 */
int nf4_dequant(const uint8_t* W_nf4, const float* absmax, int blocksize, int64_t n,
                const float* table16, uint16_t* out_bf16, void* stream);

/*
 * LoRA dropout on the adapter's input (page "微调太慢？试试Unsloth…", section
 * 3.3, configuration E trains with dropout 0.05; page "Unsloth框架：高效LLM微调
 * 与LoRA优化实践", section 2.2, passes lora_dropout = 0.1): inverted dropout
 * D = X * keep / (1 - p) feeds only the rank-r branch, the base path sees X:
 *     Y  = X W^T + s (D A^T) B^T
 *     dX = G W + s ((G B) A) * keep / (1 - p),  dA = s (G B)^T D,  dB = s G^T (D A^T).
 * keep: device bit mask [M, d_in / 8] bytes, bit b of byte (i, j) keeps element
 * (i, 8 j + b); the caller draws it (the library has no random generator) and
 * passes the same mask to the backward.  0 <= p < 1.  The masked copy of X is
 * exact and 1 / (1 - p) joins s in the rank-r panels; the masked rank-r term
 * of dX is a separate rank-r GEMM added into dX.  Other arguments, workspace
 * (op LORA_OP_DROPOUT_FWD / _BWD) and errors as lora_linear_fwd / _bwd;
 * LORA_ERR_SHAPE if p is outside [0, 1).
 */
int lora_dropout_fwd(int dtype, int64_t M, int64_t d_in, int64_t d_out, int64_t r, float scale, float p,
                     const uint8_t* keep, const void* X, const void* W, const void* A, const void* B, void* Y,
                     void* ws, size_t ws_bytes, void* stream);
int lora_dropout_bwd(int dtype, int64_t M, int64_t d_in, int64_t d_out, int64_t r, float scale, float p,
                     const uint8_t* keep, const void* X, const void* W, const void* A, const void* B,
                     const void* dY, void* dX, float* dA, float* dB, void* ws, size_t ws_bytes, void* stream);

/*
 * The dropout keep mask drawn on the device from the counter-based generator
 * Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
 * as 1, 2, 3", SC'11, section 4), so that a backward regenerates its forward's
 * mask from the same (seed, offset) instead of keeping it.  Element e of the
 * row-major [M, d_in] input takes word e mod 4 of the generator's block for
 * the counter (lo32(e / 4), hi32(e / 4), lo32(offset), hi32(offset)) under the
 * key (lo32(seed), hi32(seed)), and is kept iff that word >= floor(p 2^32).
 * keep: device output [M, d_in / 8] bytes in lora_dropout_fwd's bit order.
 * Needs d_in % 8 == 0 and 0 <= p < 1 (else LORA_ERR_SHAPE); asynchronous.
 */
int lora_dropout_mask(int64_t M, int64_t d_in, float p, uint64_t seed, uint64_t offset, uint8_t* keep,
                      void* stream);

/*
 * lora_dropout_fwd / _bwd with the mask drawn on the device as
 * lora_dropout_mask(M, d_in, p, seed, offset) draws it (one pass over X
 * writes the masked copy and, in the backward, the bits); the same
 * (seed, offset) in the forward and the backward gives the same mask.
 * Results equal lora_dropout_fwd / _bwd given that mask.  Workspace: ops
 * LORA_OP_DROPOUT_FWD / _BWD; errors as there.
 */
int lora_dropout_philox_fwd(int dtype, int64_t M, int64_t d_in, int64_t d_out, int64_t r, float scale, float p,
                            uint64_t seed, uint64_t offset, const void* X, const void* W, const void* A,
                            const void* B, void* Y, void* ws, size_t ws_bytes, void* stream);
int lora_dropout_philox_bwd(int dtype, int64_t M, int64_t d_in, int64_t d_out, int64_t r, float scale, float p,
                            uint64_t seed, uint64_t offset, const void* X, const void* W, const void* A,
                            const void* B, const void* dY, void* dX, float* dA, float* dB, void* ws,
                            size_t ws_bytes, void* stream);

/*
 * Merge for inference: W_out = W + scale * B A, one GEMM over the rank (fp32
 * accumulation) whose epilogue adds W and rounds once to the output type.
 * Page "微调太慢？试试Unsloth：实测训练速度翻倍，显存占用减半", section 5.1: for
 * inference the adapter is folded into the main weight, so no rank-r branch
 * runs per token; page "Unsloth自动化优化：无需手动调参的实现原理", section 3.2:
 * the adapter product and the original weight combined in one kernel.
 * Unmerge is the same call with -scale (it restores W up to the output type's
 * rounding, since the merge rounded).  W_out may be W (in place: every element
 * is read and written by the same thread, and by no other).  dtype LORA_F32 or
 * LORA_BF16; W, W_out [d_out, d_in], A [r, d_in], B [d_out, r]; workspace of
 * lora_workspace_bytes(LORA_OP_MERGE, dtype, 0, d_in, d_out, r) bytes (a
 * padded copy of B when r is not a multiple of 8, else none).  An NF4 weight
 * cannot absorb the adapter without re-quantising; there is no NF4 merge.
 */
int lora_merge(int dtype, int64_t d_out, int64_t d_in, int64_t r, float scale, const void* W, const void* A,
               const void* B, void* W_out, void* ws, size_t ws_bytes, void* stream);

/*
 * Groups of projections that read the same input X: q/k/v of attention,
 * gate/up of the MLP.  Page "UnSloth加速微调体验…", section RoPE缓存集成 fuses
 * q_proj with its LoRA branch; page "Unsloth框架：高效LLM微调与LoRA优化实践",
 * section 3.1 (graph rewriting), merges adjacent linear layers; page
 * "Unsloth自动化优化：无需手动调参的实现原理", section 3.3, walks the layer as
 * the segments q, k, v, o, gate, up, down.  A group call runs the
 * rank-r panels of all its members in ONE pass over X, with A_1 .. A_n stacked:
 * the forward panel s X A^T, the backward's recomputation of X A^T and the dA
 * contraction over X.  Everything else runs per member exactly as in the
 * single-projection entry points, so every member's outputs equal that
 * member's single call up to rounding order.  (fp32 groups run their members
 * one after another.)
 *
 * `members` is a HOST array of n (1 <= n <= LORA_GROUP_MAX) descriptions whose
 * pointers are device pointers.  Per member: d_out, r and the pointer rules
 * are those of one projection; `scale` is its s; `rope` = 1 gives it the RoPE
 * epilogue of lora_qk_rope_fwd with the group's head_dim / positions / caches
 * (then head_dim must be 128 and d_out a multiple of it); `W_nf4` (with
 * `absmax`, blocksize 64, d_in a multiple of 64, bf16 only, no RoPE) replaces W
 * by an NF4 base weight decoded with the HOST table `table16` as in
 * nf4_lora_linear_fwd.  Forward writes every member's Y.  Backward writes
 * every member's dA, dB and, where dX is not NULL, the member's own input
 * gradient (not summed over the group).  The rope and table arguments may be
 * NULL when no member needs them.
 * On MI355X the whole-tile GEMM reads W^T (rows of W's input dimension)
 * about 12 % faster than W with its contraction rows, so the bf16 backward
 * forms dX = G W from W^T: from `W_t` when the caller keeps one (W is frozen,
 * so one lora_transpose serves every step), else from a per-call transpose
 * in the workspace.
 */
#define LORA_GROUP_MAX 8
typedef struct lora_group_member {
  int64_t d_out, r;
  float scale;
  int rope;
  const void* W;          /* [d_out, d_in], or NULL when W_nf4 is given */
  const uint8_t* W_nf4;   /* NF4 codes [d_out * d_in / 2], or NULL */
  const float* absmax;    /* [d_out * d_in / 64] with W_nf4 */
  const void* A;          /* [r, d_in] */
  const void* B;          /* [d_out, r] */
  void* Y;                /* forward output [M, d_out] */
  const void* dY;         /* backward input [M, d_out] */
  void* dX;               /* backward output [M, d_in], or NULL */
  float* dA;              /* backward output [r, d_in] fp32 */
  float* dB;              /* backward output [d_out, r] fp32 */
  const void* W_t;        /* optional W^T [d_in, d_out] (bf16, e.g. from lora_transpose): the
                             backward's input gradient reads it instead of transposing W per call */
} lora_group_member;

/* Workspace bytes of lora_group_fwd (backward = 0) or lora_group_bwd (1); 0 for
 * invalid arguments. */
size_t lora_group_workspace_bytes(int backward, int dtype, int64_t M, int64_t d_in, int n,
                                  const lora_group_member* members);

int lora_group_fwd(int dtype, int64_t M, int64_t d_in, int n, const lora_group_member* members,
                   const void* X, int head_dim, const int32_t* positions, const float* cos_cache,
                   const float* sin_cache, int64_t max_pos, const float* table16, void* ws,
                   size_t ws_bytes, void* stream);

int lora_group_bwd(int dtype, int64_t M, int64_t d_in, int n, const lora_group_member* members,
                   const void* X, int head_dim, const int32_t* positions, const float* cos_cache,
                   const float* sin_cache, int64_t max_pos, const float* table16, void* ws,
                   size_t ws_bytes, void* stream);

/*
 * SwiGLU on a gate / up pair that reads the same X (the gated unit of the
 * Llama MLP): G and U are the two fused LoRA projections of X (each as
 * lora_linear_fwd or nf4_lora_linear_fwd), H = silu(G) * U elementwise,
 * silu(z) = z / (1 + e^-z).  Page "Unsloth框架：高效LLM微调与LoRA优化实践",
 * section 3.1: the graph rewriter merges adjacent linear layers with their
 * activation function; page "Unsloth自动化优化：无需手动调参的实现原理",
 * section 1: SwiGLU is one of the module types it optimises.
 * members[0] is the gate and members[1] the up projection (lora_group_member
 * with equal d_out, rope = 0, W or W_nf4 as in the group calls); their rank-r
 * panels run in one pass over X as in lora_group_fwd.  With bf16, M a multiple
 * of 256, d_out of 128, d_in of 64 (and for an NF4 member M >= 512, where its
 * weight is dequantised once), gate and up run as ONE GEMM whose epilogue
 * forms H from the fp32 accumulators; other shapes form G and U with the group
 * path and H in an elementwise pass from G and U rounded to the dtype.
 * H: [M, d_out] in the dtype.  members[g].Y, when not NULL, receives G (g = 0)
 * and U (g = 1) in the dtype, as the backward needs them.
 */
int lora_swiglu_fwd(int dtype, int64_t M, int64_t d_in, const lora_group_member* members, const void* X,
                    const float* table16, void* H, void* ws, size_t ws_bytes, void* stream);

/*
 * Backward of lora_swiglu_fwd for the upstream gradient dH [M, d_out]:
 * dG = dH * U * silu'(G) and dU = dH * silu(G) (G, U as the forward stored
 * them; silu'(z) = s (1 + z (1 - s)), s = 1 / (1 + e^-z)), then the LoRA
 * backward of both projections with their panels shared as in lora_group_bwd.
 * dX [M, d_in] (NULL: skipped) receives the SUM of the two input gradients;
 * members[g].dA and .dB receive each adapter's gradients (fp32, overwritten);
 * members[g].dY, .dX and .Y are not used.
 */
int lora_swiglu_bwd(int dtype, int64_t M, int64_t d_in, const lora_group_member* members, const void* X,
                    const float* table16, const void* dH, const void* G, const void* U, void* dX, void* ws,
                    size_t ws_bytes, void* stream);

/* Workspace bytes of lora_swiglu_fwd (backward = 0) or lora_swiglu_bwd (1); 0
 * for invalid arguments. */
size_t lora_swiglu_workspace_bytes(int backward, int dtype, int64_t M, int64_t d_in,
                                   const lora_group_member* members);

/*
 * One projection with bias, activation and residual in its epilogue (page
 * "Unsloth框架：高效LLM微调与LoRA优化实践", section 3.1: the graph rewriter merges
 * a linear layer with its neighbours):
 *     Z = X W^T + s (X A^T) B^T + bias,   Y = act(Z) + residual
 * Z is activated in fp32 where the product is accumulated; Y is rounded once.
 * `member` is one lora_group_member (rope = 0; W, or W_nf4 with absmax and
 * the HOST table16 as in nf4_lora_linear_fwd; W_t as in the group calls); Y is
 * member->Y.  Activations: RELU max(z, 0), SILU z / (1 + e^-z), GELU
 * z P(N(0,1) <= z), GELU_TANH z / (1 + e^(-2 u)) with
 * u = sqrt(2 / pi) (z + 0.044715 z^3).  bias [d_out], residual [M, d_out] and Z
 * [M, d_out] are of the dtype; each may be NULL.  Z, where given, receives the
 * pre-activation, which the backward of an activation needs.  residual may be
 * Y itself (the sum formed in place); Y and Z may be no other input.
 * Workspace from its own sizing call; sizes and errors as lora_linear_fwd and
 * nf4_lora_linear_fwd, and d_out <= LORA_EPI_MAX_D_OUT (2^20).
 *
 * Backward, for member->dY:
 *     dZ = dY act'(Z)  (rounded to the dtype; dY itself with LORA_ACT_NONE),
 *     dbias = sum over tokens of dZ,
 * and dX (NULL: skipped), dA, dB from dZ as lora_linear_bwd; the residual's
 * gradient is dY.  act and Z are taken from `epilogue` (its bias and residual
 * are not used).  RELU passes no gradient at 0 and below, whatever dY holds
 * there.  dbias: fp32 [d_out] (overwritten) or NULL.
 */
#define LORA_EPI_MAX_D_OUT (1 << 20)
enum { LORA_ACT_NONE = 0, LORA_ACT_RELU = 1, LORA_ACT_SILU = 2, LORA_ACT_GELU = 3, LORA_ACT_GELU_TANH = 4 };
typedef struct lora_epilogue {
  int act;
  const void* bias;
  const void* residual;
  void* Z;
} lora_epilogue;

int lora_linear_epi_fwd(int dtype, int64_t M, int64_t d_in, const lora_group_member* member,
                        const lora_epilogue* epilogue, const void* X, const float* table16, void* ws, size_t ws_bytes,
                        void* stream);
int lora_linear_epi_bwd(int dtype, int64_t M, int64_t d_in, const lora_group_member* member,
                        const lora_epilogue* epilogue, const void* X, const float* table16, float* dbias, void* ws,
                        size_t ws_bytes, void* stream);
/* Workspace bytes of the two (backward = 0 / 1; act and the member's sizes and
 * W_nf4 / W_t are read); 0 for invalid arguments. */
size_t lora_linear_epi_workspace_bytes(int backward, int dtype, int64_t M, int64_t d_in,
                                       const lora_group_member* member, const lora_epilogue* epilogue);

/*
 * dst [cols, rows] = src [rows, cols]^T for bf16 matrices (rows and cols
 * multiples of 8), e.g. the frozen W^T that the backward can take as
 * lora_group_member.W_t.  Asynchronous on `stream`.
 */
int lora_transpose(const void* src, int64_t rows, int64_t cols, void* dst, void* stream);

/*
 * Root-mean-square norm in front of a block's projections, with the residual
 * stream's addition:
 *     h = x + residual (rounded to the type; x itself without a residual)
 *     rstd = 1 / sqrt(mean of h^2 over the row + eps),   y = h rstd w
 * X [M, d] (row stride ldx >= d elements), residual [M, d] (row stride ldr, or
 * NULL) and weight [d] of the dtype.  Outputs, each of them optional (NULL; one
 * at least): H [M, d] = h, Y [M, d] = y, rstd fp32 [M], and codes [M, d] with
 * scale8 [M]: y as lora_act8_pack keeps it, rounded once (from y before its
 * rounding to the dtype).  H may be X or the residual (the stream updated in
 * place), Y may be X without a residual; with row strides of d (others are
 * refused there).  The sum of squares is kept in 64 bits, rstd in fp32 (root mean
 * squares from 2^-126 to 2^126 have one); a y past fp32's range is an infinity,
 * for the codes too.  Pointers need their element's alignment only.  1 <= d <= LORA_NORM_MAX_DIM, 0 <= M < 2^31, eps >= 0
 * (a row of zeros with eps 0 gives NaN).
 *
 * Backward, for dY [M, d] and, where the stream goes on, dH [M, d] (NULL: 0),
 * from H and rstd as the forward gave them:
 *     g = dY w,  xh = h rstd,  dX = rstd (g - xh mean(g xh)) + dH,
 *     dweight = sum over rows of dY xh
 * dX is the gradient of x and of the residual.  dX [M, d] may be NULL, or dY or
 * dH itself; dweight [d] of dweight_dtype may be NULL (then no workspace is
 * needed).  Rows are summed in fp32 in a fixed order.  M = 0: dweight is zeros.
 */
#define LORA_NORM_MAX_DIM 32768
int lora_rmsnorm_fwd(int dtype, int64_t M, int64_t d, float eps, const void* X, int64_t ldx, const void* residual,
                     int64_t ldr, const void* weight, void* H, void* Y, uint8_t* codes, float* scale8, float* rstd,
                     void* stream);
int lora_rmsnorm_bwd(int dtype, int64_t M, int64_t d, const void* H, const void* weight, const float* rstd,
                     const void* dY, const void* dH, void* dX, void* dweight, int dweight_dtype, void* ws,
                     size_t ws_bytes, void* stream);
size_t lora_rmsnorm_workspace_bytes(int64_t M, int64_t d);

/*
 * Activations kept in 8 bits between a forward and its backward (page
 * "Unsloth教程：本地微调大模型速度提升数倍，显存节省60%", section 显存优化策略).  Row t
 * of X [M, d] (row stride ldx) is codes [M, d], e4m3 (OCP: 4 exponent and 3
 * mantissa bits, largest 448), times scale8[t] = 2^e with the smallest
 * e >= -126 that keeps the row's largest finite magnitude at or below 448 (1
 * for a row of zeros):
 *     code = e4m3(x 2^-e), rounded to nearest even;   x is taken as code 2^e.
 * A value is off by at most 2^-4 of itself, or 2^(e - 10) where it is below
 * 2^(e - 6).  Infinities and NaNs become NaN codes.  lora_act8_unpack
 * writes code 2^e, [M, d]: exact in either type, but that bf16 has steps of 2^-133
 * below 2^-125, and that what was 1.9375 2^127 or more in size, rounded to 2^128,
 * is an infinity.
 *
 * lora_act8_linear_bwd is the backward of lora_linear_fwd (and of its NF4 form)
 * with the checkpoint in X's place: of the three gradients only the
 * adapter's read X, through X A^T and (dY B)^T X.  member as in
 * lora_linear_epi_bwd (W, or W_nf4 with absmax and the HOST table16; W_t; dY, dX
 * or NULL, dA, dB; with grad_dtype LORA_BF16 the latter two are bf16 arrays); codes
 * 16-byte aligned; its own sizing call; d_in <= LORA_NORM_MAX_DIM.  dX does not
 * depend on X.
 */
int lora_act8_pack(int dtype, int64_t M, int64_t d, const void* X, int64_t ldx, uint8_t* codes, float* scale8,
                   void* stream);
int lora_act8_unpack(int dtype, int64_t M, int64_t d, const uint8_t* codes, const float* scale8, void* X,
                     void* stream);
int lora_act8_linear_bwd(int dtype, int64_t M, int64_t d_in, const lora_group_member* member, const uint8_t* codes,
                         const float* scale8, const float* table16, int grad_dtype, void* ws, size_t ws_bytes,
                         void* stream);
size_t lora_act8_linear_workspace_bytes(int dtype, int64_t M, int64_t d_in, const lora_group_member* member, int grad_dtype);

/*
 * A projection whose rows each carry an adapter of their own: requests that
 * share a base weight (decode steps and packed prompts) and several adapters
 * trained at once.  n adapters of one rank (smaller ones padded with zeros),
 * A [n, r, d_in], B [n, d_out, r] of the dtype, scales fp32 [n] (s_a = alpha / r),
 * index: device int32 [M], the row's adapter; a row whose index lies outside
 * [0, n) has none:
 *     y_t = W x_t + s_a B_a (A_a x_t),   a = index[t]
 * Rows may come in any order.  What it costs grows with the number of adapters
 * that meet in 128 or 256 consecutive rows, so requests' tokens should lie together.
 * r a multiple of 8 up to LORA_MULTI_MAX_RANK, 1 <= n <= LORA_MULTI_MAX_ADAPTERS,
 * d_in and d_out as in lora_linear_fwd and at most LORA_EPI_MAX_D_OUT.
 * An infinity or NaN stays with its own: one in an adapter's A or B makes its
 * rows' outputs (dX) and its gradients NaN where the definition may leave some
 * finite, one in a row of X or dY its adapter's gradients; other adapters and rows do
 * not see it.  Y and dX overlap no input.
 * index and scales need their element's alignment only.  The forward takes any
 * M < 2^31, 2^23 rows after 2^23 rows with one workspace.  Workspace from its own
 * sizing call (with backward != 0: have_w_t whether W_t is given, need_dx
 * whether dX is).
 *
 * Backward, for dY [M, d_out]:
 *     dX_t = W^T dy_t + s_a A_a^T (B_a^T dy_t)
 *     dB_a = s_a sum_{t in a} dy_t (A_a x_t)^T,  dA_a = s_a sum_{t in a} (B_a^T dy_t) x_t^T
 * dX [M, d_in] or NULL; dA [n, r, d_in] and dB [n, d_out, r] of grad_dtype, zeros for
 * an adapter without rows, sums over rows in a fixed order.  W_t: W^T [d_in,
 * d_out] (bf16, lora_transpose) where the caller keeps one, else NULL (a bf16
 * call that needs it makes its own); fp32 calls do not read it.  The backward takes
 * LORA_MULTI_MAX_BWD_ROWS rows at most.
 */
#define LORA_MULTI_MAX_RANK 128
#define LORA_MULTI_MAX_ADAPTERS 4096
#define LORA_MULTI_MAX_BWD_ROWS (1 << 21)
size_t lora_multi_workspace_bytes(int backward, int dtype, int64_t M, int64_t d_in, int64_t d_out, int64_t n, int64_t r,
                                  int have_w_t, int need_dx);
int lora_multi_fwd(int dtype, int64_t M, int64_t d_in, int64_t d_out, int64_t n, int64_t r, const void* X, const void* W,
                   const void* A, const void* B, const float* scales, const int32_t* index, void* Y, void* ws,
                   size_t ws_bytes, void* stream);
int lora_multi_bwd(int dtype, int64_t M, int64_t d_in, int64_t d_out, int64_t n, int64_t r, const void* X, const void* W,
                   const void* W_t, const void* A, const void* B, const float* scales, const int32_t* index, const void* dY,
                   void* dX, void* dA, void* dB, int grad_dtype, void* ws, size_t ws_bytes, void* stream);

/*
 * Log-probabilities of tokens from their logits (the head projection of a
 * training step: preference and policy losses read them, and their gradient
 * goes back through the head's LoRA layer).  For row i with target t_i:
 *     logp_i = tau z_{i,t_i} - log sum_j e^(tau z_{i,j})
 *     dz_{i,j} = dlogp_i tau (1[j = t_i] - e^(tau z_{i,j}) / sum_k e^(tau z_{i,k}))
 * logits: [n, vocab] of the dtype, row stride ld >= vocab elements; targets:
 * int64 [n]; tau = inv_temp, above 0 and at most LORA_LOGP_MAX_INV_TEMP.  A target outside
 * [0, vocab) names no token: logp is 0 and the row's gradient zeros.  stats
 * [n, 2] fp32 receives each row's maximum logit m and log sum_j e^(tau (z_j - m))
 * (their sum tau m + that is the log-sum-exp); the backward takes them back.
 * Logits of -infinity (masked vocabulary) have probability 0; a row of
 * -infinities, a +infinity or a NaN gives a NaN.  The backward writes
 * dlogits [n, vocab] (row stride ld_d) in the dtype; it may be logits itself
 * (ld_d = ld).  A row whose dlogp is 0, or whose target names no token, is not
 * read and gets zeros.  Arithmetic is fp32; a logp near 0 and 1 - p of such a
 * target keep their relative accuracy.  Pointers need their element's
 * alignment only, so rows may be sliced (logits[:-1], targets[1:]).
 * 0 <= n < 2^31, 1 <= vocab < 2^31.
 */
#define LORA_LOGP_MAX_INV_TEMP 1e38f /* (tau log2 e is an fp32 number) */
int lora_token_logp_fwd(int dtype, int64_t n, int64_t vocab, const void* logits, int64_t ld, const int64_t* targets,
                        float inv_temp, float* logp, float* stats, void* stream);
int lora_token_logp_bwd(int dtype, int64_t n, int64_t vocab, const void* logits, int64_t ld, const int64_t* targets,
                        float inv_temp, const float* stats, const float* dlogp, void* dlogits, int64_t ld_d,
                        void* stream);

/*
 * Losses over packed sequences: n_tokens fp32 values, sequence s being the
 * tokens [cu[s], cu[s + 1]) (cu: device int64 [n_seq + 1], non-decreasing;
 * sequences may be empty).  mask: device bytes [n_tokens] (NULL: every token
 * counts); a token whose byte is 0 counts nowhere, whatever its values.
 * Tokens outside [cu[0], cu[n_seq]) belong to no sequence.  The host cannot
 * read cu: offsets outside [0, n_tokens] are taken as the nearer end, and
 * offsets that decrease give unspecified values but no access outside the
 * arrays.  Sums over tokens, and what is derived from them, are formed in fp64
 * in a fixed order.  Pointers need their element's alignment only (ws: 16
 * bytes, of lora_loss_workspace_bytes).  dloss: device fp32 scalar, the
 * upstream gradient of the loss (NULL: 1).  The backward writes dlogp for every
 * token of [0, n_tokens): 0 where it does not count.
 * 1 <= n_seq <= 2^30, 0 <= n_tokens < 2^40 (with 0 the token arrays may be NULL).
 */
enum { LORA_LOSS_PREFERENCE = 0, LORA_LOSS_POLICY = 1 };
size_t lora_loss_workspace_bytes(int loss, int64_t n_seq, int64_t n_tokens);

/*
 * Preference loss of `pairs` pairs: sequences 0 .. pairs-1 are the chosen
 * responses, pairs .. 2 pairs-1 the rejected ones (cu has 2 pairs + 1 entries).
 *     D_s = sum of logp - ref_logp over the counted tokens of s (over their
 *           number, if `average`; 0 for a sequence that counts none),
 *     u = D_chosen - D_rejected,
 *     SIGMOID: l = (1 - e) softplus(-beta u) + e softplus(beta u)
 *     HINGE:   l = max(0, 1 - beta u)
 *     IPO:     l = (u - 1 / (2 beta))^2
 * and the loss is the mean of l over the pairs.  e = label_smoothing in
 * [0, 1), 0 but for SIGMOID; beta > 0.  ref_logp NULL: no reference (zeros).
 * Outputs fp32: loss [1], pair_loss [pairs], rewards [2 pairs] = beta D_s,
 * coef [2 pairs] = d loss / d logp of a counted token of s, which the backward
 * spreads over the tokens.
 */
enum { LORA_PREF_SIGMOID = 0, LORA_PREF_HINGE = 1, LORA_PREF_IPO = 2 };
int lora_preference_loss_fwd(int kind, int64_t pairs, int64_t n_tokens, double beta, double label_smoothing,
                             int average, const int64_t* cu, const uint8_t* mask, const float* logp,
                             const float* ref_logp, float* loss, float* pair_loss, float* rewards, float* coef,
                             void* ws, size_t ws_bytes, void* stream);
int lora_preference_loss_bwd(int64_t pairs, int64_t n_tokens, const int64_t* cu, const uint8_t* mask,
                             const float* coef, const float* dloss, float* dlogp, void* stream);

/*
 * Clipped policy loss with a KL term.  Per counted token, with advantage A (of
 * its sequence, [n_seq], or its own, [n_tokens], if adv_per_token),
 * x = logp - old_logp (old_logp NULL: 0, the policy that sampled), r = e^x and
 * d = ref_logp - logp:
 *     l = -min(r A, clip(r, 1 - eps_low, 1 + eps_high) A) + beta (e^d - d - 1)
 *     dl / dlogp = (-r A where r A <= the clipped product, else 0) - beta (e^d - 1)
 * A = 0 leaves the KL term alone.  The clip borders are compared as
 * x > log(1 + eps_high) and x < log(1 - eps_low) in fp64.  The loss is
 * sum_t w l with w = 1 / (n_seq T_s) (SEQUENCE: mean over sequences of their
 * token mean, T_s counted tokens), 1 / sum_s T_s (TOKEN) or 1 / (n_seq norm)
 * (CONSTANT).  0 <= eps_low <= 1, eps_high >= 0, beta >= 0 (beta > 0 needs
 * ref_logp; with beta = 0 a ref_logp gives the KL statistic alone).
 * Outputs fp32: loss [1]; stats [4] = the policy part, the KL part (before
 * beta), the share of counted tokens whose clipped branch held, their number;
 * weight [n_seq] = w, which the backward takes back with the same inputs.
 */
enum { LORA_POLICY_SEQUENCE = 0, LORA_POLICY_TOKEN = 1, LORA_POLICY_CONSTANT = 2 };
int lora_policy_loss_fwd(int reduction, int64_t n_seq, int64_t n_tokens, double eps_low, double eps_high, double beta,
                         double norm, const int64_t* cu, const uint8_t* mask, const float* logp,
                         const float* old_logp, const float* ref_logp, const float* advantages, int adv_per_token,
                         float* loss, float* stats, float* weight, void* ws, size_t ws_bytes, void* stream);
int lora_policy_loss_bwd(int64_t n_seq, int64_t n_tokens, double eps_low, double eps_high, double beta,
                         const int64_t* cu, const uint8_t* mask, const float* logp, const float* old_logp,
                         const float* ref_logp, const float* advantages, int adv_per_token, const float* weight,
                         const float* dloss, float* dlogp, void* stream);

/*
 * Launch profiling (measurement hook, not part of the layer's arithmetic).
 * Between lora_profile_begin and lora_profile_end every kernel the library
 * launches is bracketed by two HIP events on its stream, and the launch's
 * algorithmic FLOP and minimum HBM bytes are recorded with its kind.  At most
 * max_launches launches are recorded (later ones are not).  Query after the
 * stream has been synchronised.  Kinds are numbered 0 .. lora_profile_kinds()-1.
 *   lora_profile_begin: LORA_ERR_SHAPE if max_launches < 1; LORA_ERR_DEVICE if
 *     event creation fails.
 *   lora_profile_query: totals over the recorded launches of `kind`:
 *     summed event time in ms, launch count, summed FLOP, summed bytes.
 *   lora_profile_only: from now on record only launches of `kind` (-1: every
 *     kind, the state at load); the others run without events, so a timed run
 *     can bracket one kernel kind without slowing the rest.  LORA_ERR_SHAPE if
 *     kind is outside [-1, lora_profile_kinds()).  No HIP call.
 */
int lora_profile_begin(int max_launches);
int lora_profile_end(void);
int lora_profile_only(int kind);
int lora_profile_kinds(void);
const char* lora_profile_kind_name(int kind);
int lora_profile_query(int kind, double* total_ms, int* count, double* total_flop, double* total_bytes);

/*
 * MFMA rate probe (measurement hook, not part of the layer's arithmetic): an
 * asynchronous launch of `blocks` workgroups of 4 waves (one per SIMD), each
 * wave running `iters` rounds of 8 independent v_mfma_f32_32x32x16_bf16 on
 * register operands, so the work is blocks * 4 * iters * 8 * 32768 FLOP; the
 * caller times it on `stream`.  This is the dense bf16 rate the chip sustains
 * under its own power and clock limits, next to the published peak.  out:
 * device fp32 [blocks * 256].  LORA_ERR_SHAPE if iters or blocks < 1.
 */
int lora_mfma_rate(int iters, int blocks, float* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_LINEAR_H */
