/*
 * muonh.h - C ABI of the MI355X (gfx950) MuonH optimizer step.
 *
 * MuonH updates a set of weight matrices with Muon's orthogonalized momentum
 * update and then puts every matrix back on the sphere of the Frobenius norm
 * it had at initialization. Sources, cited by page title and section:
 *   - digest page "Puro-2B trains for $6.9K, attention sinks hit 99%,
 *     LoopArena tops at 24.69%", section "The load-bearing tricks aren't in
 *     the abstract" and footnotes 3-4: MuonH extends Muon, fixes each matrix's
 *     Frobenius norm at its initialization value by projecting updates onto a
 *     fixed hypersphere; Muon's overhead is its Newton-Schulz iterations;
 *   - model card "Puro", section "Training": MuonH with hyperball projection
 *     and zero weight decay on the matrix group; master weights and optimizer
 *     state in FP32 or BF16 (W fp32 here; G and M fp32 or bf16 by plan flag).
 *
 * One step, per matrix (rows x cols, row-major fp32):
 *   M  <- beta*M + G                                  (heavy-ball momentum)
 *   X0  = M / (||M||_F + 1e-7), transposed when rows > cols
 *   ns_iters times:  A = X X^T;  B = b*A + c*A*A;  X <- a*X + B*X
 *                    (a, b, c) = (3.4445, -4.7750, 2.0315)
 *   O   = X (transposed back)
 *   W'  = W - lr*O
 *   W  <- (R / ||W'||_F) * W'        (W <- W' when ||W'||_F == 0)
 * with R = ||W0||_F captured once by muonh_init. The pages give neither the
 * momentum rule, nor the polynomial, nor the normalisation: the readings above
 * are the plainest ones consistent with the pages (no update scale, no weight
 * decay, no Nesterov).
 *
 * Conventions for every call below
 *   - Matrices are grouped by shape: a plan lists groups {rows, cols, count};
 *     matrix index i runs over group 0's matrices, then group 1's, etc.
 *   - W, G, M are DEVICE arrays of n_matrices DEVICE pointers (the layout of
 *     batched-BLAS pointer arrays); each points to a contiguous row-major
 *     rows x cols matrix: W in fp32; G and M in fp32, or in bf16 (bits of
 *     IEEE binary32's upper half) under the plan flags MUONH_GRAD_BF16 and
 *     MUONH_MOM_BF16 (so G and M are typed void). R is a DEVICE array of
 *     n_matrices floats. Pointers aligned to 4 elements (16 bytes fp32,
 *     8 bytes bf16) take the vector path; others work through a scalar path.
 *     W, G and M must not overlap.
 *   - The workspace is a DEVICE buffer of at least muonh_workspace_bytes(plan)
 *     bytes, 256-byte aligned, owned by the caller. It holds the
 *     Newton-Schulz operands (bf16, split bf16 or fp32 by plan flag) and the
 *     norm partials. After a step it holds that step's update O until the
 *     next call that uses it.
 *   - All device work is enqueued asynchronously on `stream` (a hipStream_t;
 *     NULL is the default stream). No call synchronises the device, except
 *     muonh_step_status, which waits for `stream`.
 *   - Calls that share a workspace must be ordered by the caller (same stream,
 *     or events). A plan itself is read-only after creation and may be shared.
 *   - All argument checks run before any work is enqueued; a call that returns
 *     an error has enqueued nothing. Negative return values are errors;
 *     muonh_last_error() gives a message for the calling thread.
 *   - Non-finite inputs are not errors: they propagate into the results. A
 *     step records in the workspace whether a norm it took was not finite
 *     (muonh_step_status reads that record).
 */
#ifndef MUONH_H
#define MUONH_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MUONH_ABI_VERSION 3

typedef struct muonh_plan muonh_plan;

typedef struct {
  int32_t rows;   /* rows of every matrix in the group, >= 1 */
  int32_t cols;   /* columns of every matrix in the group, >= 1 */
  int32_t count;  /* number of matrices in the group, >= 1 */
} muonh_group_desc;

enum {
  MUONH_OK = 0,
  MUONH_EINVAL = -1,     /* bad argument (null pointer, value out of range) */
  MUONH_ESHAPE = -2,     /* bad group description or matrix index */
  MUONH_EWORKSPACE = -3, /* workspace missing, too small or misaligned */
  MUONH_EHIP = -4,       /* a HIP runtime call failed (see muonh_last_error) */
  MUONH_ENOMEM = -5,     /* host allocation failed */
  MUONH_EALIAS = -6      /* two of the W, G, M matrices (or an fp8 call's arrays) overlap */
};

/* Newton-Schulz plan flags (at most one). Default: operands in bf16, bf16
 * MFMA with fp32 accumulation; about 1e-2 relative error of O at 5
 * iterations, about 1.8e-2 at 8. With bf16 or split operands and
 * ns_iters >= 1, X0's factor 1/(||M||_F + 1e-7) is applied inside the first
 * iteration's products rather than before rounding M to the operand format
 * (the same value up to that rounding; matrices of at most 65536 entries,
 * and momentum norms outside [2^-40, 2^40], are normalised first). For
 * matrices of more than 65536 entries the polynomial stores
 * B' = a*I + b*A + c*A*A and the update is X <- B' X: the same algebra as
 * a*X + B*X, with a better-conditioned rounding of B'. */
enum {
  /* fp32 operands and fp32 MFMA. Debug/reference mode: about 1e-6 relative
   * error, an order of magnitude slower. */
  MUONH_NS_FP32 = 1u,
  /* Split-bf16 operands: every stored value v is kept as hi = bf16(v) plus
   * lo = bf16(v - hi), and each product takes hi*hi + hi*lo + lo*hi on bf16
   * MFMA (fp32 accumulation). About 1e-4 relative error of O at 8
   * iterations, for about 3x the Newton-Schulz time and twice its
   * workspace. */
  MUONH_NS_SPLIT_BF16 = 2u
};

/* Storage plan flags (any combination with the above; model card "Puro",
 * section "Training": master weights and optimizer state in FP32 or BF16).
 * W always stays fp32. */
enum {
  /* G is bf16: its values are taken as given. */
  MUONH_GRAD_BF16 = 4u,
  /* M is stored in bf16: the new momentum is the exact beta*M + G (beta
   * as the fp32 value passed) rounded once to the nearest bf16, ties to
   * even; that stored value is the momentum whose norm and Newton-Schulz
   * update the step uses. Cuts the momentum pass from 12 to 8 bytes per parameter
   * (6 with MUONH_GRAD_BF16). */
  MUONH_MOM_BF16 = 8u
};

/* Limits. */
#define MUONH_MAX_GROUPS 4096
#define MUONH_MAX_MATRICES (1 << 20)
#define MUONH_MAX_DIM 65536      /* rows and cols */
#define MUONH_MAX_NS_ITERS 32
#define MUONH_MAX_TENSOR_ELEMS (1LL << 40) /* elements per AdamW tensor */

/* Library ABI version (MUONH_ABI_VERSION of the built library). */
int32_t muonh_abi_version(void);

/*
 * Create a plan for `n_groups` shape groups. Host-only: no HIP call.
 * flags: at most one of MUONH_NS_FP32 and MUONH_NS_SPLIT_BF16, or'd with any
 * of MUONH_GRAD_BF16 and MUONH_MOM_BF16. On success *out owns a plan
 * that must be released with muonh_plan_destroy. Errors: MUONH_EINVAL (null
 * out/groups, n_groups out of [1, MUONH_MAX_GROUPS], unknown or conflicting
 * flags), MUONH_ESHAPE (a dim out
 * of [1, MUONH_MAX_DIM], count < 1, too many matrices, or more than 2^31
 * 64x64 tiles of the 256-padded matrices in total), MUONH_ENOMEM.
 */
int muonh_plan_create(muonh_plan** out, const muonh_group_desc* groups, int32_t n_groups,
                      uint32_t flags);

/* Release a plan (NULL is ignored). The caller must not have work in flight
 * that still needs it: plans hold no device memory, so this never syncs. */
void muonh_plan_destroy(muonh_plan* plan);

/* Number of matrices, and of matrix entries (parameters), in the plan. */
int64_t muonh_plan_num_matrices(const muonh_plan* plan);
int64_t muonh_plan_num_params(const muonh_plan* plan);

/* Bytes of device workspace that muonh_init/muonh_step need. */
size_t muonh_workspace_bytes(const muonh_plan* plan);

/*
 * R[i] <- ||W[i]||_F for every matrix (fp32 result of a fixed-order
 * reduction: squares summed 4 at a time in fp32, fp64 beyond that). Capture the
 * radius once, from the initial weights. Deterministic.
 * Errors: MUONH_EINVAL (null plan/W/R), MUONH_EWORKSPACE, MUONH_EHIP.
 */
int muonh_init(const muonh_plan* plan, float* const* W, float* R, void* workspace,
               size_t workspace_bytes, void* stream);

/*
 * One MuonH step over every matrix of the plan (formula at the top of this
 * file). W and M are updated in place; G and R are read only.
 * lr: finite, >= 0 (the caller's effective rate; the model card applies a
 *     10x multiplier to the matrix group, section "Training").
 * beta: in [0, 1).  ns_iters: in [0, MUONH_MAX_NS_ITERS].
 * Results are bitwise deterministic for a given plan and input. A matrix's
 * result does not depend on the other matrices of the plan, except that bf16
 * Newton-Schulz phases whose GEMMs have few 256x256 tiles (at most 128)
 * run 128x128 tiles, which can change the last bits of the polynomial's
 * diagonal blocks and so of O (well within the tolerances).
 * Errors: MUONH_EINVAL, MUONH_EWORKSPACE, MUONH_EHIP.
 */
int muonh_step(const muonh_plan* plan, float* const* W, const void* const* G, void* const* M,
               const float* R, float lr, float beta, int32_t ns_iters, void* workspace,
               size_t workspace_bytes, void* stream);

/* Bytes of the fixed device workspace of muonh_step_noalloc (per GPU). */
#define MUONH_NOALLOC_WORKSPACE_BYTES (128u << 20)

/*
 * muonh_step for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc): the
 * same step with the same arguments, but no caller workspace. The library
 * keeps one fixed array of MUONH_NOALLOC_WORKSPACE_BYTES (128 MiB) of
 * device memory per GPU for the life of the process, and this call runs in
 * the current device's array; it calls no allocating routine. Plans whose
 * muonh_workspace_bytes exceed that size are rejected (MUONH_EWORKSPACE),
 * before anything is enqueued. `stream` must belong to the current device.
 * Every call on one GPU shares that GPU's array and leaves its contents
 * behind (the step clears what must start at zero): calls that may overlap
 * on one GPU (other streams, other threads) race and must be ordered by the
 * caller. The update O is not kept for muonh_read_update, and the
 * non-finite record is not reachable through muonh_step_status. R comes
 * from muonh_init (with a workspace, at set-up) or from a checkpoint;
 * muonh_init also looks up this device's array, so that the first
 * muonh_step_noalloc on a device need not.
 * Errors: as muonh_step.
 */
int muonh_step_noalloc(const muonh_plan* plan, float* const* W, const void* const* G,
                       void* const* M, const float* R, float lr, float beta, int32_t ns_iters,
                       void* stream);

/*
 * muonh_step plus phase timing: the same work, with hipEventRecord of the
 * caller's events on `stream` at the phase boundaries, for profiling.
 * events: host array of n_events hipEvent_t (created by the caller, with
 * timing enabled); n_events must be 3*ns_iters + 3. Recorded, in order:
 *   [0] before the momentum update,
 *   [1] after momentum, its norm and the normalised cast (Newton-Schulz input),
 *   [2+3i], [3+3i], [4+3i] after iteration i's Gram, polynomial and apply,
 *   [3*ns_iters+2] after the trial update, its norm and the projection.
 * Errors: as muonh_step, plus MUONH_EINVAL for a NULL events array, a NULL
 * event or a wrong n_events.
 */
int muonh_step_timed(const muonh_plan* plan, float* const* W, const void* const* G,
                     void* const* M, const float* R, float lr, float beta, int32_t ns_iters,
                     void* workspace, size_t workspace_bytes, void* stream, void* const* events,
                     int32_t n_events);

/*
 * The baseline MuonH is measured against: Muon with decoupled weight decay
 * (the digest page quotes MuonH's speedup against standard weight decay,
 * section "The load-bearing tricks aren't in the abstract"; the report page,
 * part 6/7, section 4.3 "Cost Estimation", its compute multiplier relative to
 * Muon; neither prints the update). The same momentum and Newton-Schulz as
 * muonh_step, then
 *   W <- (1 - lr*weight_decay) * W - lr*O
 * with no projection and no radius. Same plan, workspace and conventions as
 * muonh_step (the two may share a plan; W and M are updated in place).
 * weight_decay: finite, >= 0. Errors: as muonh_step.
 */
int muonh_step_muon_wd(const muonh_plan* plan, float* const* W, const void* const* G,
                       void* const* M, float lr, float beta, float weight_decay,
                       int32_t ns_iters, void* workspace, size_t workspace_bytes, void* stream);

/* muonh_step_muon_wd with the phase events of muonh_step_timed (the last one
 * after the decayed update). */
int muonh_step_muon_wd_timed(const muonh_plan* plan, float* const* W, const void* const* G,
                             void* const* M, float lr, float beta, float weight_decay,
                             int32_t ns_iters, void* workspace, size_t workspace_bytes,
                             void* stream, void* const* events, int32_t n_events);

/*
 * AdamW for the parameters outside the MuonH group (model card page "Puro",
 * section "Training": AdamW with weight decay 0.1; the page gives no other
 * hyperparameter). One step at step number `step` (1-based), per element of
 * every tensor, in fp32 (decoupled decay, bias-corrected moments):
 *   p <- p*(1 - lr*weight_decay)
 *   m <- beta1*m + (1 - beta1)*g ;  v <- beta2*v + (1 - beta2)*g^2
 *   p <- p - lr*(m/(1 - beta1^step)) / (sqrt(v/(1 - beta2^step)) + eps)
 * sizes: HOST array of n_tensors element counts (0 allowed, at most
 *   MUONH_MAX_TENSOR_ELEMS). P, G, M, V: DEVICE arrays of n_tensors DEVICE
 *   pointers to flat fp32 tensors (parameters, gradients, first and second
 *   moments); P, M, V are updated in place, G is read. No plan and no
 *   workspace: tensors go in grouped launches of up to 128 tensors.
 * lr, weight_decay: finite, >= 0; beta1, beta2 in [0, 1); eps finite, >= 0.
 * n_tensors == 0 is a no-op. Deterministic; asynchronous on `stream`.
 * Errors: MUONH_EINVAL (bad scalar, NULL array, step < 1, n_tensors < 0),
 * MUONH_ESHAPE (a size out of range), MUONH_EHIP.
 */
int muonh_adamw_step(int32_t n_tensors, const int64_t* sizes, float* const* P,
                     const float* const* G, float* const* M, float* const* V, float lr,
                     float beta1, float beta2, float eps, float weight_decay, int32_t step,
                     void* stream);

/*
 * Copy the update O of matrix `index` computed by the last muonh_step (or
 * muonh_step_muon_wd) that used this workspace into dst, a DEVICE buffer of
 * rows x cols fp32 (row-major, the matrix's own orientation). For inspection
 * and tests.
 * Errors: MUONH_EINVAL, MUONH_ESHAPE (index out of range), MUONH_EWORKSPACE,
 * MUONH_EHIP.
 */
int muonh_read_update(const muonh_plan* plan, int64_t index, float* dst, const void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * Non-finite report of the last muonh_step or muonh_step_muon_wd that used
 * this workspace (0 after muonh_init on it and before any step): each step
 * clears the record when it starts and then sets
 *   MUONH_NONFINITE_MOMENTUM  when ||M|| (after the momentum update) of any
 *                             matrix is NaN or infinite: its X0, O and W are
 *                             then not finite either;
 *   MUONH_NONFINITE_UPDATE    (muonh_step only) when ||W - lr*O|| of any
 *                             matrix is NaN or infinite, so the projected W
 *                             is not finite.
 * (the two norms the step divides by, formula at the top of this file). The
 * kernels that finalize the norms write the record; it never changes the
 * results. *flags (HOST) receives the bits.
 * This call copies 4 bytes to the host and waits for `stream` (the only
 * synchronising call of the library); order it after the step like any
 * other call on the workspace.
 * Errors: MUONH_EINVAL (NULL plan or flags), MUONH_EWORKSPACE, MUONH_EHIP.
 */
enum {
  MUONH_NONFINITE_MOMENTUM = 1,
  MUONH_NONFINITE_UPDATE = 2,
};
int muonh_step_status(const muonh_plan* plan, const void* workspace, size_t workspace_bytes,
                      void* stream, uint32_t* flags);

/*
 * Check that no two of the plan's W, G and M matrices overlap in memory
 * (model card "Puro", section "Training": the step updates W and M in place,
 * so W, G and M must be distinct storage). W, G and M are HOST arrays of
 * n_matrices DEVICE pointers: the values the caller puts into the device
 * pointer arrays it passes to muonh_step. Each matrix spans rows*cols
 * elements of its storage type (W fp32; G and M fp32 or bf16 by plan flag).
 * Host-only: no HIP call, nothing enqueued, and no pointer is dereferenced.
 * muonh_step itself cannot check this (its pointer arrays live in device
 * memory); a caller whose pointers change calls this before the step.
 * O(n log n) in the number of matrices.
 * Errors: MUONH_EINVAL (NULL plan or array), MUONH_EALIAS (the message names
 * the first overlapping pair, e.g. "G[3] overlaps W[3]"), MUONH_ENOMEM.
 */
int muonh_check_disjoint(const muonh_plan* plan, const void* const* W, const void* const* G,
                         const void* const* M);

/*
 * Block-scaled 8-bit matrices: the operands of the linear layers that a
 * MuonH-trained model runs in E4M3 with a scale per block of 128 (model card
 * "Puro", section "Training"; report page, part 6/7, section 4.3 "Cost
 * Estimation", blockwise FP8: linear-layer products in FP8, master weights
 * and optimizer state in FP32 or BF16). The pages give neither the rounding
 * nor the scales' type; the readings here:
 *   - codes: OCP e4m3 (sign, 4 exponent, 3 mantissa bits; largest 448,
 *     smallest normal 2^-6, smallest 2^-9; NaN, no infinity);
 *   - scales: E8M0, the byte b stands for 2^(b - 127). A block's scale is the
 *     smallest power of two 2^e, e >= -126, with max|x| <= 448 * 2^e over the
 *     block's finite entries (-126 where all are zero or none is finite), so
 *     no entry overflows. x * 2^-e is exact, so a code is x / 2^e rounded
 *     once, to the nearest e4m3 value, ties to even (fp32 entries from 248 *
 *     2^120, about 3.3e38, to 256 * 2^120, which fp32 itself does not hold).
 *     NaN and infinities become NaN codes and do not count for the maximum;
 *   - blocks: MUONH_FP8_ROWS: 128 consecutive columns of one row (the last
 *     one of a row may be shorter); MUONH_FP8_TILES: 128 x 128 entries (edge
 *     tiles smaller).
 * Storage of a rows x cols matrix: codes, row-major, row pitch
 * muonh_fp8_ld(cols) = cols rounded up to 128 bytes, zeros in the columns
 * past cols; scales, row-major, one row per matrix row (ROWS) or per 128
 * matrix rows (TILES), muonh_fp8_scale_ld(cols) = ceil(cols/128) rounded up
 * to a multiple of 4 bytes per row, zeros past ceil(cols/128). codes 16-byte,
 * scales 4-byte aligned. The quantizing calls write all of it; an operand
 * of muonh_fp8_matmul from elsewhere needs the zeros past cols; its scale bytes
 * are 0 to 254, and 255 is NaN, as in E8M0. Matrices without rows or columns
 * are allowed.
 */
enum { MUONH_FP8_ROWS = 0, MUONH_FP8_TILES = 1 };
enum { MUONH_DT_FP32 = 0, MUONH_DT_BF16 = 1 };
/* In muonh_fp8_matmul's out_dtype beside MUONH_DT_BF16: 8-bit matrix
 * instructions, twice the rate, with sums of fewer bits than fp32. */
enum { MUONH_FP8_FAST = 256 };
#define MUONH_MAX_FP8_DIM (1 << 24) /* rows and cols of a block-scaled matrix */

typedef struct {
  const void* codes;  /* DEVICE, rows x muonh_fp8_ld(cols) bytes */
  const void* scales; /* DEVICE, rows or ceil(rows/128) x muonh_fp8_scale_ld(cols) bytes */
  int64_t rows, cols; /* in [0, MUONH_MAX_FP8_DIM] */
  int32_t block;      /* MUONH_FP8_ROWS or MUONH_FP8_TILES */
} muonh_fp8_matrix;

/* Row pitches in bytes (0 for cols out of [0, MUONH_MAX_FP8_DIM]) and the
 * number of scale rows. Host-only. */
int64_t muonh_fp8_ld(int64_t cols);
int64_t muonh_fp8_scale_ld(int64_t cols);
int64_t muonh_fp8_scale_rows(int64_t rows, int32_t block);

/*
 * Quantize src (DEVICE, rows x cols of `dtype`, element (r, c) at
 * r*src_ld + c, src_ld >= cols) into codes and scales, its own orientation,
 * and/or codes_t and scales_t, the same for its transpose (cols x rows). Each
 * pair is given whole or NULL, at least one of them given. With MUONH_FP8_ROWS
 * the two forms group differently (along src's columns, and along its rows:
 * a forward product contracts over features, a weight gradient over
 * tokens); with MUONH_FP8_TILES they hold the same values. One pass over
 * src. Deterministic; asynchronous on `stream`, capturable.
 * Errors: MUONH_EINVAL (NULL or half-given pair, bad dtype or block, src_ld <
 * cols or above 2^36, misaligned output), MUONH_ESHAPE (a dim out of range, or
 * 2^24 tiles of 128 x 128 or more), MUONH_EALIAS (an output overlaps src or
 * another output), MUONH_EHIP.
 */
int muonh_fp8_quantize(const void* src, int32_t dtype, int64_t rows, int64_t cols, int64_t src_ld,
                       int32_t block, void* codes, void* scales, void* codes_t, void* scales_t,
                       void* stream);

/*
 * Quantize every weight of a plan with MUONH_FP8_TILES, in grouped launches:
 * what the forward product (codes, scales) and the data gradient (codes_t,
 * scales_t, the transposed form) read after a step. W: DEVICE array of
 * n_matrices DEVICE pointers, as for muonh_step; the others: DEVICE arrays of
 * n_matrices DEVICE pointers to outputs in the storage above. codes_t and
 * scales_t may both be NULL. No output may overlap another or W (not
 * checked: the arrays live in device memory). Deterministic; asynchronous
 * on `stream`, capturable.
 * Errors: MUONH_EINVAL (NULL argument, half-given pair), MUONH_ESHAPE (2^24
 * tiles or more in one launch of up to 16 groups), MUONH_EHIP.
 */
int muonh_fp8_weights(const muonh_plan* plan, const float* const* W, void* const* codes,
                      void* const* scales, void* const* codes_t, void* const* scales_t,
                      void* stream);

/*
 * out[i][j] = sum_k a[i][k] * b[j][k] over the values that a (m x k) and b
 * (n x k) stand for, plus out's old value if `accumulate`; out: DEVICE, m x n
 * of out_dtype, element (i, j) at i*out_ld + j, out_ld >= n. The products of
 * a linear layer Y = X W^T:
 *   Y  = matmul(X, W)           X rows; W tiles (n x k)
 *   dX = matmul(dY, W^T)        dY rows; W's transposed tiles
 *   dW = matmul(dY^T, X^T)      transposed rows forms (grouped along tokens);
 *                               fp32 or bf16 G with accumulate: micro-batches
 * k = 0 gives zeros (or leaves out as it is). out_dtype: MUONH_DT_FP32 or
 * MUONH_DT_BF16. Entries are widened to bf16: exact from 2^-130 to below 2^128 in
 * magnitude, smaller ones to within 2^-134, larger ones count as infinite
 * (fp32 does not hold them either). Their products are exact, sums are fp32,
 * and the result is rounded once to out_dtype. With
 * MUONH_DT_BF16 | MUONH_FP8_FAST, 8-bit matrix instructions multiply at twice
 * the rate: of the products that one of them adds at once (at most 16) they
 * drop the bits below 2^-13 of the largest, so beside fp32 sums a result is
 * off by up to 15 * 2^-13 * sum_k |a[i][k] * b[j][k]|, however small it is
 * itself, before it is rounded; entries of every magnitude are exact. NaN codes give NaN in their row or column of out.
 * The result does not depend on out_ld or alignment, and is deterministic.
 * workspace: DEVICE, 256-byte aligned, of at least
 * muonh_fp8_matmul_workspace_bytes(m, n, k, out_dtype) bytes (NULL if that is
 * 0): partial sums of products with few output tiles. Calls in flight at once
 * need workspaces of their own. Asynchronous on `stream`, capturable.
 * Errors: MUONH_EINVAL (NULL argument, bad block or dtype, misaligned codes or
 * scales, out_ld < n), MUONH_ESHAPE (a dim out of range, a and b of different
 * cols, or 2^21 output tiles of 128 x 128 or more), MUONH_EWORKSPACE, MUONH_EALIAS (out or
 * the workspace overlaps an operand or each other), MUONH_EHIP.
 */
size_t muonh_fp8_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t out_dtype);
int muonh_fp8_matmul(const muonh_fp8_matrix* a, const muonh_fp8_matrix* b, void* out,
                     int32_t out_dtype, int64_t out_ld, int32_t accumulate, void* workspace,
                     size_t workspace_bytes, void* stream);

/* Static description of a status code. */
const char* muonh_status_string(int status);

/* Message of the last error raised on the calling thread ("" if none). */
const char* muonh_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MUONH_H */
