/*
 * muon_rocm.h -- C ABI of the MI355X (gfx950) Muon optimizer-step library.
 *
 * The library applies, to a set of 2-D fp32 weight matrices W of shape [A, B],
 *   - the Muon step of "Muon is Scalable for LLM Training" (Sec. 2.1 Eq. 1 momentum,
 *     Eq. 2 Newton-Schulz with X0 = M / ||M||_F and coefficients a, b, c, and
 *     Sec. 2.2 Eq. 4 update W <- W - lr * (0.2 * O * sqrt(max(A,B)) + wd * W)), and
 *   - the Periodic Row-wise variant of "Scaling Muon for Diffusion Transformers"
 *     (Periodic Row-wise paragraphs): NS5 once every K steps, and on the other steps
 *     Eq. 4 with O replaced by gamma * RowNorm(M), RowNorm scaling every row of M
 *     to unit l2 norm when A <= B and every column when A > B.
 * Tall matrices (A > B) run Newton-Schulz on M^T so the Gram matrix is min(A,B)^2.
 *
 * Conventions shared by every entry point:
 *   - All matrix buffers are DEVICE pointers owned by the caller, fp32, row-major,
 *     contiguous (leading dimension = cols), 16-byte aligned.
 *   - `workspace` is a caller-owned DEVICE buffer of at least the size that
 *     muon_workspace_bytes() reports for the same shapes, 256-byte aligned. Its
 *     contents need not be initialised and are garbage after the call.
 *   - `stream` is a hipStream_t (NULL = the legacy default stream). Calls only
 *     enqueue work on it and never synchronise; results are ready when the stream
 *     reaches that point. Concurrent calls must use distinct workspaces.
 *   - Every argument is validated on the host before anything is enqueued: on any
 *     error code no kernel runs and no buffer is touched.
 *   - Matrices with rows == 0 or cols == 0 are skipped (their pointers may be NULL);
 *     count == 0 is a no-op.
 *   - NaN / Inf in the inputs propagate to the outputs; they are not checked.
 *   - Results are deterministic: identical inputs give bitwise identical outputs.
 */
#ifndef MUON_ROCM_H
#define MUON_ROCM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MUON_ABI_VERSION 4

/* Status codes returned by every entry point. */
#define MUON_OK 0
#define MUON_ERR_INVALID_ARG (-1) /* NULL where a pointer is required, negative dims,
                                     count < 0, ns_steps < 1, period_k < 1, eps <= 0,
                                     unknown scale_mode, hidden < 1 under MUON_SCALE_HIDDEN */
#define MUON_ERR_WORKSPACE (-2)   /* workspace NULL or smaller than required */
#define MUON_ERR_ALIGN (-3)       /* matrix pointer not 16-byte aligned, workspace not 256,
                                     update_rms not 4 */
#define MUON_ERR_ALIAS (-4)       /* overlapping buffers that must be distinct */
#define MUON_ERR_HIP (-5)         /* a HIP runtime call or kernel launch failed */
#define MUON_ERR_TOO_LARGE (-6)   /* a dimension above 2^30 or a matrix above 2^40 elements */

/* Update-scale rules ("Muon is Scalable for LLM Training", Sec. 3.1). The update is
 * W <- W - lr (c U + wd W) with U = O on refresh steps and U = gamma R on RowNorm
 * steps, and the factor c is
 *   MUON_SCALE_MAX_DIM: rms_scale sqrt(max(A,B))     (Eq. 4, the same as Eq. 7)
 *   MUON_SCALE_HIDDEN:  rms_scale sqrt(hidden)        (Eq. 5, H = the model's hidden size)
 *   MUON_SCALE_RMS:     rms_scale / max(RMS(O), eps)  (Eq. 6) on refresh steps, where
 *                       RMS(O) = sqrt(mean(O^2)) is measured on the device; on RowNorm
 *                       steps rms_scale sqrt(max(A,B)), since RMS(R) = 1/sqrt(max(A,B))
 *                       exactly when every row (column) norm is >= eps. */
#define MUON_SCALE_MAX_DIM 0
#define MUON_SCALE_HIDDEN 1
#define MUON_SCALE_RMS 2

/* Hyperparameters. muon_default_hparams() fills the pages' defaults:
 * lr 1e-3, weight_decay 0.1, mu 0.95 (Muon notes Sec. 2.2), a, b, c =
 * 3.4445, -4.7750, 2.0315 (Sec. 2.1), rms_scale 0.2 (Eq. 4), gamma 0.15 and
 * period_k 3 (DiT paper, K/gamma sweep), eps 1e-7, ns_steps 5 (Sec. 2.2),
 * scale_mode MUON_SCALE_MAX_DIM, hidden 0. */
typedef struct muon_hparams {
    float lr;           /* eta */
    float weight_decay; /* lambda, decoupled (Eq. 3/4) */
    float mu;           /* momentum coefficient (Eq. 1) */
    float ns_a, ns_b, ns_c; /* Newton-Schulz polynomial coefficients (Eq. 2) */
    float rms_scale;    /* the 0.2 of Eq. 4 */
    float gamma;        /* RowNorm step relative to NS5 (Periodic variant) */
    float eps;          /* norms are divided as x / max(norm, eps) */
    int32_t ns_steps;   /* N, Newton-Schulz iterations (>= 1) */
    int32_t period_k;   /* K, refresh period (>= 1; 1 = vanilla Muon) */
    int32_t scale_mode; /* MUON_SCALE_* above */
    int32_t hidden;     /* H of MUON_SCALE_HIDDEN (>= 1 there, ignored otherwise) */
} muon_hparams;

/* One weight matrix with its optimizer state. All three are [rows, cols]. */
typedef struct muon_matrix {
    int64_t rows, cols;
    float* w;       /* weights, updated in place */
    float* m;       /* momentum (M_{t-1} in, M_t out), updated in place; zeros at t = 0 */
    const float* g; /* gradient, read only */
} muon_matrix;

/* Kernel classes reported by the optional timing facility. */
#define MUON_KCLASS_CAST 0          /* momentum + Frobenius partials + bf16 working copies */
#define MUON_KCLASS_FROB 1          /* per-matrix 1 / max(||M||_F, eps) */
#define MUON_KCLASS_GRAM 2          /* A = X X^T (symmetric tiles, bf16 MFMA; with its tail fixup) */
#define MUON_KCLASS_POLY 3          /* P = a I + b A + c A A (symmetric tiles, bf16 MFMA; with its tail fixup) */
#define MUON_KCLASS_APPLY 4         /* X' = P X = a X + (b A + c A A) X, iterations 1..N-1 (with its tail fixup) */
#define MUON_KCLASS_APPLY_FINAL 5   /* last iteration: O out, or the fused Eq. 4 update */
#define MUON_KCLASS_ROWNORM_ROWS 6  /* one-pass RowNorm step, flat / square matrices */
#define MUON_KCLASS_COLNORM_PARTIAL 7  /* tall: momentum + per-column partial sums */
#define MUON_KCLASS_COLNORM_FINALIZE 8 /* tall: per-column 1 / max(norm, eps) */
#define MUON_KCLASS_COLNORM_APPLY 9    /* tall: Eq. 4 update with the column-normalised M */
#define MUON_KCLASS_RMS_FINALIZE 10    /* per-matrix RMS(U): monitor value, Eq. 6 factor */
#define MUON_KCLASS_SCALED_UPDATE 11   /* Eq. 6 refresh: W <- decay W - coef O */
#define MUON_KCLASS_ADAMW 12           /* AdamW companion (non-matrix parameters) */
#define MUON_KCLASS_SPEC_GRAM 13       /* SVD entropy: fp64 Gram matrix (fp64 MFMA) */
#define MUON_KCLASS_SPEC_HOUSE 14      /* SVD entropy: Householder reflector per column */
#define MUON_KCLASS_SPEC_PASS 15       /* SVD entropy: trailing update + matrix-vector partials */
#define MUON_KCLASS_SPEC_REDUCE 16     /* SVD entropy: matrix-vector product from the partials */
#define MUON_KCLASS_SPEC_BISECT 17     /* SVD entropy: eigenvalues by Sturm bisection */
#define MUON_KCLASS_SPEC_ENTROPY 18    /* SVD entropy: normalisation and entropy */
#define MUON_KCLASS_NORM_FORWARD 19    /* normalisation layer: rows normalised, scaled and shifted */
#define MUON_KCLASS_NORM_BACKWARD 20   /* its input gradient, with the blocks' weight-gradient sums */
#define MUON_KCLASS_NORM_WGRAD 21      /* the weight and bias gradients from those sums */
#define MUON_KCLASS_TENSOR_PLAN 22     /* descriptor tables of many-tensor calls (set-up) */
#define MUON_KCLASS_ADAMW_MULTI 23     /* AdamW over many tensors, 32- or 8-bit states */
#define MUON_KCLASS_GRAD_NORM 24       /* sums of squares of the gradients, block by block */
#define MUON_KCLASS_GRAD_TOTAL 25      /* the tensors' norms, their total and the clip factor */
#define MUON_KCLASS_GRAD_SCALE 26      /* gradients scaled in place */
#define MUON_KCLASS_QUANTISE8 27       /* matrices to 8 bits with a power of two a block */
#define MUON_KCLASS_DEQUANTISE8 28     /* and back */
#define MUON_KCLASS_MATMUL8 29         /* products of such matrices */
#define MUON_KCLASS_MATMUL8_JOIN 30    /* the sum of a product's parts along k */
#define MUON_KCLASS_ADD_NORM_FORWARD 31   /* residual addition, RMS norm and quantising */
#define MUON_KCLASS_ADD_NORM_BACKWARD 32  /* its gradients (the weight's sums count as 21) */
#define MUON_KCLASS_ROTARY 33          /* rotary positions */
#define MUON_KCLASS_COUNT 34

/* Returns MUON_ABI_VERSION. Host only. */
int muon_abi_version(void);

/* Static English text for a status code (never NULL). Host only. */
const char* muon_status_str(int status);

/* Detail of the last MUON_ERR_HIP (or other error) raised on this thread; "" if none. */
const char* muon_last_error(void);

/* Fills *hp with the defaults listed above. Host only; hp NULL is ignored. */
void muon_default_hparams(muon_hparams* hp);

/* Workspace size in bytes sufficient for muon_step, ns5_batched and rownorm_update
 * on `count` matrices of shapes rows[i] x cols[i]. Host only, touches no device.
 * Errors: INVALID_ARG (NULL bytes, count < 0, NULL rows/cols with count > 0, negative
 * dims), TOO_LARGE. */
int muon_workspace_bytes(const int64_t* rows, const int64_t* cols, int32_t count, size_t* bytes);

/* The GEMM plan of the Newton-Schulz stages (Eq. 2 of the Muon scaling paper: the Gram
 * X X^T, the polynomial P = a I + b A + c A A, the Apply P X = a X + (b A + c A A) X)
 * that ns5_batched and the refresh step of muon_step use for `count` matrices of
 * shapes rows[i] x cols[i].
 * Host only, touches no device; for tests and capacity planning. Nonempty matrices are
 * grouped as those calls group them: sorted by m = min(rows, cols), then by
 * n = max(rows, cols), both descending (stable), at most 16 per group. *groups receives
 * the number of groups. With capacity >= groups * MUON_PLAN_RECORD_INTS, `out` (host
 * array, caller-owned) receives one record of MUON_PLAN_RECORD_INTS values per group:
 *   [0]        matrices in the group;
 *   [1 .. 16]  their indices into rows / cols, -1 past that count;
 *   then 17 values for each of the Gram, the polynomial, the Apply of iterations
 *   1 .. N-1 and the last Apply, in that order: the tile width (128 or 256), then for
 *   XCD 0 .. 7 the number of its tiles that run as K chunks and the number of chunks
 *   (0 and 1 where the XCD does not split). A positive count h means the last h tiles
 *   of its sequence (tail split); a negative one, -h, its first h (head split, for a
 *   stage whose tiles fit one round and whose matrices differ in K).
 * capacity 0 only reports *groups (out may then be NULL).
 * Errors: INVALID_ARG (NULL groups, count < 0, NULL rows / cols with count > 0,
 * negative dims, capacity < 0, NULL out with capacity > 0, capacity below the
 * records), TOO_LARGE. */
#define MUON_PLAN_RECORD_INTS 85
int ns5_plan(const int64_t* rows, const int64_t* cols, int32_t count, int32_t* out, int32_t capacity,
             int32_t* groups);

/* One optimizer step at 0-based step index `step` for `count` matrices.
 * Periodic schedule (DiT paper, "NS5 once every K steps"; read here as a refresh
 * iff step % period_k == 0, so step 0 refreshes and period_k == 1 is vanilla Muon):
 *   refresh:  M <- mu M + G;  O = NS5(M);  W <- W - lr (c O + wd W), c per scale_mode
 *             (Eq. 4 and Eq. 5 fuse the update into the last Newton-Schulz GEMM;
 *             Eq. 6 writes O to the workspace, reduces RMS(O), then updates W)
 *   otherwise: exactly rownorm_update() below.
 * mats: host array of `count` descriptors.
 * update_rms: optional DEVICE array of `count` floats (NULL = not wanted). Entry i
 *   receives RMS(c U_i), the RMS of the update direction before the learning rate,
 *   weight decay excluded (about rms_scale under Eq. 4 by Lemma 1, exactly rms_scale
 *   under Eq. 6); entries of skipped empty matrices are left unchanged. It must not
 *   overlap any other buffer.
 * Errors: INVALID_ARG, ALIGN, ALIAS (any two of all w, m, g, update_rms ranges
 * overlap), WORKSPACE, TOO_LARGE, HIP. */
int muon_step(const muon_matrix* mats, int32_t count, const muon_hparams* hp, int64_t step,
              void* workspace, size_t workspace_bytes, float* update_rms, void* stream);

/* muon_step's checks alone: the status that it would refuse the same arguments with, or
 * MUON_OK. Host only. For a caller that has to know before it writes anything (a clipped
 * step scales the gradients in place first). Errors: muon_step's, but HIP. */
int muon_step_check(const muon_matrix* mats, int32_t count, const muon_hparams* hp, int64_t step, void* workspace,
                    size_t workspace_bytes, float* update_rms);

/* Newton-Schulz orthogonalisation alone ("Muon is Scalable", Sec. 2.1 Eq. 2):
 * o_out[i] = NS_N(m_in[i]) with X0 = M / max(||M||_F, eps), for [rows[i], cols[i]]
 * fp32 device matrices; the output has the input's shape and orientation. bf16 MFMA
 * products with fp32 accumulation; relative Frobenius error vs exact arithmetic is
 * about 1e-2. o_out[i] == m_in[i] (in place) is allowed; any other overlap is ALIAS.
 * m_in, o_out, rows, cols are host arrays of `count` entries. Only hp->ns_* and
 * hp->eps are used. Errors: INVALID_ARG, ALIGN, ALIAS, WORKSPACE, TOO_LARGE, HIP. */
int ns5_batched(const float* const* m_in, float* const* o_out, const int64_t* rows,
                const int64_t* cols, int32_t count, const muon_hparams* hp,
                void* workspace, size_t workspace_bytes, void* stream);

/* The Periodic variant's non-refresh step (DiT paper, Periodic Row-wise and
 * distributed-implementation paragraphs), fp32 throughout, in one pass for flat and
 * square matrices and three short kernels for tall ones:
 *   M <- mu M + G
 *   R = M / max(row l2 norms, eps)     if rows <= cols
 *   R = M / max(column l2 norms, eps)  if rows >  cols
 *   W <- W - lr (c gamma R + wd W), c = rms_scale sqrt(max(A,B)) or rms_scale sqrt(hidden)
 * update_rms as for muon_step (here RMS(c gamma R), one more small kernel when given).
 * hp->period_k is not used. Errors as muon_step. */
int rownorm_update(const muon_matrix* mats, int32_t count, const muon_hparams* hp,
                   void* workspace, size_t workspace_bytes, float* update_rms, void* stream);

/* ---- Allocation-free RowNorm step ---------------------------------------------------
 * For callers that cannot allocate device memory: code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc. The same step as rownorm_update() (the
 * same kernels in the same order: bitwise identical results), with its workspace taken
 * from a fixed array of MUON_NOALLOC_SCRATCH_BYTES in device memory that the library
 * holds: one copy on each GPU it runs on, kept until the process ends. The call
 * allocates nothing (no hipMalloc, hipFree or allocating library routine) and creates
 * no timing events.
 * Limit: the RowNorm workspace of the matrices must fit the array. Per group of up to
 * 16 matrices (the same grouping as muon_step) it is the sum over the group of
 *   tall [A, B] (A > B):  4 B (ceil(A / 64) + 2) bytes,
 *   flat [A, B]:          4 A bytes,
 * each part rounded up to 256 bytes; sixteen [30720, 5120] matrices take 158 MB. Beyond
 * it the call returns MUON_ERR_WORKSPACE and nothing runs.
 * Every call on one GPU uses that GPU's single array: calls that overlap in time on one
 * GPU (other streams, other threads) race and corrupt each other's results; serialise
 * them. The array keeps the last call's contents; no part of it needs to start at zero.
 * Errors: as rownorm_update (WORKSPACE for the limit), HIP when the current device or the
 * array's address cannot be looked up. */
#define MUON_NOALLOC_SCRATCH_BYTES ((size_t)160 << 20)
int rownorm_update_noalloc(const muon_matrix* mats, int32_t count, const muon_hparams* hp,
                           float* update_rms, void* stream);

/* ---- One GPU's share of a row-sharded RowNorm step --------------------------------
 * "Scaling Muon for Diffusion Transformers", distributed-implementation paragraph: with
 * the weights sharded by rows (dim 0) across GPUs, the rows of a flat matrix (A <= B)
 * are whole on every GPU, so rownorm_update() on a GPU's block of rows is already its
 * share of the step (the block's sqrt(max(rows, B)) = sqrt(B) is the whole matrix's
 * scale). A tall matrix (A > B) normalises columns, which span the GPUs. Its step is
 * split in two calls around the caller's reduction:
 *   1. rownorm_shard_colsq: M <- mu M + G on the block, and colsq[c] = sum over the
 *      block's rows of M[r][c]^2;
 *   2. the caller sums colsq over the GPUs holding the matrix (an all-reduce; with
 *      one block per matrix, nothing);
 *   3. rownorm_shard_apply: W <- W - lr (c gamma M / max(sqrt(total[c]), eps) + wd W)
 *      with c = rms_scale sqrt(full_rows), or rms_scale sqrt(hidden) under
 *      MUON_SCALE_HIDDEN (MUON_SCALE_RMS takes the max-dimension form, as rownorm_update).
 * Concatenating the blocks reproduces rownorm_update() on the whole matrix up to the
 * summation order of the column sums. */
typedef struct muon_shard {
    int64_t rows, cols;  /* this GPU's block: `rows` rows of the matrix, all `cols` columns */
    int64_t full_rows;   /* A of the whole matrix: must exceed cols (tall) and be >= rows */
    float* w;            /* [rows, cols] block of W, updated by rownorm_shard_apply */
    float* m;            /* [rows, cols] block of M, updated by rownorm_shard_colsq */
    const float* g;      /* [rows, cols] block of G, read by rownorm_shard_colsq (apply: unused, may be NULL) */
} muon_shard;

/* Workspace in bytes for either shard call on these blocks (about 4 cols ceil(rows / 256)
 * bytes per block for up to 16 blocks at a time). Host only.
 * Errors: INVALID_ARG (NULL bytes or shards, count < 0, negative dims, full_rows <= cols,
 * rows > full_rows), TOO_LARGE. Blocks with cols == 0 are skipped. */
int rownorm_shard_workspace_bytes(const muon_shard* shards, int32_t count, size_t* bytes);

/* Step 1 for `count` blocks (host array). colsq: host array of `count` DEVICE pointers,
 * each to cols floats (4-byte aligned), written; a block with rows == 0 writes zeros.
 * Errors: as rownorm_update, plus INVALID_ARG for NULL colsq entries. */
int rownorm_shard_colsq(const muon_shard* shards, int32_t count, const muon_hparams* hp,
                        float* const* colsq, void* workspace, size_t workspace_bytes, void* stream);

/* Step 3. colsq_total: host array of `count` DEVICE pointers to the reduced column sums
 * (cols floats each), read only. M must hold step 1's output. Blocks with rows == 0 are
 * left alone. Errors: as rownorm_shard_colsq. */
int rownorm_shard_apply(const muon_shard* shards, int32_t count, const muon_hparams* hp,
                        const float* const* colsq_total, void* workspace, size_t workspace_bytes,
                        void* stream);

/* ---- AdamW companion for the parameters Muon does not take -------------------------
 * "Scaling Muon for Diffusion Transformers" (setup paragraph) keeps biases,
 * normalisation parameters and everything outside the transformer blocks on AdamW,
 * an auxiliary group at lr 1e-4; "Muon is Scalable for LLM Training" (Sec. 2.2,
 * matching-update-RMS paragraph) pairs Muon with AdamW for non-matrix parameters.
 * The pages do not restate AdamW; this is Adam with bias-corrected moments and
 * decoupled weight decay in Eq. 3's form, at 0-based step s (t = s + 1):
 *   m <- b1 m + (1 - b1) g;  v <- b2 v + (1 - b2) g^2
 *   W <- W - lr (m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps) + wd W)
 * adamw_default_hparams(): lr 1e-4 (the DiT paper's auxiliary group), beta1 0.9,
 * beta2 0.999, eps 1e-8 (PyTorch's AdamW defaults), weight_decay 0.1 (shared with Muon). */
typedef struct adamw_hparams {
    float lr;
    float beta1, beta2; /* in [0, 1) */
    float eps;          /* > 0 */
    float weight_decay;
} adamw_hparams;

/* One parameter tensor of any shape, as `numel` contiguous fp32 elements. w, m
 * (first moment), v (second moment) are DEVICE pointers updated in place (zeros at
 * s = 0); g is read only. All four 16-byte aligned; numel == 0 entries are skipped. */
typedef struct adamw_param {
    int64_t numel;
    float* w;
    float* m;
    float* v;
    const float* g;
} adamw_param;

/* Fills *hp with the defaults above. Host only; hp NULL is ignored. */
void adamw_default_hparams(adamw_hparams* hp);

/* One AdamW step at 0-based step `step` for `count` tensors (host array of
 * descriptors), enqueued on `stream`: one launch per 48 tensors, 28 bytes of HBM
 * traffic per element. fp32 throughout; no workspace.
 * Errors: INVALID_ARG (NULL hp / params / pointers, count < 0, numel < 0, step < 0,
 * beta outside [0, 1), eps <= 0, non-finite lr or wd), ALIGN, ALIAS (any two of all
 * w, m, v, g ranges overlap), TOO_LARGE (numel above 2^40), HIP. */
int adamw_step(const adamw_param* params, int32_t count, const adamw_hparams* hp, int64_t step,
               void* stream);

/* adamw_step's checks alone, as muon_step_check's. Host only. */
int adamw_step_check(const adamw_param* params, int32_t count, const adamw_hparams* hp, int64_t step);

/* ---- Many tensors in one launch ------------------------------------------------------
 * The hybrid optimizer's AdamW side has hundreds of small tensors (238 in the 15B-scale
 * model). The calls below read their descriptors from a table in device memory that a
 * plan call writes once, so that a step is one launch whatever the count. */

/* Element types of the operators from here on. */
#define MUON_DTYPE_F32 0
#define MUON_DTYPE_BF16 1
#define MUON_DTYPE_F16 2

/* A written table. Filled by a plan call, read-only to the caller; valid while `device`
 * and the tensors that it describes live. */
typedef struct tensor_plan {
    void* device;    /* the caller's buffer */
    size_t bytes;    /* the part of it in use */
    int32_t kind;    /* which plan call filled it */
    int32_t count;   /* tensors, empty ones included */
    int32_t blocks;  /* thread blocks of a launch */
    int32_t reserved;
} tensor_plan;

/* ---- AdamW with 32-bit or 8-bit states ------------------------------------------------
 * adamw_step()'s formula with g' = grad_scale g, for each tensor on its own:
 *   m <- b1 m + (1 - b1) g',  v <- b2 v + (1 - b2) g'^2,  t = step + 1
 *   W <- (1 - lr wd) W - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
 * with lr and wd times the tensor's lr_scale and wd_scale. W is fp32; copy, if given,
 * receives the new W rounded to 16 bits (the weights of the next forward pass). g is
 * fp32, bf16 or fp16.
 * state_bits 32: m and v are numel floats.
 * state_bits 8: m and u = sqrt(v) are numel bytes of e4m3 (1 sign, 4 exponent, 3 mantissa
 * bits, largest value 448) and a float of scale for every 256 consecutive elements (the
 * last block may be shorter): m = m_scale code, v = (v_scale code)^2. The step runs in
 * fp32 on these values; W is updated from the unrounded new m and v. Then each block's
 * scale becomes its largest magnitude / 448 (0, with all codes 0, where that magnitude is
 * below 1e-30) and its values are rounded stochastically: with b2 = 0.999 a u moves by at
 * most 0.05% a step where its gradient shrinks, far below the 6% to 12% between codes, so
 * that rounding to nearest would hold it for good. A u above 0 is never rounded to 0 (the
 * update would lose its denominator). A block with a non-finite new m or v gets NaN as
 * that state's scale, and so NaN in all its 256 elements from the next step on.
 * The rounding bits are a function of (seed, step, position of the tensor in the list,
 * index of the element) alone: all 32-bit arithmetic, with
 *   mix(x): x = (x ^ x >> 16) 0x6A09E667; x = (x ^ x >> 15) 0xBB67AE85; x ^ x >> 16
 *   key = mix(mix(mix(mix(seed_lo) + seed_hi) + step_lo) + 0x510E527F tensor)
 *   bits = mix(0x9E3779B9 i_lo + 0x510E527F i_hi + key)
 * the low 16 round m, the high 16 u. A magnitude a (of 448) between two codes goes up
 * where its fraction, cut to 20 bits, plus bits / 2^16 reaches 1. */
typedef struct adamw_tensor {
    int64_t numel;
    float* w;
    void* copy;       /* numel 16-bit elements of copy_dtype, NULL = not wanted */
    const void* g;
    void* m;
    void* v;
    float* m_scale;   /* state_bits 8: ceil(numel / 256) floats each; else ignored */
    float* v_scale;
    int32_t g_dtype;    /* MUON_DTYPE_* */
    int32_t copy_dtype; /* MUON_DTYPE_BF16 or _F16 where copy is given */
    int32_t state_bits; /* 8 or 32 */
    float lr_scale;     /* finite */
    float wd_scale;     /* finite */
} adamw_tensor;

/* Bytes of the device buffer for adamw_multi_plan. Host only; reads numel and state_bits.
 * Errors: INVALID_ARG, TOO_LARGE. */
int adamw_multi_plan_bytes(const adamw_tensor* tensors, int32_t count, size_t* bytes);

/* Checks `count` tensors (host array), enqueues the table's writing into `device` (256-byte
 * aligned, `bytes` of adamw_multi_plan_bytes) on `stream` and fills *plan. Steps with this
 * plan come after it on the stream. A gradient at another address needs a new plan call
 * (into the same buffer, if it follows the last step on the stream). Plan calls are
 * refused on a stream that is being captured: what a graph records is not yet written.
 * On an error after the first launch plan->kind is 0 and steps with it are refused.
 * Errors: INVALID_ARG (NULL pointers, negative numel, unknown type or bits, non-finite
 * scale, a capture), ALIGN (w, m, v, g, copy not 16-byte aligned, scales not 4-byte), ALIAS (any two
 * of all w, copy, m, v, m_scale, v_scale, g ranges or the table overlap, gradients with each
 * other excepted), WORKSPACE (device
 * NULL or too small), TOO_LARGE (2^36 elements or 2^22 - 1 tensors and more in all), HIP. */
int adamw_multi_plan(const adamw_tensor* tensors, int32_t count, void* device, size_t bytes, tensor_plan* plan,
                     void* stream);

/* One step at 0-based step `step` over the plan's tensors: one launch.
 * grad_scale: DEVICE float (the clip factor of grad_norm, or one over a loss scale), NULL = 1;
 * outside the plan's w, copy, m, v and scales (not checked: the plan's addresses are on the device).
 * seed: of the stochastic rounding; without effect on 32-bit states. Two calls on one plan
 * at the same time race, as on the states themselves.
 * Errors: INVALID_ARG (as adamw_step, eps below 2^-126, a plan of another kind), ALIGN,
 * HIP. */
int adamw_multi_step(const tensor_plan* plan, const adamw_hparams* hp, int64_t step, uint64_t seed,
                     const float* grad_scale, void* stream);

/* The same step with its counter, and if wanted its learning rate, on the device: for steps
 * that are captured into a graph, where a host argument would stay what it was at capture
 * (with it the bias corrections and the rounding bits of 8-bit states, which have to change
 * from step to step). counter: DEVICE int64, 8-byte aligned: the 0-based step, not below 0;
 * the call uses its value and then adds one, so that every plan needs its own; a plan without
 * elements launches nothing and leaves it. lr: DEVICE float, NULL = hp->lr; both outside the
 * plan's tensors (not checked). Two launches.
 * Errors: as adamw_multi_step, INVALID_ARG for a NULL counter. */
int adamw_multi_step_device(const tensor_plan* plan, const adamw_hparams* hp, int64_t* counter, const float* lr,
                            uint64_t seed, const float* grad_scale, void* stream);

/* ---- Gradient norm and clipping --------------------------------------------------------
 * n_i = l2 norm of tensor i, total = sqrt(sum n_i^2), factor = min(1, max_norm / (total +
 * 1e-6)): on the device, for adamw_multi_step's grad_scale and grad_scale() below. Squares
 * and sums are fp64, in a fixed order. */
typedef struct grad_tensor {
    void* g;        /* DEVICE, aligned to its element; only grad_scale writes it */
    int64_t numel;  /* 0: skipped, its norm is 0 */
    int32_t dtype;  /* MUON_DTYPE_* */
    int32_t reserved;
} grad_tensor;

/* Bytes of the device buffer (table and partial sums) for grad_norm_plan. Host only. */
int grad_norm_plan_bytes(const grad_tensor* grads, int32_t count, size_t* bytes);

/* As adamw_multi_plan. The buffer also holds the sums of a running grad_norm: calls on one
 * plan must not overlap in time.
 * Errors: INVALID_ARG, ALIGN (g not aligned to its element), ALIAS (two tensors, or one and
 * the table, overlap), WORKSPACE, TOO_LARGE, HIP. */
int grad_norm_plan(const grad_tensor* grads, int32_t count, void* device, size_t bytes, tensor_plan* plan,
                   void* stream);

/* total[0] = the norm over all of the plan's tensors, total[1] = the clip factor; norms[i] =
 * tensor i's norm, NULL = not wanted. DEVICE arrays of 2 and `count` floats outside the
 * plan's tensors (not checked). A NaN gradient
 * gives NaN for both, an infinite one an infinite norm and the factor 0. Two launches.
 * Errors: INVALID_ARG (NULL plan or total, another plan's kind, max_norm not > 0 and
 * finite), ALIGN, ALIAS (total and norms overlap each other or the table), HIP. */
int grad_norm(const tensor_plan* plan, float max_norm, float* total, float* norms, void* stream);

/* g <- factor g in place, rounded to g's type, for the plan's tensors; factor: DEVICE float
 * outside these tensors (not checked).
 * Nothing is read or written where factor is 1. One launch. Errors: INVALID_ARG, ALIGN, HIP. */
int grad_scale(const tensor_plan* plan, const float* factor, void* stream);

/* ---- Normalisation layers and their gradients ---------------------------------------
 * The layers whose parameters the hybrid optimizer keeps on AdamW (affine layer norm, the
 * query and key RMS norms), and the modulated norm whose scale and shift the blocks'
 * [6H, H] adaLN matrices produce for every sample. Rows of `cols` elements, split evenly
 * into `groups` of consecutive rows; row r in group g = r / (rows / groups):
 *   mean = (1/cols) sum x              (0 under MUON_NORM_RMS)
 *   rstd = 1 / sqrt((1/cols) sum (x - mean)^2 + eps)
 *   h = (x - mean) rstd,   y = h (weight_offset + w[g]) + b[g]
 * One group is an affine norm, one group a sample is adaLN (there weight_offset 1: the
 * projection gives 1 + scale). Backward, from dy with a = dy (weight_offset + w[g]):
 *   dx = rstd (a - (1/cols) sum a - h (1/cols) sum a h)   (RMS: without the first sum)
 *   dw[g] = sum over the group's rows of dy h,   db[g] = sum of dy
 * Arithmetic and statistics are fp32 whatever the types; each output is rounded once.
 * Sums run in a fixed order: identical calls give identical bits. */
#define MUON_NORM_LAYER 0
#define MUON_NORM_RMS 1
#define MUON_NORM_MAX_COLS 16384

typedef struct norm_desc {
    int64_t rows, cols, groups; /* groups >= 1 divides rows */
    int64_t inner;              /* >= 1, divides rows: see norm_rows */
    int32_t kind;               /* MUON_NORM_* */
    int32_t dtype;              /* of x, y, dy, dx */
    int32_t wdtype;             /* of w, b, dw, db: MUON_DTYPE_F32 or dtype */
    float eps;                  /* finite, > 0 */
    float weight_offset;        /* finite; without effect where w is NULL */
} norm_desc;

/* A [rows, cols] tensor whose row r starts at data + (r / inner) stride0 +
 * (r % inner) stride1 elements (a query view [tokens, heads, cols] of a fused
 * projection: inner = heads). Elements of a row are adjacent. Strides are >= 0; rows that
 * are written must not overlap each other. data: aligned to its element. */
typedef struct norm_rows {
    void* data;
    int64_t stride0, stride1;
} norm_rows;

/* A [groups, cols] parameter tensor, group g at data + g stride elements; data NULL =
 * absent. data: aligned to its element. */
typedef struct norm_param {
    void* data;
    int64_t stride;
} norm_param;

/* y from x. w and b may be absent (factor 1, shift 0). mean and rstd: DEVICE arrays of
 * `rows` floats that receive the rows' statistics for the backward pass, each NULL when
 * not wanted; mean is not written under MUON_NORM_RMS. y may be x itself (same pointer
 * and strides). One launch.
 * Errors: INVALID_ARG, ALIGN, ALIAS (y, mean or rstd overlaps another buffer, by the
 * span from its first to its last element), TOO_LARGE (cols above MUON_NORM_MAX_COLS,
 * rows or groups above 2^30, groups that take 2^32 threads, a span above 2^46 elements), HIP. rows == 0 or cols == 0 is
 * a no-op. */
int norm_forward(const norm_desc* desc, const norm_rows* x, const norm_param* w, const norm_param* b,
                 const norm_rows* y, float* mean, float* rstd, void* stream);

/* Workspace in bytes of norm_backward with dw or db. Host only. Errors: as norm_forward's
 * for desc, INVALID_ARG for NULL bytes. */
int norm_backward_workspace_bytes(const norm_desc* desc, size_t* bytes);

/* dx, dw and db from dy and the forward pass's x, mean (LAYER) and rstd. dw and db are
 * overwritten, zeros where rows == 0; absent ones are not computed, and without both no
 * workspace is needed. dw without w is INVALID_ARG. dx may be dy or x itself. One launch,
 * and a second that adds the blocks' sums where a group spans several blocks.
 * desc->eps is not used. Errors: as norm_forward, and WORKSPACE. */
int norm_backward(const norm_desc* desc, const norm_rows* dy, const norm_rows* x, const norm_param* w,
                  const float* mean, const float* rstd, const norm_rows* dx, const norm_param* dw,
                  const norm_param* db, void* workspace, size_t workspace_bytes, void* stream);

/* ---- Matrices in 8 bits and their products ------------------------------------------------
 * For the layers whose weights Muon steps: activations, weights and gradients as e4m3 codes
 * (1 sign, 4 exponent, 3 mantissa bits, largest value 448) with a power of two for every block
 * of MUON_BLOCK8 = 128 elements of a row, or for every 128 x 128 elements (`tiles`, for
 * weights: the transposed matrix then has the same codes and powers). A block's power is the
 * least 2^e with max |x| <= 448 2^e over its finite elements (e >= -127), kept as the byte
 * e + 127 (255 stands for NaN and is never written); its codes are x 2^-e rounded to nearest,
 * ties to even. Infinities and NaN become NaN codes, each for itself. A value is
 * code 2^(byte - 127), for a byte of 0 as for the others. */
#define MUON_BLOCK8 128
#define MUON_BLOCKS8_MAX_COLS (1 << 22)

typedef struct blocks8 {
    int64_t rows, cols;
    uint8_t* codes;    /* DEVICE, 16-byte aligned: row r at codes + r ld, cols codes and zeros up
                          to the next multiple of 128 (quantise8 writes them, products take
                          them for zeros) */
    uint8_t* scales;   /* DEVICE, 4-byte aligned: byte j of row r (of row block r / 128 with
                          tiles) at scales + r scale_ld + j, one for each 128 columns; read in
                          fours, the rest of the last four without effect */
    int64_t ld;        /* multiple of 16, at least cols rounded up to 128 */
    int64_t scale_ld;  /* multiple of 4, at least cols / 128 rounded up */
    int32_t tiles;     /* 0: a power for 1 x 128 elements, 1: for 128 x 128 */
    int32_t reserved;
} blocks8;

/* direct [rows, cols] and / or transposed [cols, rows] (either NULL = not wanted) from x
 * [rows, cols] of `dtype` with rows `stride` elements apart (aligned to its element, stride
 * >= 0). Blocks run along each result's own rows: the transposed one's are 128 rows of x. Both
 * have the same `tiles`. One read of x, one launch. rows == 0 or cols == 0 is a no-op.
 * Errors: INVALID_ARG, ALIGN, ALIAS (an output overlaps another buffer, by spans), TOO_LARGE
 * (rows or cols above 2^30, a row of a result above MUON_BLOCKS8_MAX_COLS, a span above 2^46
 * elements, 2^24 blocks of 128 x 128 and more), HIP. */
int quantise8(const void* x, int64_t rows, int64_t cols, int64_t stride, int32_t dtype, const blocks8* direct,
              const blocks8* transposed, void* stream);

/* y [rows, cols] of `dtype`, rows `stride` elements apart: the values of q, rounded to dtype
 * (exact in fp32, and in bf16 but for what has bits below 2^-133, in blocks below 2^-116). Errors: as quantise8. */
int dequantise8(const blocks8* q, void* y, int64_t stride, int32_t dtype, void* stream);

/* c[i][j] = sum_k a[i][k] b[j][k] for a [m, k], b [n, k], c [m, n] of `dtype`, rows ldc
 * elements apart; plus the old c with accumulate != 0. Sums are fp32, rounded to dtype once;
 * parts of k that blocks of the launch took are added in their order: identical calls give
 * identical bits. m == 0 or n == 0 is a no-op, k == 0 gives zeros. With
 *   y = x w^T           a = x (direct),             b = w (direct)
 *   dx = dy w           a = dy (direct),            b = w (transposed)
 *   dw = dy^T x         a = dy (transposed),        b = x (transposed)
 * products: 8 = by the 8-bit matrix instructions, which drop, in every eight products that
 *   follow each other along k, bits below 2^-13 of the largest: the result is off by 2^-16 of
 *   it, root mean square, on normally distributed values, and by 2^-10 of the sum of
 *   magnitudes at most (above a 16-bit c's own rounding where sums cancel); 16 = the codes are
 *   widened to bf16 (as exactly as dequantise8 does) and the sums are those of fp32 additions,
 *   at half the rate; 0 = 16 for an fp32 c, 8 for others.
 * Workspace (matmul8_workspace_bytes, 256-byte aligned; none needed where that gives 0): the
 * partial sums of products with few tiles.
 * Errors: INVALID_ARG (and a->cols != b->cols), ALIGN, ALIAS (c or the workspace overlaps
 * another buffer, rows of c overlap), WORKSPACE, TOO_LARGE (as quantise8, 2^21 tiles of 128 x
 * 128 of c and more, 2^35 elements of c and more), HIP. */
int matmul8_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t dtype, int32_t products, size_t* bytes);
int matmul8(const blocks8* a, const blocks8* b, void* c, int64_t ldc, int32_t dtype, int32_t products,
            int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream);

/* How matmul8 cuts a product [m, k] x [n, k]. Host only, touches no device; for tests and
 * capacity planning. `out` (host array of MUON_MATMUL8_PLAN_INTS) receives
 *   [0] the side of a block's tile of c, 128 or 256; 0 with m <= 64
 *   [1] the parts of k, one after another in the workspace where there are several
 * and with m <= 64 (else 0)
 *   [2] the groups of 16 rows of a that a wave takes: 1, 2 or 4
 *   [3] 1 = b streams through LDS, 128 of its rows a block; 0 = straight to registers, then
 *   [4] the waves of a block, and
 *   [5] those of them that take turns along k at the same 16 rows of b.
 * All are 0 where m == 0 or n == 0. Errors: INVALID_ARG, TOO_LARGE, as matmul8_workspace_bytes. */
#define MUON_MATMUL8_PLAN_INTS 6
int matmul8_plan(int64_t m, int64_t n, int64_t k, int32_t dtype, int32_t products, int32_t* out);

/* ---- Residual addition with RMS norm ----------------------------------------------------
 * The step between two layers of a pre-norm block. For rows of `cols` elements:
 *   h = x + residual, rounded to the residual's type;  rstd = 1 / sqrt((1/cols) sum h^2 + eps)
 *   y = h rstd (weight_offset + w)
 * with y in x's type and / or in 8 bits for matmul8, both from the same fp32 values. Without a
 * residual h is x and is not written. Backward, from dy and the gradient dh of h itself (what
 * comes down the residual stream; NULL = 0), with n = h rstd and a = dy (weight_offset + w):
 *   d = dh + rstd (a - n (1/cols) sum a n)        the gradient of x and of the residual
 *   dw = sum over rows of dy n
 * Quantising y counts as the identity there. Arithmetic is fp32, each output rounded once;
 * sums run in a fixed order. */
typedef struct add_norm_desc {
    int64_t rows, cols;
    int32_t dtype;        /* of x, y, dy, dx */
    int32_t rdtype;       /* of residual, h, dh, dr: MUON_DTYPE_F32 or dtype */
    int32_t wdtype;       /* of w, dw: MUON_DTYPE_F32 or dtype */
    float eps;            /* finite, > 0 */
    float weight_offset;  /* finite; without effect where w is NULL */
    int32_t reserved;
} add_norm_desc;

/* norm_rows here: row r at data + r stride0 (stride1 is not used); norm_param: one row. h may
 * be residual or x (same pointer, stride and type). residual, w, y, codes, rstd: NULL (or data
 * NULL) = absent or not wanted; h goes with residual. codes: [rows, cols], tiles 0. One launch.
 * rows == 0 or cols == 0 is a no-op.
 * Errors: INVALID_ARG, ALIGN, ALIAS (an output overlaps another buffer, by spans), TOO_LARGE
 * (cols above MUON_NORM_MAX_COLS, rows above 2^30, a span above 2^46 elements), HIP. */
int add_rms_norm_forward(const add_norm_desc* desc, const norm_rows* x, const norm_rows* residual, const norm_param* w,
                         const norm_rows* h, const norm_rows* y, const blocks8* codes, float* rstd, void* stream);

/* Workspace in bytes of add_rms_norm_backward with dw. Host only. */
int add_rms_norm_backward_workspace_bytes(const add_norm_desc* desc, size_t* bytes);

/* dr [rows, cols] of rdtype receives d; dx, wanted only where dtype is not rdtype, d in dtype.
 * dr and dx may be dy, dh or h where pointer, stride and type are the same. dw is overwritten
 * (zeros where rows == 0), NULL = not wanted; dw without w is INVALID_ARG. desc->eps is not
 * used. One launch, and a second for dw where the rows took several blocks.
 * Errors: as add_rms_norm_forward, and WORKSPACE (256-byte aligned; none needed without dw). */
int add_rms_norm_backward(const add_norm_desc* desc, const norm_rows* dy, const norm_rows* dh, const norm_rows* h,
                          const norm_param* w, const float* rstd, const norm_rows* dr, const norm_rows* dx,
                          const norm_param* dw, void* workspace, size_t workspace_bytes, void* stream);

/* ---- Rotary positions over several axes ---------------------------------------------------
 * For the query and key heads, after their RMS norms: time, height and width of an image or
 * video token, or one axis for text. Each head has `dim` elements, of which 2 pairs are turned:
 * pair i is elements (i, i + pairs) under MUON_ROTARY_HALVES and (2 i, 2 i + 1) under
 * MUON_ROTARY_ADJACENT, turned by the angle 2 pi freq[i] position[axis[i]] of its token:
 *   p' = p cos - q sin,  q' = p sin + q cos
 * elements from 2 pairs on are copied. inverse != 0 turns back, which is also the gradient.
 * The angle's fraction of a turn is fp64, its sine and cosine and the products are fp32,
 * rounded once. */
#define MUON_ROTARY_HALVES 0
#define MUON_ROTARY_ADJACENT 1
#define MUON_ROTARY_MAX_DIM 1024
#define MUON_ROTARY_MAX_HEADS 65536
#define MUON_POSITION_I32 0
#define MUON_POSITION_I64 1
#define MUON_POSITION_F32 2

typedef struct rotary_desc {
    int64_t batch, tokens, heads, dim;
    int32_t pairs, axes;     /* >= 1; 2 pairs <= dim */
    int32_t dtype;           /* of x and y */
    int32_t layout;          /* MUON_ROTARY_* */
    int32_t position_type;   /* MUON_POSITION_* */
    int32_t inverse;
} rotary_desc;

/* Head h of token t of batch b at data + b stride_batch + t stride_token + h stride_head
 * elements, its elements adjacent. Strides are >= 0. */
typedef struct rotary_rows {
    void* data;
    int64_t stride_batch, stride_token, stride_head;
} rotary_rows;

/* The token's `axes` positions, adjacent, at data + b stride_batch + t stride_token elements
 * (stride_batch 0: the same for every batch). */
typedef struct rotary_positions {
    const void* data;
    int64_t stride_batch, stride_token;
} rotary_positions;

/* freq (DEVICE, pairs doubles): turns per unit of position, theta^(-i / n) / (2 pi) for a
 * ladder of n pairs. axis (DEVICE, pairs ints in 0 .. axes - 1; others are taken for the last).
 * y may be x itself (same pointer and strides). One launch; batch, tokens, heads or dim == 0 is
 * a no-op.
 * Errors: INVALID_ARG, ALIGN (a pointer not aligned to its element), ALIAS (y overlaps another
 * buffer, by spans, or itself), TOO_LARGE (dim above MUON_ROTARY_MAX_DIM, heads above
 * MUON_ROTARY_MAX_HEADS, batch tokens above 2^30, a span above 2^46 elements), HIP. */
int rotary_apply(const rotary_desc* desc, const rotary_rows* x, const rotary_positions* positions, const double* freq,
                 const int32_t* axis, const rotary_rows* y, void* stream);

/* ---- Singular-spectrum diagnostic ----------------------------------------------------
 * SVD entropy of "Muon is Scalable for LLM Training", Sec. 3.4 (Dynamics of Singular
 * Spectrum): for W [A, B] with singular values sigma_1..sigma_n, n = min(A, B),
 *   q_i = sigma_i^2 / sum_j sigma_j^2,   H = -(1 / log n) sum_i q_i log q_i,
 * 1 for a flat spectrum and 0 for rank one. Zero singular values contribute 0; n = 1
 * gives 0; an all-zero matrix gives NaN (nothing to normalise).
 * Computed in fp64 on the device: sigma_i^2 are the eigenvalues of the Gram matrix
 * X X^T (X = W, or W^T when A > B), reduced to tridiagonal form by Householder
 * reflections and solved by Sturm-count bisection. The cost is about
 * min(A,B)^2 max(A,B) fp64 MFMA flops plus 8 min(A,B)^3 / 3 bytes of memory traffic
 * (the upper triangle of the shrinking trailing block, read and written once per
 * column), so this is an occasional diagnostic, not a per-step call. */

/* Workspace in bytes for svd_entropy on `count` matrices of shapes rows[i] x cols[i]
 * (about 8.25 min(A,B)^2 bytes per matrix for up to 16 matrices at a time). Host only.
 * Errors: INVALID_ARG (NULL bytes, count < 0, NULL rows/cols with count > 0, negative
 * dims), TOO_LARGE (as muon_workspace_bytes, or min(A, B) above 65536). */
int svd_entropy_workspace_bytes(const int64_t* rows, const int64_t* cols, int32_t count, size_t* bytes);

/* entropy[i] = H(w[i]) for the fp32 DEVICE matrices w[i] of shape rows[i] x cols[i]
 * (host arrays of `count` entries; row-major, 16-byte aligned, read only).
 * entropy: DEVICE array of `count` doubles, 8-byte aligned.
 * sigma_sq: optional DEVICE array (NULL = not wanted) of sum_i min(rows[i], cols[i])
 *   doubles, 8-byte aligned; matrix i's sigma^2 in descending order start at
 *   sum_{k<i} min(rows[k], cols[k]). Eigenvalues below 0 by rounding are reported as 0.
 * Empty matrices are skipped (their entropy entry is left unchanged). Outputs must not
 * overlap each other, the inputs or the workspace.
 * Errors: INVALID_ARG, ALIGN, ALIAS, WORKSPACE, TOO_LARGE, HIP. */
int svd_entropy(const float* const* w, const int64_t* rows, const int64_t* cols, int32_t count,
                void* workspace, size_t workspace_bytes, double* entropy, double* sigma_sq,
                void* stream);

/* ---- Attainable ceilings ------------------------------------------------------------
 * Yardsticks for the two rooflines the step is measured against, timed by the caller
 * (HIP events on `stream`) on the same GPU; neither is part of the optimizer step.
 * muon_ceiling_copy: dst[i] = src[i] for n fp32 elements (DEVICE pointers, 16-byte
 *   aligned, not overlapping), streamed as the step's HBM-bound passes stream: 256
 *   threads, 32 KiB contiguous per block, all loads of a thread before its stores,
 *   non-temporal hints. 8 n bytes of HBM traffic. Errors: INVALID_ARG, ALIGN, ALIAS,
 *   TOO_LARGE, HIP.
 * muon_ceiling_mfma: `blocks` blocks of four waves; every wave issues `iters` rounds of
 *   16 independent v_mfma_f32_32x32x16_bf16 on register operands into 16 fp32 32 x 32
 *   accumulators (the register budget of a Newton-Schulz GEMM wave), then writes one
 *   checksum to out[4 block + wave] (DEVICE, 4 blocks floats, 4-byte aligned). *flops
 *   (host, may be NULL) receives the dense flop count, blocks * 4 * iters * 16 * 32768.
 *   One block per compute unit (256 blocks) keeps one wave on every SIMD, as the GEMMs
 *   do. Errors: INVALID_ARG, ALIGN, HIP. */
int muon_ceiling_copy(const float* src, float* dst, int64_t n, void* stream);
int muon_ceiling_mfma(float* out, int32_t blocks, int32_t iters, double* flops, void* stream);

/* Optional per-kernel-class timing. While enabled (enable != 0), every kernel the
 * library enqueues is bracketed by HIP events recorded on the caller's stream (a GEMM
 * stage that splits its last tiles over K is bracketed together with its fixup
 * launch, and counts as one launch).
 * muon_timing_read() waits for the recorded events, adds their durations into
 * ms[MUON_KCLASS_COUNT] and launch counts into launches[MUON_KCLASS_COUNT] (either
 * may be NULL), and clears the record. muon_timing_enable(0) discards the record.
 * Process-global; not meant for concurrent callers. Errors: HIP. */
int muon_timing_enable(int enable);
int muon_timing_read(double* ms, int64_t* launches);

#ifdef __cplusplus
}
#endif

#endif /* MUON_ROCM_H */
