/*
 * muon.h -- C ABI of the MI355X (gfx950) Muon optimizer step.
 *
 * One call runs the whole Muon step over a list of 2-D weight matrices:
 *   M' = beta*M + G                        (momentum, no dampening)
 *   U  = M'   (or beta*M' + G with MUON_FLAG_NESTEROV)
 *   X0 = U / (||U||_F + eps)               (Frobenius normalization)
 *   X  <- a_k X + (b_k A + c_k A A) X,  A = X X^T,  k = 1..ns_steps
 *         (on the smaller side: matrices with rows > cols are transposed)
 *   W' = (1 - lr*wd) W - lr * s_rule(rows, cols) * X
 * It also runs the AdamW step for the other parameters (muon_adamw_step),
 * the Muon-Cayley step on the Stiefel manifold (muon_cayley_step), and the
 * operators that make the gradients in a preference or policy step: norms
 * around a block (muon_block_norm), token log-probabilities over a vocabulary
 * head (muon_token_logp) and two losses on them (muon_preference_loss,
 * muon_policy_loss).
 * Sources, cited by page title and section:
 *   [Muon优化器] linsight.cn/f25d614e.html -- the industrial Muon class
 *     (momentum, Nesterov, decay and apply), zeropower_via_newtonschulz
 *     (normalization, transposition, the quintic iteration) and section
 *     "缩放因子：从初始化到更新尺度" (the four scale rules);
 *   [DeepSeek V4 summary] prism.simon-ai.net/article/8795, section
 *     "Muon的训练效率与DeepSeek V4的混合优化策略" -- per-step coefficients
 *     (8 fast iterations, then 2 stable ones);
 *   [Adam vs Muon essay] guanweilu.cn/article/354.html -- the step as
 *     muon_step(weight, grad, momentum, lr, beta).
 *
 * Conventions for every entry point:
 *  - Matrices are dense, row-major, contiguous, rows = d_out, cols = d_in
 *    (the PyTorch Linear layout), in device memory of the current HIP
 *    device.  All matrices of one call share one dtype (hp->dtype).
 *  - The caller owns every device buffer, including the workspace; the
 *    library never allocates device memory in these calls and keeps no
 *    pointer once the enqueued work has finished.  Host arrays (mats,
 *    hp->schedule) are read during the call only.
 *  - `stream` is a hipStream_t passed as void*; NULL means the default
 *    stream.  Work is enqueued asynchronously; device buffers must stay
 *    alive until the stream reaches that point.
 *  - Argument validation is synchronous and happens before anything is
 *    enqueued; on any error nothing is modified.  Faults during kernel
 *    execution surface at the caller's next synchronization.
 *  - NaN/Inf in G or M are not checked; they stay inside their own matrix.
 *  - Not re-entrant on one workspace: concurrent calls need separate
 *    workspaces (and, if they must overlap, separate streams).
 */
#ifndef MUON_MI355X_H
#define MUON_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MUON_OK = 0,
    MUON_ERR_INVALID_ARG = -1,  /* bad pointer, shape, enum, non-finite scalar, overlap */
    MUON_ERR_UNSUPPORTED = -2,  /* device is not gfx950, or a size beyond the limits below */
    MUON_ERR_WORKSPACE = -3,    /* workspace NULL, too small or not 256-byte aligned */
    MUON_ERR_HIP = -4           /* a HIP runtime call or kernel launch failed */
} muon_status;

typedef enum { MUON_F32 = 0, MUON_BF16 = 1 } muon_dtype;

/* [Muon优化器] section "缩放因子：从初始化到更新尺度" (d_out = rows, d_in = cols):
 *   NAIVE         1
 *   KELLER_JORDAN sqrt(max(1, d_out/d_in))
 *   MUP           sqrt(d_out/d_in)
 *   MOONLIGHT     0.2 * sqrt(max(d_out, d_in))                               */
typedef enum {
    MUON_SCALE_NAIVE = 0,
    MUON_SCALE_KELLER_JORDAN = 1,
    MUON_SCALE_MUP = 2,
    MUON_SCALE_MOONLIGHT = 3
} muon_scale_rule;

/* One Newton-Schulz step's coefficients: X <- a X + (b A + c A A) X. */
typedef struct { float a, b, c; } muon_ns_coeffs;

/* Nesterov form: the iteration runs on beta*M' + G instead of M'
 * ([Muon优化器], industrial Muon class, nesterov branch). */
#define MUON_FLAG_NESTEROV 1u

/* Upper limits of this build. */
#define MUON_MAX_NS_STEPS 64
#define MUON_MAX_MATRICES 65536
#define MUON_MAX_DIM      (1 << 20)

typedef struct {
    void*       weight;    /* in/out, rows x cols */
    const void* grad;      /* in; NULL => the matrix is skipped entirely (state untouched) */
    void*       momentum;  /* in/out optimizer state, same dtype and shape */
    int64_t     rows, cols;
} muon_matrix;

typedef struct {
    float lr;                         /* finite */
    float beta;                       /* finite */
    float weight_decay;               /* finite */
    float eps;                        /* finite, >= 0; added to the Frobenius norm */
    int32_t scale_rule;               /* muon_scale_rule */
    int32_t ns_steps;                 /* 0..MUON_MAX_NS_STEPS; 0 => X = X0 */
    const muon_ns_coeffs* schedule;   /* host array of ns_steps triples (finite) */
    int32_t dtype;                    /* muon_dtype of weight, grad and momentum */
    uint32_t flags;                   /* MUON_FLAG_NESTEROV or 0 */
} muon_hparams;

/* Bytes of device workspace muon_step needs for this list (0 on invalid
 * arguments; the reason is in muon_last_error_message()).  Host-only. */
size_t muon_workspace_bytes(const muon_matrix* mats, int32_t n, const muon_hparams* hp);

/* One Muon step over `n` matrices, grouped: one launch per phase covers all
 * of them.  `workspace` is device memory of at least muon_workspace_bytes()
 * bytes, 256-byte aligned; its contents need not be initialized.
 * Writes weight and momentum of every matrix whose grad is non-NULL. */
muon_status muon_step(const muon_matrix* mats, int32_t n, const muon_hparams* hp,
                      void* workspace, size_t workspace_bytes, void* stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): muon_step
 * with its workspace in a library-owned device array of
 * MUON_NOALLOC_SCRATCH_BYTES bytes per GPU.  The array is part of the
 * library's device code; its address is looked up on the first call on each
 * device, and each GPU the library runs on holds it until the process ends.
 * The call allocates nothing, on the device or the host: the descriptors
 * travel as kernel arguments.
 *  - A list whose muon_workspace_bytes() exceeds MUON_NOALLOC_SCRATCH_BYTES is
 *    rejected with MUON_ERR_WORKSPACE before anything is enqueued (128 MiB
 *    holds, for example, any one 2048 x 8192 matrix in bf16).
 *  - Every call on one GPU uses that GPU's one array, which keeps the last
 *    call's contents (nothing in it has to start at zero).  Calls that overlap
 *    on one GPU, from other streams or threads, race: the caller serializes them.
 *  - Validation, results and errors are otherwise those of muon_step. */
#define MUON_NOALLOC_SCRATCH_BYTES ((size_t)128 << 20)
muon_status muon_step_noalloc(const muon_matrix* mats, int32_t n, const muon_hparams* hp, void* stream);

/* Orthogonalization only (the zeropower_via_newtonschulz contract of
 * [Muon优化器]): out = NS(in / (||in||_F + eps)) with hp's schedule.
 * `in` has hp->dtype; `out` is fp32, same shape, row-major; in and out must
 * not overlap.  hp's lr, beta, weight_decay, scale_rule and flags are ignored. */
typedef struct {
    const void* in;
    float*      out;
    int64_t     rows, cols;
} muon_ns_matrix;

size_t muon_ns_workspace_bytes(const muon_ns_matrix* mats, int32_t n, const muon_hparams* hp);
muon_status muon_ns(const muon_ns_matrix* mats, int32_t n, const muon_hparams* hp,
                    void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * AdamW for the parameters Muon does not take (embeddings, heads, biases,
 * norms), as one grouped launch over a list of tensors:
 *   m' = beta1 m + (1 - beta1) g
 *   v' = beta2 v + (1 - beta2) g^2
 *   p' = (1 - lr wd) p - lr (m' / (1 - beta1^t)) / (sqrt(v' / (1 - beta2^t)) + eps)
 * Sources: [Muon优化器] section "AdamW的问题" (moments, bias corrections, the
 * step); [DeepSeek V4 summary] section "Adam优化器的机制与AdamW的改进" (decay
 * apart from the gradient update); [Muon在Stiefel流形上的精确闭式更新解析]
 * section 4.3 (decay first, moments start at zero, t counts calls).
 * Arithmetic is fp32; p' is rounded once (RNE) to the parameter dtype.
 * --------------------------------------------------------------------------- */
typedef struct {
    void*       param;       /* in/out, numel elements of hp->dtype, contiguous */
    const void* grad;        /* in, same dtype; NULL => the tensor is skipped (state untouched) */
    float*      exp_avg;     /* in/out first moment, numel fp32 (zero before the first step) */
    float*      exp_avg_sq;  /* in/out second moment, numel fp32 (zero before the first step) */
    int64_t     numel;       /* >= 1, <= MUON_MAX_ADAMW_NUMEL */
} muon_adamw_tensor;

#define MUON_MAX_ADAMW_TENSORS 65536
#define MUON_MAX_ADAMW_NUMEL   ((int64_t)1 << 40)

typedef struct {
    float lr;            /* finite */
    float beta1, beta2;  /* in [0, 1) */
    float eps;           /* finite, >= 0 */
    float weight_decay;  /* finite */
    int32_t step;        /* t >= 1: this call is the t-th step of these tensors */
    int32_t dtype;       /* muon_dtype of param and grad */
} muon_adamw_hparams;

/* Device workspace bytes muon_adamw_step needs (0 on invalid arguments). */
size_t muon_adamw_workspace_bytes(const muon_adamw_tensor* tensors, int32_t n, const muon_adamw_hparams* hp);
/* One AdamW step over `n` tensors; the same validation, workspace and stream
 * rules as muon_step.  Tensors must not overlap each other or the workspace. */
muon_status muon_adamw_step(const muon_adamw_tensor* tensors, int32_t n, const muon_adamw_hparams* hp,
                            void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Muon-Cayley: the closed-form update that keeps a weight on the Stiefel
 * manifold ([Muon在Stiefel流形上的精确闭式更新解析], sections 1.3, 3.1-3.3, 6.2).
 * For W with orthonormal columns (W^T W = I; for rows < cols, orthonormal rows,
 * handled as the transpose):
 *   M' = beta M + (1 - beta) (G - 1 mean(G)^T)      mean over the rows
 *   V  = M' - W sym(W^T M'),   sym(S) = (S + S^T) / 2
 *   W' = (I + c A)^-1 (I - c A) W,  A = V W^T - W V^T,  c = lr / 2
 * computed through a 2k x 2k linear system (A has rank at most 2k,
 * k = min(rows, cols)).  fp32 buffers; the 2k x 2k solve runs in fp64.  For
 * k <= 128 it eliminates by k x k blocks and inverts the two diagonal blocks
 * by Gauss-Jordan without pivoting (on the manifold the symmetric part of each
 * is positive definite), switching to partial pivoting for a block whose
 * pivot falls below 1/2; for k > 128 it is an LU factorization with partial
 * pivoting.  No weight decay on this path.
 * --------------------------------------------------------------------------- */
typedef struct {
    float*       weight;    /* in/out rows x cols, fp32, row-major */
    const float* grad;      /* in; NULL => the matrix is skipped */
    float*       momentum;  /* in/out, same shape (zero before the first step) */
    int64_t      rows, cols;
} muon_cayley_matrix;

#define MUON_CAYLEY_MAX_K 256   /* min(rows, cols) limit of this build */

typedef struct {
    float lr;      /* finite */
    float beta;    /* in [0, 1) */
} muon_cayley_hparams;

size_t muon_cayley_workspace_bytes(const muon_cayley_matrix* mats, int32_t n, const muon_cayley_hparams* hp);
/* One Muon-Cayley step over `n` matrices (grouped launches).  Same workspace,
 * stream and validation rules as muon_step; min(rows, cols) above
 * MUON_CAYLEY_MAX_K is MUON_ERR_UNSUPPORTED. */
muon_status muon_cayley_step(const muon_cayley_matrix* mats, int32_t n, const muon_cayley_hparams* hp,
                             void* workspace, size_t workspace_bytes, void* stream);

/* ===========================================================================
 * Training operators: what runs between a model's last block and the
 * optimizer step, and makes the gradients that muon_step and muon_adamw_step
 * consume.  The conventions at the top of this header hold, with these
 * additions:
 *  - matrices are row-major with a row pitch `ld_*` in elements (>= cols) and
 *    unit column stride; vectors are contiguous;
 *  - every output element is written by every call (nothing accumulates into
 *    what a buffer held before), and results are the same bits on every run;
 *  - sums, softmax statistics and norms are held in fp32, the losses' sums in fp64;
 *    an output is rounded once (RNE) to its dtype;
 *  - the calls allocate nothing and copy nothing from the host, so they can be
 *    captured in a HIP graph.
 * =========================================================================== */

/* --- Norms around a block, with its gate and residual scale -----------------
 *   a  = x * rstd0 * post_weight,    rstd0 = 1 / sqrt(mean(x^2) + eps)
 *        (post_weight NULL: a = x)
 *   r' = residual_scale * residual + gate * a         (gate NULL: 1)
 *   n  = r' * rstd1 * pre_weight,    rstd1 = 1 / sqrt(mean(r'^2) + eps)
 * x is the block's output, residual the stream it joins, n the next block's
 * input.  n is formed from the fp32 value of r', not from the stored one. */
#define MUON_GATE_NONE    0
#define MUON_GATE_CHANNEL 1   /* gate[cols], weight_dtype */
#define MUON_GATE_FULL    2   /* gate[rows][cols], dtype, pitch ld_gate */

#define MUON_MAX_NORM_COLS 32768
#define MUON_MAX_TOKENS    ((int64_t)1 << 30)

typedef struct {
    const void* x;            /* rows x cols */
    const void* residual;     /* rows x cols */
    const void* post_weight;  /* cols, or NULL: x is not normalized */
    const void* gate;         /* by gate_kind; NULL for MUON_GATE_NONE */
    const void* pre_weight;   /* cols; NULL exactly if out_norm is */
    void*  out_residual;      /* rows x cols; may be `residual` itself (same pitch) */
    void*  out_norm;          /* rows x cols, or NULL */
    float* rstd;              /* 2 x rows (rstd0, rstd1) for the backward pass, or NULL; an absent norm writes 1 */
    int64_t rows, cols;       /* rows >= 0, 1 <= cols <= MUON_MAX_NORM_COLS */
    int64_t ld_x, ld_residual, ld_gate, ld_out_residual, ld_out_norm;
    float   residual_scale;   /* finite */
    float   eps;              /* finite, >= 0 */
    int32_t dtype;            /* muon_dtype of the matrices */
    int32_t weight_dtype;     /* muon_dtype of post_weight, pre_weight and a channel gate */
    int32_t gate_kind;
} muon_block_norm_args;

muon_status muon_block_norm(const muon_block_norm_args* args, void* stream);

/* Its gradients.  grad_norm (of n) and grad_out_residual (of r') may each be
 * NULL (no gradient there), not both; out_residual and rstd are the forward
 * pass's.  Weight gradients are sums over the rows, in weight_dtype, each NULL
 * exactly if its weight is. */
typedef struct {
    const void* x;
    const void* out_residual;
    const float* rstd;               /* 2 x rows */
    const void* grad_norm;           /* rows x cols or NULL */
    const void* grad_out_residual;   /* rows x cols or NULL */
    const void* post_weight;
    const void* gate;
    const void* pre_weight;          /* NULL only if grad_norm is */
    void* grad_x;                    /* rows x cols */
    void* grad_residual;             /* rows x cols; may be grad_out_residual itself (same pitch) */
    void* grad_post_weight;          /* cols */
    void* grad_gate;                 /* cols or rows x cols */
    void* grad_pre_weight;           /* cols */
    int64_t rows, cols;
    int64_t ld_x, ld_out_residual, ld_grad_norm, ld_grad_out_residual, ld_gate, ld_grad_x, ld_grad_residual,
        ld_grad_gate;
    float   residual_scale;
    int32_t dtype, weight_dtype, gate_kind;
} muon_block_norm_backward_args;

size_t muon_block_norm_backward_workspace_bytes(const muon_block_norm_backward_args* args);
muon_status muon_block_norm_backward(const muon_block_norm_backward_args* args, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* --- Log-probabilities of target tokens under a vocabulary head -------------
 *   z_ij = scale * sum_k hidden[i][k] head[j][k]
 *   lse_i = log sum_j exp(z_ij),   logp_i = z_i,target_i - lse_i
 * The tokens x vocab logits are not formed as an output.  A negative target
 * marks a token that is not scored: logp = lse = 0, its gradients are zero and
 * its hidden row is not used, whatever it holds.  A target >= vocab gives
 * logp = NaN. */
#define MUON_MAX_VOCAB (1 << 24)

typedef struct {
    const void*    hidden;    /* tokens x cols */
    const void*    head;      /* vocab x cols */
    const int64_t* targets;   /* tokens */
    float* logp;              /* tokens */
    float* lse;               /* tokens */
    void*  saved;             /* muon_token_logp_saved_bytes() bytes, 256-byte aligned, or NULL: keeps what lets
                                 the backward pass skip forming the logits again */
    int64_t tokens, cols, vocab;   /* tokens >= 0, cols >= 1, vocab >= 1 */
    int64_t ld_hidden, ld_head;
    float   scale;            /* finite */
    int32_t dtype;            /* muon_dtype of hidden and head */
} muon_token_logp_args;

size_t muon_token_logp_saved_bytes(const muon_token_logp_args* args);
size_t muon_token_logp_workspace_bytes(const muon_token_logp_args* args);
muon_status muon_token_logp(const muon_token_logp_args* args, void* workspace, size_t workspace_bytes, void* stream);

/* With c_i = scale * grad_logp_i and p_ij = exp(z_ij - lse_i):
 *   dz_ij = c_i ([j = target_i] - p_ij),  grad_hidden = dz head,  grad_head = dz^T hidden
 * grad_hidden or grad_head may be NULL (not wanted), not both.  `saved` is what
 * muon_token_logp kept for the same inputs, or NULL: then the logits are formed
 * again, and lse with them (a rounded lse does not hold a certain token's
 * 1 - p; what the argument holds is not used).
 *
 * Precision.  Up to 64 tokens: dz as two bf16 parts (2^-16) in bf16 calls; in fp32
 * dz, hidden and head as three (24 bits for values down to 2^-109; hidden is scaled
 * for them first in a backward pass and in a forward pass with `saved`).
 * More tokens: dz as fp16 under a power-of-two scale for each token, in bf16 calls
 * one part (11 bits), in fp32 calls two (22), and hidden and head, for the gradients'
 * products, as one part (exact for bf16 values) or two under one scale each; all
 * this for values down to 2^-28 of the operand's largest finite one (of the token's
 * largest in dz; in grad_head a token counts so down to 2^-28 of the largest
 * token), fewer bits below and none below 2^-39.  bf16 calls form dz from
 * exp(z - M) in fp16, M the maximum of up to 256 neighbouring entries without the
 * target: 11 bits down to 2^-14, none below 2^-25.  The logits' product takes
 * bf16 operands as they are.  fp32 operands of scored tokens have to be finite: an
 * infinity makes NaN of its logits. */
typedef struct {
    const void*    hidden;
    const void*    head;
    const int64_t* targets;
    const float*   lse;         /* tokens, as muon_token_logp wrote it for the same inputs */
    const float*   grad_logp;
    const void*    saved;
    void* grad_hidden;        /* tokens x cols or NULL, dtype */
    void* grad_head;          /* vocab x cols or NULL, dtype */
    int64_t tokens, cols, vocab;
    int64_t ld_hidden, ld_head, ld_grad_hidden, ld_grad_head;
    float   scale;
    int32_t dtype;
} muon_token_logp_backward_args;

size_t muon_token_logp_backward_workspace_bytes(const muon_token_logp_backward_args* args);
muon_status muon_token_logp_backward(const muon_token_logp_backward_args* args, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* --- Losses over per-token log-probabilities --------------------------------
 * Tokens of `sequences` sequences lie one after the other: sequence s is
 * tokens offsets[s] .. offsets[s + 1) - 1, with offsets in device memory,
 * 0 <= offsets[0] and non-decreasing up to at most `tokens` (values outside are
 * taken as the nearest bound; empty sequences are fine).  Tokens of no
 * sequence, and tokens with mask 0, count for nothing and get gradient 0,
 * whatever their log-probabilities hold.  The gradient of the loss with respect
 * to logp, times grad_scale, comes with the same call. */

/* Preference loss over pairs (sequence 2p preferred to sequence 2p + 1), over the
 * pairs' mean:
 *   r_s = sum_t mask_t (logp_t - ref_logp_t)   [/ number of counted tokens]
 *   u = r_2p - r_2p+1,  h = beta u - margin
 *   SIGMOID  -(1 - e) log sigma(h) - e log sigma(-h)     e = label_smoothing; a
 *            term whose share is 0 is 0 for infinite h too
 *   HINGE    max(0, 1 - h)
 *   SQUARED  (u - 1 / (2 beta))^2                        beta != 0, margin unused */
typedef enum { MUON_PREFERENCE_SIGMOID = 0, MUON_PREFERENCE_HINGE = 1, MUON_PREFERENCE_SQUARED = 2 } muon_preference_kind;

typedef struct {
    const void*    logp;       /* tokens, dtype */
    const void*    ref_logp;   /* tokens, dtype, or NULL (0) */
    const uint8_t* mask;       /* tokens, or NULL (all count) */
    const int64_t* offsets;    /* sequences + 1 */
    float* loss;               /* 1 (0 for no pairs) */
    float* rewards;            /* sequences: beta * r_s, or NULL */
    void*  grad_logp;          /* tokens, dtype, or NULL */
    int64_t tokens, sequences; /* sequences even */
    float   beta, margin, label_smoothing, grad_scale;   /* finite; 0 <= label_smoothing <= 1 */
    int32_t kind;              /* muon_preference_kind */
    int32_t average;           /* nonzero: r_s is a mean over the counted tokens (0 if there are none) */
    int32_t dtype;
} muon_preference_args;

size_t muon_preference_loss_workspace_bytes(const muon_preference_args* args);
muon_status muon_preference_loss(const muon_preference_args* args, void* workspace, size_t workspace_bytes,
                                 void* stream);

/* Clipped policy loss with a KL term.  Per counted token, with
 * rho = exp(logp - old_logp), lo = 1 - clip_low, hi = 1 + clip_high:
 *   gain = min(rho A, clamp(rho, lo, hi) A);  for A < 0 and dual_clip > 0, at least dual_clip A
 *   KL   K1: logp - ref   K2: (logp - ref)^2 / 2   K3: exp(ref - logp) - (ref - logp) - 1
 *   l    = -gain + kl_coef KL
 * A token whose gain is held at a bound gets no gradient from it.
 * REDUCE_TOKEN:    mean of l over all counted tokens
 * REDUCE_SEQUENCE: mean over the sequences of each one's mean over its counted
 *                  tokens (a sequence without any adds 0) */
typedef enum { MUON_KL_NONE = 0, MUON_KL_K1 = 1, MUON_KL_K2 = 2, MUON_KL_K3 = 3 } muon_kl_kind;
typedef enum { MUON_REDUCE_TOKEN = 0, MUON_REDUCE_SEQUENCE = 1 } muon_loss_reduction;

typedef struct {
    const void*    logp;        /* tokens, dtype */
    const void*    old_logp;    /* tokens, dtype */
    const void*    ref_logp;    /* tokens, dtype; NULL exactly if kl is MUON_KL_NONE */
    const float*   advantages;  /* tokens, or sequences (advantage_per_sequence) */
    const uint8_t* mask;        /* tokens, or NULL */
    const int64_t* offsets;     /* sequences + 1 */
    float* loss;                /* 1 */
    float* stats;               /* 4: mean KL, share of tokens held at a bound, mean rho (over the counted
                                   tokens), number of counted tokens; or NULL */
    void*  grad_logp;           /* tokens, dtype, or NULL */
    int64_t tokens, sequences;
    float   clip_low, clip_high;   /* >= 0, finite */
    float   dual_clip;             /* 0 (off), or >= 1, finite */
    float   kl_coef, grad_scale;   /* finite */
    int32_t kl, reduction, advantage_per_sequence, dtype;
} muon_policy_args;

size_t muon_policy_loss_workspace_bytes(const muon_policy_args* args);
muon_status muon_policy_loss(const muon_policy_args* args, void* workspace, size_t workspace_bytes, void* stream);

/* Static description of a status code. */
const char* muon_status_string(int32_t status);
/* Detail of the calling thread's last failure ("" if none). */
const char* muon_last_error_message(void);

/* Optional per-kernel timing with HIP events recorded on the launch stream.
 * While enabled, every launch is bracketed by two
 * events; reading synchronizes them and returns, per kernel class,
 * the summed duration in milliseconds and the number of launches, then
 * resets the counters of all classes.  muon_profile_read returns the first
 * MUON_KCLASS_COUNT classes, those of the optimizer steps (its struct does not
 * grow), muon_profile_read_classes the first `classes` into two arrays of that
 * length (either may be NULL).  Classes: 0 momentum+norm, 1 norm finalize, 2 Gram,
 * 3 polynomial, 4 update, 5 apply, 6 AdamW, 7 Muon-Cayley (all its kernels),
 * 8 the last update of muon_step, which also applies decay and the step to W,
 * 9 block norm (both directions), 10 token log-probabilities (both directions),
 * 11 preference loss, 12 policy loss.
 * Host-side bookkeeping only. */
#define MUON_KCLASS_COUNT 9
#define MUON_KCLASS_ALL   13
typedef struct {
    double  ms[MUON_KCLASS_COUNT];
    int64_t launches[MUON_KCLASS_COUNT];
} muon_profile;

muon_status muon_profile_enable(int32_t on);
muon_status muon_profile_read(muon_profile* out);
muon_status muon_profile_read_classes(int32_t classes, double* ms, int64_t* launches);

/* Library version as major*10000 + minor*100 + patch. */
int32_t muon_version(void);

#ifdef __cplusplus
}
#endif
#endif /* MUON_MI355X_H */
