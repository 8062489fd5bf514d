/*
 * falcon.h -- C ABI of the MI355X (gfx950) Falcon fast-weight library.
 *
 * The library computes the read-after-write, prefix-shifted, NLMS-normalised
 * delta rule of "Fast Weight Attention for Continual Learning" (arXiv
 * 2608.27763; section and equation numbers below are the paper's) and its
 * inner-product and per-column relatives.  For every (batch b, head h) the
 * fast state S in R^{dk x dv} evolves over t = 1..T as
 *
 *     x_t   = phi(k_{t-1})             x_1 = k_prev, or 0 on a fresh start
 *     eta_t = beta_t / (||x_t||^2 + lam_t + eps)          (Eq. 3.4)
 *             eta_t := 0 if the denominator is 0, and eta_1 := 0 on a fresh
 *             start (Section 3, indexing and causality conventions)
 *     alpha_t = min(eta_t lam_t, 1 - eps_gamma),  gamma_t = 1 - alpha_t
 *             (Section 4.3, "Decay positivity"; applied in every entry point)
 *     FALCON_1 : S_t = gamma_t S_{t-1} + eta_t x_t r_t^T, r_t = v_t - S_{t-1}^T x_t
 *     FALCON_1A: S_t = gamma_t S_{t-1} + eta_t x_t v_t^T            (Section 4.3)
 *     FALCON_2 : per-column gains beta_{t,j}: column j of S follows FALCON_1
 *                with eta_{t,j}, gamma_{t,j}                       (Section 4.2)
 *     FALCON_2A: per-column gains, additive write                  (Eq. 4.7)
 *     o_t = S_t^T phi(q_t)              (read after write, Section 4 summary)
 *
 * Conventions shared by every entry point
 *  - All tensor pointers are DEVICE pointers owned by the caller, contiguous
 *    row-major with the last axis fastest, 16-byte aligned.  Layouts:
 *      phi_k, phi_q : [B, H, T, dk]     io dtype
 *      v, o         : [B, H, T, dv]     io dtype
 *      beta         : [B, H, T] (FALCON_1, FALCON_1A) or [B, H, T, dv]
 *                     (FALCON_2, FALCON_2A), float32
 *      lam          : [B, H, T]         float32
 *      S0, S_T, S   : [B, H, dk, dv]    float32 (dv fastest)
 *      k_prev       : [B, H, dk]        io dtype
 *  - Calls are asynchronous and stream-ordered on `stream` (a hipStream_t;
 *    NULL means the legacy default stream).  The library never synchronises
 *    the device, allocates no device memory in these entry points, and keeps
 *    no global mutable state besides two process-wide settings
 *    (falcon_set_wait_limit, falcon_set_f1_launch_form), so concurrent calls
 *    on different streams are safe as long as their output buffers and
 *    workspaces do not overlap.
 *  - Every argument is validated before anything is launched; on error the
 *    call returns a negative falcon_status and touches no memory.
 *  - Launch failures reported by the HIP runtime return FALCON_ERR_HIP.
 *  - Values outside the paper's domain (beta outside (0,2), lam < 0,
 *    non-finite data) are not checked on the device: they propagate
 *    arithmetically (NaN in, NaN out).
 *  - Supported sizes: dk, dv in {16, 32, 64, 128}; chunk C in {16, 32, 64};
 *    any T >= 0 (the last chunk may be ragged); B, H >= 0.
 *  - Arithmetic: the state and every accumulation are float32.  With bf16
 *    I/O the matrix products of the chunked path take bf16 operands with
 *    float32 accumulation; with float32 I/O everything is float32.
 */
#ifndef FALCON_H_
#define FALCON_H_

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FALCON_ABI_VERSION 1

typedef enum {
  FALCON_OK = 0,
  FALCON_ERR_NULL = -1,      /* a required pointer is NULL                    */
  FALCON_ERR_SHAPE = -2,     /* B, H, T < 0, or dk / dv not supported         */
  FALCON_ERR_DTYPE = -3,     /* io_dtype not a falcon_dtype                   */
  FALCON_ERR_CHUNK = -4,     /* chunk size not supported                      */
  FALCON_ERR_ALIGN = -5,     /* a pointer is not 16-byte aligned              */
  FALCON_ERR_WORKSPACE = -6, /* workspace missing or smaller than required   */
  FALCON_ERR_VARIANT = -7,   /* variant not a falcon_variant                  */
  FALCON_ERR_HIP = -8,       /* the HIP runtime reported an error at launch  */
  FALCON_ERR_VALUE = -9,     /* eps < 0 / not finite, eps_gamma not in (0,1) */
  FALCON_ERR_ALIAS = -10,    /* an output or the workspace overlaps another
                                argument                                     */
  FALCON_ERR_SCRATCH = -11   /* falcon_fwd_chunked_noalloc: one sequence needs
                                more than FALCON_NOALLOC_SCRATCH_BYTES        */
} falcon_status;

typedef enum {
  FALCON_1 = 1,   /* scalar NLMS regression rule (Section 4, Falcon-1)      */
  FALCON_1A = 2,  /* scalar inner-product rule   (Section 4.3, Falcon-1A)   */
  FALCON_2 = 3,   /* per-column regression rule  (Section 4.2, Falcon-2)    */
  FALCON_2A = 4   /* per-column inner-product    (Section 4.3, Falcon-2A)   */
} falcon_variant;

typedef enum {
  FALCON_F32 = 0,  /* float32 features, values and outputs */
  FALCON_BF16 = 1  /* bfloat16 features, values and outputs (RNE on store) */
} falcon_dtype;

/* Problem description (plain int32 fields so that every language binds it
 * the same way). */
typedef struct {
  int32_t B, H, T;      /* batch, heads, sequence length                    */
  int32_t dk, dv;       /* key-feature and value widths                     */
  int32_t variant;      /* a falcon_variant                                 */
  int32_t io_dtype;     /* a falcon_dtype                                   */
  float eps;            /* step-size stabiliser, >= 0 (Eq. 3.4)             */
  float eps_gamma;      /* positive-decay clamp, in (0, 1) (Section 4.3);
                           the pages give no value, 1e-6 is the default    */
} falcon_problem;

/* Version of this ABI (FALCON_ABI_VERSION of the built library). */
int32_t falcon_abi_version(void);

/* Human-readable name of a status code (static storage, never NULL). */
const char* falcon_status_string(int32_t status);

/*
 * falcon_set_wait_limit -- a process-wide setting of the library.  Some
 * kernels hand data between waves or workgroups through flags in memory;
 * every such wait is bounded and gives up after `polls` polls (default
 * 4194304, about 0.1-0.2 s).  A call in which a wait gave up does not hang:
 * it finishes and reports the failure in its results, every output element
 * and every final-state element of the affected sequences being NaN.
 * falcon_scan_fwd works the tokens concerned out again where nothing waits
 * instead: its results are the same whether or not a wait gave up.
 * Meant for tests of that path and for debugging; calls made while it
 * changes read either value.  polls = 0 makes every such wait give up at
 * once.  Returns the previous limit, or -1 (nothing changed) for polls < 0.
 */
int32_t falcon_set_wait_limit(int32_t polls);

/*
 * falcon_set_f1_launch_form -- the other process-wide setting: how
 * falcon_fwd_chunked runs its Falcon-1 fast path (bf16 I/O, dk = dv = 64,
 * C = 64; every other case ignores it).  Both forms compute the same chunk
 * form with the same roundings and give bit-identical results (paper,
 * Section 4.2, chunk-parallel implementation; Eq. 3.3 per chunk):
 *   FALCON_F1_ONE_LAUNCH (default): one kernel in which chunk workgroups
 *     build the chunk matrices while per-sequence chain workgroups, started
 *     first, carry the state through announced chunks (plus a small fill of
 *     the hand-over flags).  Batches of more than 256 sequences (B H) run the
 *     two-launch form instead: their chains would hold too many workgroup
 *     slots;
 *   FALCON_F1_TWO_LAUNCH: the chunk matrices of all chunks, then the chains.
 * The workspace size is the same for both.  Meant for comparison and
 * debugging; calls made while it changes use either form.  Returns the
 * previous form, or -1 (nothing changed) for any other value.
 */
#define FALCON_F1_ONE_LAUNCH 0
#define FALCON_F1_TWO_LAUNCH 1
int32_t falcon_set_f1_launch_form(int32_t form);

/*
 * falcon_fwd_recurrent -- the recurrent form (paper, Section 4.6 and the
 * complexity table of the juhoplayground post: O(N) sequential scan, O(1)
 * state).  One pass over T per (b, h) with the state held on-chip.
 *
 *  S0      : initial state, or NULL for S_0 = 0.
 *  k_prev  : phi(k_0), the key feature preceding token 1, for continuing a
 *            sequence; NULL selects the fresh-start boundary x_1 = 0,
 *            eta_1 = 0 (even when S0 is not NULL).
 *  o       : output, must not overlap any input.
 *  S_T     : final state, or NULL to skip; may alias S0 exactly.
 */
falcon_status falcon_fwd_recurrent(const falcon_problem* p,
                                   const void* phi_k, const void* phi_q, const void* v,
                                   const float* beta, const float* lam,
                                   const float* S0, const void* k_prev,
                                   void* o, float* S_T, hipStream_t stream);

/*
 * falcon_fwd_chunked -- the chunk-parallel form (paper, Section 4.2
 * "Chunk-parallel implementation" and the SSD-style chunking of the
 * rainbus review: intra-chunk work in parallel, only the fixed-size state
 * passed between chunks).  Same arguments and result as
 * falcon_fwd_recurrent up to float rounding, plus the chunk size C.
 *
 *  C         : chunk length, 16, 32 or 64.
 *  workspace : device scratch of at least falcon_workspace_bytes(p, C)
 *              bytes (may be NULL when that is 0); the bytes the call uses
 *              may overlap no input and no output (FALCON_ERR_ALIAS).
 */
falcon_status falcon_fwd_chunked(const falcon_problem* p,
                                 const void* phi_k, const void* phi_q, const void* v,
                                 const float* beta, const float* lam,
                                 const float* S0, const void* k_prev,
                                 void* o, float* S_T,
                                 int32_t C, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/* Device scratch needed by falcon_fwd_chunked for this problem and C;
 * returns (size_t)-1 for an invalid problem. */
size_t falcon_workspace_bytes(const falcon_problem* p, int32_t C);

/* Size of the static device buffer behind falcon_fwd_chunked_noalloc. */
#define FALCON_NOALLOC_SCRATCH_BYTES (64u << 20)

/*
 * falcon_fwd_chunked_noalloc -- falcon_fwd_chunked for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  Same arguments and results as
 * falcon_fwd_chunked, without the workspace: the kernels that need scratch
 * use a static device buffer of FALCON_NOALLOC_SCRATCH_BYTES (64 MiB) that the
 * library holds on every GPU it runs on until the process ends.  When the
 * problem needs more scratch than that, the sequences are processed in
 * groups that fit, one group after another on `stream`; a problem in which a
 * single sequence needs more returns FALCON_ERR_SCRATCH (with bf16 I/O,
 * dk = dv = 64 and C = 64: Falcon-1 beyond T = 130880 tokens, Falcon-1A
 * beyond T = 1048064).  The call allocates nothing.
 *
 * The buffer of a GPU is shared by every call on that GPU and keeps the last
 * call's contents; no part of it needs to start at zero.  Calls that overlap
 * in time on one GPU (different streams or threads without ordering) race on
 * it and must not be made.  `stream` must belong to the current device, whose
 * buffer is used.  The first call on a device looks the buffer up (the HIP
 * runtime's symbol lookup, no allocation); FALCON_ERR_HIP if that fails.
 */
falcon_status falcon_fwd_chunked_noalloc(const falcon_problem* p,
                                         const void* phi_k, const void* phi_q, const void* v,
                                         const float* beta, const float* lam,
                                         const float* S0, const void* k_prev,
                                         void* o, float* S_T, int32_t C, hipStream_t stream);

/*
 * falcon_decode_step -- one read-after-write token for every (b, h) from a
 * carried state: the rule of the paper's Section 4 naming summary (Falcon-1:
 * residual against the state before the write, Eq. 3.3; step size Eq. 3.4;
 * decay clamp of Section 4.3) applied to a single token, which is the
 * recurrent form run at inference with O(1) state per head (complexity table
 * of the juhoplayground post).  The read o = S_t^T phi(q_t) comes after the
 * write.  p->T is ignored.  Validation, status codes and stream semantics are
 * those of the forward entry points; S is both read and written, so it may
 * overlap no other argument.
 *
 *  phi_k_prev : [B, H, dk] io dtype, the PREVIOUS token's key feature x_t.
 *  phi_q, v   : [B, H, dk] / [B, H, dv] io dtype, this token's query, value.
 *  beta       : [B, H] (FALCON_1, 1A) or [B, H, dv] (FALCON_2, 2A), float32.
 *  lam        : [B, H] float32.
 *  S          : [B, H, dk, dv] float32, updated IN PLACE to S_t.
 *  is_first   : [B] bytes or NULL; a nonzero entry marks a sequence whose
 *               current token is t = 1, where eta := 0 and gamma := 1.
 *  o          : [B, H, dv] io dtype, o_t = S_t^T phi(q_t).
 */
falcon_status falcon_decode_step(const falcon_problem* p,
                                 const void* phi_k_prev, const void* phi_q, const void* v,
                                 const float* beta, const float* lam,
                                 float* S, const uint8_t* is_first,
                                 void* o, hipStream_t stream);

/*
 * falcon_bwd_chunked -- gradients of the FALCON_1 forward.  Training
 * differentiates through the update itself (paper, Section 3); this entry
 * point returns, for the scalar loss
 *
 *     L = <dO, o> + <dS_T, S_T>     (o, S_T the result of falcon_fwd_*),
 *
 * the derivatives of L with respect to every input.  It recomputes the
 * forward in 32-token chunks (Section 4.2's chunk-parallel form), runs the
 * state chain forward and the adjoint chain backward, and then the chunk-local
 * reverse mode in parallel over chunks.  All arithmetic is float32.
 *
 * Supported: variant FALCON_1, dk = dv = 64, io dtype float32 or bfloat16,
 * any T >= 0.  Other variants return FALCON_ERR_VARIANT, other widths
 * FALCON_ERR_SHAPE.  The clamp of Section 4.3 is part of the forward: where it
 * binds (eta lam > 1 - eps_gamma) gamma is constant and passes no gradient.
 *
 *  phi_k .. k_prev : the forward's inputs, as in falcon_fwd_chunked.
 *  dO      : [B, H, T, dv] io dtype, dL/do.
 *  dS_T    : [B, H, dk, dv] float32, dL/dS_T, or NULL for zero.
 *  dphi_k, dphi_q : [B, H, T, dk] float32.  dphi_k[..., T-1, :] is 0 (the
 *            last key is read by no token of this call).
 *  dv      : [B, H, T, dv] float32.
 *  dbeta, dlam : [B, H, T] float32.
 *  dS0     : [B, H, dk, dv] float32, dL/dS_0, or NULL to skip.
 *  dk_prev : [B, H, dk] float32, dL/dk_prev, or NULL to skip; ignored (not
 *            written) when k_prev is NULL.
 *  Every output must not overlap any input or another output
 *  (FALCON_ERR_ALIAS).
 *  workspace : device scratch of at least falcon_bwd_workspace_bytes(p)
 *              bytes, 16-byte aligned (per 32-token chunk per (b, h): the
 *              chunk maps, the state entering the chunk, the adjoint
 *              leaving it, the forward factors W, U, T, the gates and
 *              each row's decay gamma; 103,552 bytes).
 */
falcon_status falcon_bwd_chunked(const falcon_problem* p,
                                 const void* phi_k, const void* phi_q, const void* v,
                                 const float* beta, const float* lam,
                                 const float* S0, const void* k_prev,
                                 const void* dO, const float* dS_T,
                                 float* dphi_k, float* dphi_q, float* dv,
                                 float* dbeta, float* dlam, float* dS0, float* dk_prev,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Device scratch needed by falcon_bwd_chunked; (size_t)-1 for an invalid or
 * unsupported problem. */
size_t falcon_bwd_workspace_bytes(const falcon_problem* p);

/*
 * ---- around the recurrence ---------------------------------------------------
 *
 * What a fast-weight block runs before and after its recurrence, and the
 * recurrence's sibling with a decay of its own for every channel and state:
 *   falcon_conv_*  the short causal convolution of the projections;
 *   falcon_norm_*  the group norm with an activation, a token's head at a time:
 *                  it makes phi(k) and phi(q) in the [B, H, T, dk] layout that
 *                  falcon_fwd_* read, and norms the [B, H, T, dv] outputs;
 *   falcon_scan_*  the selective state space scan;
 *   falcon_linear_*  linear attention with a decay for each head;
 *   falcon_residual_*  the residual update between two blocks: norm of the block's
 *                  output, gate, scale, sum, norm for the next block.
 * Status codes, streams, the order of checks and launches and the absence of
 * allocation are those of the entry points above.  Also:
 *  - "Rows" tensors are channels last, [B, T, width].  Where a field *_row is
 *    named for an input, row (b, t) starts at element (b T + t) *_row, so the
 *    input may be some of the columns of a wider projection (*_row >= width);
 *    every other tensor is contiguous.  Base pointers are 16-byte aligned.
 *    An input's range, for the check of overlaps, runs from its first row's
 *    first element to its last row's last one: columns of one projection may
 *    interleave among inputs, but an output may not lie between them.
 *  - lengths, [B] int32 or NULL, gives each sequence's number of tokens
 *    (clamped to [0, T]).  Rows behind a sequence's end are never read.
 *    Forward calls leave the output rows behind it as they were (where a problem
 *    has zero_behind and it is not 0: clear them) and take the carried state at
 *    the end; backward calls write zero gradients there.
 *  - Parameters (weights, biases, A, D) and states of the scan are float32;
 *    gradients are float32.  Incoming gradients dy have dy_dtype, a
 *    falcon_dtype of its own (falcon_bwd_chunked gives float32 ones).
 *  - Sums over tokens (parameter gradients) are made in a fixed order: results
 *    are the same from call to call.
 *  - A call has at most 2^30 tokens (B T) and 2^40 elements of one tensor, a
 *    single-token call 2^31 elements of x (the scan's 2^27).  Scans and
 *    gradients that would take more than 2^24 - 1 workgroups return
 *    FALCON_ERR_HIP, with nothing launched.
 */

typedef enum {
  FALCON_ACT_NONE = 0,  /* f(p) = p                                   */
  FALCON_ACT_SILU = 1,  /* f(p) = p / (1 + exp(-p))                   */
  FALCON_ACT_ELU1 = 2,  /* f(p) = p + 1 for p > 0, exp(p) otherwise;
                           falcon_norm_* only                         */
  FALCON_ACT_SIGMOID = 3 /* f(p) = 1 / (1 + exp(-p));
                           falcon_residual_* only                     */
} falcon_activation;

/*
 * falcon_conv_fwd -- the short causal convolution, a channel at a time:
 *
 *     y_t = f( bias + sum_{j < W} weight_j x_{t - (W - 1) + j} )
 *
 * where the rows before the first token are those of `state` (the last W - 1
 * rows that came before, oldest first), or zero.
 *
 *  x          : [B, T, C] io dtype, rows of x_row elements.
 *  weight     : [C, W] float32, W in {2, 3, 4}; the last tap is this token's.
 *  bias       : [C] float32 or NULL for zero.
 *  state      : [B, W - 1, C] io dtype, or NULL for zero rows.
 *  y          : [B, T, C] io dtype.
 *  state_out  : [B, W - 1, C] io dtype: the last W - 1 rows up to each
 *               sequence's end (rows of `state` among them where it has fewer
 *               tokens), to go on from; or NULL.  May not overlap `state`.
 */
typedef struct {
  int32_t B, T, C, W;
  int32_t io_dtype;     /* a falcon_dtype                     */
  int32_t activation;   /* FALCON_ACT_NONE or FALCON_ACT_SILU */
  int64_t x_row;        /* elements from one row of x to the next */
} falcon_conv_problem;

falcon_status falcon_conv_fwd(const falcon_conv_problem* p, const void* x, const float* weight,
                              const float* bias, const void* state, const int32_t* lengths,
                              void* y, void* state_out, hipStream_t stream);

/*
 * falcon_conv_step -- one token of every sequence.  p->T is ignored; x is
 * [B, C] with rows of x_row, y is [B, C], and `state` ([B, W - 1, C] io dtype)
 * moves on by this token IN PLACE.  is_first, [B] bytes or NULL: a nonzero
 * entry marks a sequence whose rows before this token count as zero,
 * whatever `state` holds.
 */
falcon_status falcon_conv_step(const falcon_conv_problem* p, const void* x, const float* weight,
                               const float* bias, void* state, const uint8_t* is_first, void* y,
                               hipStream_t stream);

/*
 * falcon_conv_bwd -- gradients of <dy, y> + <dstate_out, state_out>.
 *  dy         : [B, T, C] dy_dtype.
 *  dstate_out : [B, W - 1, C] float32, or NULL for zero.
 *  dx         : [B, T, C] float32.
 *  dweight    : [C, W] float32;  dbias : [C] float32, or NULL to skip.
 *  dstate     : [B, W - 1, C] float32, the gradient of `state`, or NULL to
 *               skip (it may be asked for where `state` is NULL, too).
 *  workspace  : at least falcon_conv_bwd_workspace_bytes(p) bytes, 16-byte
 *               aligned, overlapping nothing else.
 */
falcon_status falcon_conv_bwd(const falcon_conv_problem* p, const void* x, const float* weight,
                              const float* bias, const void* state, const int32_t* lengths,
                              const void* dy, int32_t dy_dtype, const float* dstate_out,
                              float* dx, float* dweight, float* dbias, float* dstate,
                              void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Device scratch of falcon_conv_bwd; (size_t)-1 for an invalid problem. */
size_t falcon_conv_bwd_workspace_bytes(const falcon_conv_problem* p);

/*
 * falcon_norm_fwd -- group norm with an activation.  Every token's C = G d
 * channels are G groups (the heads) of d, and each group is normed by itself:
 *
 *     xhat = (x - mu) / sqrt( mean((x - mu)^2) + eps ),   mu = mean(x) if center, else 0
 *     y    = scale f( weight xhat + bias )
 *
 * (a group of zeros needs eps > 0 to stay finite; with center, a group's sum has
 * to be a float32 number).  With center = 0 this is the
 * root-mean-square norm (the paper's QK-RMSNorm), with f = FALCON_ACT_ELU1 a positive feature map phi.
 *
 *  x          : rows [B, T, C] of x_row elements, or heads [B, G, T, d]
 *               (x_heads; contiguous, x_row is ignored), io dtype.
 *  weight     : [C] float32, or NULL for one;  bias : [C] float32, or NULL.
 *  y          : rows [B, T, C] or heads [B, G, T, d] (y_heads), contiguous.
 *  1 <= d <= 4096.
 */
typedef struct {
  int32_t B, T, G, d;
  int32_t io_dtype;
  int32_t activation;
  int32_t center;             /* 0 or 1 */
  int32_t x_heads, y_heads;   /* 0: rows, 1: heads */
  float eps;                  /* >= 0, finite */
  float scale;                /* finite */
  int64_t x_row;
} falcon_norm_problem;

falcon_status falcon_norm_fwd(const falcon_norm_problem* p, const void* x, const float* weight,
                              const float* bias, void* y, hipStream_t stream);

/*
 * falcon_norm_bwd -- gradients of <dy, y>.
 *  dy         : dy_dtype, in y's layout;  dx : float32, contiguous, in x's.
 *  dweight, dbias : [C] float32, or NULL to skip either (they may be asked for
 *               where weight or bias is NULL, too).
 *  workspace  : at least falcon_norm_bwd_workspace_bytes(p) bytes.
 */
falcon_status falcon_norm_bwd(const falcon_norm_problem* p, const void* x, const float* weight,
                              const float* bias, const void* dy, int32_t dy_dtype, float* dx,
                              float* dweight, float* dbias, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);

size_t falcon_norm_bwd_workspace_bytes(const falcon_norm_problem* p);

/*
 * falcon_scan_fwd -- the selective state space scan.  Channel c of D, in group
 * g = c / (D / G), has a state S of N numbers:
 *
 *     delta_t = softplus(dt_t + dt_bias), or dt_t + dt_bias
 *     S_t     = exp(delta_t A_c) * S_{t-1} + delta_t x_t B_{t,g}
 *     y_t     = ( <C_{t,g}, S_t> + D_c x_t ) silu(z_t)
 *
 * (products of vectors of N elementwise).  The read comes after the write.
 *
 *  x, dt, z   : [B, T, D] io dtype, rows of x_row, dt_row, z_row elements; z
 *               may be NULL (no gate).  Rows have at most 2^22 elements.
 *  A          : [D, N] float32, N in {8, 16, 32, 64}.
 *  Bm, Cm     : [B, T, G, N] io dtype, rows of b_row, c_row elements; G
 *               divides D.
 *  Dskip, dt_bias : [D] float32, or NULL for zero.
 *  S0         : [B, D, N] float32, or NULL for zero.
 *  y          : [B, T, D] io dtype.
 *  S_T        : [B, D, N] float32, the state at each sequence's end, or NULL;
 *               may alias S0 exactly.
 *  workspace  : at least falcon_scan_workspace_bytes(p) bytes (may be NULL
 *               when that is 0), 16-byte aligned, overlapping nothing else.
 * Arithmetic is float32 throughout.  The scan is meant for states that decay
 * (delta A <= 0); where they grow past float32 the results are not finite.  A
 * wait between waves that gives up (falcon_set_wait_limit) costs time only: one
 * wave then runs its channels' tokens by itself, to the same bits.
 */
typedef struct {
  int32_t B, T, D, N, G;
  int32_t io_dtype;
  int32_t softplus;           /* 0 or 1 */
  int64_t x_row, dt_row, z_row, b_row, c_row;
} falcon_scan_problem;

falcon_status falcon_scan_fwd(const falcon_scan_problem* p, const void* x, const void* dt,
                              const float* A, const void* Bm, const void* Cm, const float* Dskip,
                              const float* dt_bias, const void* z, const float* S0,
                              const int32_t* lengths, void* y, float* S_T, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);

size_t falcon_scan_workspace_bytes(const falcon_scan_problem* p);

/*
 * falcon_scan_step -- one token of every sequence: x, dt, z, y are [B, D], Bm
 * and Cm [B, G, N] (rows as above, p->T is ignored), S [B, D, N] float32 moves
 * on IN PLACE.  is_first, [B] bytes or NULL: a nonzero entry marks a sequence
 * whose state before this token counts as zero, whatever S holds.
 */
falcon_status falcon_scan_step(const falcon_scan_problem* p, const void* x, const void* dt,
                               const float* A, const void* Bm, const void* Cm, const float* Dskip,
                               const float* dt_bias, const void* z, float* S,
                               const uint8_t* is_first, void* y, hipStream_t stream);

/*
 * falcon_scan_bwd -- gradients of <dy, y> + <dS_T, S_T>; the forward is
 * recomputed.
 *  dy         : [B, T, D] dy_dtype;  dS_T : [B, D, N] float32 or NULL.
 *  dx, ddt    : [B, T, D] float32;  dz : the same, required where z is given,
 *               ignored where it is not.
 *  dA         : [D, N] float32;  dB, dC : [B, T, G, N] float32, summed over
 *               the channels of each group.
 *  dD, ddt_bias : [D] float32, or NULL to skip.
 *  dS0        : [B, D, N] float32, or NULL to skip.
 *  workspace  : at least falcon_scan_bwd_workspace_bytes(p) bytes.
 */
falcon_status falcon_scan_bwd(const falcon_scan_problem* p, const void* x, const void* dt,
                              const float* A, const void* Bm, const void* Cm, const float* Dskip,
                              const float* dt_bias, const void* z, const float* S0,
                              const int32_t* lengths, const void* dy, int32_t dy_dtype,
                              const float* dS_T, float* dx, float* ddt, float* dz, float* dA,
                              float* dB, float* dC, float* dD, float* ddt_bias, float* dS0,
                              void* workspace, size_t workspace_bytes, hipStream_t stream);

size_t falcon_scan_bwd_workspace_bytes(const falcon_scan_problem* p);

/*
 * falcon_linear_fwd -- linear attention with a decay for each head.  Head h of H
 * has a state S of dk x dv numbers and forgets at one rate:
 *
 *     S_t = exp(log_decay_h) S_{t-1} + k_t v_t^T
 *     o_t = scale S_t^T q_t
 *
 * The read comes after the write.  It is the recurrences' plain relative: no shift,
 * no step size, a decay that does not depend on the token.
 *
 *  q, k       : heads [B, H, T, dk] (qk_heads; contiguous, q_row and k_row are
 *               ignored) or rows [B, T, H dk] of q_row and k_row elements, io dtype.
 *  v          : heads [B, H, T, dv] (v_heads) or rows [B, T, H dv] of v_row.
 *               Rows are a multiple of 16 bytes apart (FALCON_ERR_ALIGN).
 *  log_decay  : [H] float32, at most 0; -infinity leaves each token to itself, 0
 *               forgets nothing.  Not checked.
 *  S0         : [B, H, dk, dv] float32, or NULL for zero.
 *  o          : heads [B, H, T, dv] (o_heads) or rows [B, T, H dv], io dtype.
 *  S_T        : [B, H, dk, dv] float32, the state at each sequence's end, or NULL;
 *               may alias S0 exactly.
 *  workspace  : at least falcon_linear_workspace_bytes(p) bytes (may be NULL when
 *               that is 0), 16-byte aligned, overlapping nothing else.
 * dk, dv in {16, 32, 64, 128}; at most 2^21 heads (B H) and 2^22 elements of a
 * row.  The prompt is worked on in
 * chunks of 64 tokens: float32 throughout with float32 inputs, and with bf16 inputs
 * by bf16 products with float32 sums in which every float32 operand is a sum of three
 * bf16 numbers, which hold all its bits, so results are those of float32 arithmetic,
 * rounded once.  A value that is not finite reaches what depends on it and nothing else:
 * the outputs of its own and of later tokens, the state at the end; gradients the other
 * way round (dlog_decay, a sum over all of a head's tokens, from any of them).
 */
typedef struct {
  int32_t B, H, T, dk, dv;
  int32_t io_dtype;
  int32_t qk_heads, v_heads, o_heads;   /* 0: rows, 1: heads */
  float scale;                          /* finite */
  int64_t q_row, k_row, v_row;
  int32_t zero_behind;                  /* zeros in the rows of o behind the ends  */
} falcon_linear_problem;

falcon_status falcon_linear_fwd(const falcon_linear_problem* p, const void* q, const void* k,
                                const void* v, const float* log_decay, const float* S0,
                                const int32_t* lengths, void* o, float* S_T, void* workspace,
                                size_t workspace_bytes, hipStream_t stream);

size_t falcon_linear_workspace_bytes(const falcon_linear_problem* p);

/*
 * falcon_linear_step -- one token of every sequence: q and k are [B, H dk] with rows of
 * q_row and k_row, v is [B, H dv] with rows of v_row, o [B, H dv]; p->T and the layouts
 * are ignored, S ([B, H, dk, dv] float32) moves on IN PLACE.  is_first, [B] bytes or
 * NULL: a nonzero entry marks a sequence whose state before this token counts as zero,
 * whatever S holds.  Arithmetic is float32.
 */
falcon_status falcon_linear_step(const falcon_linear_problem* p, const void* q, const void* k,
                                 const void* v, const float* log_decay, float* S,
                                 const uint8_t* is_first, void* o, hipStream_t stream);

/*
 * falcon_linear_bwd -- gradients of <dO, o> + <dS_T, S_T>; the states are recomputed.
 *  dO         : io dtype, in o's layout;  dS_T : [B, H, dk, dv] float32 or NULL.
 *  dq, dk, dv : float32, contiguous, in the layouts of q and k, and of v.
 *  dlog_decay : [H] float32, or NULL to skip.  A sum of terms each decayed as often as it
 *               counts, so a head's error is float32's of its own terms, however fast it
 *               forgets; 0 for -infinity.
 *  dS0        : [B, H, dk, dv] float32, or NULL to skip.
 *  workspace  : at least falcon_linear_bwd_workspace_bytes(p) bytes.
 */
falcon_status falcon_linear_bwd(const falcon_linear_problem* p, const void* q, const void* k,
                                const void* v, const float* log_decay, const float* S0,
                                const int32_t* lengths, const void* dO, const float* dS_T,
                                float* dq, float* dk, float* dv, float* dlog_decay, float* dS0,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

size_t falcon_linear_bwd_workspace_bytes(const falcon_linear_problem* p);

/*
 * falcon_residual_fwd -- from a block's output to the next block's input.  A token's
 * C = G d channels are G groups (the heads) of d:
 *
 *     z     = post_weight y / sqrt( mean over the group(y^2) + eps ),  or y without post_norm
 *     h_out = h + alpha f(gate) z                       (f(gate) = 1 without a gate)
 *     n     = pre_weight h_out / sqrt( mean over the row(h_out^2) + eps ),  with pre_norm
 *
 * in float32, each result rounded once (n is made from h_out before its rounding).
 * Without h and pre_norm it is the gated norm of the heads' outputs ahead of the output
 * projection; without post_norm and gate, the plain pre-norm residual.  A group of zeros
 * needs eps > 0 to stay finite.
 *
 *  y, gate    : [B, T, C] io dtype, rows of y_row and gate_row elements; gate may be NULL
 *               (gate_row is then ignored).
 *  h          : [B, T, C] stream dtype, or NULL for zero.
 *  post_weight, alpha, pre_weight : [C] float32, or NULL for one.
 *  h_out      : [B, T, C] stream dtype; may alias h exactly.
 *  n          : [B, T, C] io dtype; required with pre_norm, ignored without.
 *  saved      : NULL, or where to leave y and gate in 8 bits for falcon_residual_bwd:
 *               codes [B, T, C], steps [B, T, ceil(C / 32)].  Every 32 adjacent channels
 *               (fewer at a row's end) share a step 2^(byte - 127), the smallest power of
 *               two (from 2^-126 on) of which 127 reach their largest magnitude; a
 *               value is code times step, the multiple nearest to it (ties to even).
 *               Channels that are not all finite get byte 255 and come back as NaN.
 *               The gate's arrays are required where there is a gate, ignored else.
 * 1 <= C <= 8192.
 */
typedef struct {
  int32_t B, T, G, d;
  int32_t io_dtype;
  int32_t stream_dtype;       /* of h and h_out: a falcon_dtype                  */
  int32_t activation;         /* of the gate: FALCON_ACT_NONE, _SILU or _SIGMOID */
  int32_t post_norm, pre_norm;
  float eps;                  /* >= 0, finite */
  int64_t y_row, gate_row;
  int32_t zero_behind;        /* zeros in the forward's rows behind the ends    */
} falcon_residual_problem;

typedef struct {
  int8_t* y_codes;
  uint8_t* y_steps;
  int8_t* gate_codes;
  uint8_t* gate_steps;
} falcon_saved;

falcon_status falcon_residual_fwd(const falcon_residual_problem* p, const void* y, const void* gate,
                                  const void* h, const float* post_weight, const float* alpha,
                                  const float* pre_weight, const int32_t* lengths, void* h_out,
                                  void* n, const falcon_saved* saved, hipStream_t stream);

/*
 * falcon_residual_bwd -- gradients of <dh_out, h_out> + <dn, n>.
 *  y, gate    : the forward's; NULL where `saved` holds them in 8 bits instead (a gate
 *               where saved->gate_codes is not NULL).  y_row and gate_row are then ignored.
 *  h_out      : the forward's, required with pre_norm.
 *  dh_out     : [B, T, C] dh_out_dtype, or NULL for zero;  dn : [B, T, C] dn_dtype, required
 *               with pre_norm, ignored without.
 *  dy, dgate  : [B, T, C] float32; dgate is required where there is a gate, ignored else.
 *  dh         : [B, T, C] float32, or NULL to skip; may alias a float32 dh_out exactly.
 *  dalpha, dpost_weight, dpre_weight : [C] float32, or NULL to skip each (they may be asked
 *               for where alpha or the weights are NULL, too; dpost_weight without
 *               post_norm and dpre_weight without pre_norm are not written).
 *  workspace  : at least falcon_residual_bwd_workspace_bytes(p) bytes, 16-byte aligned.
 */
falcon_status falcon_residual_bwd(const falcon_residual_problem* p, const void* y, const void* gate,
                                  const falcon_saved* saved, const void* h_out,
                                  const float* post_weight, const float* alpha,
                                  const float* pre_weight, const int32_t* lengths,
                                  const void* dh_out, int32_t dh_out_dtype, const void* dn,
                                  int32_t dn_dtype, float* dy, float* dgate, float* dh,
                                  float* dalpha, float* dpost_weight, float* dpre_weight,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream);

size_t falcon_residual_bwd_workspace_bytes(const falcon_residual_problem* p);

#ifdef __cplusplus
}
#endif

#endif /* FALCON_H_ */
