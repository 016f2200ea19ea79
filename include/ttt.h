/*
 * ttt.h — C ABI of libttt_amd.so: forward scan of a test-time-training (TTT)
 * layer on an AMD Instinct MI355X (gfx950).
 *
 * What the library computes
 * -------------------------
 * A TTT layer carries, per (batch, head), a fast-weight state that is itself a
 * small model; reading the sequence trains that model one gradient step at a
 * time (PaperTrace "5 · TestingTime 训练与长上下文" §1.1 and §2.1: an initial
 * state W0, an update rule W_t = W_{t-1} - eta * grad l(W_{t-1}; x_t) and an
 * output rule y_t = f(q_t; W_t); keys, queries and values arrive already
 * projected).  The loss is the key-to-value reconstruction
 * l = 1/2 ||f(k_t) - v_t||^2 (same page §2.3).  Tokens are taken in chunks of
 * `chunk` tokens (same page §1.1, "b = 16"); every gradient in a chunk is taken
 * at the chunk-start state, token t reads with the chunk's updates up to and
 * including its own, and the state then advances by the eta-weighted sum of the
 * chunk's gradients.  eta_s scales the gradient of token s (the writer).
 *
 *   TTT-Linear  f_W(k) = W k,               W  : d x d            (§2.3)
 *   TTT-MLP     f(k) = W2 gelu(W1 k + b1) + b2, W1 : 4d x d, b1 : 4d,
 *               W2 : d x 4d, b2 : d; GELU in its exact erf form
 *               (diosapp "Test-Time Training (TTT) guide" §3: two layers,
 *               hidden width 4x, GELU)
 *
 * Inside a chunk the kernels use the dual form (diosapp guide §3; PaperTrace
 * §1.1): for TTT-Linear, with the chunk's keys/queries/values as columns,
 *   E = W K - V,   Z = W Q - E diag(eta) triu(K^T Q),   W <- W - E diag(eta) K^T.
 *
 * Conventions for every entry point
 * ---------------------------------
 *  - All tensor pointers are DEVICE pointers, row-major and contiguous.
 *    K, Q, V, Z, W0/W_out, W1/W2 and their outputs must be 16-byte aligned;
 *    eta and the bias vectors 4-byte aligned.
 *  - K, Q, V  : [B, H, T, d] in `io_dtype` (one row of d features per token).
 *    Z        : [B, H, T, d] in `io_dtype` (fp32 -> bf16 rounds to nearest even).
 *    eta      : [B, H, T] fp32 per-token learning rate, or NULL to use
 *               `eta_scalar` for every token.
 *    states   : always fp32; row index = output feature.
 *  - Any T >= 1; a last chunk shorter than `chunk` is processed with the
 *    tokens it has.
 *  - Ownership: the caller allocates every buffer, including the workspace.
 *    The library allocates no device memory, keeps no state between calls and
 *    may be called from several host threads at once.
 *  - Streams: all work is enqueued on `stream` (a hipStream_t; NULL = the
 *    default stream).  It is declared `void*` so that this header compiles
 *    without the HIP headers; the calling convention is that of the pointer
 *    hipStream_t is.  The call returns before the work completes; outputs are
 *    valid once the stream has been synchronised.  The library never
 *    synchronises.
 *  - `io_dtype` and `plan` take the ttt_dtype and ttt_plan values (passed as
 *    int, the enums' own calling convention).
 *  - Aliasing: the final-state outputs may alias the matching initial-state
 *    inputs (W_out == W0 updates in place).  Z must not overlap any input.
 *  - Errors: arguments are checked on the host before any HIP call; a failed
 *    check returns a negative ttt_status and enqueues nothing.  A kernel
 *    launch failure returns TTT_ERR_LAUNCH.  Non-finite values inside tensors
 *    are not checked: they propagate (IEEE) within their own (batch, head)
 *    slice only.
 */
#ifndef TTT_H
#define TTT_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TTT_OK = 0,
    TTT_ERR_INVALID_ARG = -1,   /* null/misaligned pointer, non-positive size, bad enum,
                                   non-finite eta_scalar with eta == NULL */
    TTT_ERR_UNSUPPORTED = -2,   /* valid arguments outside what the kernels implement */
    TTT_ERR_WORKSPACE = -3,     /* workspace missing or smaller than required */
    TTT_ERR_LAUNCH = -4         /* the HIP runtime rejected a kernel launch */
} ttt_status;

typedef enum {
    TTT_DTYPE_F32 = 0,          /* K, Q, V, Z in fp32 */
    TTT_DTYPE_BF16 = 1          /* K, Q, V, Z in bf16; arithmetic accumulates in fp32 */
} ttt_dtype;

/* Kernel plans.  AUTO picks the fastest plan that supports the shape; the others
 * force one (TTT_ERR_UNSUPPORTED if it cannot run the shape) so that tests can
 * compare plans on the same inputs. */
typedef enum {
    TTT_PLAN_AUTO = 0,
    TTT_PLAN_GENERIC = 1,       /* fp32 vector ALU, any chunk, fp32 or bf16 I/O */
    TTT_PLAN_MFMA = 2,          /* matrix cores, inclusive read.  bf16 I/O: bf16 matrix
                                   cores, d in {32, 64, 128}, chunk <= 16 or a multiple
                                   of 16.  fp32 I/O: fp32 matrix cores, d in {16, 32,
                                   64, 128}, any chunk (not for packed documents) */
    TTT_PLAN_BIGCHUNK = 3,      /* bf16 matrix cores, three stages, d in {64, 128}, chunk a
                                   multiple of 32 >= 128 */
    TTT_PLAN_SPLIT = 4          /* bf16 matrix cores, inclusive read, d = 64, chunk 16,
                                   T >= 2048, at most 64 (batch, head) slices (AUTO
                                   takes it up to 32 slices, and from 33 to 64 when
                                   T >= 4096): each sequence in S ~ 256 / slices + 1
                                   segments; segment 0 scans while segments 1 .. S-2
                                   form their affine maps, a combine gives every
                                   segment its start state, and segments 1 .. S-1
                                   scan again from it (workspace: 3 S d^2 fp32 per
                                   slice) */
} ttt_plan;

/* Read order of a chunk's tokens.  INCLUSIVE: token t reads with the chunk's
 * updates up to and including its own (the dual form above).  CHUNK_START:
 * every token of a chunk reads with the chunk-start state, z_t = W_c q_t (apply,
 * then update: the large-chunk ordering that leaves in-chunk dependencies to
 * window attention, PaperTrace "5 · TestingTime 训练与长上下文" §1.1, and the
 * read/write-order passage of its §2.4; with chunk == 1 the read-before-write
 * delta rule).  The state update is the same in both. */
typedef enum {
    TTT_READ_INCLUSIVE = 0,
    TTT_READ_CHUNK_START = 1
} ttt_read_mode;

/* Order of the axes of token tensors, where a call takes one. */
typedef enum {
    TTT_LAYOUT_BHTD = 0,        /* [B, H, T, d]; per-token scalars [B, H, T] */
    TTT_LAYOUT_BTHD = 1         /* [B, T, H, d]; per-token scalars [B, T, H] */
} ttt_layout;

/* Activations of ttt_groupnorm_fwd. */
typedef enum {
    TTT_ACT_NONE = 0,
    TTT_ACT_SILU = 1,           /* v / (1 + exp(-v)) */
    TTT_ACT_GELU = 2            /* the exact erf form */
} ttt_act;

/* ------------------------------------------------------------------------ */
/* TTT-Linear                                                                */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace ttt_linear_fwd needs for this shape: the largest size any
 * plan needs for either I/O dtype (0 when none does).  A workspace of this size
 * serves ttt_linear_fwd and ttt_linear_fwd_ex for the shape whatever their
 * dtype and plan. */
size_t ttt_linear_workspace_bytes(int B, int H, int T, int d, int chunk);

/* Bytes of workspace for this shape, dtype and plan exactly (0 when none, and
 * for shapes the plan cannot run). */
size_t ttt_linear_workspace_bytes_ex(int B, int H, int T, int d, int chunk,
                                     int io_dtype, int plan);

/* Plan that ttt_linear_fwd would run for this shape (never TTT_PLAN_AUTO), or a
 * negative ttt_status if no plan supports it. */
int ttt_linear_select_plan(int B, int H, int T, int d, int chunk, int io_dtype, int plan);

/* Forward scan of TTT-Linear (plan AUTO, inclusive read).
 *   W0    : [B, H, d, d] fp32 initial state.
 *   W_out : [B, H, d, d] fp32 state after the last token (may alias W0).
 *   d     : 16, 32, 64 or 128.   chunk : >= 1.
 *   workspace / workspace_bytes : device scratch of at least
 *           ttt_linear_workspace_bytes_ex(..., io_dtype, TTT_PLAN_AUTO) bytes
 *           (ttt_linear_workspace_bytes(...) always suffices), 256-byte aligned
 *           (may be NULL when that is 0).
 * The state update follows PaperTrace "5 · TestingTime 训练与长上下文" §1.1/§2.3;
 * with chunk == 1 it is the delta rule of the same page §2.1. */
int ttt_linear_fwd(const void* K, const void* Q, const void* V,
                   const float* eta, float eta_scalar,
                   const float* W0,
                   void* Z, float* W_out,
                   int B, int H, int T, int d, int chunk, int io_dtype,
                   void* workspace, size_t workspace_bytes,
                   void* stream);

/* TTT-Linear with a momentum state (the E2-TTT passage of "Test-Time Training
 * (TTT)", §2.3 and §5.1: fast weights and a momentum evolve per chunk from the
 * gradient at the chunk start).  With grad_c the eta-weighted sum of chunk c's
 * token gradients at its start state W_c:
 *   Mom_{c+1} = beta Mom_c + (1 - beta) grad_c,   W_{c+1} = W_c - Mom_{c+1},
 * and every token of a chunk reads with W_c (z_t = W_c q_t), as the passage
 * states the update per chunk only.  beta = 0 is ttt_linear_fwd_ex with
 * TTT_READ_CHUNK_START.
 *   Mom0     : [B, H, d, d] fp32 initial momentum, or NULL for zero.
 *   Mom_out  : [B, H, d, d] fp32 final momentum (may alias Mom0).
 *   beta     : 0 <= beta < 1.
 *   Plans: GENERIC (any chunk) and BIGCHUNK (as ttt_linear_fwd; its workspace);
 *   MFMA is TTT_ERR_UNSUPPORTED.  Other arguments as ttt_linear_fwd. */
int ttt_linear_fwd_momentum(const void* K, const void* Q, const void* V,
                            const float* eta, float eta_scalar, const float* W0,
                            const float* Mom0, float beta,
                            void* Z, float* W_out, float* Mom_out,
                            int B, int H, int T, int d, int chunk, int io_dtype,
                            void* workspace, size_t workspace_bytes, void* stream, int plan);

/* TTT-Linear with the inner bias as part of the state and, when ln_weight is
 * given, LayerNorm and a residual inside the inner model:
 *   f(x) = x + LN(W x + b),  LN(u) = ln_weight * (u - mean(u)) / sqrt(var(u) + eps)
 *                                    + ln_bias   (over the d features),
 * or f(x) = W x + b when ln_weight == ln_bias == NULL (diosapp "Test-Time
 * Training (TTT) guide" §3 gives f(x) = W x + b; the LN-and-residual ablation
 * is the one of PaperTrace "5 · TestingTime 训练与长上下文" §3.1).  W and b
 * take the chunked gradient step of ttt_linear_fwd (loss 1/2 ||f(k) - v||^2,
 * gradients at the chunk-start state, inclusive read); ln_weight and ln_bias
 * are fixed (outer-model parameters).
 *   b0, b_out            : [B, H, d] fp32 (b_out may alias b0; b0 may be zeros).
 *   ln_weight, ln_bias   : [H, d] fp32, shared by the batch, or both NULL.
 *   eps                  : > 0, finite.
 *   Others as ttt_linear_fwd; d : 16, 32, 64 or 128; any chunk; fp32 arithmetic
 *   on the fp32 matrix cores, one workgroup per (batch, head); no workspace. */
int ttt_linear_ln_fwd(const void* K, const void* Q, const void* V,
                      const float* eta, float eta_scalar, const float* W0, const float* b0,
                      const float* ln_weight, const float* ln_bias, float eps,
                      void* Z, float* W_out, float* b_out,
                      int B, int H, int T, int d, int chunk, int io_dtype, void* stream);

/* Packed documents with a reset at every document (variable-length batches).
 * Each document of every head is its own TTT-Linear scan from its own initial
 * state: no state, gradient or output crosses a document boundary, and chunks
 * are counted from the document's first token (PaperTrace "5 · TestingTime
 * 训练与长上下文" §2.4, the cross-sequence reset passage: each independent
 * document needs its own W0 and state).
 *   K, Q, V, Z  : [H, total_T, d] in io_dtype, head-major: document n of head h is
 *                 rows cu_seqlens[n] .. cu_seqlens[n+1]-1 of head h's block.
 *   eta         : [H, total_T] fp32 or NULL (eta_scalar).
 *   W0, W_out   : [n_docs, H, d, d] fp32 (W_out may alias W0).
 *   cu_seqlens  : DEVICE int32 [n_docs + 1], non-decreasing offsets into
 *                 [0, total_T] (read on the GPU; values outside are clamped, so a
 *                 malformed table gives wrong documents, never an out-of-range
 *                 access).  An empty document passes W0 through.  Rows that no
 *                 document covers are not written in Z.
 *   d : 16, 32, 64 or 128;  chunk >= 1;  plans: GENERIC, and MFMA for bf16 with
 *   chunk <= 16 (AUTO picks it); no workspace. */
int ttt_linear_fwd_varlen(const void* K, const void* Q, const void* V,
                          const float* eta, float eta_scalar, const float* W0,
                          void* Z, float* W_out, const int* cu_seqlens,
                          int n_docs, int H, int total_T, int d, int chunk, int io_dtype,
                          void* stream, int plan);

/* Plan that ttt_linear_fwd_varlen would run (never TTT_PLAN_AUTO), or a negative
 * ttt_status. */
int ttt_linear_select_plan_varlen(int n_docs, int H, int total_T, int d, int chunk,
                                  int io_dtype, int plan);

/* Bytes of workspace ttt_linear_bwd needs: the chunk-start states
 * (B*H*(ceil(T/chunk)+1)*d*d fp32) and one fp32 plane of dK, dQ and deta per
 * 16-row block of the state ((d/16)*B*H*T*(2d+1) fp32), each piece rounded up
 * to 256 bytes; the same for either I/O type.  0 for an unsupported shape. */
size_t ttt_linear_bwd_workspace_bytes(int B, int H, int T, int d, int chunk, int io_dtype);

/* Backward pass (vector-Jacobian product) of ttt_linear_fwd: for the scalar
 * L = <dZ, Z> + <dW_T, W_out> it writes the gradients with respect to K, Q, V,
 * each token's eta and W0.  The forward scan is recomputed from W0 (nothing is
 * kept from a ttt_linear_fwd call).  Same chunking and semantics as
 * ttt_linear_fwd (PaperTrace "5 · TestingTime 训练与长上下文" §1.1, §2.1, §2.3).
 *   K, Q, V, dZ    : [B, H, T, d] in io_dtype (dZ: the cotangent of Z).
 *   eta            : [B, H, T] fp32 or NULL (eta_scalar for every token).
 *   W0             : [B, H, d, d] fp32.
 *   dW_T           : [B, H, d, d] fp32 cotangent of W_out, or NULL for zero.
 *   dK, dQ, dV     : [B, H, T, d] in io_dtype (outputs).
 *   deta           : [B, H, T] fp32, the gradient for each token's eta (also
 *                    when eta is NULL: the gradient of eta_scalar is then the
 *                    sum of deta), or NULL to skip it.
 *   dW0            : [B, H, d, d] fp32 (output).
 *   d : 16, 32, 64 or 128;  chunk >= 1.
 *   workspace      : at least ttt_linear_bwd_workspace_bytes(...) bytes,
 *                    256-byte aligned.
 * Arithmetic is fp32 (inputs in bf16 are widened exactly).  dK, dQ and deta
 * are sums over the state's 16-row blocks, each block's terms kept in its own
 * fp32 plane of the workspace and the planes added in a fixed order: every
 * output is the same bits on every call.  Outputs must not overlap inputs or
 * each other. */
int ttt_linear_bwd(const void* K, const void* Q, const void* V,
                   const float* eta, float eta_scalar, const float* W0,
                   const void* dZ, const float* dW_T,
                   void* dK, void* dQ, void* dV, float* deta, float* dW0,
                   int B, int H, int T, int d, int chunk, int io_dtype,
                   void* workspace, size_t workspace_bytes, void* stream);

/* Streaming continuation of the TTT-Linear scan: n more tokens of every
 * (batch, head) sequence, from a carried state, with the same chunking as
 * ttt_linear_fwd over the whole sequence (token i of the sequence belongs to
 * chunk floor(i / chunk)).  Inside a chunk every gradient is taken at the
 * chunk-start state and a token reads with the chunk's updates up to and
 * including its own (PaperTrace "5 · TestingTime 训练与长上下文" §1.1, §2.1,
 * §2.3), so the carried state is a pair:
 *   W_chunk : [B, H, d, d] fp32, the state at the start of the current chunk;
 *   G       : [B, H, d, d] fp32, the sum over the chunk's tokens so far of
 *             eta_s (W_chunk k_s - v_s) k_s^T;
 *   pos     : how many tokens of the current chunk came before this call,
 *             0 <= pos < chunk (the caller tracks it: after the call it is
 *             (pos + n) % chunk).
 * The state after the last token read so far is W_chunk - G.  Both are updated
 * in place; when a chunk completes W_chunk becomes W_chunk - G and G is zeroed.
 * A stream starts from W_chunk = W0, G = 0, pos = 0; ttt_linear_fwd over a
 * prefix whose length is a multiple of chunk hands over W_out with G = 0.
 *   K, Q, V : [B, H, n, d] in io_dtype;  eta : [B, H, n] fp32 or NULL;
 *   Z       : [B, H, n, d] in io_dtype;  d : 16, 32, 64 or 128;  n >= 1.
 * W_chunk and G must not overlap each other or any other argument.  Arithmetic
 * is fp32 on the vector ALUs; no workspace. */
int ttt_linear_step(const void* K, const void* Q, const void* V,
                    const float* eta, float eta_scalar,
                    float* W_chunk, float* G, int pos,
                    void* Z, int B, int H, int n, int d, int chunk, int io_dtype,
                    void* stream);

/* ttt_linear_fwd with a kernel plan (ttt_plan) and a choice of read order
 * (ttt_read_mode); ttt_linear_fwd is this call with TTT_PLAN_AUTO and
 * TTT_READ_INCLUSIVE.  CHUNK_START runs on the GENERIC and BIGCHUNK plans (MFMA:
 * TTT_ERR_UNSUPPORTED); an unknown read_mode is TTT_ERR_INVALID_ARG.  Workspace
 * sizes are those of ttt_linear_workspace_bytes_ex for the plan that runs. */
int ttt_linear_fwd_ex(const void* K, const void* Q, const void* V,
                      const float* eta, float eta_scalar,
                      const float* W0,
                      void* Z, float* W_out,
                      int B, int H, int T, int d, int chunk, int io_dtype,
                      void* workspace, size_t workspace_bytes,
                      void* stream, int plan, int read_mode);

/* ttt_linear_fwd for callers that cannot allocate device memory: code being
 * captured into a HIP graph, tight serving loops, harnesses that forbid
 * hipMalloc.  Same arguments as ttt_linear_fwd without the workspace: the plans
 * that need one (TTT_PLAN_BIGCHUNK for chunks of 128+ tokens, TTT_PLAN_SPLIT for
 * a few long chunk-16 heads, at most 12 MiB) run in a static device array of the
 * library, TTT_NOALLOC_SCRATCH_BYTES (64 MiB) per GPU.  The array is part of the
 * library's code object: each GPU holds it from the library's first use there
 * until the process ends.  The call allocates nothing and frees nothing.
 *   - Shapes whose workspace (ttt_linear_workspace_bytes_ex for the AUTO plan)
 *     exceeds 64 MiB return TTT_ERR_WORKSPACE before any HIP call (for example
 *     16 heads x 131072 tokens at d = 128, chunk 2048, which needs 160 MiB: use
 *     ttt_linear_fwd with a caller workspace there).
 *   - The scratch of the caller's current device is used; `stream` must belong
 *     to that device.
 *   - Every call on one GPU shares that GPU's array: calls that overlap in time
 *     on one GPU (other streams, other host threads) race and give wrong
 *     results.  Calls serialised on one stream are safe; each call writes every
 *     scratch byte it reads, so nothing depends on what an earlier call left.
 *   - A failure to find the array's device address returns TTT_ERR_LAUNCH. */
#define TTT_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
int ttt_linear_fwd_noalloc(const void* K, const void* Q, const void* V,
                           const float* eta, float eta_scalar,
                           const float* W0,
                           void* Z, float* W_out,
                           int B, int H, int T, int d, int chunk, int io_dtype,
                           void* stream);

/* Size in bytes of ttt_linear_fwd_noalloc's per-GPU scratch array. */
size_t ttt_linear_noalloc_scratch_bytes(void);

/* Plan that ttt_linear_fwd_ex would run for this shape and read order. */
int ttt_linear_select_plan_ex(int B, int H, int T, int d, int chunk, int io_dtype, int plan,
                              int read_mode);

/* ------------------------------------------------------------------------ */
/* TTT-MLP (hidden width 4d)                                                 */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace ttt_mlp_fwd needs for this shape: the largest size any plan
 * needs for either I/O dtype (0 when none does). */
size_t ttt_mlp_workspace_bytes(int B, int H, int T, int d, int chunk);

/* Bytes of workspace for this shape, dtype and plan exactly. */
size_t ttt_mlp_workspace_bytes_ex(int B, int H, int T, int d, int chunk, int io_dtype, int plan);

int ttt_mlp_select_plan(int B, int H, int T, int d, int chunk, int io_dtype, int plan);

/* Forward scan of TTT-MLP, f(k) = W2 gelu(W1 k + b1) + b2 (plan AUTO).
 *   W1_0 : [B, H, 4d, d]   b1_0 : [B, H, 4d] or NULL (model without b1)
 *   W2_0 : [B, H, d, 4d]   b2_0 : [B, H, d]  or NULL (model without b2)
 *   W1_out, W2_out : final states (may alias W1_0, W2_0);
 *   b1_out / b2_out: final biases, NULL exactly when b1_0 / b2_0 is NULL.
 *   d : 16, 32 or 64 (hidden 4d).  chunk : >= 1.
 *   workspace : at least ttt_mlp_workspace_bytes(...) bytes, 256-byte aligned.
 * A present bias is part of the state and takes the same gradient step; an
 * absent one is a model without that bias.
 * Operand range of the matrix-core plan (bf16 I/O, d = 64, chunk <= 16, which
 * AUTO picks): its products take fp16 operands with fp32 accumulation.  The fp16
 * operands are K, Q, the states W1 and W2, the activations gelu(W1 k + b1), the
 * prediction error E = f(k) - v, the eta-scaled gradients eta E and
 * eta (W2^T E) * gelu', and the token scores k_s . q_t.  Each of them must stay
 * below 65504 in magnitude: past it the operand overflows and the outputs turn
 * non-finite.  Values of at least 2^-14 keep their bf16 value exactly; smaller
 * ones are rounded to fp16's subnormal spacing of 2^-24 (so a tiny eta with a
 * tiny error loses precision).  For data outside that range, call ttt_mlp_fwd_ex
 * with TTT_PLAN_GENERIC (fp32 vector ALU, any magnitude). */
int ttt_mlp_fwd(const void* K, const void* Q, const void* V,
                const float* eta, float eta_scalar,
                const float* W1_0, const float* b1_0,
                const float* W2_0, const float* b2_0,
                void* Z, float* W1_out, float* b1_out, float* W2_out, float* b2_out,
                int B, int H, int T, int d, int chunk, int io_dtype,
                void* workspace, size_t workspace_bytes,
                void* stream);

/* ttt_mlp_fwd with a kernel plan (ttt_plan); the workspace is
 * ttt_mlp_workspace_bytes_ex for the plan that runs. */
int ttt_mlp_fwd_ex(const void* K, const void* Q, const void* V,
                   const float* eta, float eta_scalar,
                   const float* W1_0, const float* b1_0,
                   const float* W2_0, const float* b2_0,
                   void* Z, float* W1_out, float* b1_out, float* W2_out, float* b2_out,
                   int B, int H, int T, int d, int chunk, int io_dtype,
                   void* workspace, size_t workspace_bytes,
                   void* stream, int plan);

/* ------------------------------------------------------------------------ */
/* Gated linear recurrence                                                   */
/* ------------------------------------------------------------------------ */

/* The recurrence of a gated sequence layer, one scalar state per channel:
 *   h_t = exp(g_t) h_{t-1} + x_t,   z_t = h_t,   t = 0 .. T-1,
 * over [B, H, T, d] like the scan above, every (batch, head, feature) a channel of
 * its own.  g_t is the logarithm of the gate: it carries gates close to 1 in bf16,
 * where the gate itself could not.
 *   - g_t <= 0 is required.  Values above 0 are not checked; the results are then
 *     unspecified (no access depends on them).
 *   - g_t = -inf, or any g_t <= -1e30 (a type's lowest value as a mask), forgets:
 *     h_t = x_t whatever h_{t-1} is, infinite and NaN included.  Documents packed in
 *     one row start anew that way.
 *   - Under any other gate an infinite state stays infinite, however small exp(g_t) is.
 *     Of a finite state, what factors (of one gate, or of several in a row) below 2^-126
 *     would leave is taken as 0.
 *   - g_t = 0 with x_t = 0 carries the state through (padding of a shorter sequence:
 *     h_out is then the state at its own end).
 * Arithmetic is fp32 whatever the I/O type; every output is the same bits on every
 * call.
 *   X, G    : [B, H, T, d] in io_dtype.
 *   h0      : [B, H, d] fp32 state before the first token, or NULL for zero.
 *   Z       : [B, H, T, d] in io_dtype (output; must not overlap an input).
 *   h_out   : [B, H, d] fp32 state after the last token (may alias h0), or NULL.
 *   1 <= d <= 2^26, 1 <= T <= 2^30, T d <= 2^34; all pointers 16-byte aligned.
 *   workspace : at least ttt_gated_workspace_bytes(...) bytes, 256-byte aligned (NULL
 *           where that is 0).  Calls that may overlap in time need one each, graph
 *           replays included; its contents need not be kept between calls. */
int ttt_gated_fwd(const void* X, const void* G, const float* h0, void* Z, float* h_out,
                  int B, int H, int T, int d, int io_dtype,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace ttt_gated_fwd and ttt_gated_bwd need for this shape (0 for few
 * tokens, and for shapes they refuse). */
size_t ttt_gated_workspace_bytes(int B, int H, int T, int d, int io_dtype);

/* Streaming continuation (decode): n more tokens of every sequence, the state updated
 * in place.  The same as ttt_gated_fwd from h0 = h to h_out = h; no workspace, so n is
 * meant to be small (any n >= 1 is right).
 *   X, G, Z : [B, H, n, d] in io_dtype;  h : [B, H, d] fp32. */
int ttt_gated_step(const void* X, const void* G, float* h, void* Z,
                   int B, int H, int n, int d, int io_dtype, void* stream);

/* Backward pass (vector-Jacobian product) of ttt_gated_fwd: the gradients of
 * L = <dZ, Z> + <dh_T, h_out>.  With lambda_T = dh_T,
 *   lambda_t = dz_t + exp(g_{t+1}) lambda_{t+1}   (g_T taken as 0),
 *   dx_t = lambda_t,   dg_t = exp(g_t) lambda_t h_{t-1},   dh0 = exp(g_0) lambda_0,
 * where a gate that forgets gives dg_t = 0 and passes nothing back.
 *   G       : as given to ttt_gated_fwd.
 *   Z       : what ttt_gated_fwd returned (h_{t-1} is read from it, in io_dtype).
 *   h0      : as given to ttt_gated_fwd (NULL for zero).
 *   dZ      : [B, H, T, d] in io_dtype;  dh_T : [B, H, d] fp32 or NULL for zero.
 *   dX, dG  : [B, H, T, d] in io_dtype (outputs).
 *   dh0     : [B, H, d] fp32 (output), or NULL.
 * Outputs must not overlap inputs or each other.  Workspace as ttt_gated_fwd. */
int ttt_gated_bwd(const void* G, const void* Z, const float* h0, const void* dZ,
                  const float* dh_T, void* dX, void* dG, float* dh0,
                  int B, int H, int T, int d, int io_dtype,
                  void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Root-mean-square norm with the residual's addition                        */
/* ------------------------------------------------------------------------ */

/* Over each of `rows` rows of D features:
 *   r = x + residual,   y = r / sqrt(mean(r^2) + eps) * weight.
 * The sum, the mean and y are formed in fp32 from the unrounded r (sums of squares past
 * fp32's range give the k = 0 of an infinite mean).
 *   X        : [rows, D] in io_dtype.
 *   residual : [rows, D] in io_dtype, or NULL (r = x).
 *   weight   : [D] fp32, or NULL for ones.
 *   Y        : [rows, D] in io_dtype (output; may alias X).
 *   R        : [rows, D] in io_dtype (output: r, the residual of what follows; may alias
 *              residual or X, but not Y), or NULL to leave it out.
 *   eps      : > 0, finite and no denormal number.  rows >= 0 (0 does nothing),
 *              1 <= D <= 2^26; X, residual, Y and R 16-byte aligned, weight 4-byte. */
int ttt_rmsnorm_fwd(const void* X, const void* residual, const float* weight, float eps,
                    void* Y, void* R, long long rows, int D, int io_dtype, void* stream);

/* The same with y in 8-bit floating point (OCP e4m3: largest value 448) and one scale
 * per row: scale = max|y| / 448, Y8 = y / (max|y| / 448) rounded to nearest even, as the
 * formula's value in fp64 is (a few 2^-52 off), whatever scale is rounded to.  A row of zeros
 * has scale 0 and Y8 0; a row whose r has a NaN or an infinity in it has a NaN scale, and
 * its Y8 is NaN throughout.
 *   Y8 : [rows, D] bytes (16-byte aligned);  scale : [rows] fp32. */
int ttt_rmsnorm_q8_fwd(const void* X, const void* residual, const float* weight, float eps,
                       void* Y8, float* scale, void* R, long long rows, int D, int io_dtype,
                       void* stream);

/* Backward pass of ttt_rmsnorm_fwd.  With k = 1 / sqrt(mean(r^2) + eps), n = k r and
 * u = dy * weight:
 *   dx = k (u - n mean(u n)) + dr,   dweight = sum over the rows of dy n.
 * dx is the gradient for x and for the residual alike.
 *   R        : [rows, D] in io_dtype, r as the forward pass stored it (X where there was
 *              no residual).
 *   dY       : [rows, D] in io_dtype.
 *   dR       : [rows, D] in io_dtype, the gradient that reaches r by itself, or NULL.
 *   dX       : [rows, D] in io_dtype (output; may alias dY or dR).
 *   dweight  : [D] fp32 (output), or NULL.
 *   workspace: at least ttt_rmsnorm_bwd_workspace_bytes(...) bytes, 256-byte aligned
 *              (may be NULL when dweight is NULL).
 * The rows' terms of dweight are added in a fixed order: the same bits on every call. */
int ttt_rmsnorm_bwd(const void* R, const float* weight, const void* dY, const void* dR,
                    float eps, void* dX, float* dweight, long long rows, int D, int io_dtype,
                    void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace ttt_rmsnorm_bwd needs for this shape (0 for shapes it refuses). */
size_t ttt_rmsnorm_bwd_workspace_bytes(long long rows, int D, int io_dtype);

/* ------------------------------------------------------------------------ */
/* Gradient norm over many tensors, and clipping                             */
/* ------------------------------------------------------------------------ */

/* norm = sqrt(sum of the squares of every element of every tensor), in fp64, and
 *   outs[i] = grads[i] * min(1, max_norm / (norm + eps)).
 * A norm that is not finite scales as the formula says (NaN: everything NaN; inf: finite
 * elements 0): the caller looks at *norm.
 *   n        : number of tensors, >= 0.  The four arrays are HOST arrays of n entries,
 *              read before the call returns.
 *   grads    : device pointers, contiguous, aligned to their element.
 *   outs     : device pointers; outs[i] may be grads[i] (in place), else it overlaps no
 *              tensor of the call; or NULL for the norm alone.  No two outputs overlap
 *              (TTT_ERR_INVALID_ARG), so a gradient that is listed twice is refused.
 *   sizes    : elements of each (0 allowed);  dtypes : ttt_dtype of each.
 *   max_norm : >= 0 (inf allowed);  eps : > 0, finite.
 *   norm     : DEVICE fp32 [1] (output; overlaps no tensor of the call).
 *   workspace: at least ttt_clip_workspace_bytes() bytes, 256-byte aligned; one for each
 *              call that may overlap in time.
 * Sums run in a fixed order: the same bits on every call. */
int ttt_clip_grad_norm(int n, const void* const* grads, void* const* outs,
                       const long long* sizes, const int* dtypes, float max_norm, float eps,
                       float* norm, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace ttt_clip_grad_norm needs, whatever the tensors. */
size_t ttt_clip_workspace_bytes(void);

/* ------------------------------------------------------------------------ */
/* Gated delta rule                                                          */
/* ------------------------------------------------------------------------ */

/* The fast-weight state of TTT-Linear with one gradient step per token, taken at the
 * state right before it, and a decay of the state:
 *   u_t = v_t - exp(g_t) W_{t-1} k_t,
 *   W_t = exp(g_t) W_{t-1} + eta_t u_t k_t^T,      z_t = W_t q_t.
 * With g = 0 it is ttt_linear_fwd with chunk = 1 (and any widths of keys and values).
 *   K, Q    : tokens of Hk heads of dk features, in io_dtype;  H must be a multiple of Hk:
 *             head h of values uses head h / (H / Hk) of keys and queries.
 *   V, Z    : tokens of H heads of dv features, in io_dtype (Z: output).
 *   layout  : a ttt_layout, for every token tensor of the call (eta and g too).
 *   eta     : fp32 step size of each token and head, or NULL to use eta_scalar (finite).
 *             A token with eta = 0 writes nothing.
 *   g       : fp32 logarithm of each token's decay, or NULL for none.  g_t <= 0 is meant;
 *             values above 0 grow the state and are not checked.  g_t = -inf, or any
 *             g_t <= -1e30, forgets a finite state entirely: documents packed in one row
 *             start anew that way.  eta_t = 0 with g_t = 0 carries the state through the
 *             padding of a shorter sequence (whose keys and values have to be finite).
 *   W0      : [B, H, dv, dk] fp32 state before the first token, or NULL for zero.
 *   W_out   : [B, H, dv, dk] fp32 state after the last token (may be W0), or NULL.
 *   1 <= dk <= 128, 1 <= dv <= 256 (TTT_ERR_UNSUPPORTED past that), 1 <= T <= 2^30; B H
 *   ceil(dv / 16) and (H / Hk) ceil(T / 64) below 2^24; token tensors and states 16-byte
 *   aligned, eta and g 4-byte.
 *   workspace : at least ttt_delta_workspace_bytes(...) bytes, 256-byte aligned; one for
 *             each call that may overlap in time, graph replays included.
 * Sums, states and products are fp32 (operands that are not exact in bf16 go to the matrix
 * cores in three bf16 parts), and a bf16 Z is rounded once from them.  Magnitudes below 1e-33
 * lose their last digits, and those above 3.38e38 turn NaN.  Non-finite values spread within
 * their (batch, head) and may turn NaN.  Every output is the same bits on every call. */
int ttt_delta_fwd(const void* K, const void* Q, const void* V, const float* eta, float eta_scalar,
                  const float* g, const float* W0, void* Z, float* W_out,
                  int B, int H, int Hk, int T, int dk, int dv, int layout, int io_dtype,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace ttt_delta_fwd needs (0 for shapes it refuses and for few tokens). */
size_t ttt_delta_workspace_bytes(int B, int H, int Hk, int T, int dk, int dv, int io_dtype);

/* Streaming continuation (decode): n more tokens of every sequence, the state W
 * [B, H, dv, dk] fp32 updated in place.  The same as ttt_delta_fwd from W0 = W to W_out = W,
 * token by token without a workspace, so n is meant to be small (any n >= 1 is right). */
int ttt_delta_step(const void* K, const void* Q, const void* V, const float* eta, float eta_scalar,
                   const float* g, float* W, void* Z,
                   int B, int H, int Hk, int n, int dk, int dv, int layout, int io_dtype,
                   void* stream);

/* Backward pass (vector-Jacobian product) of ttt_delta_fwd: the gradients of
 * L = <dZ, Z> + <dW_T, W_out>.  The forward scan is run again from W0 (nothing is kept from
 * a ttt_delta_fwd call).
 *   K, Q, V, eta, eta_scalar, g, W0, layout : as given to ttt_delta_fwd.
 *   dZ         : like Z;  dW_T : [B, H, dv, dk] fp32, or NULL for zero.
 *   dK, dQ     : like K (outputs; summed over the heads that share them, in fp32).
 *   dV         : like V (output).
 *   deta, dg   : like eta and g, fp32 (outputs, also where eta or g is NULL), or NULL to
 *                leave them out.  dg is 0 where g_t forgets.
 *   dW0        : [B, H, dv, dk] fp32 (output), or NULL.
 *   workspace  : at least ttt_delta_bwd_workspace_bytes(...) bytes, 256-byte aligned.
 * Outputs must not overlap inputs or each other.  Every output is the same bits on every
 * call. */
int ttt_delta_bwd(const void* K, const void* Q, const void* V, const float* eta, float eta_scalar,
                  const float* g, const float* W0, const void* dZ, const float* dW_T,
                  void* dK, void* dQ, void* dV, float* deta, float* dg, float* dW0,
                  int B, int H, int Hk, int T, int dk, int dv, int layout, int io_dtype,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace ttt_delta_bwd needs (0 for shapes it refuses). */
size_t ttt_delta_bwd_workspace_bytes(int B, int H, int Hk, int T, int dk, int dv, int io_dtype);

/* ------------------------------------------------------------------------ */
/* Group norm with an activation                                             */
/* ------------------------------------------------------------------------ */

/* Over channels-last tensors [N, S, C]: each row's S places and the C / G neighbouring
 * channels of a group are normed together,
 *   y = act((x - mean) / sqrt(var + eps) * weight + bias),   var = mean((x - mean)^2).
 * S = 1 is the norm of each of G heads' features of each of N tokens.
 *   X, Y         : [N, S, C] in io_dtype (Y: output; may be X).
 *   weight, bias : [C] fp32, or NULL for ones and zeros.
 *   mean, rstd   : [N, G] fp32 (outputs: the mean and 1 / sqrt(var + eps)).
 *   act          : a ttt_act.  eps : > 0 and finite (no denormal number).
 *   N, S >= 0 (0 does nothing), C a multiple of G, C <= 2^20, N G and N ceil(C / 256) below
 *   2^31; X and Y 16-byte aligned, the others 4-byte.
 *   workspace    : at least ttt_groupnorm_workspace_bytes(...) bytes, 256-byte aligned.
 * Arithmetic is fp32, sums in a fixed order: the same bits on every call. */
int ttt_groupnorm_fwd(const void* X, const float* weight, const float* bias, float eps, int act,
                      void* Y, float* mean, float* rstd, long long N, long long S, int C, int G,
                      int io_dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace ttt_groupnorm_fwd needs (0 for shapes it refuses and where a group is
 * small enough to be read once). */
size_t ttt_groupnorm_workspace_bytes(long long N, long long S, int C, int G, int io_dtype);

/* Backward pass of ttt_groupnorm_fwd.  With n = (x - mean) rstd, v = n weight + bias and
 * u = dy act'(v) weight,
 *   dx = rstd (u - mean(u) - n mean(u n)),  dweight = sum of dy act'(v) n,
 *   dbias = sum of dy act'(v).
 *   X, weight, bias, act : as given to ttt_groupnorm_fwd;  mean, rstd : as it returned them.
 *   dY      : [N, S, C] in io_dtype;  dX : [N, S, C] in io_dtype (output; may be dY or X).
 *   dweight, dbias : [C] fp32 (outputs; zeros where N or S is 0), or NULL.
 *   workspace : at least ttt_groupnorm_bwd_workspace_bytes(...) bytes, 256-byte aligned. */
int ttt_groupnorm_bwd(const void* X, const float* weight, const float* bias, int act,
                      const float* mean, const float* rstd, const void* dY, void* dX,
                      float* dweight, float* dbias, long long N, long long S, int C, int G,
                      int io_dtype, void* workspace, size_t workspace_bytes, void* stream);

size_t ttt_groupnorm_bwd_workspace_bytes(long long N, long long S, int C, int G, int io_dtype);

/* ------------------------------------------------------------------------ */
/* Dropout                                                                   */
/* ------------------------------------------------------------------------ */

/* y_i = keep_i x_i / (1 - p) + residual_i (no residual where NULL), where a dropped x_i
 * leaves 0 whatever it is.  keep_i holds where a 32-bit number is at least p 2^32 (to the
 * nearest): word i mod 4 of Philox 4x32 (10 rounds) of the key rng[0] and the counter
 * rng[1] + floor(i / 4), a 64-bit number in the counter's lower words.  The gradient for x is
 * the same call on dy without a residual, so no mask is kept; the next call's counter is this
 * one's plus ceil(n / 4).
 *   X, residual, Y : n elements in io_dtype, 16-byte aligned (Y: output; may be X or
 *                    residual).  n >= 0.
 *   p   : 0 <= p < 1.
 *   rng : DEVICE int64 [2], 8-byte aligned: seed and first counter, read by the kernel, so
 *         replays of a captured graph draw anew when it changes between them. */
int ttt_dropout(const void* X, const void* residual, void* Y, long long n, double p,
                const long long* rng, int io_dtype, void* stream);

/* Static string for a ttt_status value (or "unknown status"). */
const char* ttt_status_string(int status);

/* Static string naming a plan ("generic", "mfma", "bigchunk", ...). */
const char* ttt_plan_name(int plan);

#ifdef __cplusplus
}
#endif
#endif /* TTT_H */
