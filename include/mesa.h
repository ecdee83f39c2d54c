/*
 * mesa.h -- C ABI of the MI355X (gfx950) Mesa-layer library (libmesa.so).
 *
 * The operation is the Mesa layer of the MesaNet summary page
 * (gist.science, paper 2506.05233), section "A Camada Mesa":
 *   - displayed objective: Phi_t = argmin 1/2 sum_{t'<=t} zeta_{tt'}
 *     |v_t' - Phi k_t'|^2 + 1/2 Tr(Phi Lambda Phi^T), zeta_{tt'} the cumulative
 *     forget factors, Lambda symmetric positive definite;
 *   - output Delta_t = Phi_t q_t = G_t q*_t, q*_t = (H_t + Lambda)^{-1} q_t,
 *     solved by Conjugate Gradient;
 *   - bullet "Paralelizacao": CG over all time steps is a gated-linear-attention
 *     pass, run chunk-parallel with the states H_t, G_t (O(T) forward, O(1)
 *     per decoded token);
 *   - bullet "Computacao Dinamica": the CG iteration count needed to meet a
 *     stopping criterion varies per token.
 *
 * Concretely, per batch row b, head h and token t (readings of the page):
 *   H_t = gamma_t H_{t-1} + k_t k_t^T,  G_t = gamma_t G_{t-1} + v_t k_t^T,
 *   H_0 = G_0 = 0  (i.e. zeta_{tt'} = prod_{s=t'+1..t} gamma_s);
 *   Lambda = diag(lambda[h, :]);
 *   x = CG on (H_t + Lambda) x = q_t from x0 = 0, at most max_iters updates;
 *       when tol > 0 a token stops before an update once
 *       |r|_2 / |q_t|_2 < tol (r the recursively updated residual);
 *       tol == 0 makes exactly max_iters updates; r^T r == 0 or p^T A p <= 0
 *       also stop; q_t == 0 gives x = 0 and 0 iterations;
 *   out_t = G_t x,  iters_t = number of CG updates made.
 *
 * Conventions for every entry point:
 *   - Tensor pointers are DEVICE pointers (hipMalloc / torch CUDA memory),
 *     contiguous row-major, 16-byte aligned.  The caller owns every buffer;
 *     the library allocates nothing and keeps no state between calls, except
 *     the optional profiling records below.
 *   - Work is enqueued asynchronously on `stream` (a hipStream_t; NULL = the
 *     default stream).  Results are valid once the caller synchronises.
 *   - All arguments are validated on the host before anything is enqueued;
 *     on error nothing is enqueued.  Device data preconditions (0 < gamma <= 1,
 *     lambda > 0, finite inputs) are documented, not checked.
 *   - Outputs must not alias inputs.  Nothing aborts; no C++ exception
 *     crosses the ABI.  Errors return a mesa_status; the thread-local text
 *     from mesa_last_error_message() says which argument was wrong.
 *   - Supported sizes: d_k == d_v in {16, 32, 64, 128}; chunk in {16, 32, 64};
 *     any T >= 0 (a ragged last chunk is handled); 0 <= max_iters <= 4096.
 */
#ifndef MESA_H
#define MESA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MESA_ABI_VERSION 1

typedef enum {
    MESA_OK = 0,
    MESA_ERR_INVALID_ARGUMENT = 1,   /* null pointer, bad size, tol < 0 or NaN, misaligned */
    MESA_ERR_UNSUPPORTED = 2,        /* valid but not built: d, chunk or d_k != d_v      */
    MESA_ERR_WORKSPACE_TOO_SMALL = 3,
    MESA_ERR_HIP = 4                 /* a HIP runtime call failed (text in the message)  */
} mesa_status;

typedef enum {
    MESA_DTYPE_F32 = 0,              /* q, k, v stored as float32                        */
    MESA_DTYPE_BF16 = 1              /* q, k, v stored as bfloat16; vectors, states and
                                        sums in fp32.  The chunk states' products are exact
                                        (bf16 MFMAs on three-part bf16 splits).  The CG and
                                        output products (d >= 32, either dtype) run as fp16
                                        MFMAs on two-part splits: each operand group is
                                        scaled by a power of two and held as hi + lo to 22
                                        bits, and a product is hi.hi + hi.lo + lo.hi, within
                                        about 3 * 2^-22 of the float product                 */
} mesa_dtype;

/* Kernel ids for the optional profiling records. */
typedef enum {
    MESA_KERNEL_CHUNK_STATES = 0,    /* chunk-boundary states S^H_c, S^G_c (+ final)     */
    MESA_KERNEL_CG_OUTPUT = 1,       /* all CG iterations of a chunk + output contraction */
    MESA_KERNEL_DECODE = 2,          /* one recurrent decode step                        */
    MESA_KERNEL_QK_PREPROCESS = 3,   /* q/k convolution + normalisation                  */
    MESA_KERNEL_BWD_ADJOINT = 4,     /* backward: adjoint CG solve, per-token totals     */
    MESA_KERNEL_BWD_STATES = 5,      /* backward: reverse chunk states                   */
    MESA_KERNEL_BWD_KV = 6,          /* backward: key and value gradients                */
    MESA_KERNEL_BWD_GATE = 7,        /* backward: gate and regulariser gradients         */
    MESA_KERNEL_HAWK = 8,            /* Hawk layer recurrence (all its kernels)          */
                                     /* 9..15 are not used: 9 was the first id that was  */
                                     /* refused, and callers may count on it             */
    MESA_KERNEL_DELTA_PREP = 16,     /* delta rule: the chunks' state-free matrices      */
    MESA_KERNEL_DELTA_SCAN = 17,     /* delta rule: the pass over the chunks             */
    MESA_KERNEL_DELTA_STEP = 18,     /* delta rule: one token                            */
    MESA_KERNEL_DELTA_BWD_SCAN = 19, /* delta rule: the backward's passes over the chunks */
    MESA_KERNEL_DELTA_GRADS = 20,    /* delta rule: gradients per chunk, sums over heads */
    MESA_KERNEL_GATE_NORM = 21,      /* norm and gate of a layer's outputs               */
    MESA_KERNEL_GATE_NORM_BWD = 22,
    MESA_KERNEL_RESIDUAL_NORM = 23,  /* residual scale, addition and norm                */
    MESA_KERNEL_RESIDUAL_NORM_BWD = 24,
                                     /* 25..31 are not used, as 9..15                    */
    MESA_KERNEL_CAUSAL_CONV = 32,    /* causal convolution over rows                     */
    MESA_KERNEL_CAUSAL_CONV_BWD = 33,
    MESA_KERNEL_SSM_SCAN = 34,       /* state space scan: the passes over the chunks     */
    MESA_KERNEL_SSM_STATES = 35,     /* state space scan: the backward's chunk states    */
    MESA_KERNEL_SSM_GRADS = 36,      /* state space scan: gradients per chunk, their sums */
    MESA_KERNEL_SSM_STEP = 37,       /* state space scan: one token                      */
    MESA_KERNEL_QK_ROTATE = 38,      /* norm and rotation of queries and keys            */
    MESA_KERNEL_QK_ROTATE_BWD = 39,
    MESA_KERNEL_COUNT = 40
} mesa_kernel_id;

/* Library ABI version (MESA_ABI_VERSION of the build). */
int mesa_abi_version(void);

/* Static text for a status code; never NULL. */
const char *mesa_status_string(int status);

/* Thread-local detail about the last error returned on this thread ("" if none). */
const char *mesa_last_error_message(void);

/*
 * Bytes of device workspace mesa_forward needs for these sizes: the
 * chunk-boundary states S^H_c = H_{c*chunk-1} (symmetric; its upper triangle
 * of 16x16 blocks, dk (dk + 16) / 2 floats) and S^G_c (dv * dk floats), fp32,
 * per chunk and head, plus a 256-byte tail (the CG kernel's chunk-claim
 * counter).  Returns 0 if the sizes are invalid or T == 0.
 */
size_t mesa_forward_workspace_bytes(int B, int H, int T, int dk, int dv, int chunk);

/*
 * Mesa-layer forward over a whole sequence (the "Paralelizacao" bullet:
 * chunkwise-parallel CG; every CG matvec over all t is one gated-linear-
 * attention pass with query p and key = value = k).
 *
 *   q, k      [B, H, T, dk]   qkv_dtype
 *   v         [B, H, T, dv]   qkv_dtype
 *   gamma     [B, H, T]       float32, 0 < gamma <= 1 (gamma at the first
 *                             token has no effect: H_0 = 0)
 *   lambda    [H, dk]         float32, lambda > 0 (shared over the batch)
 *   chunk                     GPU chunk length; results do not depend on it
 *                             beyond rounding
 *   max_iters, tol            CG cap and residual tolerance (see top)
 *   out       [B, H, T, dv]   float32, written
 *   iters     [B, H, T]       int32 CG update counts, or NULL
 *   final_H   [B, H, dk, dk]  float32 H_T, or NULL   (prefill -> decode
 *   final_G   [B, H, dv, dk]  float32 G_T, or NULL    hand-off)
 *   workspace, workspace_bytes  at least mesa_forward_workspace_bytes(...);
 *                             may be NULL/0 when max_iters == 0
 *   stream                    hipStream_t or NULL
 */
mesa_status mesa_forward(const void *q, const void *k, const void *v, int qkv_dtype,
                         const float *gamma, const float *lambda,
                         int B, int H, int T, int dk, int dv, int chunk,
                         int max_iters, float tol,
                         float *out, int32_t *iters, float *final_H, float *final_G,
                         void *workspace, size_t workspace_bytes, void *stream);

/*
 * mesa_forward for training: the same computation (without final states),
 * and also the CG solutions the backward pass needs:
 *   x_out     [B, H, T, dk]   float32, x_t = the k-step CG solution of
 *                             (H_t + Lambda) x = q_t (0 when max_iters == 0)
 */
mesa_status mesa_forward_train(const void *q, const void *k, const void *v, int qkv_dtype,
                               const float *gamma, const float *lambda,
                               int B, int H, int T, int dk, int dv, int chunk,
                               int max_iters, float tol, float *out, int32_t *iters, float *x_out,
                               void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of the device array that mesa_forward_noalloc keeps its chunk
 * states in (64 MiB on every GPU the library runs on). */
#define MESA_NOALLOC_SCRATCH_BYTES (64u << 20)

/*
 * mesa_forward for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same computation and arguments without the workspace.  The chunk
 * states live in a device array of MESA_NOALLOC_SCRATCH_BYTES built into
 * the library; sizes whose mesa_forward_workspace_bytes(...) exceeds it
 * return MESA_ERR_WORKSPACE_TOO_SMALL before anything is enqueued.  The
 * call allocates nothing and records no profiling events.  Every call on a
 * GPU shares that GPU's array (the chunk-state kernel rewrites all of it
 * that a call reads, including the claim counter), so calls that overlap on
 * one GPU -- on different streams or host threads -- race; serialise them.
 */
mesa_status mesa_forward_noalloc(const void *q, const void *k, const void *v, int qkv_dtype,
                                 const float *gamma, const float *lambda,
                                 int B, int H, int T, int dk, int dv, int chunk,
                                 int max_iters, float tol,
                                 float *out, int32_t *iters, float *final_H, float *final_G,
                                 void *stream);

/*
 * Bytes of device workspace mesa_backward needs: the forward chunk states
 * (as mesa_forward_workspace_bytes counts them, without its tail), two
 * d x d reverse states per chunk and head (d^2 floats each, with d/16
 * exponents each), two floats per token, d floats per chunk, head and 16
 * tokens of the chunk, and a 256-byte tail (the adjoint kernel's chunk-claim
 * counter).  0 if invalid.
 */
size_t mesa_backward_workspace_bytes(int B, int H, int T, int dk, int dv, int chunk);

/*
 * Backward pass of the layer for a loss L with dL/d(out) = grad_out.  The
 * page says the layer trains in parallel but gives no gradient (section "A
 * Camada Mesa", bullet "Paralelizacao").  Reading: o_t = G_t A_t^{-1} q_t
 * (A_t = H_t + Lambda) is differentiated implicitly at the forward's CG
 * solution x_t, with the adjoint system solved by the same k-step CG:
 *   z_t = CG(A_t, G_t^T g_t)                        dL/dq_t = z_t
 *   dL/dv_i = sum_{t>=i} zeta_ti (x_t . k_i) g_t
 *   dL/dk_i = sum_{t>=i} zeta_ti [(g_t . v_i) x_t - (x_t . k_i) z_t - (z_t . k_i) x_t]
 *   dL/dlambda = -sum_{b,t} z_t (.) x_t
 *   dL/dgamma_s = (1/gamma_s) sum_{t>=s} (beta_t - a_t),
 *     beta_t = g_t . o_t - z_t . (H_t x_t),  a_i = (v_i . dL/dv_i + k_i . dL/dk_i) / 2
 * (g_t = grad_out_t).  The adjoint solve stops like the forward's, relative
 * to |G_t^T g_t|.
 *
 *   k         [B, H, T, dk]   qkv_dtype (q itself is not needed)
 *   v         [B, H, T, dv]   qkv_dtype
 *   gamma, lambda             as mesa_forward
 *   x         [B, H, T, dk]   float32, x_out of mesa_forward_train
 *   out       [B, H, T, dv]   float32, out of the same forward
 *   grad_out  [B, H, T, dv]   float32
 *   chunk, max_iters, tol     as mesa_forward (use the forward's values)
 *   grad_q, grad_k [B, H, T, dk], grad_v [B, H, T, dv], grad_gamma [B, H, T],
 *   grad_lambda [H, dk]       float32, written (grad_lambda sums the batch)
 *   z_iters   [B, H, T]       int32 update counts of the adjoint solve, or NULL
 *   workspace, workspace_bytes  at least mesa_backward_workspace_bytes(...)
 * Sizes and errors as mesa_forward.  Outputs must not alias inputs.
 */
mesa_status mesa_backward(const void *k, const void *v, int qkv_dtype,
                          const float *gamma, const float *lambda,
                          const float *x, const float *out, const float *grad_out,
                          int B, int H, int T, int dk, int dv, int chunk, int max_iters, float tol,
                          float *grad_q, float *grad_k, float *grad_v, float *grad_gamma,
                          float *grad_lambda, int32_t *z_iters,
                          void *workspace, size_t workspace_bytes, void *stream);

/*
 * One recurrent decode step for N x H independent heads (the "Paralelizacao"
 * bullet: O(1) per-token inference on the states H_t, G_t; "Computacao
 * Dinamica": per-head dynamic stopping).  For each (n, h):
 *   H <- gamma H + k k^T;  G <- gamma G + v k^T   (in place)
 *   x  = CG on (H + diag lambda[h]) x = q  (max_iters, tol as above)
 *   out = G x
 *
 *   q, k      [N, H, dk]      qkv_dtype
 *   v         [N, H, dv]      qkv_dtype
 *   gamma     [N, H]          float32
 *   lambda    [H, dk]         float32
 *   state_H   [N, H, dk, dk]  float32, read and overwritten
 *   state_G   [N, H, dv, dk]  float32, read and overwritten
 *   out       [N, H, dv]      float32, written
 *   iters     [N, H]          int32, or NULL
 */
mesa_status mesa_decode_step(const void *q, const void *k, const void *v, int qkv_dtype,
                             const float *gamma, const float *lambda,
                             float *state_H, float *state_G,
                             int N, int H, int dk, int dv, int max_iters, float tol,
                             float *out, int32_t *iters, void *stream);

/* Start points of the warm-started decode solve. */
typedef enum {
    MESA_WARM_COLD = 0,       /* x0 = 0: the solve of mesa_decode_step                 */
    MESA_WARM_PREVIOUS = 1,   /* x0 = x_prev                                           */
    MESA_WARM_PROJECTED = 2   /* x0 = c x_prev, c = x_prev.q / x_prev.(H+Lambda) x_prev
                                 (0 when that denominator is not positive)            */
} mesa_warm_mode;

/*
 * One decode step whose CG starts from each head's previous solution: the
 * warm start that the page names as future work for the solver's cost
 * (section "Significancia e Alegacoes").  Arguments as mesa_decode_step, plus
 *   state_x   [N, H, dk]      float32, read and overwritten: on entry the
 *                             previous step's solution x of each head (zeros
 *                             at the start of a sequence), on exit this step's
 *   warm_mode                 a mesa_warm_mode
 * From x0 the CG is the same method with r0 = q - (H + Lambda) x0; the stop
 * test still compares |r| with |q|, a zero q still gives x = 0 and 0
 * iterations, and iters counts the updates made after x0.  The projected
 * start is the multiple of x_prev closest to the solution in the energy
 * norm, so it is never further from it, in that norm, than the cold start.
 * out = G x as before.  state_x must not alias any other argument.
 */
mesa_status mesa_decode_step_warm(const void *q, const void *k, const void *v, int qkv_dtype,
                                  const float *gamma, const float *lambda,
                                  float *state_H, float *state_G, float *state_x,
                                  int N, int H, int dk, int dv, int max_iters, float tol,
                                  int warm_mode, float *out, int32_t *iters, void *stream);

/*
 * Query/key pre-processing before the layer (section "Arquitetura (MesaNet)",
 * bullet "Pre-processamento": keys and queries are normalised and convolved
 * with a small window before the Mesa layer).  Reading: per head h, token t
 * and feature f, a causal convolution of width W over the tokens followed by
 * L2 normalisation of each token's vector,
 *   c_t[f] = sum_{j<W} conv_w[h][j][f] x_{t-j}[f],   y_t = c_t / |c_t|_2
 * (y_t = 0 when c_t = 0), in one pass: one read of x, one write of y.  Call
 * it once for q and once for k (each with its own weights).
 *
 *   x         [B, H, T, d]    in_dtype (mesa_dtype)
 *   conv_w    [H, W, d]       float32; j = 0 weighs the current token
 *   width     W, 1 <= W <= 8 (this build: W <= 4, else MESA_ERR_UNSUPPORTED)
 *   hist      [B, H, W-1, d]  in_dtype, the W-1 input rows before t = 0
 *                             (oldest first), or NULL for zeros
 *   hist_out  [B, H, W-1, d]  in_dtype, or NULL: receives the last W-1 rows
 *                             of hist followed by x, the hist of the next
 *                             piece (prefill, then one token per decode step)
 *   y         [B, H, T, d]    out_dtype (mesa_dtype; bfloat16 rounds to
 *                             nearest even)
 * d in {16, 32, 64, 128}; T >= 0.  y must not alias x, and hist_out must not
 * alias hist or x.  Inputs must be finite.
 */
mesa_status mesa_qk_preprocess(const void *x, int in_dtype, const float *conv_w, int width,
                               const void *hist, void *hist_out, int B, int H, int T, int d,
                               void *y, int out_dtype, void *stream);

/*
 * Recurrence of the Hawk layer that the hybrid "Hawk-Mesa" model alternates
 * with Mesa layers (section "Arquitetura (MesaNet)", bullet "Variante
 * Hibrida": LRU (Hawk) layers).  The page names the layer only; this is
 * Hawk's published real-gated linear recurrent unit, per channel d:
 *   r_t = sigmoid(ga_t),  i_t = sigmoid(gx_t),  a_t = sigmoid(lam_d)^(c r_t)
 *   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t,   y_t = h_t
 * The gate pre-activations come from the layer's input projections, which are
 * plain matrix products outside this call.
 *
 *   x, ga, gx [B, T, D]       in_dtype (mesa_dtype)
 *   lam       [D]             float32
 *   c                         the gate's exponent scale (Hawk uses 8)
 *   h0        [B, D]          float32 state before t = 0, or NULL for zeros
 *   y         [B, T, D]       float32, written
 *   h_final   [B, D]          float32 state after the last token, or NULL
 *   workspace, workspace_bytes  at least mesa_hawk_workspace_bytes(B, T, D)
 * T >= 0; y must not alias the inputs.  Wide shapes (B * ceil(D / 64) >= 128)
 * run as one pass that reads each input once and leaves the workspace
 * untouched; narrower ones run a two-pass chunked scan that keeps per-chunk
 * summaries in the workspace.
 */
size_t mesa_hawk_workspace_bytes(int B, int T, int D);
mesa_status mesa_hawk_scan(const void *x, const void *ga, const void *gx, int in_dtype, const float *lam,
                           float c, const float *h0, int B, int T, int D, float *y, float *h_final,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * Gated delta rule over a whole sequence: the linear-attention layer that
 * takes, per token, one decayed gradient step on the objective the Mesa layer
 * solves to the end.  Per batch row and head, with the state S (a map from
 * keys to values, like the Mesa layer's G):
 *   S_t = gamma_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,
 *   out_t = S_t q_t,     S_0 = state0 (zeros when NULL)
 *
 *   q, k       [B, Hk, T, dk]   dtype (mesa_dtype)
 *   v          [B, H, T, dv]    dtype; H a multiple of Hk: value head h uses
 *                               key and query head h / (H / Hk)
 *   gamma,beta [B, H, T]        float32.  0 < gamma <= 1; gamma = 0 is taken
 *                               too and forgets the state (a sequence start in
 *                               a packed row).  beta is the write strength:
 *                               0 writes nothing, so a padded token is gamma =
 *                               1, beta = 0 and leaves the state as it is.
 *                               The rule is a contraction for beta |k|^2 <= 2;
 *                               beyond that states may grow without bound.
 *   state0     [B, H, dv, dk]   float32, or NULL
 *   out        [B, H, T, dv]    dtype, written (bfloat16 rounds to nearest even)
 *   final_state [B, H, dv, dk]  float32 S_T, or NULL; may be state0 itself
 *   workspace                   at least mesa_delta_workspace_bytes(...), which
 *                               never decreases with B, H or T: one for the
 *                               largest batch and longest sequence serves all
 * dk in {16, 32, 64, 128}, dv in {16, 32, 64, 128, 256}, T >= 0.  Sums, states
 * and decays are float32 (prefix sums of ln gamma float64); products run as
 * fp16 MFMAs on two-part splits (see mesa_dtype; of a bfloat16 output's decayed
 * scores the second part is a byte, which leaves them 2^-14).  A split shares
 * its scale among a chunk of 64 tokens and keeps 2^-39 of its largest element,
 * so that a value 2^-17 and more below the largest of its chunk and column (also
 * one of a token with beta = 0) is met with fewer bits.  The sizes of v, states
 * and gradients are otherwise free, from 2^-60 to 2^60.  Values are taken as finite:
 * a NaN or infinity reaches its chunk of 64 tokens and what follows in its head
 * (other heads and rows never), also from a token with beta = 0.
 *
 * Here and in the calls below, outputs and workspace share no memory with an
 * input or with one another but where it says "may be"; others are refused.
 */
size_t mesa_delta_workspace_bytes(int B, int H, int T, int dk, int dv, int dtype);
mesa_status mesa_delta_forward(const void *q, const void *k, const void *v, int dtype, const float *gamma,
                               const float *beta, const float *state0, int B, int Hk, int H, int T, int dk,
                               int dv, void *out, float *final_state, void *workspace,
                               size_t workspace_bytes, void *stream);

/*
 * Gradients of the gated delta rule, from the forward's inputs (the chunk
 * states are formed again), for L = <out, grad_out> + <final_state, grad_final>:
 *   grad_out   [B, H, T, dv]    dtype
 *   grad_final [B, H, dv, dk]   float32, or NULL for zeros
 *   grad_q, grad_k [B, Hk, T, dk], grad_v [B, H, T, dv]  dtype, written;
 *                               shared heads' gradients are summed in float32
 *   grad_gamma, grad_beta [B, H, T]  float32, written.  Where gamma is 0, a
 *                               sequence start and not a decay, grad_gamma is
 *                               written 0 (the derivative there need not be)
 *   grad_state [B, H, dv, dk]   float32 gradient of state0, or NULL; may be
 *                               grad_final itself
 *   workspace                   at least mesa_delta_backward_workspace_bytes(...)
 * Products of a gradient with a value or a state keep their bits down to 2^-110.
 * Sums are taken in a fixed order: results do not change from run to run.
 */
size_t mesa_delta_backward_workspace_bytes(int B, int Hk, int H, int T, int dk, int dv, int dtype);
mesa_status mesa_delta_backward(const void *q, const void *k, const void *v, int dtype, const float *gamma,
                                const float *beta, const float *state0, const void *grad_out,
                                const float *grad_final, int B, int Hk, int H, int T, int dk, int dv,
                                void *grad_q, void *grad_k, void *grad_v, float *grad_gamma, float *grad_beta,
                                float *grad_state, void *workspace, size_t workspace_bytes, void *stream);

/*
 * One token of the gated delta rule for N sequences, states updated in place:
 *   q, k [N, Hk, dk], v [N, H, dv] dtype; gamma, beta [N, H] float32;
 *   state [N, H, dv, dk] float32 in/out; out [N, H, dv] dtype.
 * Sizes and heads as mesa_delta_forward; its final_state is this state.
 */
mesa_status mesa_delta_step(const void *q, const void *k, const void *v, int dtype, const float *gamma,
                            const float *beta, float *state, int N, int Hk, int H, int dk, int dv, void *out,
                            void *stream);

/*
 * Norm and gate of a layer's outputs, per token and head:
 *   y = x / sqrt(mean(x^2) + eps) * w * silu(gate),   silu(g) = g / (1 + e^-g)
 *   x     [B, H, T, d]   x_dtype: a layer's output (mesa_forward, mesa_delta_forward)
 *   gate  [B, T, H, d]   dtype, or NULL for no gate: rows of an input projection
 *   w     [H, d]         float32
 *   y     [B, T, H, d]   dtype: rows of the output projection's input
 * d in {16, 32, 64, 128, 256}; eps > 0.  A row of zeros gives zeros.  Squares
 * are summed in float32: |x| up to about 1e18.
 *
 * Backward, for grad_y = dL/dy [B, T, H, d] dtype, from the forward's inputs:
 *   grad_x [B, H, T, d] x_dtype, grad_gate [B, T, H, d] dtype (NULL exactly
 *   when gate is), grad_w [H, d] float32; workspace at least
 *   mesa_gate_norm_backward_workspace_bytes(...).  Sums are taken in a fixed
 *   order: results do not change from run to run.
 */
mesa_status mesa_gate_norm(const void *x, int x_dtype, const void *gate, int dtype, const float *w, float eps,
                           int B, int H, int T, int d, void *y, void *stream);
size_t mesa_gate_norm_backward_workspace_bytes(int B, int H, int T, int d);
mesa_status mesa_gate_norm_backward(const void *x, int x_dtype, const void *gate, int dtype, const float *w,
                                    float eps, const void *grad_y, int B, int H, int T, int d, void *grad_x,
                                    void *grad_gate, float *grad_w, void *workspace, size_t workspace_bytes,
                                    void *stream);

/*
 * Residual scale, addition and the next block's norm, per row:
 *   h_out = h + scale * y,   n = h_out / sqrt(mean(h_out^2) + eps) * w
 *   h      [R, D]  h_dtype: the residual
 *   y      [R, D]  dtype: the block's output, or NULL (n = the norm of h;
 *                  h_out must then be NULL too)
 *   scale  [D]     float32, or NULL for 1
 *   w      [D]     float32
 *   h_out  [R, D]  h_dtype; may be h itself
 *   n      [R, D]  dtype; from h_out before its rounding
 * 1 <= D <= 16384 (rows of a multiple of 8 elements move in 16-byte pieces),
 * R >= 0, eps > 0; |h_out| up to about 1e18.
 *
 * Backward, for grad_n = dL/dn and grad_h_out = dL/d(h_out) through the rest
 * of the network (h_dtype, NULL for zeros), from the forward's inputs:
 *   grad_h [R, D] h_dtype, grad_y [R, D] dtype (NULL exactly when y is),
 *   grad_w [D] float32, grad_scale [D] float32 (NULL exactly when scale is);
 *   workspace at least mesa_residual_norm_backward_workspace_bytes(...).
 */
mesa_status mesa_residual_norm(const void *h, int h_dtype, const void *y, int dtype, const float *scale,
                               const float *w, float eps, int R, int D, void *h_out, void *n, void *stream);
size_t mesa_residual_norm_backward_workspace_bytes(int R, int D);
mesa_status mesa_residual_norm_backward(const void *h, int h_dtype, const void *y, int dtype, const float *scale,
                                        const float *w, float eps, const void *grad_n, const void *grad_h_out,
                                        int R, int D, void *grad_h, void *grad_y, float *grad_w,
                                        float *grad_scale, void *workspace, size_t workspace_bytes,
                                        void *stream);

/*
 * Strided tensors.  In the calls below some tensors may be views: slices of the
 * rows of a projection, of a convolution's output, of one buffer of gradients.
 * `*_strides` then holds their element strides {batch, head, token} (of a
 * [B, T, D] tensor {batch, token}), NULL says contiguous in the order given.
 * The last dimension is always contiguous; a view needs the alignment of an
 * element only.  Strides are not negative; an input's may be 0 (the same rows for
 * several), an output's rows may not share memory.  Outputs that lie between one
 * another in the same rows are told apart where they have a stride in common.
 * All other pointers, and contiguous tensors, are 16-byte aligned as everywhere.
 *
 * Lengths.  `lens` [B] int32, or NULL: the tokens that each row of a padded batch
 * has (taken as 0 below 0 and as T above T).  What is behind them is not read;
 * outputs and gradients there are written as zeros, and states and histories are
 * those after the row's own last token.
 */

/*
 * Short causal convolution over the rows of an input projection, with its
 * activation, as it stands before the state space scan.  Per channel,
 *   z_t = bias + sum_{j<W} w[j] x_{t-j},   y_t = silu(z_t), or z_t when silu is 0
 *
 *   x         [B, T, D]       dtype, x_strides
 *   w         [W, D]          float32; j = 0 weighs the current token
 *   width     W, 1 <= W <= 4
 *   bias      [D]             float32, or NULL
 *   hist      [B, W-1, D]     dtype, the W-1 rows before t = 0 (oldest first), or
 *                             NULL for zeros
 *   hist_out  [B, W-1, D]     dtype, or NULL: the last W-1 rows of hist followed by
 *                             x, the hist of the next piece (prefill, then one
 *                             token per decode step); may be hist itself
 *   y         [B, T, D]       dtype
 * Any D >= 1 and T >= 0.
 */
mesa_status mesa_causal_conv(const void *x, const int64_t *x_strides, int dtype, const float *w, int width,
                             const float *bias, int silu, const void *hist, void *hist_out, const int32_t *lens,
                             int B, int T, int D, void *y, void *stream);

/*
 * Gradients of mesa_causal_conv from its inputs and grad_y = dL/dy [B, T, D]:
 *   grad_x [B, T, D] dtype, grad_x_strides; grad_hist [B, W-1, D] dtype, or NULL;
 *   grad_w [W, D] float32; grad_bias [D] float32 (NULL exactly when bias is).
 * hist_out is not differentiated.  Sums are taken in a fixed order.
 */
size_t mesa_causal_conv_backward_workspace_bytes(int B, int T, int D, int width);
mesa_status mesa_causal_conv_backward(const void *x, const int64_t *x_strides, int dtype, const float *w, int width,
                                      const float *bias, int silu, const void *hist, const int32_t *lens,
                                      const void *grad_y, int B, int T, int D, void *grad_x,
                                      const int64_t *grad_x_strides, float *grad_w, float *grad_bias,
                                      void *grad_hist, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Selective state space scan over whole sequences: the gated linear layer whose
 * state decays by what each token says, one number a head, and takes the token's
 * outer product without looking at what it holds (the delta rule looks).  Per batch
 * row and head, with the state S (a map from keys to values, like the delta rule's),
 *   step_t = softplus(dt_t + dt_bias), or dt_t + dt_bias when softplus is 0
 *   S_t = exp(A step_t) S_{t-1} + step_t x_t b_t^T,   S_0 = state0 (zeros when NULL)
 *   out_t = S_t c_t + D x_t
 *
 *   x          [B, H, T, dv]    dtype, x_strides: the values
 *   b, c       [B, Hk, T, dk]   dtype, b_strides, c_strides: the key's and the
 *                               query's part; H a multiple of Hk, head h uses
 *                               b and c of h / (H / Hk)
 *   dt         [B, H, T]        dt_dtype, dt_strides; steps are >= 0.  A token of
 *                               step 0 (raw -infinity, or the storage type's
 *                               lowest value) leaves the state as it is
 *   A          [H]              float32, A <= 0
 *   D, dt_bias [H]              float32, or NULL
 *   state0     [B, H, dv, dk]   float32, or NULL
 *   out        [B, H, T, dv]    dtype, written (bfloat16 rounds to nearest even)
 *   final_state [B, H, dv, dk]  float32, or NULL; may be state0 itself
 *   workspace                   at least mesa_ssm_workspace_bytes(...) (0 where
 *                               none is needed), which never decreases with B, H
 *                               or T
 * dk and dv in {16, 32, 64, 128}, T >= 0, token strides of x, b and c below 2^23.
 * Sums and states are float32, prefix sums of the decays float64.  Rows stored as
 * bfloat16 enter the products exactly; what is formed in float32 enters as two
 * bfloat16 parts where only bfloat16 outputs follow (2^-18 of a term, below their
 * rounding unless terms cancel by more than about 2^9) and as three (2^-27) where the
 * state does.  Values are taken as finite: a NaN or infinity reaches its chunk of 64
 * tokens and what follows in its head, other heads never (of b and c: of the heads
 * that share them).
 */
size_t mesa_ssm_workspace_bytes(int B, int H, int T, int dk, int dv, int dtype);
mesa_status mesa_ssm_forward(const void *x, const int64_t *x_strides, const void *b, const int64_t *b_strides,
                             const void *c, const int64_t *c_strides, int dtype, const void *dt,
                             const int64_t *dt_strides, int dt_dtype, const float *A, const float *D,
                             const float *dt_bias, int softplus, const float *state0, const int32_t *lens, int B,
                             int Hk, int H, int T, int dk, int dv, void *out, float *final_state, void *workspace,
                             size_t workspace_bytes, void *stream);

/*
 * Gradients of the scan, from the forward's inputs (the chunk states are formed
 * again), for L = <out, grad_out> + <final_state, grad_final>:
 *   grad_out   [B, H, T, dv]    dtype
 *   grad_final [B, H, dv, dk]   float32, or NULL for zeros
 *   grad_x [B, H, T, dv], grad_b, grad_c [B, Hk, T, dk] dtype, with strides; shared
 *                               heads' gradients are summed in float32
 *   grad_dt    [B, H, T]        dt_dtype, strides: of the raw dt
 *   grad_A, grad_D, grad_dt_bias [H]  float32; grad_D and grad_dt_bias NULL exactly
 *                               when D and dt_bias are
 *   grad_state [B, H, dv, dk]   float32 gradient of state0, or NULL; may be
 *                               grad_final itself
 * Sums are taken in a fixed order: results do not change from run to run.
 */
size_t mesa_ssm_backward_workspace_bytes(int B, int Hk, int H, int T, int dk, int dv, int dtype);
mesa_status mesa_ssm_backward(const void *x, const int64_t *x_strides, const void *b, const int64_t *b_strides,
                              const void *c, const int64_t *c_strides, int dtype, const void *dt,
                              const int64_t *dt_strides, int dt_dtype, const float *A, const float *D,
                              const float *dt_bias, int softplus, const float *state0, const int32_t *lens,
                              const void *grad_out, const float *grad_final, int B, int Hk, int H, int T, int dk,
                              int dv, void *grad_x, const int64_t *grad_x_strides, void *grad_b,
                              const int64_t *grad_b_strides, void *grad_c, const int64_t *grad_c_strides,
                              void *grad_dt, const int64_t *grad_dt_strides, float *grad_A, float *grad_D,
                              float *grad_dt_bias, float *grad_state, void *workspace, size_t workspace_bytes,
                              void *stream);

/*
 * One token of the scan for N sequences, states updated in place: x [N, H, dv],
 * b, c [N, Hk, dk], dt [N, H] with strides {batch, head} (NULL for contiguous);
 * state [N, H, dv, dk] float32 in/out; out [N, H, dv] dtype.  The rest as
 * mesa_ssm_forward, whose final_state is this state.
 */
mesa_status mesa_ssm_step(const void *x, const int64_t *x_strides, const void *b, const int64_t *b_strides,
                          const void *c, const int64_t *c_strides, int dtype, const void *dt,
                          const int64_t *dt_strides, int dt_dtype, const float *A, const float *D,
                          const float *dt_bias, int softplus, float *state, int N, int Hk, int H, int dk, int dv,
                          void *out, void *stream);

/*
 * Angles per token of the rot / 2 pairs of features that mesa_qk_rotate turns, into
 * HOST memory: freqs[i] = base^(-2 i / rot), and *amplitude, the factor on the
 * rotated features (1 unless said).  For contexts longer than the one trained on,
 * stretched `factor` >= 1 times:
 *   MESA_ROTARY_PLAIN    as above (factor must be 1)
 *   MESA_ROTARY_LINEAR   all angles divided by factor
 *   MESA_ROTARY_BASE     base times factor^(rot / (rot - 2)): the fastest pair keeps
 *                        its angle, the slowest is divided by factor
 *   MESA_ROTARY_PARTS    pairs that turn more than `fast` times over `context` tokens
 *                        keep their angle, those that turn less than `slow` times
 *                        are divided by factor, in between the angles are mixed
 *                        linearly in the turns; amplitude 1 + 0.1 ln(factor)
 * `fast` > `slow` >= 0 and `context` > 0 are read by the last only.
 */
typedef enum {
    MESA_ROTARY_PLAIN = 0,
    MESA_ROTARY_LINEAR = 1,
    MESA_ROTARY_BASE = 2,
    MESA_ROTARY_PARTS = 3
} mesa_rotary_scaling;
mesa_status mesa_rotary_frequencies(int rot, double base, int scaling, double factor, double context, double fast,
                                    double slow, double *freqs, float *amplitude);

/*
 * Per-head RMS norm of queries and keys and the rotation by their positions, in one
 * pass; also of the state space scan's c and b.  Per token at position p and head:
 *   n = x / sqrt(mean(x^2) + eps) * w   (norm 1),   n = x   (norm 0)
 *   (y_a, y_b) = amplitude (n_a cos - n_b sin, n_b cos + n_a sin),  angle p freqs[i]
 * for the pairs i < rot / 2 of features (a, b) = (i, i + rot / 2), or (2 i, 2 i + 1)
 * when interleaved; features rot and up are n.
 *
 *   q, k      [B, Hq, T, d], [B, Hk, T, d]  dtype, with strides; k NULL with Hk = 0
 *   freqs     [rot / 2]       float64, on the device (mesa_rotary_frequencies)
 *   rot       a multiple of 16, 16 <= rot <= d
 *   positions [B, T] int64 (or [T], positions_stride 0), batch stride
 *             positions_stride; NULL: token t is at position0 + t.  Angles are
 *             formed as pairs of float64 values: float32's accuracy at
 *             positions up to 2^50 to either side (of frequencies up to 1);
 *             farther ones turn by some angle
 *   wq, wk    [d]             float32 weights of the norm, or NULL for 1
 *   yq, yk    [B, Hq, T, d], [B, Hk, T, d]  dtype
 * d in {16, 32, 64, 128, 256}; eps > 0.  A row of zeros gives zeros.  Squares are
 * summed in float32: |x| up to about 1e18.
 *
 * Backward, for grad_yq, grad_yk (contiguous), from the forward's inputs: grad_q,
 * grad_k dtype, with strides; grad_wq, grad_wk [d] float32 (NULL exactly when wq, wk
 * are).  q and k are not read without the norm, but must be given.  Sums are taken
 * in a fixed order.
 */
mesa_status mesa_qk_rotate(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                           int dtype, const double *freqs, int rot, int interleaved, float amplitude,
                           const int64_t *positions, int64_t positions_stride, int64_t position0, const float *wq,
                           const float *wk, int norm, float eps, int B, int Hq, int Hk, int T, int d, void *yq,
                           void *yk, void *stream);
size_t mesa_qk_rotate_backward_workspace_bytes(int d);
mesa_status mesa_qk_rotate_backward(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                                    int dtype, const double *freqs, int rot, int interleaved, float amplitude,
                                    const int64_t *positions, int64_t positions_stride, int64_t position0,
                                    const float *wq, const float *wk, int norm, float eps, const void *grad_yq,
                                    const void *grad_yk, int B, int Hq, int Hk, int T, int d, void *grad_q,
                                    const int64_t *grad_q_strides, void *grad_k, const int64_t *grad_k_strides,
                                    float *grad_wq, float *grad_wk, void *workspace, size_t workspace_bytes,
                                    void *stream);

/*
 * Optional per-kernel timing (not part of the method).  While enabled, each
 * kernel launch made by the library is bracketed by two hipEvents recorded on
 * its stream.  mesa_profile_read synchronises on the recorded events, returns
 * the summed milliseconds and launch count for one kernel id since the last
 * reset, and mesa_profile_reset drops all records.  Records are process-wide
 * and guarded by a mutex.
 */
mesa_status mesa_profile_enable(int on);
mesa_status mesa_profile_read(int kernel_id, double *total_ms, int64_t *launches);
mesa_status mesa_profile_reset(void);
const char *mesa_kernel_name(int kernel_id);

#ifdef __cplusplus
}
#endif

#endif /* MESA_H */
