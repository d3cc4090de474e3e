/*
 * cfc.h -- C ABI of the batched CfC K-loop library for one NVIDIA GB300 (sm_103a).
 *
 * The three operations of the method:
 *
 *   cfc_kloop_forward   the three-head closed-form continuous-time (CfC) cell
 *                       run over K steps for B independent samples;
 *   cfc_kloop_backward  backward through time: parameter gradients summed over
 *                       the batch, grad_h0 and (optionally) grad_x;
 *   reduce_axis0        deterministic, atomic-free column sum [B, N] -> [N];
 *
 * and around them:
 *
 *   reduce_axis0_multi  reduce_axis0 for a list of matrices in few launches;
 *   cfc_tau_kloop_*     the pages' single-head tau-cell K loop (FP32);
 *   cfc_grn_*           the multi-horizon GRN heads on every K position (FP32);
 *   cfc_kloop_forward_backward_static
 *                       forward + backward for callers that cannot allocate
 *                       device memory (fixed workspace inside the library);
 *   cfc_gdr_*           the gated delta rule, a matrix-state recurrence for long
 *                       sequences: forward, backward, and its form for the next
 *                       tokens of decoding sequences (FP32, bf16);
 *   cfc_rmsnorm_*       root-mean-square norm of a residual stream, forward
 *                       (optionally to 8 bits with scales) and backward;
 *   cfc_layernorm_*     layer norm of a residual stream, forward and backward;
 *   cfc_conv_*          the short causal convolution of each channel over its
 *                       sequence: forward, backward, next tokens;
 *   cfc_ssm_*           the selective state space scan, a recurrence with a state of
 *                       N values a channel: forward, backward, next tokens;
 *   cfc_grad_norm, cfc_grad_clip
 *                       the norm of many gradients together, and clipping to it;
 *   helpers             workspace sizes, status strings, the device error
 *                       word and its self-test, per-kernel event tracing.
 *
 * Cell (per sample, step k = 0..K-1, heads c = f, g, h~ in that order):
 *   A_c    = b[c] + W_in[c] x_k + W_rec[c] h_k
 *   g      = tanh(A_g),  hh = tanh(A_h~),  gate = sigmoid(-A_f * dt) = 1/(1+exp(A_f dt))
 *   h_{k+1} = gate * g + (1 - gate) * hh,   h_seq[:, k] = h_{k+1}
 * The per-sample pre-activation over row-major [n_hid, n_in] / [n_hid, n_hid]
 * weights, tanh as the squashing function, the argument order of the backward,
 * overwrite-vs-accumulate rules and the optional grad_x follow "K-loop
 * Parallelization Implementation Plan", Tasks 2 and 3 (cfc_step_batched and
 * cfc_step_backward_batched).  The reducer follows Task 1 of that page
 * (reduce_axis0: argument order, overwrite, summation order).
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers unless stated otherwise; the caller owns
 *     every buffer.  Nothing is allocated, freed or synchronised inside a call.
 *   - Work is enqueued on `stream` (a cudaStream_t passed as void*; NULL is the
 *     legacy default stream) and runs asynchronously in stream order.
 *   - A non-zero return value means the arguments were rejected (nothing was
 *     launched) or a launch failed; cfc_status_string() names the reason.
 *   - Results are bit-identical from run to run for the same inputs,
 *     configuration and GPU model: no atomics, fixed summation orders.
 *   - Layouts are dense row-major with the last index fastest.
 *
 * Precision modes (`math`):
 *   CFC_MATH_FP32  x, h0, W_in, W_rec, h_seq are float; all arithmetic fp32.
 *   CFC_MATH_TF32  same storage as FP32; every operand of the projections and
 *                  gradient contractions (x, h, W, dA) is rounded to TF32 (10
 *                  mantissa bits, nearest, ties away from zero), products are
 *                  accumulated in fp32.  Activations and state stay fp32.
 *   CFC_MATH_BF16  x, h0, W_in, W_rec and h_seq are bfloat16 (raw 16-bit);
 *                  b, dt, y, grad inputs and all gradient outputs are float.
 *                  h_{k+1} is rounded to bf16 (nearest even) and that value is
 *                  stored and carried; dA is rounded to bf16 before the
 *                  gradient contractions; accumulation is fp32.
 */
#ifndef CFC_H_
#define CFC_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  CFC_OK = 0,
  CFC_ERR_NULL = -1,      /* a required pointer is NULL                        */
  CFC_ERR_SHAPE = -2,     /* a size is negative, zero where not allowed, or too large */
  CFC_ERR_ALIGN = -3,     /* a pointer is not aligned to its element size      */
  CFC_ERR_WORKSPACE = -4, /* workspace NULL or smaller than cfc_kloop_workspace_bytes() */
  CFC_ERR_MODE = -5,      /* unknown math mode or gradient path                */
  CFC_ERR_LAUNCH = -6,    /* a kernel launch failed (cudaGetLastError != 0)    */
  CFC_ERR_DEVICE = -7,    /* no usable CUDA device / unsupported architecture  */
  CFC_ERR_TOO_LARGE = -8, /* sizes need more than CFC_STATIC_WORKSPACE_BYTES   */
  CFC_ERR_OVERLAP = -9    /* buffers that must not overlap do                  */
} cfc_status;

typedef enum { CFC_MATH_FP32 = 0, CFC_MATH_TF32 = 1, CFC_MATH_BF16 = 2 } cfc_math;

/* How the per-sample parameter gradients are summed over the batch.
 *   CFC_GRAD_SCRATCH: each sample's packed gradient row (length N, below) is
 *     written once to a caller-provided per_sample_scratch[B, N] (overwrite;
 *     the K steps are summed on chip), then reduce_axis0 sums the B rows.
 *     This is the pages' per-batch scratch + reducer scheme ("K-loop
 *     Parallelization Implementation Plan", Tasks 3-5).
 *   CFC_GRAD_GEMM: the gradients are contracted directly over all B*K rows
 *     (dW = dA^T [x; h; 1]) as one batch-dimension GEMM with a fixed split
 *     over row blocks; the split partials live in the workspace and are summed
 *     by reduce_axis0 ("kernel-optimization" plan, Task 2 Step 3: weight
 *     gradient as a batch-dimension GEMM).
 * Packed per-sample layout, N = 3*(n_in + n_hid + 1)*n_hid floats:
 *   [ gW_in (c, i, j) : 3*n_hid*n_in | gW_rec (c, i, j) : 3*n_hid*n_hid | gb (c, i) : 3*n_hid ] */
typedef enum { CFC_GRAD_SCRATCH = 0, CFC_GRAD_GEMM = 1 } cfc_grad_path;

/* Human-readable name of a status code (static string, never NULL). */
const char* cfc_status_string(int status);

/* N = 3*(n_in + n_hid + 1)*n_hid, or 0 for invalid sizes. Host-only. */
long long cfc_per_sample_length(int n_in, int n_hid);

/* Bytes of device workspace that cfc_kloop_forward and cfc_kloop_backward
 * need for these sizes (the same value for both calls).  Host-only; returns 0
 * for invalid arguments.  The forward stores the activations of every step
 * there and the backward reads them, so the same workspace, untouched, must be
 * passed to the backward of the same inputs. */
size_t cfc_kloop_workspace_bytes(int B, int K, int n_in, int n_hid, int math, int grad_path);

/* Number of rows S of the gradient partials [S, N] that the backward sums with
 * reduce_axis0 (B for CFC_GRAD_SCRATCH; a fixed split of the B*K rows for
 * CFC_GRAD_GEMM).  Host-only; 0 for invalid arguments. */
int cfc_kloop_grad_splits(int B, int K, int n_in, int n_hid, int math, int grad_path);

/* Device-side error word of the library (host-blocking diagnostic: waits for
 * all work on the device).  Returns 0 if no kernel has reported an error,
 * 1 if a tensor-core kernel gave up a bounded wait (its outputs are then not
 * valid), or CFC_ERR_DEVICE if the word cannot be read.  clear != 0 resets it. */
int cfc_device_error(int clear);

/* Diagnostic of the timeout path: launches one kernel whose bounded mbarrier
 * wait (the wait helper of the K-loop kernels) runs out after max_polls polls
 * (1 .. 2^20) because nothing completes the barrier; the kernel then sets the
 * device error words (the K loop's and those of the gated delta rule) and
 * returns, so cfc_device_error reports 1 until it clears them.  No other state
 * changes; the context stays usable.  CFC_ERR_SHAPE for max_polls
 * out of range. */
int cfc_selftest_timeout(int max_polls, void* stream);

/* Forward K-loop.
 *   x      [B, K, n_in]      (float or bf16 by `math`)
 *   h0     [B, n_hid]        (float or bf16)
 *   W_in   [3, n_hid, n_in]  heads f, g, h~ (float or bf16)
 *   W_rec  [3, n_hid, n_hid] (float or bf16)
 *   b      [3, n_hid]        float
 *   dt     [B] float if dt_stride == 1, or one float broadcast if dt_stride == 0
 *   h_seq  [B, K, n_hid]     OUTPUT, overwrite: h_seq[:, k] = h_{k+1}
 *   workspace / workspace_bytes: see cfc_kloop_workspace_bytes.
 * Requirements: B >= 1, K >= 1, 1 <= n_in, 1 <= n_hid <= 1024, n_in + n_hid <= 1024;
 * every pointer aligned to 16 bytes. */
int cfc_kloop_forward(const void* x, const void* h0, const void* W_in, const void* W_rec,
                      const float* b, const float* dt, int dt_stride,
                      int B, int K, int n_in, int n_hid, int math,
                      void* h_seq, void* workspace, size_t workspace_bytes, void* stream);

/* Backward through the K loop of the forward that wrote `workspace`.
 * Inputs as in the forward, plus
 *   h_seq        [B, K, n_hid] as written by that forward
 *   grad_h_seq   [B, K, n_hid] float or NULL: upstream gradient of every h_seq[:, k]
 *   grad_h_last  [B, n_hid] float or NULL: extra upstream gradient of h_K
 *   y            [B, n_hid] float or NULL: target of the loss 0.5*||h_K - y||^2;
 *                adds h_K - y to the gradient of h_K
 * Outputs (all overwrite; the three parameter gradients are summed over B):
 *   grad_W_in [3, n_hid, n_in], grad_W_rec [3, n_hid, n_hid], grad_b [3, n_hid]
 *   grad_h0   [B, n_hid] or NULL
 *   grad_x    [B, K, n_in] or NULL (as in the pages' backward, grad_x is optional)
 *   per_sample_scratch [B, N] float: required for CFC_GRAD_SCRATCH (it then
 *                holds each sample's packed gradient), ignored (may be NULL)
 *                for CFC_GRAD_GEMM.
 * At least one upstream gradient (grad_h_seq, grad_h_last or y) must be given. */
int cfc_kloop_backward(const void* x, const void* h0, const void* W_in, const void* W_rec,
                       const float* b, const float* dt, int dt_stride,
                       int B, int K, int n_in, int n_hid, int math,
                       const void* h_seq, const float* grad_h_seq, const float* grad_h_last,
                       const float* y,
                       float* grad_W_in, float* grad_W_rec, float* grad_b,
                       float* grad_h0, float* grad_x,
                       float* per_sample_scratch, int grad_path,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Column sum of a row-major [n_batch, n_tail] float matrix into out[n_tail]
 * (overwrite), atomic-free, in a fixed association order that is bit-identical
 * to the pages' reference reducer ("K-loop Parallelization Implementation
 * Plan", Task 1): with 256 partial sums,
 *   p[t] = ((0.0f + in[t]) + in[t+256]) + in[t+512] + ...,  t = 0..255,
 * then p[t] += p[t+s] for s = 128, 64, ..., 1 and t < s;  out[j] = p[0].
 * n_batch == 0 writes +0.0f.  n_batch >= 0, 0 <= n_tail <= 2^35; per_batch and
 * out must be 4-byte aligned and must not overlap (16-byte alignment and
 * n_tail % 4 == 0 select the float4 path; otherwise scalar, same order). */
int reduce_axis0(const float* per_batch, int n_batch, long long n_tail, float* out, void* stream);

/* ---------------------------------------------------------------------------
 * The pages' single-head tau-cell ("K-loop Parallelization Implementation
 * Plan", Task 2: cfc_step_batched, Task 3: cfc_step_backward_batched), FP32:
 *   pre = b + W_in x_k + W_rec h_k,  s = tanh(pre),
 *   decay_i = exp(-dt / max(tau_i, 1e-6)),  h_{k+1} = h_k * decay + (1 - decay) * s,
 *   h_seq[:, k] = h_{k+1}.
 * Backward (dh = gradient reaching h_{k+1}): d_pre = dh (1 - decay)(1 - s^2);
 * gb += d_pre, gW_in += d_pre (x) x_k, gW_rec += d_pre (x) h_k,
 * gtau += dh (h_k - s) decay dt / max(tau, 1e-6)^2 where tau > 1e-6 (else 0);
 * grad h_k = W_rec^T d_pre + dh decay, grad x_k = W_in^T d_pre.
 * Shapes: x [B, K, n_in], h0 [B, n_hid], W_in [n_hid, n_in], W_rec [n_hid, n_hid],
 * b [n_hid], tau [n_hid], dt [B] (dt_stride 1) or [1] (dt_stride 0).  Every
 * pointer 16-byte aligned.  Sizes: 1 <= n_in, n_hid <= 1024 and the sample's
 * weights and gradient, 2 n_hid ((n_in + n_hid) | 1) floats, within one SM's
 * shared memory (about 28 K floats each; n_in = 64, n_hid = 128 fits) —
 * otherwise CFC_ERR_SHAPE. */

/* Packed per-sample gradient length (n_in + n_hid + 2) * n_hid, layout
 * [gW_in (i, j) | gW_rec (i, j) | gb (i) | gtau (i)]; 0 if unsupported. */
long long cfc_tau_per_sample_length(int n_in, int n_hid);

/* Workspace bytes of the tau-cell forward/backward pair (the saved s values),
 * 0 for unsupported sizes. */
size_t cfc_tau_kloop_workspace_bytes(int B, int K, int n_in, int n_hid);

/* Forward K loop: h_seq [B, K, n_hid] (overwrite) and s in the workspace. */
int cfc_tau_kloop_forward(const float* x, const float* h0, const float* W_in, const float* W_rec, const float* b,
                          const float* tau, const float* dt, int dt_stride, int B, int K, int n_in, int n_hid,
                          float* h_seq, void* workspace, size_t workspace_bytes, void* stream);

/* Backward through the K loop of the forward that filled `workspace`.
 * Upstream gradients as for cfc_kloop_backward (at least one of grad_h_seq
 * [B, K, n_hid], grad_h_last [B, n_hid], y [B, n_hid]).  Outputs (overwrite):
 * grad_W_in [n_hid, n_in], grad_W_rec [n_hid, n_hid], grad_b [n_hid],
 * grad_tau [n_hid] summed over the batch by reduce_axis0 from
 * per_sample_scratch [B, cfc_tau_per_sample_length] (written, required);
 * grad_h0 [B, n_hid] and grad_x [B, K, n_in] optional (NULL). */
int cfc_tau_kloop_backward(const float* x, const float* h0, const float* W_in, const float* W_rec,
                           const float* b, const float* tau, const float* dt, int dt_stride, int B, int K,
                           int n_in, int n_hid, const float* h_seq, const float* grad_h_seq,
                           const float* grad_h_last, const float* y, float* grad_W_in, float* grad_W_rec,
                           float* grad_b, float* grad_tau, float* grad_h0, float* grad_x,
                           float* per_sample_scratch, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Multi-horizon GRN heads on every K position of the trunk state, FP32.
 * Forward per horizon j of a row h (the ml-alpha commit history, commit "wire
 * TFT GRN heads into PerceptionTrainer (Phase 1.7)"):
 *   z1 = W1[j] h + b1[j],  a1 = GELU(z1) (exact: z Phi(z)),  z2 = W2[j] a1 + b2[j],
 *   gate = w_gate[j].z2 + b_gate[j],  main = w_main[j].z2 + b_main[j],
 *   skip = w_skip[j].h + b_skip[j],   p[j] = sigmoid(skip + sigmoid(gate) main).
 * Backward ("K-loop Parallelization Implementation Plan", Commit 2 / Task 11):
 * the chain rule of that forward from dL/dp, with
 *   grad_h = grad_h_carry + sum_j lambda[j] (W1[j]^T dz1_j + dskip_j w_skip[j])
 * (lambda scales the trunk gradient only) and every parameter gradient summed
 * per sample over its K rows (k = K-1 .. 0), then over the batch by
 * reduce_axis0.
 * Sizes: hidden (Hd) a multiple of 4 in [4, 256], head_mid (M) a multiple of 4
 * in [4, 64], n_horizons (J) in [1, 8]; otherwise CFC_ERR_SHAPE.  Rows are
 * r = b*K + k, so h may be the K loop's h_seq [B, K, Hd] and grad_h its
 * grad_h_seq.  Parameters (and gradients) are one packed vector of
 * cfc_grn_param_length floats, the ten tensors in this order, horizon-major:
 * [W1 (J,M,Hd) | b1 (J,M) | W2 (J,M,M) | b2 (J,M) | w_gate (J,M) | b_gate (J) |
 *  w_main (J,M) | b_main (J) | w_skip (J,Hd) | b_skip (J)].
 * Every pointer 16-byte aligned (CFC_ERR_ALIGN). */

/* Packed parameter / per-sample gradient length; 0 if unsupported. */
long long cfc_grn_param_length(int hidden, int head_mid, int n_horizons);

/* Floats per row of the forward's saved intermediates (z1, a1, z2 [J, M],
 * gate, main [J]): J (3 M + 2); 0 if unsupported. */
long long cfc_grn_saved_per_row(int head_mid, int n_horizons);

/* Workspace bytes of cfc_grn_backward for B*K rows; 0 if unsupported. */
size_t cfc_grn_workspace_bytes(int B, int K, int hidden, int head_mid, int n_horizons);

/* Forward over `rows` rows: probs [rows, J] and saved [rows, saved_per_row]
 * (both overwrite).  rows = 0 is a no-op. */
int cfc_grn_forward(const float* h, long long rows, int hidden, int head_mid, int n_horizons,
                    const float* params, float* probs, float* saved, void* stream);

/* Backward of the forward that wrote probs and saved for h [B*K, Hd]:
 * grad_probs [B*K, J] = dL/dp, lambda [J], grad_h_carry [B*K, Hd] (optional,
 * NULL = zero).  Outputs (overwrite): grad_h [B*K, Hd], per_sample_scratch
 * [B, cfc_grn_param_length] (each sample's gradient), grad_params
 * [cfc_grn_param_length] (their sum in reduce_axis0's order). */
int cfc_grn_backward(const float* h, int B, int K, int hidden, int head_mid, int n_horizons, const float* params,
                     const float* probs, const float* saved, const float* grad_probs, const float* lambda,
                     const float* grad_h_carry, float* grad_h, float* per_sample_scratch, float* grad_params,
                     void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * The gated delta rule (FP32 and BF16 modes; CFC_MATH_TF32 gives CFC_ERR_MODE).
 * Each sequence and value head h keeps a state S [d_k, d_v], zero or
 * initial_state at first, and per token t does
 *   S <- exp(g_t) S,  u = beta_t (v_t - S^T k_t),  S <- S + k_t u^T,
 *   o_t = scale S^T q_t.
 * Value head h uses query and key head h / (n_v_heads / n_k_heads).  g <= 0 is
 * the log-decay (-inf, and anything below -110, is a factor of zero: a reset);
 * for a bounded state beta |k|^2 stays in [0, 2].
 *
 * Shapes, rows being all tokens of all sequences one after another:
 *   q, k  [rows, n_k_heads, d_k], v [rows, n_v_heads, d_v]: float (FP32) or
 *         bfloat16 (BF16); the head and width axes are dense, rows are
 *         *_stride elements apart (at least heads * width, a multiple of 16
 *         bytes), so they may be parts of one projection's output
 *   g, beta [rows, n_v_heads]: float in both modes
 *   o, grad_o, grad_v like v but dense; grad_q, grad_k like q, k but dense;
 *   grad_g, grad_beta [rows, n_v_heads] in the type of q (float or bfloat16)
 *   states [n_seq, n_v_heads, d_k, d_v]: float in both modes
 * Sequences: with seq_offsets NULL, n_seq sequences of rows / n_seq tokens;
 * else seq_offsets is a DEVICE array of n_seq + 1 non-decreasing row numbers,
 * seq_offsets[0] = 0 and seq_offsets[n_seq] = rows, and sequence i has the rows
 * from seq_offsets[i] up to seq_offsets[i + 1] (none is allowed).  Offsets
 * outside [0, rows] are held to it: nothing outside the tensors is touched.
 * Sizes: d_k a multiple of 8 in [8, 128], d_v a multiple of 8 in [8, 256],
 * n_v_heads a multiple of n_k_heads and at most 4096, 1 <= n_seq <= 2^20,
 * 0 <= rows <= 2^30.  q, k, v, o, states, grad_o, grad_q, grad_k, grad_v and
 * the workspace are 16-byte aligned, the rest 4-byte aligned.
 *
 * FP32: products of two TF32 values an operand, fp32-accurate.  BF16: products
 * take bf16 operands and sum in fp32, and the running state is fp32.  Where a
 * final_state is asked for, every operand on the way to it and to o keeps 17
 * significant bits: the state is good to about 1e-5, o to its own rounding (2e-3).
 * Without one (training), the state, the corrections u and the chunk's inverse are
 * rounded to bf16 where they enter a product, and what the backward reads of them is
 * kept in bf16: o and the gradients are good to 3e-3 to 5e-3 of their norm.  The
 * roundings grow where little decays and beta |k|^2 is near 2, since the terms then
 * nearly cancel: without any decay o to 1.6e-2 with random keys at 2, and with one
 * key at every token to 5e-3 at 1, 4e-2 at 1.7, and 0.4 at 1.9 (with decays of 0.025
 * a token on average 1e-2); grad_q, grad_g and grad_beta, differences of such terms,
 * to several times that.  Ask for a final_state (o) or use FP32 where it matters.
 *
 * A NaN or an infinity at a token reaches o of that token and, through the
 * state, of its sequence's later ones, as in the recurrence; no earlier token, no
 * other sequence or head, and from v no other column.  The gradients of a
 * sequence and head in which anything is not finite are not specified. */

/* Device workspace of the two calls (save != 0: of a forward that a backward
 * follows, and of that backward).  Host-only; 0 for unsupported sizes. */
size_t cfc_gdr_workspace_bytes(long long rows, int n_seq, int n_k_heads, int n_v_heads, int d_k, int d_v, int math,
                               int save);

/* Forward over whole sequences.  initial_state and final_state may be NULL, or
 * the same buffer.  save != 0: keeps in the workspace what the backward reads. */
int cfc_gdr_forward(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                    long long v_stride, const float* g, const float* beta, const int* seq_offsets, int n_seq,
                    long long rows, int n_k_heads, int n_v_heads, int d_k, int d_v, float scale, int math,
                    const float* initial_state, void* o, float* final_state, int save, void* workspace,
                    size_t workspace_bytes, void* stream);

/* Backward of the forward that filled `workspace` (same inputs, save != 0).
 * grad_final_state may be NULL (zero), grad_initial_state too (not written).
 * All outputs are overwritten; grad_q and grad_k are summed over the value
 * heads of a group in a fixed order. */
int cfc_gdr_backward(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                     long long v_stride, const float* g, const float* beta, const int* seq_offsets, int n_seq,
                     long long rows, int n_k_heads, int n_v_heads, int d_k, int d_v, float scale, int math,
                     const void* grad_o, const float* grad_final_state, void* grad_q, void* grad_k, void* grad_v,
                     void* grad_g, void* grad_beta, float* grad_initial_state, void* workspace,
                     size_t workspace_bytes, void* stream);

/* The next `tokens` tokens of each of n_seq sequences (rows = n_seq * tokens):
 * sequence i's state is slots[i] of `state` [n_slots, n_v_heads, d_k, d_v]
 * (slots NULL: i), updated in place.  No two sequences may share a slot.  A
 * sequence whose slot is outside [0, n_slots) has no state: its o is zero and
 * nothing is kept.  All tokens are applied and no state in between is kept: who
 * may have to take tokens back (rejected drafts) copies the slots before the
 * call.  All arithmetic is fp32. */
int cfc_gdr_step(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                 long long v_stride, const float* g, const float* beta, int n_seq, int tokens, int n_k_heads,
                 int n_v_heads, int d_k, int d_v, float scale, int math, float* state, long long n_slots,
                 const int* slots, void* o, void* stream);

/* ---------------------------------------------------------------------------
 * Root-mean-square norm of a residual stream (FP32 and BF16 modes).
 *   s = x + residual rounded to the stored type (s = x where residual is NULL),
 *   rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd weight.
 * x, residual, y, residual_out, grad_y, grad_residual_out, grad_x [rows, d] in
 * the mode's type; weight, grad_weight [d], rstd [rows] float.  1 <= d <= 32768.
 * Pointers 16-byte aligned (rstd and y8_scale: 4).
 *
 * Forward: y and/or y8 (at least one); residual_out (= s) and rstd optional,
 * both needed by the backward.  y8 [rows, d] holds e4m3 values y / c with one
 * scale c for each group of y8_group columns (a divisor of d; d: one a row),
 * y8_scale [rows, d / y8_group] float, c = max |y| of the group / 448, from y
 * before its own rounding; c = 1 for a group of zeros.  residual_out may be
 * the buffer of x or residual. */
int cfc_rmsnorm_forward(const void* x, const void* residual, const float* weight, long long rows, int d, float eps,
                        int math, void* y, void* residual_out, float* rstd, void* y8, float* y8_scale, int y8_group,
                        void* stream);

/* Device workspace of the backward; 0 for unsupported sizes.  Host-only. */
size_t cfc_rmsnorm_workspace_bytes(long long rows, int d);

/* Backward from the stream s and rstd of the forward: grad_x is the gradient
 * of s, hence of x and of residual: the norm's own plus grad_residual_out (the
 * gradient that reaches s from later layers; NULL: none).  grad_weight is the
 * sum over rows (0 for rows = 0), its partial sums added by reduce_axis0.
 * grad_x may be the buffer of grad_y or grad_residual_out. */
int cfc_rmsnorm_backward(const void* s, const float* weight, const float* rstd, const void* grad_y,
                         const void* grad_residual_out, long long rows, int d, int math, void* grad_x,
                         float* grad_weight, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Layer norm of a residual stream (FP32 and BF16 modes).
 *   s = x + residual rounded to the stored type (s = x where residual is NULL),
 *   mean = sum(s) / d,  rstd = 1 / sqrt(sum((s - mean)^2) / d + eps),
 *   y = (s - mean) rstd weight + bias.
 * x, residual, y, residual_out, grad_y, grad_residual_out, grad_x [rows, d] in
 * the mode's type; weight, bias, grad_weight, grad_bias [d], mean, rstd [rows]
 * float.  1 <= d <= 32768.  Pointers 16-byte aligned (mean and rstd: 4).
 *
 * Forward: bias NULL: none.  residual_out (= s), mean and rstd are optional, and
 * all needed by the backward.  residual_out may be the buffer of x or residual. */
int cfc_layernorm_forward(const void* x, const void* residual, const float* weight, const float* bias, long long rows,
                          int d, float eps, int math, void* y, void* residual_out, float* mean, float* rstd, void* stream);

/* Device workspace of the backward; 0 for unsupported sizes.  Host-only. */
size_t cfc_layernorm_workspace_bytes(long long rows, int d);

/* Backward from the stream s, mean and rstd of the forward: grad_x is the
 * gradient of s, hence of x and of residual: the norm's own plus
 * grad_residual_out (NULL: none).  grad_weight and grad_bias (NULL: not wanted)
 * are sums over rows (0 for rows = 0), their partial sums added by
 * reduce_axis0.  grad_x may be the buffer of grad_y or grad_residual_out. */
int cfc_layernorm_backward(const void* s, const float* weight, const float* mean, const float* rstd, const void* grad_y,
                           const void* grad_residual_out, long long rows, int d, int math, void* grad_x,
                           float* grad_weight, float* grad_bias, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * The short causal convolution (FP32 and BF16 modes): each channel c over the
 * last `width` rows of its sequence,
 *   pre_t = bias[c] + sum_j weight[c, j] x_{t - width + 1 + j}[c],
 *   y_t = pre sigmoid(pre) where silu != 0, else pre.
 * The rows before a sequence's first are those of its initial_state, or zeros; its
 * final_state are its last width - 1 inputs, those of initial_state among them
 * where it is shorter.
 *   x [rows, channels], rows x_stride elements apart (at least channels, a multiple of
 *         16 bytes), in the mode's type; y, grad_y, grad_x like x but dense
 *   states [n_seq, width - 1, channels] in the mode's type
 *   weight, grad_weight [channels, width], bias, grad_bias [channels]: float
 * Sequences: seq_offsets NULL, n_seq sequences of rows / n_seq rows, else a DEVICE
 * array of n_seq + 1 non-decreasing row numbers from 0, sequence i having the rows
 * from seq_offsets[i] up to seq_offsets[i + 1] (none is allowed).  Rows from
 * seq_offsets[n_seq] on are nobody's: not read, and left as they are in every
 * output, so that a batch may be padded.  Nothing outside the tensors is touched
 * whatever the array holds.
 * Sizes: channels a multiple of 8, 2 <= width <= 8, 1 <= n_seq <= 2^20,
 * 0 <= rows <= 2^30.  Pointers 16-byte aligned (bias, seq_offsets, slots: 4).  Outputs,
 * a step's pool and the workspace among them, overlap neither inputs nor one another:
 * CFC_ERR_OVERLAP (rows that are parts of wider ones count by what they hold).
 *
 * Sums are fp32.  A NaN or an infinity reaches the `width` rows that see it, of
 * its own channel and sequence. */

/* Forward.  bias, initial_state and final_state may be NULL. */
int cfc_conv_forward(const void* x, long long x_stride, const float* weight, const float* bias, const int* seq_offsets,
                     int n_seq, long long rows, int channels, int width, int silu, int math, const void* initial_state,
                     void* y, void* final_state, void* stream);

/* Device workspace of the backward; 0 for unsupported sizes.  Host-only. */
size_t cfc_conv_workspace_bytes(long long rows, int channels, int width, int math);

/* Backward, from the forward's inputs alone.  grad_final_state NULL: zero;
 * grad_initial_state and grad_bias NULL: not written.  grad_weight and grad_bias
 * are sums over all rows, their partial sums added by reduce_axis0. */
int cfc_conv_backward(const void* x, long long x_stride, const float* weight, const float* bias, const int* seq_offsets,
                      int n_seq, long long rows, int channels, int width, int silu, int math, const void* initial_state,
                      const void* grad_y, const void* grad_final_state, void* grad_x, float* grad_weight, float* grad_bias,
                      void* grad_initial_state, void* workspace, size_t workspace_bytes, void* stream);

/* The next `tokens` rows of each of n_seq sequences (rows = n_seq * tokens):
 * sequence i's last inputs are slot slots[i] of `state` [n_slots, width - 1,
 * channels] (slots NULL: i), updated in place.  No two sequences may share a
 * slot.  A sequence whose slot is outside [0, n_slots) has no state: its y is
 * zero and nothing is kept. */
int cfc_conv_step(const void* x, long long x_stride, const float* weight, const float* bias, int n_seq, int tokens,
                  int channels, int width, int silu, int math, void* state, long long n_slots, const int* slots, void* y,
                  void* stream);

/* ---------------------------------------------------------------------------
 * The selective state space scan (FP32 and BF16 modes).  Each sequence and
 * channel c keeps a state h [n_states], zero or initial_state at first, and per
 * token t does
 *   dt = softplus(delta_t[c] + delta_bias[c]),
 *   h[n] <- exp(dt A[c, n]) h[n] + dt x_t[c] B_t[group, n],
 *   y_t[c] = (sum_n C_t[group, n] h[n] + D[c] x_t[c]) z_t[c] sigmoid(z_t[c]),
 * group = c / (channels / groups).  delta_bias, D and z may be NULL: 0, 0, and no
 * gate.  For a bounded state A is negative.
 *   x, delta, z [rows, channels], rows *_stride elements apart (at least channels, a
 *         multiple of 16 bytes); B, C [rows, groups, n_states], rows *_stride elements
 *         apart (at least groups * n_states); all in the mode's type
 *   A [channels, n_states], D, delta_bias [channels]: float
 *   y, grad_y, grad_x, grad_delta, grad_z, grad_B, grad_C like x, B and C but dense
 *   grad_A, grad_D, grad_delta_bias: float, summed over all rows
 *   states [n_seq, channels, n_states]: float in both modes
 * Sequences as for cfc_conv_forward.  Sizes: channels / groups a multiple of 8,
 * 1 <= n_states <= 64, groups * n_states <= 65536, 1 <= n_seq <= 2^20, 0 <= rows
 * <= 2^30.  x, delta, z, y, states, gradients and the workspace are 16-byte aligned;
 * B and C to their type (rows of whole 16-byte vectors, with 8, 16, 32 or 64
 * states, are read faster); grad_B, grad_C, A, D, delta_bias and their gradients 4
 * bytes.  Nothing that is written overlaps anything else, as for cfc_conv_forward.
 *
 * All arithmetic is fp32: states are good to about 1e-6 of their size times the
 * number of tokens that they remember, outputs as their sums of states, with |z| 6e-8
 * of the gate and their rounding on top.  A NaN or an infinity
 * at a token reaches that token's and, through the state, its sequence's later
 * outputs (of x, delta and z of its own channel); no earlier token and no other
 * sequence.  The gradients of a sequence in which anything is not finite are
 * not specified, nor those that sums over sequences share with it. */

/* Device workspace of the two calls (save != 0: of a forward that a backward
 * follows, and of that backward).  Host-only; 0 for unsupported sizes. */
size_t cfc_ssm_workspace_bytes(long long rows, int n_seq, int channels, int groups, int n_states, int math, int save);

/* Forward.  initial_state and final_state may be NULL.  save != 0: keeps in
 * the workspace what the backward reads, a state for every 16 rows. */
int cfc_ssm_forward(const void* x, long long x_stride, const void* delta, long long delta_stride, const float* A,
                    const void* B, long long B_stride, const void* C, long long C_stride, const float* D, const void* z,
                    long long z_stride, const float* delta_bias, const int* seq_offsets, int n_seq, long long rows,
                    int channels, int groups, int n_states, int math, const float* initial_state, void* y,
                    float* final_state, int save, void* workspace, size_t workspace_bytes, void* stream);

/* Backward of the forward that filled `workspace` (same inputs, save != 0).
 * grad_final_state NULL: zero.  grad_z is required with z; grad_D,
 * grad_delta_bias and grad_initial_state NULL: not written.  All outputs are
 * overwritten; grad_B and grad_C are summed over the channels of a group, grad_A,
 * grad_D and grad_delta_bias over rows, in a fixed order. */
int cfc_ssm_backward(const void* x, long long x_stride, const void* delta, long long delta_stride, const float* A,
                     const void* B, long long B_stride, const void* C, long long C_stride, const float* D, const void* z,
                     long long z_stride, const float* delta_bias, const int* seq_offsets, int n_seq, long long rows,
                     int channels, int groups, int n_states, int math, const float* initial_state, const void* grad_y,
                     const float* grad_final_state, void* grad_x, void* grad_delta, float* grad_A, void* grad_B,
                     void* grad_C, float* grad_D, void* grad_z, float* grad_delta_bias, float* grad_initial_state,
                     void* workspace, size_t workspace_bytes, void* stream);

/* The next `tokens` tokens of each of n_seq sequences (rows = n_seq * tokens):
 * sequence i's state is slots[i] of `state` [n_slots, channels, n_states] (slots
 * NULL: i), updated in place.  No two sequences may share a slot.  A sequence
 * whose slot is outside [0, n_slots) has no state: its y is zero and nothing is
 * kept. */
int cfc_ssm_step(const void* x, long long x_stride, const void* delta, long long delta_stride, const float* A,
                 const void* B, long long B_stride, const void* C, long long C_stride, const float* D, const void* z,
                 long long z_stride, const float* delta_bias, int n_seq, int tokens, int channels, int groups, int n_states,
                 int math, float* state, long long n_slots, const int* slots, void* y, void* stream);

/* ---------------------------------------------------------------------------
 * The norm of many gradients together, and clipping to it:
 *   norm = sqrt(sum of the squares of all values),
 *   out = grad min(1, max_norm / (norm + 1e-6)).
 * grads, out, n_values and math are HOST arrays of `count` entries, read before the
 * call returns: entry i is a device tensor of n_values[i] values (0 <= n_values[i] <=
 * 2^35; none is skipped), float for CFC_MATH_FP32 and bfloat16 for CFC_MATH_BF16,
 * aligned to its type (to 16 bytes is faster).  norm: one float on the device.
 * 0 <= count <= 65536.  Squares are fp32 where that holds them and 64 bits
 * elsewhere, their sums 64 bits: values from the smallest to the largest of their
 * type are counted.  A NaN makes the norm and the result NaN; a norm that is
 * infinite, or too large for a float, makes the factor 0 (for a finite max_norm). */

/* Device workspace of the two calls; 0 for unsupported counts.  Host-only. */
size_t cfc_grad_clip_workspace_bytes(int count);

int cfc_grad_norm(const void* const* grads, const long long* n_values, const int* math, int count, float* norm,
                  void* workspace, size_t workspace_bytes, void* stream);

/* out[i] may be grads[i]; otherwise no out overlaps a gradient or another out,
 * and no gradient may be named twice where it is its own out; norm overlaps
 * neither, and in both calls the workspace nothing at all (CFC_ERR_OVERLAP).  max_norm >= 0
 * (infinity: no clipping, whatever the norm but a NaN); otherwise CFC_ERR_SHAPE. */
int cfc_grad_clip(const void* const* grads, void* const* out, const long long* n_values, const int* math, int count,
                  float max_norm, float* norm, void* workspace, size_t workspace_bytes, void* stream);

/* reduce_axis0 for `count` independent matrices with one launch per kernel
 * configuration (the pages' training step calls the reducer 17 times, once per
 * scratch buffer: "K-loop Parallelization Implementation Plan", Self-Review).
 * per_batch, n_batch, n_tail and out are HOST arrays of `count` entries; entry
 * i is a device matrix [n_batch[i], n_tail[i]] and its device output
 * out[i][n_tail[i]] (overwrite), with the rules of reduce_axis0.  Every out[i]
 * receives exactly the bits reduce_axis0 would write.  0 <= count <= 4096;
 * entries with n_tail 0 are skipped; matrices and outputs must not overlap.
 * All entries are checked before anything is launched. */
int reduce_axis0_multi(const float* const* per_batch, const int* n_batch, const long long* n_tail,
                       float* const* out, int count, void* stream);

/* Forward + backward without allocation.  This entry point has no counterpart
 * in the pages; it exists for callers that cannot allocate device memory
 * when they run the K loop (code running under an allocator it does not own,
 * plugins barred from cudaMalloc, real-time loops where an allocation would
 * stall).  It computes what cfc_kloop_forward followed by cfc_kloop_backward
 * with CFC_GRAD_GEMM computes, but keeps the whole workspace in a fixed device
 * array inside the library and always runs the CUDA-core (SIMT) kernels: the
 * SIMT forward and backward K loops, the SIMT weight-gradient tiles and
 * reduce_axis0, in every precision mode.  The regular entry points choose
 * cluster or tensor-core kernels, which sum in other orders, so the two
 * agree within the parity tolerances (fp32: 1e-4 relative; TF32 / bf16:
 * 2e-3 normwise), not bit for bit; each is run-to-run bit-identical.
 *   - The array holds CFC_STATIC_WORKSPACE_BYTES bytes on every device that
 *     loads the library, until the process exits.  Sizes whose SIMT workspace
 *     (the W_cat^T copy, the [B,K,3H] activations and dA, and the weight
 *     gradient's split partials) is larger are rejected with
 *     CFC_ERR_TOO_LARGE before anything is launched.
 *   - The caller passes all inputs and outputs (same meaning, layout and
 *     overwrite rules as the two calls it replaces); nothing is allocated or
 *     freed by the call.
 *   - The first call on a device looks up the array's device address (once
 *     per device, with that device current); make that first call before any
 *     stream capture.  The address is kept for the life of the process: a
 *     device reset after that first call is not supported.
 *   - All calls share the one array, which keeps the last call's contents.
 *     Nothing in it has to start at zero (every part that is read is written
 *     earlier in the same call), but calls whose work overlaps on the GPU
 *     (for example on two streams) race on it and must be serialised. */
#define CFC_STATIC_WORKSPACE_BYTES (16u << 20)
int cfc_kloop_forward_backward_static(const void* x, const void* h0, const void* W_in,
                                      const void* W_rec, const float* b, const float* dt,
                                      int dt_stride, int B, int K, int n_in, int n_hid, int math,
                                      const float* grad_h_seq, const float* grad_h_last,
                                      const float* y,
                                      void* h_seq, float* grad_W_in, float* grad_W_rec,
                                      float* grad_b, float* grad_h0, float* grad_x, void* stream);

/* Kernel tracing (diagnostics, off by default).  While enabled, every kernel
 * that this library launches is bracketed by two CUDA events recorded on its
 * launch stream, so per-kernel device time can be read back afterwards.
 * Host-side state, not thread-safe; the events are created by the library
 * (the only resources it creates), so do not enable tracing inside CUDA-graph
 * capture.
 *   cfc_trace_enable(on): clears all records; on != 0 starts recording.
 *   cfc_trace_count():    number of recorded launches.
 *   cfc_trace_get(i, &name, &ms): kernel name (static string) and device time
 *                         in milliseconds of record i; waits for that record's
 *                         stop event.  Returns CFC_OK or CFC_ERR_SHAPE for a
 *                         bad index. */
int cfc_trace_enable(int on);
int cfc_trace_count(void);
int cfc_trace_get(int i, const char** name, float* ms);

#ifdef __cplusplus
}
#endif

#endif /* CFC_H_ */
