/*
 * gsdpa.h -- C ABI of the GB300 gated softmax attention library (libgsdpa.so).
 *
 * The operation: for each batch b, query head h and query row i,
 *
 *     O[b,i,h,:] = softmax_j( Q[b,i,h,:] . K[b,j,kv(h),:] / sqrt(d_k)  + causal mask )
 *                  @ V[b,:,kv(h),:]
 *                  (.) sigmoid( X[b,i,:] W_g[:, cols(h)] )
 *
 * Sources (page title and section):
 *   - SDPA, rows non-negative and summing to one:
 *       "GatedAttention [2025]", sec. 1.2.1 (the Attention(Q,K,V) equation).
 *   - The gate Y' = Y (.) sigma(X W_theta), X the hidden state after
 *     pre-normalisation, sigma the logistic sigmoid, multiplicative and
 *     head-specific by default:
 *       "GatedAttention [2025]", sec. 1.2.2.
 *   - Position G1 (on the SDPA output of each head, before the heads are
 *     concatenated), elementwise gate (n x q x d_k) and headwise gate (n x q):
 *       "GatedAttention [2025]", sec. 1.2.2 and 1.3.2; "10 . 门控", sec. 3.2
 *       (position table, Table 1 excerpt rows 5 and 10, and the G1 module with
 *       no bias and head-major gate columns).
 *   - Grouped-query K/V heads: "GatedAttention [2025]", sec. 1.3.1.
 *   - Causal sums over j <= i: "GatedAttention [2025]", sec. 1.4.1.
 *   - First-token attention share: "10 . 门控", sec. 3.4; "GatedAttention
 *     [2025]", sec. 1.4.3 (the F-Attn column).
 *
 * Readings where the pages are silent (the library's choices):
 *   - kv(h) = h / (H_q / H_kv): query heads form contiguous groups.
 *   - When L_q < L_k the causal mask is aligned bottom-right: query i sits at
 *     absolute position L_k - L_q + i and sees keys 0 .. L_k - L_q + i. A single
 *     decode query therefore sees the whole cache (the current token included).
 *   - The gate has no bias. cols(h) = h*d_k .. h*d_k + d_k - 1 (elementwise)
 *     or the single column h (headwise).
 *   - The first-token share is measured on the ungated attention weights and
 *     averaged over query rows: sink[b,h] = mean_i p(i -> key 0).
 *
 * Layouts (all row-major, contiguous, no padding):
 *   X    [B, L_q, d_model]
 *   Q    [B, L_q, H_q,  d_k]
 *   K, V [B, L_k, H_kv, d_k]
 *   W_g  [d_model, H_q*d_k] (elementwise) or [d_model, H_q] (headwise)
 *   O    [B, L_q, H_q,  d_k]  == the concatenated [B, L_q, H_q*d_k]
 *   sink [B, H_q] float32
 * The element type of X, Q, K, V, W_g and O is float32 (GSDPA_F32) or
 * bfloat16 (GSDPA_BF16); sink is always float32.
 *
 * Ownership: the caller owns every buffer (inputs, outputs, workspace) and
 * the stream. All pointers passed to gated_sdpa_fwd are DEVICE pointers of
 * the current device. The library never allocates device memory and never
 * synchronises inside gated_sdpa_fwd: the call enqueues kernels (and small
 * memset nodes on the workspace) on `stream` and returns.
 *
 * Errors: every function returns a gsdpa_status. Argument errors are detected
 * on the host before anything is enqueued. Kernels never wait without a limit:
 * a wait that runs out records a device error word and the kernel returns;
 * gsdpa_check_device_error() reads that word.
 */
#ifndef GSDPA_H_
#define GSDPA_H_

#include <stddef.h>

#if defined(__GNUC__)
#define GSDPA_API __attribute__((visibility("default")))
#else
#define GSDPA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GSDPA_GATE_NONE = 0,         /* plain SDPA, W_g and X may be NULL */
    GSDPA_GATE_HEADWISE = 1,     /* one sigmoid per (token, head)     */
    GSDPA_GATE_ELEMENTWISE = 2,  /* one sigmoid per (token, head, c)  */
    /* gated_sdpa_fwd_variant only: */
    GSDPA_GATE_HEADWISE_SHARED = 3,     /* W_g [d_model, 1]: one gate per token, every head */
    GSDPA_GATE_ELEMENTWISE_SHARED = 4,  /* W_g [d_model, d_k]: one gate per (token, c), every head */
    GSDPA_GATE_STATIC = 5,              /* W_g holds theta [H_q, d_k]: the gate does not read X */
    GSDPA_GATE_HEADWISE_AVERAGED = 6,   /* W_g [d_model, H_q]: the H_q heads' gate values averaged,
                                           one gate per token for every head */
    GSDPA_GATE_ELEMENTWISE_AVERAGED = 7 /* W_g [d_model, H_q d_k]: the heads' gate values averaged
                                           over the heads, one gate per (token, c) for every head */
} gsdpa_gate_mode;

/* How the gate's logit gl acts on the SDPA output y (gated_sdpa_fwd_variant). */
typedef enum {
    GSDPA_FN_SIGMOID_MUL = 0,    /* y * sigma(gl)               (gated_sdpa_fwd's gate) */
    GSDPA_FN_NS_SIGMOID_MUL = 1, /* y * (0.5 + 0.5 sigma(gl))                          */
    GSDPA_FN_SIGMOID_ADD = 2,    /* y + sigma(gl)                                      */
    GSDPA_FN_SILU_ADD = 3,       /* y + gl sigma(gl)                                   */
    GSDPA_FN_IDENTITY_ADD = 4,   /* y + gl                                             */
    GSDPA_FN_SILU_SELF = 5,      /* y * sigma(y), no gate (gate_mode NONE)             */
    GSDPA_FN_RMSNORM = 6         /* per head: y / sqrt(mean_c y^2 + eps) * gamma[h, c],
                                    no gate (gate_mode NONE); W_g holds gamma [H_q, d_k]
                                    or is NULL for gamma = 1                            */
} gsdpa_gate_fn;

typedef enum {
    GSDPA_F32 = 0,               /* float32 in/out, float32 arithmetic (SIMT) */
    GSDPA_BF16 = 1               /* bfloat16 in/out, fp32 accumulation (tcgen05) */
} gsdpa_dtype;

typedef enum {
    GSDPA_OK = 0,
    GSDPA_ERR_INVALID_ARG = -1,      /* a size, mode or pointer is invalid      */
    GSDPA_ERR_UNSUPPORTED = -2,      /* valid, but not built (d_k, device, ...) */
    GSDPA_ERR_ALIGNMENT = -3,        /* a pointer is not 16-byte aligned        */
    GSDPA_ERR_WORKSPACE = -4,        /* workspace NULL or smaller than needed   */
    GSDPA_ERR_LAUNCH = -5,           /* the CUDA runtime refused a launch       */
    GSDPA_ERR_DEVICE_TIMEOUT = -6,   /* a kernel wait ran out (see below)       */
    GSDPA_ERR_CACHE_RANGE = -7       /* a length on the device lay outside its cache (see below) */
} gsdpa_status;

/*
 * Bytes of device workspace gated_sdpa_fwd needs for this problem, or 0 if
 * none. Same arguments as gated_sdpa_fwd (want_sink != 0 when a sink pointer
 * will be passed). Returns (size_t)-1 for arguments gated_sdpa_fwd would
 * reject. Host-only; touches no device.
 */
GSDPA_API size_t gsdpa_workspace_bytes(int B, int L_q, int L_k, int d_model, int H_q, int H_kv, int d_k,
                             int gate_mode, int want_sink, int dtype);

/*
 * The gated attention forward (prefill when L_q > 1, decode when L_q == 1).
 *
 *   X, Q, K, V, W_g : device inputs in the layouts above. X and W_g may be
 *                     NULL when gate_mode == GSDPA_GATE_NONE.
 *   O               : device output [B, L_q, H_q, d_k], same dtype as inputs.
 *   sink            : device float32 [B, H_q] or NULL (not computed). With
 *                     bf16 prefill the rows' shares are added in fixed point
 *                     with 43 - ceil(log2(L_q + 1)) fraction bits, so the sum
 *                     does not depend on the order of the additions and
 *                     repeated calls give the same bits; there L_q <= 2^24
 *                     (GSDPA_ERR_UNSUPPORTED otherwise).
 *   B, L_q, L_k     : batch, query rows, key rows; 1 <= L_q <= L_k. B, L_q == 0
 *                     is an empty problem: nothing is enqueued, GSDPA_OK.
 *   d_model         : width of X (>= 1 when a gate is used; for bf16 a
 *                     multiple of 8, since every row must start on 16 bytes).
 *   H_q, H_kv       : query and K/V heads, H_q % H_kv == 0 (bf16 headwise
 *                     gate: H_q a multiple of 8, for the same reason).
 *   d_k             : head dimension, 64 or 128.
 *   gate_mode       : gsdpa_gate_mode.
 *   causal          : nonzero for the bottom-right causal mask.
 *   dtype           : gsdpa_dtype. GSDPA_BF16 needs an sm_103 device.
 *   workspace       : device scratch of at least gsdpa_workspace_bytes(...)
 *                     bytes, 256-byte aligned; contents need not be
 *                     initialised and are overwritten. NULL allowed when 0.
 *   stream          : a cudaStream_t (NULL = legacy default stream).
 *
 * X, Q, K, V, W_g and O must be 16-byte aligned and sink 4-byte aligned
 * (GSDPA_ERR_ALIGNMENT otherwise).
 * Calls that share a workspace must not overlap on the device.
 */
GSDPA_API int gated_sdpa_fwd(const void* X, const void* Q, const void* K, const void* V, const void* W_g,
                   void* O, float* sink,
                   int B, int L_q, int L_k, int d_model, int H_q, int H_kv, int d_k,
                   int gate_mode, int causal, int dtype,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * The forward with one of the gate variants of "GatedAttention [2025]"
 * (sec. 1.2.2 items (3)-(5): head-shared gates, additive gating with sigmoid
 * or SiLU; sec. 1.4.1: SiLU of the output with no parameters, additive gating
 * without SiLU, per-head RMSNorm before concatenation; sec. 1.4.2: an
 * input-independent gate, NS-sigmoid). The gate shape is gate_mode, how the
 * gate acts on the SDPA output y is gate_fn:
 *   gate_mode HEADWISE, ELEMENTWISE and the two _SHARED shapes: logit
 *     gl = X W_g for the columns the shape gives; gate_fn one of
 *     SIGMOID_MUL .. IDENTITY_ADD;
 *   gate_mode STATIC: gl = theta[h, c] from W_g ([H_q, d_k], same dtype as
 *     the call); X is not read and may be NULL; gate_fn as above;
 *   gate_mode HEADWISE_AVERAGED, ELEMENTWISE_AVERAGED: the head-shared gate
 *     read as an average over the query heads (sec. 1.3.2 (ii)): the
 *     head-specific gate values v_h = f(gl_h) of every head h (gl = X W_g as
 *     for HEADWISE, ELEMENTWISE; f the gate_fn's function of the logit) are
 *     averaged, vbar = (1/H_q) sum_h v_h, and every head combines the same
 *     vbar with its y (multiplied or added as gate_fn says); prefill only
 *     (L_q == 1 decode calls return GSDPA_ERR_UNSUPPORTED);
 *   gate_mode NONE: gate_fn SIGMOID_MUL (plain SDPA), SILU_SELF or RMSNORM
 *     (W_g = gamma [H_q, d_k] or NULL; eps >= 0 is added to the mean square).
 * Other combinations return GSDPA_ERR_INVALID_ARG. The gate's value is kept
 * as fp16 between the gate pass and the attention kernel (bf16 path), as for
 * gated_sdpa_fwd. Workspace: gsdpa_workspace_bytes_variant. All other
 * arguments, alignment and errors as for gated_sdpa_fwd; gate_fn
 * SIGMOID_MUL with gate_mode 0..2 is gated_sdpa_fwd.
 */
GSDPA_API size_t gsdpa_workspace_bytes_variant(int B, int L_q, int L_k, int d_model, int H_q, int H_kv, int d_k,
                                               int gate_mode, int gate_fn, int want_sink, int dtype);
GSDPA_API int gated_sdpa_fwd_variant(const void* X, const void* Q, const void* K, const void* V, const void* W_g,
                                     void* O, float* sink, int B, int L_q, int L_k, int d_model, int H_q, int H_kv,
                                     int d_k, int gate_mode, int gate_fn, float eps, int causal, int dtype,
                                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * gated_sdpa_fwd that also measures the gate's scores ("GatedAttention
 * [2025]", sec. 1.4.2: the mean gating score of Table 4, the score
 * distribution of Figure 3, and the fraction of scores below a threshold):
 *   stats     : device array of 3 + n_bins unsigned 64-bit counters, 8-byte
 *               aligned, overwritten by the call:
 *               [0] number of scores (B L_q H_q d_k elementwise, B L_q H_q headwise),
 *               [1] the sum of the scores times 2^32 in fixed point: exactly
 *                   the sum of round(score * 2^32) for the headwise gate, the
 *                   decode kernel and the float32 path; the bf16 elementwise
 *                   prefill rounds each thread's float32 partial sums (of at
 *                   most 256 scores) once, so its mean is within 2^-18 of the
 *                   exact mean of the scores,
 *               [2] number of scores < threshold,
 *               [3 + k] scores s with min(floor(s n_bins), n_bins - 1) = k.
 *               Integer counters: the result does not depend on the order in
 *               which threads add them (two calls give the same bits). The
 *               score is the value the call multiplies by (bf16 path: the
 *               fp16 value of the elementwise gate; the fp32 value of the
 *               headwise gate).
 *   n_bins    : 1 .. 64.   threshold : in [0, 1].
 * gate_mode HEADWISE or ELEMENTWISE (GSDPA_ERR_INVALID_ARG otherwise); other
 * arguments, workspace and errors as for gated_sdpa_fwd (an empty problem
 * enqueues nothing and leaves stats as they are).
 */
GSDPA_API int gated_sdpa_fwd_stats(const void* X, const void* Q, const void* K, const void* V, const void* W_g,
                                   void* O, float* sink, unsigned long long* stats, int n_bins, float threshold,
                                   int B, int L_q, int L_k, int d_model, int H_q, int H_kv, int d_k, int gate_mode,
                                   int causal, int dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The whole layer around the attention ("GatedAttention [2025]", sec. 1.2.1:
 * Q, K, V projected from the hidden state X; sec. 1.2.2: the gate reads X
 * too; the heads' gated outputs concatenated and projected by W_O):
 *   [Q | K | V | GL] = X W_in                    one GEMM (the four share X)
 *   Y = (softmax(Q K^T / sqrt(d_k) + causal) V (.) sigma(GL)) W_O
 * with the attention of gated_sdpa_fwd in between. Self-attention (L_q = L_k
 * = L) without a cache.
 *   X      : device bf16 [B, L, d_model].
 *   W_in   : device bf16 [d_model, (H_q + 2 H_kv) d_k + G] with G = H_q d_k
 *            (elementwise gate), H_q (headwise gate) or 0 (no gate);
 *            columns: the Q heads, the K heads, the V heads, then the gate's
 *            columns (head-major, like gated_sdpa_fwd's W_g).
 *   W_O    : device bf16 [H_q d_k, d_model].
 *   Y      : device bf16 [B, L, d_model] out.
 *   gate_mode NONE, HEADWISE or ELEMENTWISE (GSDPA_ERR_INVALID_ARG
 *   otherwise); bf16, d_k = 128, L >= 2, d_model a multiple of 8 and >= 256,
 *   H_q a multiple of 8 with the headwise gate (GSDPA_ERR_UNSUPPORTED
 *   otherwise).
 * Q, K, V and the pre-W_O output live in the workspace (bf16), the gate as
 * fp16 values (elementwise) or float32 logits (headwise), as in
 * gated_sdpa_fwd. Pointers 16-byte aligned; asynchronous on `stream`; errors
 * as for gated_sdpa_fwd.
 */
GSDPA_API size_t gsdpa_layer_workspace_bytes(int B, int L, int d_model, int H_q, int H_kv, int d_k, int gate_mode);
GSDPA_API int gated_attention_layer(const void* X, const void* W_in, const void* W_O, void* Y, int B, int L,
                                    int d_model, int H_q, int H_kv, int d_k, int gate_mode, int causal,
                                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * The forward a training step runs: gated_sdpa_fwd, and also, for every
 * batch b, query head h and query row i, the natural log of the softmax
 * denominator, lse[b, h, i] = log sum_j exp(s_j) over the row's visible
 * scores s_j = Q.K / sqrt(d_k) ("GatedAttention [2025]", sec. 1.2.1: the
 * softmax of the SDPA equation; the backward rebuilds the weights from it).
 *
 *   lse : device float32 [B, H_q, L_q] (head-major), 4-byte aligned; required.
 *   Other arguments and the workspace as for gated_sdpa_fwd.
 * bf16 prefill only (L_q != 1): GSDPA_ERR_UNSUPPORTED otherwise.
 */
GSDPA_API int gated_sdpa_fwd_train(const void* X, const void* Q, const void* K, const void* V, const void* W_g,
                   void* O, float* sink, float* lse,
                   int B, int L_q, int L_k, int d_model, int H_q, int H_kv, int d_k,
                   int gate_mode, int causal, int dtype,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * gated_sdpa_fwd_train for the elementwise gate that also saves the gate's
 * values for the backward pass (gated_sdpa_bwd_saved_gate then skips their
 * recomputation, a GEMM of the size of the gate's):
 *   gate_out : device fp16 [B * L_q, H_q * d_k], 16-byte aligned, overwritten
 *              with sigma(X W_g) exactly as the forward multiplied by it.
 * gate_mode ELEMENTWISE and gate_out non-NULL (GSDPA_ERR_INVALID_ARG
 * otherwise); other arguments, workspace and errors as for
 * gated_sdpa_fwd_train. The values are copied from the workspace after the
 * call's kernels, on the same stream.
 */
GSDPA_API int gated_sdpa_fwd_train_save_gate(const void* X, const void* Q, const void* K, const void* V,
                   const void* W_g, void* O, float* sink, float* lse, void* gate_out,
                   int B, int L_q, int L_k, int d_model, int H_q, int H_kv, int d_k,
                   int gate_mode, int causal, int dtype,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * Workspace bytes gated_sdpa_bwd needs for this problem (bf16, d_k = 128);
 * (size_t)-1 for an invalid or unsupported shape, 0 for an empty one.
 */
GSDPA_API size_t gsdpa_bwd_workspace_bytes(int B, int L_q, int L_k, int d_model, int H_q, int H_kv, int d_k,
                   int gate_mode);

/*
 * The backward pass of the layer: given dO = dL/dO, the gradients of the
 * loss with respect to Q, K, V and, with a gate, W_g and X (the gate path's
 * share of dX; X also feeds projections this library does not own).
 * The chain rule of the forward ("GatedAttention [2025]", sec. 1.2.1 and
 * 1.2.2); the gate's part as in "解密NeurIPS最佳论文：Gated Attention…",
 * sec. 2.2: the gradient on the gate's input is dO times the ungated output
 * times sigma (1 - sigma).
 *
 *   X, Q, K, V, W_g : the forward's inputs (same layouts as gated_sdpa_fwd).
 *   O, lse          : the forward's output [B, L_q, H_q, d_k] and its
 *                     log-denominators [B, H_q, L_q] (gated_sdpa_fwd_train).
 *   dO              : device [B, L_q, H_q, d_k], same dtype.
 *   dQ              : out, like Q.   dK, dV : out, like K and V (each the sum
 *                     over the query heads of the kv head's group).
 *   dX, dW_g        : out, like X and W_g (gated only; NULL allowed without a gate).
 *   workspace       : gsdpa_bwd_workspace_bytes(...) bytes, 256-byte aligned.
 * Every output is overwritten. bf16, d_k = 128 and gate_mode NONE, HEADWISE
 * or ELEMENTWISE with the sigmoid gate only (GSDPA_ERR_UNSUPPORTED otherwise:
 * the variants of gated_sdpa_fwd_variant have no backward); sm_103 device.
 * Tensors 16-byte aligned, lse 4-byte aligned.
 * Asynchronous on `stream`; errors as for gated_sdpa_fwd.
 */
GSDPA_API int gated_sdpa_bwd(const void* X, const void* Q, const void* K, const void* V, const void* W_g,
                   const void* O, const void* dO, const float* lse,
                   void* dX, void* dQ, void* dK, void* dV, void* dW_g,
                   int B, int L_q, int L_k, int d_model, int H_q, int H_kv, int d_k,
                   int gate_mode, int causal, int dtype,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * gated_sdpa_bwd for the elementwise gate with the gate's values taken from
 * gate_saved (what gated_sdpa_fwd_train_save_gate wrote: fp16
 * [B * L_q, H_q * d_k], 16-byte aligned) instead of recomputed from X and
 * W_g. With the forward's own values the outputs equal gated_sdpa_bwd's bit
 * for bit. gate_mode ELEMENTWISE and gate_saved non-NULL
 * (GSDPA_ERR_INVALID_ARG otherwise); other arguments, workspace (the same
 * gsdpa_bwd_workspace_bytes) and errors as for gated_sdpa_bwd.
 */
GSDPA_API int gated_sdpa_bwd_saved_gate(const void* X, const void* Q, const void* K, const void* V,
                   const void* W_g, const void* O, const void* dO, const float* lse,
                   const void* gate_saved,
                   void* dX, void* dQ, void* dK, void* dV, void* dW_g,
                   int B, int L_q, int L_k, int d_model, int H_q, int H_kv, int d_k,
                   int gate_mode, int causal, int dtype,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * Per-head RMS norm of queries and keys, and rotary positions, in one pass:
 * what stands between the projection and the attention ("GatedAttention
 * [2025]", sec. 1.2.1 takes Q and K as given). For one head's row x at
 * position p:
 *     y_c = x_c gamma_c / sqrt(mean_c x_c^2 + eps)      (norm; else y = x)
 *     (y_a, y_b) -> t (y_a cos(p w_i) - y_b sin(p w_i),
 *                      y_b cos(p w_i) + y_a sin(p w_i))  for each pair i < rotary_dim / 2
 * with (a, b) = (i, i + rotary_dim / 2) (half layout) or (2i, 2i + 1)
 * (interleaved), w_i the pair's frequency and t = attn_scale; the columns from
 * rotary_dim on are not rotated. Everything in float32, rounded once; the angle
 * p w_i is that of the float64 frequency to |p| 2^-59 rad, modulo a turn, for every
 * 32-bit position (before it is rounded to float32).
 *
 * gsdpa_rope is the plan, made once on the host by one of the two init
 * functions and passed to every call (its contents are copied at the call).
 *   rotary_dim : a multiple of 16, 16 .. 128 (and at most the call's d_k).
 *   theta      : > 1; w_i = theta^(-2i / rotary_dim).
 *   scaling    : PLAIN; LINEAR, w_i / factor; BASE, theta replaced by
 *                theta factor^(rotary_dim / (rotary_dim - 2)); PARTS (the
 *                "NTK-by-parts" interpolation of the YaRN paper), pairs that
 *                turn more than beta_fast times in orig_len positions keep
 *                their frequency, those under beta_slow turns are divided by
 *                factor, a linear ramp over the pair's index between. factor
 *                >= 1 (unused with PLAIN), orig_len >= 1 and beta_fast >=
 *                beta_slow > 0 with PARTS.
 *   attn_scale : t; 0 for the default, 1 (PARTS: 0.1 ln(factor) + 1).
 * gsdpa_rope_init_freqs takes any finite frequencies (rotary_dim / 2 of them,
 * radians per position) and t as it is.
 */
typedef enum { GSDPA_ROPE_HALF = 0, GSDPA_ROPE_INTERLEAVED = 1 } gsdpa_rope_layout;
typedef enum {
    GSDPA_ROPE_PLAIN = 0,
    GSDPA_ROPE_LINEAR = 1,
    GSDPA_ROPE_BASE = 2,
    GSDPA_ROPE_PARTS = 3
} gsdpa_rope_scaling;
typedef struct {
    int rotary_dim, layout;
    float attn_scale;
    int reserved;
    unsigned long long turn[64];   /* each pair's frequency in turns per position, times 2^64, modulo 2^64 */
} gsdpa_rope;
GSDPA_API int gsdpa_rope_init(gsdpa_rope* rope, int rotary_dim, int layout, double theta, int scaling, double factor,
                              double orig_len, double beta_fast, double beta_slow, double attn_scale);
GSDPA_API int gsdpa_rope_init_freqs(gsdpa_rope* rope, int rotary_dim, int layout, const double* inv_freq,
                                    double attn_scale);

/*
 * The forward. Q [B, L, H_q, d_k] and K [B, L, H_kv, d_k], heads contiguous in
 * a token's row, rows ld elements apart (ld_q >= H_q d_k, ...), so that Q and K
 * may be column blocks of one projection's output; likewise the outputs Qo, Ko.
 *   gamma_q, gamma_k : [d_k], same dtype, or NULL for 1 (NULL without norm).
 *   positions        : device int32 [B, L] (any values), or NULL for 0 .. L - 1.
 *   norm             : 1 or 0.    eps : finite, >= 0 (norm only).
 *   rope             : the plan (host pointer), or NULL for no rotation.
 *   dtype            : GSDPA_F32 or GSDPA_BF16 (Q, K, gammas and outputs).
 * d_k 64 or 128 (GSDPA_ERR_UNSUPPORTED otherwise); any H_q, H_kv >= 1. In place
 * (Qo == Q with ld_qo == ld_q, the same for K) is allowed, other overlaps are
 * not. Tensors 16-byte aligned, row lengths a multiple of 16 bytes. sm_103
 * device. No workspace. B or L == 0: nothing is enqueued, GSDPA_OK.
 */
GSDPA_API int gsdpa_qk_norm_rope(const void* Q, const void* K, const void* gamma_q, const void* gamma_k,
                   const int* positions, void* Qo, void* Ko,
                   long long ld_q, long long ld_k, long long ld_qo, long long ld_ko,
                   int B, int L, int H_q, int H_kv, int d_k, int norm, float eps, const gsdpa_rope* rope, int dtype,
                   void* stream);

/*
 * The backward of gsdpa_qk_norm_rope: from dQo, dKo (the loss's gradients with
 * respect to its outputs: gated_sdpa_bwd's dQ and dK) and the forward's inputs,
 * the gradients with respect to Q, K, gamma_q and gamma_k.
 *   Q, K             : the forward's inputs; not read (may be NULL) without norm.
 *   dQ, dK           : out, each may be dQo, dKo (same row length).
 *   dgamma_q, dgamma_k : out, [d_k] in the call's dtype, 16-byte aligned, summed in
 *                      float32 over all rows in a fixed order (repeated calls give
 *                      the same bits), or NULL for one that is not wanted; NULL
 *                      without norm. With gamma NULL they are the gradients at 1.
 *   workspace        : gsdpa_qk_norm_rope_bwd_workspace_bytes(...) bytes, 256-byte
 *                      aligned (0 without norm).
 * Other arguments, alignment and errors as for the forward. An empty problem
 * enqueues nothing and leaves dgamma_q and dgamma_k as they are.
 */
GSDPA_API size_t gsdpa_qk_norm_rope_bwd_workspace_bytes(int B, int L, int d_k, int norm);
GSDPA_API int gsdpa_qk_norm_rope_bwd(const void* Q, const void* K, const void* gamma_q, const void* gamma_k,
                   const int* positions, const void* dQo, const void* dKo, void* dQ, void* dK,
                   void* dgamma_q, void* dgamma_k,
                   long long ld_q, long long ld_k, long long ld_dqo, long long ld_dko, long long ld_dq,
                   long long ld_dk, int B, int L, int H_q, int H_kv, int d_k, int norm, float eps,
                   const gsdpa_rope* rope, int dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * A K/V cache held in 8 bits, with one scale per block of 64 tokens and head
 * ("GatedAttention [2025]", sec. 1.3.1: the grouped-query cache is what decode
 * reads). The caller owns every buffer; the struct (on the host) describes them
 * and its contents are copied at each call.
 *   k8      : [B, H_kv, capacity / 64, 64, d_k] codes of the keys
 *   v8      : [B, H_kv, capacity / 64, d_k, 64] codes of the values (transposed)
 *   k_scale, v_scale : float32 [B, H_kv, capacity / 64], >= 0 (or NaN): a code stands
 *             for code * scale
 *   k_tail  : bf16 [B, H_kv, 2, 64, d_k], v_tail : bf16 [B, H_kv, 2, d_k, 64]: the
 *             tokens of a block that is not full yet wait here unrounded, block j in
 *             buffer j % 2. Token p is token p % 64 of block p / 64.
 *   kind    : GSDPA_CACHE_INT8 (signed integers) or GSDPA_CACHE_E4M3 (8-bit floating
 *             point, 4 exponent and 3 mantissa bits, no infinities).
 *   capacity: tokens per sequence, a multiple of 64.   d_k : 64 or 128.
 * A sequence of T tokens has T / 64 full blocks in 8 bits and T % 64 tokens in its
 * open block's buffer; the lengths belong to the caller (one array serves every
 * layer of a model). Nothing needs to be initialised for T = 0. Codes and scales
 * written elsewhere in this format may be used as well. Tensors 16-byte aligned,
 * scales 4-byte aligned.
 */
typedef enum { GSDPA_CACHE_INT8 = 0, GSDPA_CACHE_E4M3 = 1 } gsdpa_cache_kind;
typedef struct {
    int kind, B, H_kv, d_k, capacity;
    void *k8, *v8;
    float *k_scale, *v_scale;
    void *k_tail, *v_tail;
} gsdpa_cache8;

/*
 * Appends a step's keys and values. Sequence b holds lens[b] tokens before the
 * call; its first n_new[b] rows of K and V become tokens lens[b] .. (rows past
 * them are not read). lens is not changed: add n_new to it once, after the last
 * layer's attention.
 *   K, V   : device bf16 [B, L, H_kv, d_k], heads contiguous, rows ld_k, ld_v elements
 *            apart (multiples of 8, >= H_kv d_k).
 *   lens   : device int32 [B].    n_new : device int32 [B], or NULL for L each.
 * A block that becomes full is written in 8 bits: with amax its largest |x|,
 *   int8: scale = amax (1 / 127), reciprocal and product rounded to float32, code =
 *         x / scale to nearest, ties to even (+-127 at most);
 *   e4m3: scale = 2^e, the least e >= -126 with amax <= 448 scale, code = x / scale
 *         to nearest, ties to even.
 * amax = 0: scale and codes 0. A block that holds a NaN or an infinity: scale NaN,
 * codes 0 (every row that sees one of its tokens becomes NaN). Each token is rounded
 * once: the contents do not depend on how tokens were split over calls. Tokens may be
 * taken back (drafts that were not accepted) by lowering lens, repeatedly, to no less
 * than 64 below the longest length that the sequence has had since the tokens that stay
 * were appended: further back the open block's tokens have been written over, which no
 * call can see.
 * A sequence with lens[b] < 0, n_new[b] outside 0 .. L or more tokens than capacity
 * is left as it was, and the next gsdpa_check_device_error returns
 * GSDPA_ERR_CACHE_RANGE. Asynchronous on `stream`; sm_103 device.
 */
GSDPA_API int gsdpa_cache8_append(const gsdpa_cache8* cache, const void* K, const void* V, long long ld_k,
                   long long ld_v, const int* lens, const int* n_new, int L, void* stream);

/*
 * The gated attention of a step's tokens against the cache, after their keys and
 * values have been appended: query row i of sequence b sees tokens 0 .. lens[b] + i.
 *   Q, O   : device bf16 [B, L_q, H_q, d_k]; O overlaps no input.   X : bf16 [B, L_q, d_model].
 *   W_g    : as for gated_sdpa_fwd; gate_mode NONE, HEADWISE or ELEMENTWISE.
 *   lens   : device int32 [B], the tokens BEFORE this step (as passed to the append).
 *   n_new  : device int32 [B], rows of this step, or NULL for L_q each. Rows i >=
 *            n_new[b] of O are zero.
 * H_q a multiple of H_kv with (H_q / H_kv) L_q <= 128 (a decoding step, or a few
 * drafted tokens; GSDPA_ERR_UNSUPPORTED otherwise); d_model and the headwise gate's
 * H_q multiples of 8. A sequence that does not fit its cache (as above) gives zero
 * rows and GSDPA_ERR_CACHE_RANGE from the next gsdpa_check_device_error. Tokens past
 * a sequence's end are not seen whatever their bytes; a NaN or infinity among the
 * step's own keys is seen by the rows that may see it, one among its values in the
 * open block, or a NaN code in v8, by every row of the step.
 * Scores, softmax statistics and sums are float32; before they multiply V the weights
 * are rounded to fp16 (11 bits down to 2^-26 of the row's largest product of a weight
 * and a block's value scale, fewer below, nothing from 2^-37 on), the open block's to
 * 16 bits. The sums hold values up to 2^100 in magnitude.
 * workspace: gsdpa_cache8_workspace_bytes(...) bytes, 256-byte aligned; calls that
 * share one must not overlap on the device. Asynchronous on `stream`; other errors
 * as for gated_sdpa_fwd.
 */
GSDPA_API size_t gsdpa_cache8_workspace_bytes(const gsdpa_cache8* cache, int L_q, int d_model, int H_q,
                   int gate_mode);
GSDPA_API int gated_sdpa_cache8(const void* X, const void* Q, const gsdpa_cache8* cache, const int* lens,
                   const int* n_new, const void* W_g, void* O, int L_q, int d_model, int H_q, int gate_mode,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * A K/V cache held in 4 bits, in pages of 64 tokens that any sequence may take
 * ("GatedAttention [2025]", sec. 1.3.1: the grouped-query cache is what decode
 * reads). The caller owns the pool; the struct (on the host) describes it and its
 * contents are copied at each call.
 *   pool    : device uint8 [n_pages, H_kv, 72 d_k], 16-byte aligned. Nothing needs to be
 *             initialised. Token p % 64 of page s / 64 is slot s = 64 page + p % 64.
 *   kind    : GSDPA_CACHE_INT4 (integers -7 .. 7) or GSDPA_CACHE_E2M1 (4-bit floating
 *             point: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).
 *   k_exp, v_exp : -64 .. 64. Every 16 columns of a token's key (value) have a scale
 *             with 4 exponent and 3 mantissa bits (e4m3, up to 448): a code stands for
 *             code * scale * 2^k_exp (2^v_exp), which is exact in bfloat16. They put the
 *             data's largest magnitudes, over 6 or 7, below 448: larger ones are cut off
 *             there, groups whose largest magnitude is under 2^exp 2^-10 times 6 or 7 become
 *             zero.   d_k : 64 or 128.
 * Of one page and head, in bytes: key codes [64][d_k / 2], key scales [64][d_k / 16],
 * value codes [4][d_k / 64][8][4][4] words, value scales [4][4][d_k / 16] words. A key's
 * byte t d_k / 8 + 2 j + p (e2m1) holds columns 16 j + 4 t + 2 p and the one after it,
 * the first in the low 4 bits; int4 has bit 16 s + 4 (2 (j % 2) + p) of the 32-bit
 * word at t d_k / 8 + 4 (j / 2) for column 16 j + 4 t + 2 p + s, and code + 8. The value
 * word [n / 16][j / 4][g][t][j % 4] has columns 16 j + g (low 4 bits) and 16 j + 8 + g of
 * tokens n % 16 = 2 t, 2 t + 1, 2 t + 8, 2 t + 9 in bytes 0, 1, 2, 3 (e2m1) or 0, 2, 1, 3
 * (int4), the scale word [n / 16][t][j] their scales in bytes 0, 1, 2, 3.
 */
typedef enum { GSDPA_CACHE_INT4 = 0, GSDPA_CACHE_E2M1 = 1 } gsdpa_cache4_kind;
typedef struct {
    int kind, n_pages, H_kv, d_k, k_exp, v_exp;
    void* pool;
} gsdpa_cache4;

/*
 * The plan of a step: pages for the tokens that the requests bring, the block table
 * brought up to date, and for every token of the step, packed request after request,
 * its slot and position. Request b holds lens[b] tokens; it goes back to keep[b] of
 * them (drafts that were not accepted; 0 ends it) and then takes n_new[b] more.
 *   lens, n_new : device int32 [B].    keep : device int32 [B], or NULL for lens.
 *   table       : device int32 [B, max_pages], in and out: the pages of request b in
 *                 the order of its tokens. Entries past a request's pages mean nothing.
 *   free_pages  : device int32 [n_pages], n_free : device int32 [1]: the pages that no
 *                 request has, free_pages[0 .. n_free), last in first out. n_free_out,
 *                 device int32 [1], is what is left; it may be n_free.
 *   cu          : out, int32 [B + 1]: request b's tokens are rows cu[b] .. cu[b + 1].
 *   granted     : out, int32 [B]: n_new[b], or 0 where the pages did not suffice. Pages
 *                 are taken in the requests' order: a request gets its own if it needs
 *                 none or if the needs up to and with it fit what is free (pages given
 *                 back in this call among it, request after request, in order).
 *   slots       : out, int64 [n_rows], -1 for tokens that were not granted and rows from
 *                 cu[B] on.    positions : out, int32 [n_rows], keep and on, granted or not (0 from
 *                 cu[B] on, and where lens, keep or n_new is out of range), or NULL.
 * lens is not changed: set it to keep + granted once, after the last layer's attention
 * (until then keep is what the attention takes as lens). A request whose numbers are out of range
 * (negative, keep > lens, more than 64 max_pages tokens, rows past n_rows) is left as
 * it was, with granted 0 (a negative n_new has no rows), and the next
 * gsdpa_check_device_error returns GSDPA_ERR_CACHE_RANGE; so does a page number
 * outside the pool, whose tokens get slot -1 (one that is given back is reported then, and
 * goes on the stack as it is). B <= 8192 (GSDPA_ERR_UNSUPPORTED
 * otherwise). Repeated on the same contents it gives the same result, bit for bit.
 * Asynchronous on `stream`; sm_103 device; no workspace.
 */
GSDPA_API int gsdpa_pages_step(const int* lens, const int* keep, const int* n_new, int* table, int* free_pages,
                   const int* n_free, int* n_free_out, int* cu, int* granted, long long* slots, int* positions,
                   int B, int max_pages, int n_pages, int n_rows, void* stream);

/*
 * Writes keys and values of n_rows tokens to their slots.
 *   K, V  : device bf16 [n_rows, H_kv, d_k], heads contiguous, rows ld_k, ld_v elements
 *           apart (multiples of 8, >= H_kv d_k), 16-byte aligned.
 *   slots : device int64 [n_rows], different ones (of two equal ones either may be
 *           kept, or bytes of both); negative ones are passed over.
 * Every 16 columns of a token, with amax their largest |x| and top = 7 (int4) or 6
 * (e2m1): scale = e4m3 nearest to amax 2^-exp (1 / top), reciprocal and product rounded to
 * float32, ties to even, at most 448; code = x / (scale 2^exp) to nearest (the exact
 * quotient), ties to even, at most top (e2m1: zero with the sign of x). Scale 0: codes 0. A
 * group with a NaN or an infinity: scale NaN, codes 0 (every row that sees its token
 * becomes NaN). A token is rounded by itself: the contents do not depend on how tokens
 * were split over calls, and other tokens' bytes are left as they were. A slot past the
 * pool is passed over, and the next gsdpa_check_device_error returns
 * GSDPA_ERR_CACHE_RANGE. Asynchronous on `stream`; sm_103 device.
 */
GSDPA_API int gsdpa_cache4_append(const gsdpa_cache4* cache, const void* K, const void* V, long long ld_k,
                   long long ld_v, const long long* slots, int n_rows, void* stream);

/*
 * Reads keys and values back from slots, as the bfloat16 numbers that their codes
 * stand for, exactly: what gated_sdpa_fwd takes for a later piece of a prompt, whose
 * queries are too many for gated_sdpa_cache4. K, V : out, as for the append (rows
 * ld_k, ld_v elements apart); rows of negative slots are zero; a slot past the pool
 * gives a zero row and GSDPA_ERR_CACHE_RANGE from the next gsdpa_check_device_error.
 */
GSDPA_API int gsdpa_cache4_read(const gsdpa_cache4* cache, const long long* slots, void* K, void* V,
                   long long ld_k, long long ld_v, int n_rows, void* stream);

/*
 * The gated attention of a step's tokens against the cache through the block table,
 * after their keys and values have been appended. The step's tokens are packed:
 * request b has rows cu[b] .. cu[b + 1] of Q, X and O, and its row i sees its tokens
 * 0 .. lens[b] + i.
 *   Q, O  : device bf16 [n_rows, H_q, d_k]; O overlaps no input.   X : bf16 [n_rows, d_model].
 *   W_g   : as for gated_sdpa_fwd; gate_mode NONE, HEADWISE or ELEMENTWISE.
 *   table : device int32 [B, max_pages].   lens : device int32 [B], the tokens BEFORE
 *           this step.   cu : device int32 [B + 1].   n_new : device int32 [B] (the plan's
 *           granted), rows of a request that count, or NULL for all. Rows that
 *           do not count, and rows from cu[B] on, are zero.
 *   max_new : most rows of a request; (H_q / H_kv) max_new <= 128
 *           (GSDPA_ERR_UNSUPPORTED otherwise).
 * H_q a multiple of H_kv; d_model and the headwise gate's H_q multiples of 8. A request
 * whose numbers are out of range (cu decreasing or past n_rows, more than max_new rows,
 * more than 64 max_pages tokens) gives zero rows and GSDPA_ERR_CACHE_RANGE from the
 * next gsdpa_check_device_error; so does a page number outside the pool, and rows that
 * see one of its tokens become NaN. A page may be in several requests' tables. Tokens
 * past a request's end are not seen whatever their bytes; a NaN scale among the step's
 * own keys is seen by the rows that may see it, one among its values by every row of
 * the request.
 * Scores, softmax statistics and sums are float32; queries are exact (bf16; elements
 * under 2^-31 of the row's largest lose bits that weigh less than 2^-39 of it). Finite queries
 * have finite scores: where these would leave float32, the largest has all the weight. (A query
 * with infinities gives NaN, or zero if it makes all scores -infinity.) The
 * weights are rounded to fp16 twice, before and after they take the value's scale, 11 bits
 * each. fp16's range ends at 2^-38 W, W the row's largest product of a weight and a page's
 * largest value scale (rounded up to a power of two, at least 1): a weight is off by no
 * less than that, nor is its product with a scale.
 * workspace: gsdpa_cache4_workspace_bytes(...) bytes, 256-byte aligned; calls that
 * share one must not overlap on the device. Asynchronous on `stream`; other errors as
 * for gated_sdpa_fwd.
 */
GSDPA_API size_t gsdpa_cache4_workspace_bytes(const gsdpa_cache4* cache, int B, int max_pages, int n_rows, int max_new,
                   int d_model, int H_q, int gate_mode);
GSDPA_API int gated_sdpa_cache4(const void* X, const void* Q, const gsdpa_cache4* cache, const int* table,
                   const int* lens, const int* cu, const int* n_new, const void* W_g, void* O, int B, int max_pages,
                   int n_rows, int max_new, int d_model, int H_q, int gate_mode, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * Synchronises `stream`, then reads and clears the device error word that
 * bounded waits inside the kernels set when they run out, and the kernels of
 * the 8-bit and 4-bit caches when a sequence's length or token count, a slot or a
 * page number does not fit its cache. Returns GSDPA_OK, GSDPA_ERR_DEVICE_TIMEOUT, GSDPA_ERR_CACHE_RANGE (where
 * both have occurred the timeout, and the range error from the next call), or
 * GSDPA_ERR_LAUNCH if the stream itself reports a CUDA error.
 */
GSDPA_API int gsdpa_check_device_error(void* stream);

/* A static, human-readable name for a gsdpa_status value. */
GSDPA_API const char* gsdpa_status_string(int status);

/*
 * gated_sdpa_decode_noalloc -- the decode call (one query row per sequence,
 * L_q == 1) for callers that cannot allocate device memory. (The pages
 * describe no such entry point; it belongs to this library's interface only.)
 *
 * Some callers cannot hand the library a workspace: code that must never make
 * the device synchronise (cudaMalloc and cudaFree can), plugin or callback
 * hooks that provide no allocator, or processes with a device memory budget
 * fixed in advance. This entry point takes no workspace: its scratch (the
 * split-K partials, the gate-logit partials and the arrival counters) lives
 * in a 16 MiB array inside the library that every GPU loading the library
 * holds until the process exits (see gsdpa_decode_noalloc_max_scratch()).
 *
 *   Arguments are those of gated_sdpa_fwd with L_q = 1, causal, bf16 implied.
 *   Covered gate modes: GSDPA_GATE_NONE, GSDPA_GATE_HEADWISE and
 *   GSDPA_GATE_ELEMENTWISE (sigmoid gate); the head-shared and input-independent
 *   modes return GSDPA_ERR_UNSUPPORTED, values outside gsdpa_gate_mode
 *   GSDPA_ERR_INVALID_ARG. Covered shapes: d_k == 128 and H_q / H_kv a multiple
 *   of 4 (the dedicated decode kernel); others return GSDPA_ERR_UNSUPPORTED. A
 *   problem whose scratch exceeds the fixed array returns GSDPA_ERR_WORKSPACE
 *   (the size a problem needs is gsdpa_workspace_bytes(B, 1, L_k, ...,
 *   dtype = GSDPA_BF16)).
 *
 * The first call on a device resolves the array's device address (a runtime
 * query, no allocation); make that first call before any stream capture. The
 * address is kept for the life of the process: no call may follow a
 * cudaDeviceReset (or any reset of the device's primary context) in the same
 * process. The array is shared by all calls on a device and keeps the last
 * call's contents; counters are cleared at the start of each call. Calls that
 * overlap on the device race on the array: serialise them.
 */
GSDPA_API int gated_sdpa_decode_noalloc(const void* X, const void* Q, const void* K, const void* V,
                                        const void* W_g, void* O, float* sink,
                                        int B, int L_k, int d_model, int H_q, int H_kv, int d_k,
                                        int gate_mode, void* stream);

/* Size in bytes of the fixed scratch array used by gated_sdpa_decode_noalloc. */
GSDPA_API size_t gsdpa_decode_noalloc_max_scratch(void);

/*
 * Test hook, not part of the operation: sets the wait limit, in nanoseconds,
 * that every bounded wait inside the kernels uses from the next launch on
 * (0 restores the default of 2 s). Lets a test make a wait run out quickly.
 */
GSDPA_API int gsdpa_set_wait_limit_ns(unsigned long long ns);

/*
 * Diagnostic, not part of the operation: enqueues on `stream` one thread that
 * waits, with the current wait limit, on a barrier that nothing ever
 * completes. The wait gives up and records the timeout in the device error
 * word, which the next gsdpa_check_device_error() returns as
 * GSDPA_ERR_DEVICE_TIMEOUT (and clears). Lets a test exercise the bounded-wait
 * path without faulting or hanging the device. Returns GSDPA_OK or
 * GSDPA_ERR_LAUNCH.
 */
GSDPA_API int gsdpa_wait_self_test(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GSDPA_H_ */
