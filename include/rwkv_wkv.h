/*
 * rwkv_wkv.h — C ABI of the B200 (sm_100a) WKV operator library.
 *
 * The operator is RWKV's WKV:
 *
 *   RWKV-4 ("RWKV - Transformer 시대에 RNN을 재발명하다", Method / (2) Time-mixing
 *   (WKV); same formula in "RWKV: Reinventing RNNs for the Transformer Era",
 *   3. How It Works / The WKV Operator), per channel c:
 *
 *     wkv_t = ( Σ_{i<t} e^{-(t-1-i) w + k_i} v_i + e^{u + k_t} v_t )
 *           / ( Σ_{i<t} e^{-(t-1-i) w + k_i}     + e^{u + k_t} )
 *
 *   and its recurrent form with state (a_t, b_t):
 *     wkv_t = (a_{t-1} + e^{u+k_t} v_t) / (b_{t-1} + e^{u+k_t}),
 *     a_t = e^{-w} a_{t-1} + e^{k_t} v_t,   b_t = e^{-w} b_{t-1} + e^{k_t}.
 *
 *   Eagle / RWKV-5 ("RWKV-5 Eagle과 RWKV-6 Finch", section Eagle), per head:
 *     y_t = r_t · (s + diag(u) k_tᵀ v_t),   s ← diag(w) s + k_tᵀ v_t,
 *     w = exp(-exp(ω)),  s[i][j] with i = key index (row), j = value index.
 *
 *   Finch / RWKV-6 (same page, section Finch): the Eagle update with a
 *   data-dependent decay, w_t = exp(-exp(ω_t)) for every token t:
 *     y_t = r_t · (s + diag(u) k_tᵀ v_t),   s ← diag(w_t) s + k_tᵀ v_t.
 *
 * Conventions for every call
 *   - All tensor arguments are DEVICE pointers owned by the caller, on the
 *     current CUDA device; the library never allocates, frees or keeps them.
 *     Work is enqueued on `stream` (NULL = the legacy default stream) and the
 *     call returns without synchronising.  Inputs must stay valid and outputs
 *     untouched until the stream has run the work.
 *   - Layouts are dense row-major: WKV-4 k, v, y, gy, gk, gv are [B, T, C]
 *     (C fastest); w, u, gw, gu are [C] fp32.  WKV-5 r, k, v, y are
 *     [B, T, H, N] bf16; omega, u are [H, N] fp32; s is [B, H, N, N] fp32.
 *     Finch takes the same with omega [B, T, H, N] fp32 (step: [B, H, N]).
 *   - `w` (WKV-4) is the positive decay RATE of the formula above (the raw
 *     parameter mapped through -exp(.) by the model), not a factor.
 *   - WKV-4 state: [3, B, C] fp32 planes (a, b, p) meaning A = a·2^p,
 *     B = b·2^p (p an exponent of two).  A zero state is a = b = 0 (any p).
 *     Any finite (A, B) with A, B within fp32 range may be passed as (A, B, 0).
 *     The representation is not unique: compare states through a/b and
 *     log2(b) + p.
 *   - Returns RWKV_OK or an error status; nothing throws or aborts.
 *     Negative sizes or a NULL required pointer give RWKV_ERR_INVALID_ARG
 *     before anything is enqueued.  A launch failure gives RWKV_ERR_CUDA.
 *     Zero-sized problems are a successful no-op (T = 0 copies the state).
 *   - Values are data: no range validation; NaN and Inf propagate.
 *   - Alignment.  WKV-4 [B,T,C] tensors (k, v, y, gy, gk, gv, r, o, go, gr)
 *     whose bases are all 16-byte aligned, with C·sizeof(element) a multiple
 *     of 16, move through TMA; any other element-aligned bases or C take the
 *     plain-access instances of the same kernels (same results, fewer bytes
 *     in flight).  A pointer not aligned to its element size (4 bytes fp32,
 *     2 bytes bf16) gives RWKV_ERR_UNSUPPORTED.  The WKV-5/6 tensors r, k, v,
 *     y (and Finch's omega) must be 16-byte aligned (their rows are whole
 *     heads of 64), else RWKV_ERR_UNSUPPORTED; rwkv_wkv4_backward_noalloc
 *     keeps to the TMA conditions.
 */
#ifndef RWKV_WKV_H
#define RWKV_WKV_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define RWKV_API __attribute__((visibility("default")))
#else
#define RWKV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st *rwkv_stream_t;

typedef enum {
    RWKV_OK = 0,
    RWKV_ERR_INVALID_ARG = 1,    /* bad size, NULL required pointer, bad enum */
    RWKV_ERR_UNSUPPORTED = 2,    /* valid request this build does not handle */
    RWKV_ERR_WORKSPACE = 3,      /* workspace NULL or smaller than the query */
    RWKV_ERR_CUDA = 4,           /* a CUDA runtime call or launch failed */
    RWKV_ERR_DEVICE_TIMEOUT = 5  /* a kernel's bounded wait gave up */
} rwkv_status;

/* Element type of WKV-4 k, v, y, gy, gk, gv (arithmetic is fp32 either way). */
typedef enum { RWKV_F32 = 0, RWKV_BF16 = 1 } rwkv_dtype;

/* WKV-4 forward schedule.  SEQUENTIAL: one thread scans one channel over all
 * of T.  CHUNKED: time is cut into segments scanned in parallel from a zero
 * state, joined by an associative carry pass, then rescanned for outputs
 * (for problems with too few channels to fill the GPU).  AUTO picks. */
typedef enum { RWKV_ALGO_AUTO = 0, RWKV_ALGO_SEQUENTIAL = 1, RWKV_ALGO_CHUNKED = 2 } rwkv_algo;

/* Human-readable name of a status code (static string). */
RWKV_API const char *rwkv_status_string(rwkv_status s);

/* Library ABI version, (major << 16) | minor. */
RWKV_API int rwkv_version(void);

/* Number of WKV-4 checkpoints for T steps at interval chunk_len:
 * ceil(T / chunk_len); -1 if chunk_len is not a positive multiple of 16. */
RWKV_API int64_t rwkv_wkv4_num_checkpoints(int64_t T, int64_t chunk_len);

/* Workspace bytes rwkv_wkv4_forward needs for this shape and algo (0 if none). */
RWKV_API size_t rwkv_wkv4_forward_workspace_bytes(int64_t B, int64_t T, int64_t C, int algo);

/*
 * WKV-4 forward (time-parallel training form; the recurrent form gives the
 * same values).
 *   k, v      [B,T,C] dtype, read.           y [B,T,C] dtype, written.
 *   w, u      [C] fp32, read.
 *   state_in  [3,B,C] or NULL (zero state).  state_out [3,B,C] or NULL:
 *             the state after the last token; may equal state_in.
 *   ckpt      [num_checkpoints(T, chunk_len), 3, B, C] or NULL: ckpt[j] is
 *             the state before token j·chunk_len (ckpt[0] = state_in), in
 *             the state format, with p chosen at least ceil(k·log2 e) for
 *             every key of that chunk and b < 1; rwkv_wkv4_backward reads it
 *             and relies on that choice.  chunk_len must be 16 today.
 *   algo      rwkv_algo.   workspace: device scratch of
 *             rwkv_wkv4_forward_workspace_bytes() bytes (may be NULL if 0).
 */
RWKV_API rwkv_status rwkv_wkv4_forward(int64_t B, int64_t T, int64_t C, rwkv_dtype dtype,
                              const float *w, const float *u, const void *k, const void *v, void *y,
                              const float *state_in, float *state_out, float *ckpt, int64_t chunk_len,
                              int algo, void *workspace, size_t workspace_bytes, rwkv_stream_t stream);

/*
 * Receptance-gated WKV-4 forward: the time-mixing output of the same page,
 * o_t = W_o (σ(r_t) ⊙ WKV_t) ((2) and (4) Receptance Gating), without the
 * projection W_o (a GEMM outside the operator):
 *   o = σ(r) ⊙ WKV,   σ(x) = 1 / (1 + e^{-x}),
 * in one pass: the same arguments as rwkv_wkv4_forward plus
 *   r         [B,T,C] dtype, read (required);
 *   o         [B,T,C] dtype, written (required; replaces y).
 * state_out and ckpt are those of the ungated forward over the same k, v (the
 * gate does not enter the recurrence), so rwkv_wkv4_backward_gated reads the
 * same checkpoints.  Workspace: rwkv_wkv4_forward_workspace_bytes().
 */
RWKV_API rwkv_status rwkv_wkv4_forward_gated(int64_t B, int64_t T, int64_t C, rwkv_dtype dtype,
                                    const float *w, const float *u, const void *k, const void *v,
                                    const void *r, void *o, const float *state_in, float *state_out,
                                    float *ckpt, int64_t chunk_len, int algo, void *workspace,
                                    size_t workspace_bytes, rwkv_stream_t stream);

/* Workspace bytes rwkv_wkv4_backward needs; have_ckpt = 0 adds room to
 * recompute the checkpoints. */
RWKV_API size_t rwkv_wkv4_backward_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t chunk_len, int have_ckpt);

/*
 * WKV-4 backward: gradients of L = Σ gy·y with respect to k, v, w, u.
 * The pages print no backward; this is the derivative of the formula above.
 *   k, v, gy  [B,T,C] dtype, read.          gk, gv [B,T,C] dtype, written.
 *   gw, gu    [C] fp32, OVERWRITTEN with the sum over batch and time.
 *   state_in  the forward's initial state, or NULL (zero); used only when
 *             ckpt is NULL.
 *   ckpt      the checkpoints written by rwkv_wkv4_forward with the same
 *             inputs and chunk_len (16), or NULL to recompute them into the
 *             workspace.
 *   Deterministic: the same inputs give bit-identical outputs.
 */
RWKV_API rwkv_status rwkv_wkv4_backward(int64_t B, int64_t T, int64_t C, rwkv_dtype dtype,
                               const float *w, const float *u, const void *k, const void *v,
                               const void *gy, const float *state_in, const float *ckpt,
                               int64_t chunk_len, void *gk, void *gv, float *gw, float *gu,
                               void *workspace, size_t workspace_bytes, rwkv_stream_t stream);

/*
 * Backward of the receptance-gated forward: gradients of L = Σ go·o with
 * o = σ(r) ⊙ WKV.  The same arguments as rwkv_wkv4_backward with gy replaced
 * by r and go, plus gr:
 *   r, go     [B,T,C] dtype, read (required).
 *   gr        [B,T,C] dtype, written: go · WKV · σ(r)(1 - σ(r)).
 *   gk, gv, gw, gu as rwkv_wkv4_backward with gy = σ(r) ⊙ go.
 * Workspace: rwkv_wkv4_backward_workspace_bytes().  Deterministic.
 */
RWKV_API rwkv_status rwkv_wkv4_backward_gated(int64_t B, int64_t T, int64_t C, rwkv_dtype dtype,
                                     const float *w, const float *u, const void *k, const void *v,
                                     const void *r, const void *go, const float *state_in,
                                     const float *ckpt, int64_t chunk_len, void *gk, void *gv, void *gr,
                                     float *gw, float *gu, void *workspace, size_t workspace_bytes,
                                     rwkv_stream_t stream);

/*
 * WKV-4 recurrent decode: one token for each of B independent streams.
 *   k, v, y   [B,C] dtype.   w, u [C] fp32.
 *   state_in  [3,B,C] or NULL (zero).  state_out [3,B,C]; may equal
 *             state_in (in-place update).
 */
RWKV_API rwkv_status rwkv_wkv4_step(int64_t B, int64_t C, rwkv_dtype dtype, const float *w, const float *u,
                           const void *k, const void *v, void *y, const float *state_in,
                           float *state_out, rwkv_stream_t stream);

/* Workspace bytes rwkv_wkv5_forward needs (0 if none): with two or more 64-token chunks per head,
 * a 64 x 64 fp32 summary and a flag for each of up to 296 CTAs (the heads' chunks are dealt out
 * evenly to two CTAs per SM; a CTA whose chunks end inside a head publishes the state they reach
 * from a zero state, and the CTAs holding the rest of that head fold it into their start). */
RWKV_API size_t rwkv_wkv5_forward_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t N);

/*
 * Eagle / RWKV-5 multi-head matrix-state WKV forward.
 *   r, k, v   [B,T,H,N] bf16, read.      y [B,T,H,N] bf16, written.
 *   omega, u  [H,N] fp32 (w = exp(-exp(omega)) is formed inside).
 *   s_in      [B,H,N,N] fp32 or NULL (zero).  s_out [B,H,N,N] fp32 or NULL;
 *             may equal s_in.
 *   workspace device scratch of rwkv_wkv5_forward_workspace_bytes() bytes, 16-byte aligned
 *             (RWKV_ERR_WORKSPACE if NULL or smaller, RWKV_ERR_UNSUPPORTED if misaligned;
 *             may be NULL if the query gives 0).  Calls that share one workspace must be
 *             ordered (the same stream): it holds flags the kernel waits on.
 *   N must be 64 (RWKV_ERR_UNSUPPORTED otherwise).
 */
RWKV_API rwkv_status rwkv_wkv5_forward(int64_t B, int64_t T, int64_t H, int64_t N,
                              const void *r, const void *k, const void *v,
                              const float *omega, const float *u, void *y,
                              const float *s_in, float *s_out,
                              void *workspace, size_t workspace_bytes, rwkv_stream_t stream);

/* Workspace bytes rwkv_wkv5_backward needs (0 for an empty problem or N != 64). */
RWKV_API size_t rwkv_wkv5_backward_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t N);

/*
 * Eagle / RWKV-5 backward: gradients of L = Σ gy·y + Σ gs_out ∘ s_out for the
 * forward above ("RWKV-5 Eagle과 RWKV-6 Finch", section Eagle; the pages print
 * no backward, this is the chain rule through its recurrence).  With
 * G_T = gs_out and G_t = diag(w) G_{t+1} + r_tᵀ gy_t (the gradient of the
 * state after token t-1):
 *   gr_t = s_t gy_tᵀ + u ⊙ k_t (v_t·gy_t),   gk_t = G_{t+1} v_tᵀ + u ⊙ r_t (v_t·gy_t),
 *   gv_t = G_{t+1}ᵀ k_t + (Σ r_t u k_t) gy_t,  gs_in = G_0,
 *   gomega_d = Σ_{b,t} (Σ_j G_{t+1}[d][j] s_t[d][j]) · dw_d/dω_d,  gu_d = Σ_{b,t} r_t[d] k_t[d] (v_t·gy_t).
 *   r, k, v, gy   [B,T,H,N] bf16, read.      gr, gk, gv [B,T,H,N] bf16, written.
 *   omega, u      [H,N] fp32, read.          gomega, gu [H,N] fp32, OVERWRITTEN with the sums over
 *                                            batch and time.
 *   s_in          [B,H,N,N] fp32, the forward's initial state, or NULL (zero).
 *   gs_out        [B,H,N,N] fp32, the gradient of the final state, or NULL (zero).
 *   gs_in         [B,H,N,N] fp32, written with the gradient of s_in, or NULL (not wanted).
 *   workspace     device scratch of rwkv_wkv5_backward_workspace_bytes() bytes (the forward
 *                 states at every 64th token, per-row sums).
 *   N must be 64; the [B,T,H,N] tensors 16-byte aligned (RWKV_ERR_UNSUPPORTED otherwise).
 *   Any decay w in [0, 1]: channels decaying faster than exp(omega) = 2
 *   (w < 0.135) are summed over lags up to 15 where the rest stays on the
 *   chunked tensor-core form.  The reversed forward pass (gv, gs_in) runs on an
 *   internal non-blocking stream per device, ordered after and before the
 *   caller's stream with events (capture-safe once a first call has made it).
 *   Deterministic.
 */
RWKV_API rwkv_status rwkv_wkv5_backward(int64_t B, int64_t T, int64_t H, int64_t N, const void *r, const void *k,
                               const void *v, const float *omega, const float *u, const float *s_in,
                               const void *gy, const float *gs_out, void *gr, void *gk, void *gv,
                               float *gomega, float *gu, float *gs_in, void *workspace, size_t workspace_bytes,
                               rwkv_stream_t stream);

/*
 * Eagle / RWKV-5 recurrent decode: one token for each of B independent
 * streams ("RWKV-5 Eagle과 RWKV-6 Finch", section Eagle): per head,
 *   y = r·(s + diag(u)·kᵀv),   then   s <- diag(w)·s + kᵀv,  w = exp(-exp(ω)),
 * which is rwkv_wkv5_forward with T = 1.
 *   r, k, v, y  [B,H,N] bf16 (the token of every stream and head).
 *   omega, u    [H,N] fp32.
 *   s_in        [B,H,N,N] fp32, or NULL (zero state).
 *   s_out       [B,H,N,N] fp32, required; may equal s_in (in-place update).
 *   N must be 64 (RWKV_ERR_UNSUPPORTED otherwise); s_in and s_out must be
 *   16-byte aligned (RWKV_ERR_UNSUPPORTED otherwise).
 */
RWKV_API rwkv_status rwkv_wkv5_step(int64_t B, int64_t H, int64_t N, const void *r, const void *k,
                           const void *v, const float *omega, const float *u, void *y,
                           const float *s_in, float *s_out, rwkv_stream_t stream);

/* Workspace bytes rwkv_wkv6_forward needs (0 if none). */
RWKV_API size_t rwkv_wkv6_forward_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t N);

/*
 * Finch / RWKV-6 multi-head matrix-state WKV forward with a per-token decay
 * ("RWKV-5 Eagle과 RWKV-6 Finch", section Finch: Eagle's recurrence with the
 * decay made data dependent).  Per head, for t = 0 .. T-1:
 *   y_t = r_t · (s + diag(u) k_tᵀ v_t),   then   s <- diag(w_t) s + k_tᵀ v_t,
 *   w_t = exp(-exp(omega_t)),
 * so token i < t reaches token t decayed by w_{i+1} ⋯ w_{t-1}.
 *   r, k, v   [B,T,H,N] bf16, read.      y [B,T,H,N] bf16, written.
 *   omega     [B,T,H,N] fp32 (one value per token and channel), read.
 *   u         [H,N] fp32.
 *   s_in      [B,H,N,N] fp32 or NULL (zero).  s_out [B,H,N,N] fp32 or NULL;
 *             may equal s_in.
 *   N must be 64 (RWKV_ERR_UNSUPPORTED otherwise); omega follows the
 *   alignment rule of the [B,T,.] tensors.
 */
RWKV_API rwkv_status rwkv_wkv6_forward(int64_t B, int64_t T, int64_t H, int64_t N,
                              const void *r, const void *k, const void *v,
                              const float *omega, const float *u, void *y,
                              const float *s_in, float *s_out,
                              void *workspace, size_t workspace_bytes, rwkv_stream_t stream);

/*
 * Finch / RWKV-6 recurrent decode: one token for each of B independent
 * streams, rwkv_wkv6_forward with T = 1.
 *   r, k, v, y  [B,H,N] bf16.   omega [B,H,N] fp32 (this token's decay).
 *   u           [H,N] fp32.
 *   s_in        [B,H,N,N] fp32, or NULL (zero state).
 *   s_out       [B,H,N,N] fp32, required; may equal s_in (in-place update).
 *   N must be 64; s_in and s_out must be 16-byte aligned
 *   (RWKV_ERR_UNSUPPORTED otherwise).
 */
RWKV_API rwkv_status rwkv_wkv6_step(int64_t B, int64_t H, int64_t N, const void *r, const void *k,
                           const void *v, const float *omega, const float *u, void *y,
                           const float *s_in, float *s_out, rwkv_stream_t stream);

/* Workspace bytes rwkv_wkv6_backward needs (0 for an empty problem or N != 64). */
RWKV_API size_t rwkv_wkv6_backward_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t N);

/*
 * Finch / RWKV-6 backward: gradients of L = Σ gy·y + Σ gs_out ∘ s_out for
 * rwkv_wkv6_forward ("RWKV-5 Eagle과 RWKV-6 Finch", section Finch; the pages
 * print no backward, this is the chain rule through its recurrence).  With s_t
 * the state before token t, G_T = gs_out and G_t = diag(w_t) G_{t+1} + r_tᵀ gy_t:
 *   gr_t = s_t gy_tᵀ + u ⊙ k_t (v_t·gy_t),   gk_t = G_{t+1} v_tᵀ + u ⊙ r_t (v_t·gy_t),
 *   gv_t = G_{t+1}ᵀ k_t + (Σ r_t u k_t) gy_t,  gs_in = G_0,
 *   gomega_t[d] = (Σ_j G_{t+1}[d][j] s_t[d][j]) · dw_t[d]/dω_t[d]   (dw/dω = -e^ω w),
 *   gu_d = Σ_{b,t} r_t[d] k_t[d] (v_t·gy_t).
 *   r, k, v, gy   [B,T,H,N] bf16, read.      gr, gk, gv [B,T,H,N] bf16, written.
 *   omega         [B,T,H,N] fp32, read.      gomega [B,T,H,N] fp32, written (one value per
 *                                            token and channel, as omega).
 *   u             [H,N] fp32, read.          gu [H,N] fp32, OVERWRITTEN with the sum over
 *                                            batch and time.
 *   s_in          [B,H,N,N] fp32, the forward's initial state, or NULL (zero).
 *   gs_out        [B,H,N,N] fp32, the gradient of the final state, or NULL (zero).
 *   gs_in         [B,H,N,N] fp32, written with the gradient of s_in, or NULL (not wanted).
 *   workspace     device scratch of rwkv_wkv6_backward_workspace_bytes() bytes (the forward
 *                 states at every 64th token, per-CTA scratch, the gu parts);
 *                 RWKV_ERR_WORKSPACE if smaller.
 *   N must be 64 and every tensor 16-byte aligned, and B·H·ceil(T/64) (one CTA per
 *   64-token chunk) and 2·B·H (two per head for the boundary scans) at most 2^31 - 1
 *   (RWKV_ERR_UNSUPPORTED otherwise).
 *   Any decay w in [0, 1]: the recurrence runs token by token on the CUDA cores,
 *   so no factorization range applies.  Deterministic (gu is reduced in a fixed
 *   order).  Runs on `stream` only; allocates nothing.
 */
RWKV_API rwkv_status rwkv_wkv6_backward(int64_t B, int64_t T, int64_t H, int64_t N, const void *r, const void *k,
                               const void *v, const float *omega, const float *u, const float *s_in,
                               const void *gy, const float *gs_out, void *gr, void *gk, void *gv,
                               float *gomega, float *gu, float *gs_in, void *workspace, size_t workspace_bytes,
                               rwkv_stream_t stream);

/* ---------------------------------------------------------------------------
 * The operators around the recurrence: a short causal convolution, a selective
 * state space scan and the layer norm.  The conventions above hold (device
 * pointers, caller-owned memory, no synchronisation, status codes, zero-sized
 * problems are a no-op), and:
 *   - dtype (fp32 or bf16) is the element type of the activations and their
 *     gradients; parameters, their gradients and the scan's states are fp32.
 *     Arithmetic and sums are fp32, each output is rounded once.
 *   - `ld*` is the distance in elements between the rows of an input (one row
 *     per token: element (b, t, c) of x is x[(b T + t) ldx + c]), at least the
 *     row's length, so that a part of a wider tensor can be passed without a
 *     copy.  Tensors without an ld are dense.
 *   - Pointers aligned to their element size are served; where every base is
 *     16-byte aligned and every row length and ld a multiple of 16 bytes the
 *     accesses are wide.  The scan's states and checkpoints and every workspace must be
 *     16-byte aligned (RWKV_ERR_UNSUPPORTED otherwise).
 *   - Outputs must not overlap inputs or one another, except where a call says
 *     that a state may be updated in place.
 *   - A workspace belongs to one call until the stream has run it: calls that
 *     may overlap (other streams, graphs replayed together) need their own.
 *   - Deterministic: no atomics, sums in a fixed order.
 *   - Sizes whose launches would pass 2^31 - 1 blocks give RWKV_ERR_UNSUPPORTED, and so do T above
 *     2^31 - 65 and C above 2^31 - 129 (the convolution and the scan).
 * ------------------------------------------------------------------------- */

/* Activation behind the causal convolution: none, or silu(p) = p / (1 + e^{-p}). */
typedef enum { RWKV_ACT_NONE = 0, RWKV_ACT_SILU = 1 } rwkv_act;

/*
 * Causal convolution over time, one filter of W taps (2, 3 or 4;
 * RWKV_ERR_UNSUPPORTED otherwise) per channel:
 *   y_t[c] = act(bias[c] + sum_{j<W} weight[c][j] x_{t-W+1+j}[c]).
 * The token shift mu x_t + (1 - mu) x_{t-1} is W = 2 with weight (1 - mu, mu).
 *   weight    [C,W] fp32.   bias [C] fp32 or NULL (zero).
 *   x         [B,T,C] dtype, rows ldx apart.   y [B,T,C] dtype, written.
 *   state_in  [B,W-1,C] dtype: the W-1 tokens before the first, oldest first,
 *             or NULL (zeros).   state_out [B,W-1,C] or NULL: the last W-1
 *             tokens (of state_in too, when T < W-1); may equal state_in.
 */
RWKV_API rwkv_status rwkv_causal_conv_forward(int64_t B, int64_t T, int64_t C, int64_t W, rwkv_dtype dtype,
                                     const float *weight, const float *bias, int act, const void *x,
                                     int64_t ldx, void *y, const void *state_in, void *state_out,
                                     rwkv_stream_t stream);

/* Workspace bytes rwkv_causal_conv_backward needs (0 for an empty problem). */
RWKV_API size_t rwkv_causal_conv_backward_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t W);

/*
 * Backward of the causal convolution for L = sum gy y + sum gstate_out state_out;
 * with g_t = gy_t act'(pre_t) (pre is formed again from x):
 *   gx_t = sum_j weight[.][j] g_{t+W-1-j} (+ gstate_out's row of that token),
 *   gweight[c][j] = sum_{b,t} g_t x_{t-W+1+j},   gbias = sum_{b,t} g_t.
 *   gy        [B,T,C] dtype.   gstate_out [B,W-1,C] dtype or NULL (zero).
 *   gx        [B,T,C] dtype, written.
 *   gweight   [C,W], gbias [C] fp32, OVERWRITTEN; gbias may be NULL (not wanted).
 *   gstate_in [B,W-1,C] dtype, written, or NULL (not wanted).
 */
RWKV_API rwkv_status rwkv_causal_conv_backward(int64_t B, int64_t T, int64_t C, int64_t W, rwkv_dtype dtype,
                                      const float *weight, const float *bias, int act, const void *x,
                                      int64_t ldx, const void *state_in, const void *gy,
                                      const void *gstate_out, void *gx, float *gweight, float *gbias,
                                      void *gstate_in, void *workspace, size_t workspace_bytes,
                                      rwkv_stream_t stream);

/* One token for each of B streams: rwkv_causal_conv_forward with T = 1.  x [B,C] (rows ldx apart),
 * y [B,C], state_in [B,W-1,C] or NULL (zeros), state_out required; may equal state_in. */
RWKV_API rwkv_status rwkv_causal_conv_step(int64_t B, int64_t C, int64_t W, rwkv_dtype dtype, const float *weight,
                                  const float *bias, int act, const void *x, int64_t ldx, void *y,
                                  const void *state_in, void *state_out, rwkv_stream_t stream);

/* Workspace bytes rwkv_selective_scan_forward needs for this shape and algo (0 if none). */
RWKV_API size_t rwkv_selective_scan_forward_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t N, int algo);

/*
 * Selective scan forward: a recurrence with a diagonal state of N values per
 * channel, whose step size, input and output weights come from the tokens.
 *   D_t = log(1 + exp(dt_t + dt_bias)),   A = -exp(a_log),
 *   h_t[c][n] = exp(D_t[c] A[c][n]) h_{t-1}[c][n] + D_t[c] x_t[c] b_t[n],
 *   p_t[c] = sum_n c_t[n] h_t[c][n] + d[c] x_t[c],
 *   y_t = p_t, or with a gate z: y_t = p_t z_t / (1 + e^{-z_t}).
 *   a_log     [C,N] fp32.   d, dt_bias [C] fp32 or NULL (zero).
 *   x, dt     [B,T,C] dtype.   b, c [B,T,N] dtype.   z [B,T,C] dtype or NULL (no gate; ldz unused).
 *   y         [B,T,C] dtype, written, or NULL (states only).
 *   h_in      [B,C,N] fp32 or NULL (zero).   h_out [B,C,N] or NULL; may equal h_in.
 *   ckpt      [ceil(T/chunk_len),B,C,N] fp32 or NULL: ckpt[j] is the state before token
 *             j chunk_len (ckpt[0] = h_in), for the backward.  chunk_len must be 16 today.
 *   algo      rwkv_algo: CHUNKED cuts time into segments that run in parallel (for few channels and
 *             long sequences); needs the workspace.
 *   N         8, 16, 32 or 64 (RWKV_ERR_UNSUPPORTED otherwise).
 */
RWKV_API rwkv_status rwkv_selective_scan_forward(int64_t B, int64_t T, int64_t C, int64_t N, rwkv_dtype dtype,
                                        const float *a_log, const float *d, const float *dt_bias,
                                        const void *x, int64_t ldx, const void *dt, int64_t lddt,
                                        const void *b, int64_t ldb, const void *c, int64_t ldc,
                                        const void *z, int64_t ldz, void *y, const float *h_in,
                                        float *h_out, float *ckpt, int64_t chunk_len, int algo,
                                        void *workspace, size_t workspace_bytes, rwkv_stream_t stream);

/* Workspace bytes rwkv_selective_scan_backward needs (0 for an empty problem); have_ckpt = 0 adds
 * room to form the checkpoints again. */
RWKV_API size_t rwkv_selective_scan_backward_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t N,
                                                    int64_t chunk_len, int have_ckpt);

/*
 * Backward of the selective scan for L = sum gy y + sum gh_out h_out.  With g_t = gy_t silu(z_t)
 * (gy_t without a gate), e_t = exp(D_t A), G_t = c_t g_t + e_{t+1} G_{t+1} (gh_out behind the end):
 *   gc_t[n] = sum_c g_t h_t[.][n],   gb_t[n] = sum_c G_t[.][n] D_t x_t,
 *   s1 = sum_n G_t b_t,   q_t = G_t e_t h_{t-1},
 *   gx_t = D_t s1 + d g_t,   gdt_t = (x_t s1 + sum_n q_t A) / (1 + e^{-(dt_t + dt_bias)}),
 *   gdt_bias = sum_{b,t} gdt_t,   ga_log = A sum_{b,t} q_t D_t,   gd = sum_{b,t} g_t x_t,
 *   gz_t = gy_t p_t silu'(z_t),   gh_in = e_0 G_0.
 *   gy        [B,T,C] dtype.   h_in the forward's (used only when ckpt is NULL).
 *   gh_out    [B,C,N] fp32 or NULL (zero).
 *   ckpt      the forward's checkpoints (same inputs, chunk_len 16), or NULL to form them again in
 *             the workspace.
 *   gx, gdt   [B,T,C] dtype, gb, gc [B,T,N] dtype, written.   gz [B,T,C] dtype, required with z.
 *   ga_log    [C,N], gd, gdt_bias [C] fp32, OVERWRITTEN; gd and gdt_bias may be NULL (not wanted).
 *   gh_in     [B,C,N] fp32 or NULL (not wanted); may equal gh_out.
 */
RWKV_API rwkv_status rwkv_selective_scan_backward(int64_t B, int64_t T, int64_t C, int64_t N, rwkv_dtype dtype,
                                         const float *a_log, const float *d, const float *dt_bias,
                                         const void *x, int64_t ldx, const void *dt, int64_t lddt,
                                         const void *b, int64_t ldb, const void *c, int64_t ldc,
                                         const void *z, int64_t ldz, const void *gy, const float *h_in,
                                         const float *gh_out, const float *ckpt, int64_t chunk_len, void *gx,
                                         void *gdt, void *gb, void *gc, void *gz, float *ga_log, float *gd,
                                         float *gdt_bias, float *gh_in, void *workspace,
                                         size_t workspace_bytes, rwkv_stream_t stream);

/* One token for each of B streams: rwkv_selective_scan_forward with T = 1.  x, dt, z [B,C] and
 * b, c [B,N] (rows ld* apart), y [B,C]; h_in [B,C,N] or NULL (zero), h_out required; may equal
 * h_in. */
RWKV_API rwkv_status rwkv_selective_scan_step(int64_t B, int64_t C, int64_t N, rwkv_dtype dtype, const float *a_log,
                                     const float *d, const float *dt_bias, const void *x, int64_t ldx,
                                     const void *dt, int64_t lddt, const void *b, int64_t ldb,
                                     const void *c, int64_t ldc, const void *z, int64_t ldz, void *y,
                                     const float *h_in, float *h_out, rwkv_stream_t stream);

/*
 * Layer norm over the N columns of each of G groups of M rows, with an optional gate:
 *   xh = (x - mean x) / sqrt(var x + eps),   l = xh weight + bias,
 *   y = l, or with a gate: y = l gate / (1 + e^{-gate}).
 * var is the mean of (x - mean)^2.  G = 1 is the norm in front of a block's mixers; G = H, N = 64
 * with a gate is the head-wise norm and SiLU gate behind the Eagle and Finch operators, on their
 * y [B,T,H,N] with M = B T.
 *   x, gate, y   [M,G,N] dtype; gate may be NULL; y may equal neither.
 *   weight, bias [G,N] fp32; bias may be NULL (zero).
 *   eps          >= 0 and finite (RWKV_ERR_INVALID_ARG otherwise); G N at most 2^30 - 1.
 */
RWKV_API rwkv_status rwkv_layer_norm_forward(int64_t M, int64_t G, int64_t N, rwkv_dtype dtype, const float *weight,
                                    const float *bias, float eps, const void *x, const void *gate,
                                    void *y, rwkv_stream_t stream);

/* Workspace bytes rwkv_layer_norm_backward needs (0 for an empty problem). */
RWKV_API size_t rwkv_layer_norm_backward_workspace_bytes(int64_t M, int64_t G, int64_t N, rwkv_dtype dtype);

/*
 * Backward of the layer norm for L = sum gy y.  With g = gy silu(gate) (gy without a gate) and
 * u = g weight, per row and group:
 *   gx = (u - mean u - xh mean(u xh)) / sqrt(var x + eps),
 *   gweight = sum_rows g xh,   gbias = sum_rows g,   ggate = gy l silu'(gate).
 *   gx, ggate    [M,G,N] dtype, written; ggate required with gate.
 *   gweight, gbias [G,N] fp32, OVERWRITTEN; gbias may be NULL (not wanted).
 */
RWKV_API rwkv_status rwkv_layer_norm_backward(int64_t M, int64_t G, int64_t N, rwkv_dtype dtype, const float *weight,
                                     const float *bias, float eps, const void *x, const void *gate,
                                     const void *gy, void *gx, void *ggate, float *gweight,
                                     float *gbias, void *workspace, size_t workspace_bytes,
                                     rwkv_stream_t stream);

/* Largest B * C that rwkv_wkv4_backward_noalloc accepts. */
#define RWKV_NOALLOC_MAX_LANES 262144

/*
 * WKV-4 backward that allocates nothing and needs no workspace.
 * The pages have no counterpart: this is a library convenience for callers
 * that cannot allocate device memory where they run the backward (device
 * memory owned in full by another allocator, latency-critical loops that
 * must not pay cudaMalloc's implicit synchronisation, systems that allocate
 * only at start-up).  Same arguments and results as rwkv_wkv4_backward with
 * ckpt required (the forward's checkpoints), no workspace, and the TMA
 * alignment (16-byte bases, C·sizeof(element) a multiple of 16; else
 * RWKV_ERR_UNSUPPORTED); the per-lane
 * scratch lives in a fixed array inside the library (RWKV_NOALLOC_MAX_LANES
 * lanes, 4 MiB, held on every GPU that loads the library until exit).
 *   - B * C > RWKV_NOALLOC_MAX_LANES returns RWKV_ERR_WORKSPACE (too big for
 *     the fixed scratch); ckpt == NULL returns RWKV_ERR_INVALID_ARG.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current and caches it for the
 *     device's current context; the first call after that context is
 *     replaced (cudaDeviceReset) looks it up again.  Make the first call on
 *     a device before any stream capture.
 *   - All calls share the array: calls whose GPU work overlaps (other
 *     streams, other threads) race and must be ordered by the caller.
 *   - Calls no cudaMalloc, cudaFree or allocating library routine.
 */
RWKV_API rwkv_status rwkv_wkv4_backward_noalloc(int64_t B, int64_t T, int64_t C, rwkv_dtype dtype,
                                                const float *w, const float *u, const void *k,
                                                const void *v, const void *gy, const float *ckpt,
                                                int64_t chunk_len, void *gk, void *gv, float *gw,
                                                float *gu, rwkv_stream_t stream);

/*
 * Synchronises `stream`, then reports and clears the device error word that
 * kernels set when a bounded wait gives up (RWKV_ERR_DEVICE_TIMEOUT), or
 * RWKV_ERR_CUDA if the stream itself failed.
 * The error word is one per device and process, shared by every call on that
 * device whatever its stream or host thread: a timeout in work on one stream
 * is reported to (and cleared by) the first caller that checks, on any
 * stream.  Callers that run the library from several streams and need to
 * know which call timed out must check after each call, in stream order.
 */
RWKV_API rwkv_status rwkv_check_device_error(rwkv_stream_t stream);

/*
 * Test hooks for the failure path of the bounded waits (the pages have no
 * counterpart; they exist so that a test can watch a wait give up without
 * faulting or hanging the GPU).  Both act on the current device, synchronise
 * it first, and hold until changed; they are not meant for production use.
 *
 * rwkv_debug_set_wait_limit_ns: how long every bounded wait of the library's
 *   kernels polls before giving up (it then sets RWKV_ERR_DEVICE_TIMEOUT in
 *   the device error word and the CTA leaves at its next barrier, after
 *   waiting, bounded again, for the copies and MMAs it had issued).  ns = 0
 *   restores the default of one second.
 * rwkv_debug_withhold_loads: on != 0 makes the thread that issues a kernel's
 *   TMA loads arm its barrier and issue none, so the first wait of every CTA
 *   runs out with nothing in flight; on = 0 restores normal operation.
 *   Calls return RWKV_OK meanwhile and their outputs are undefined.
 */
RWKV_API rwkv_status rwkv_debug_set_wait_limit_ns(uint64_t ns);
RWKV_API rwkv_status rwkv_debug_withhold_loads(int on);

#ifdef __cplusplus
}
#endif

#endif /* RWKV_WKV_H */
