/*
 * kdn.h -- C ABI of libkdn, the B200 (sm_100a) Kalman Delta Network layer.
 *
 * The model (from "Kalman Delta Networks: Uncertainty-aware Associative
 * Memory", abstract, and "Kalman Delta Networks: 不确定性感知的联想记忆",
 * 方法): per batch element b and head h the memory S (d_v x d_k) is the
 * latent state of a linear-Gaussian model, S_t = a_t S_{t-1} + noise(w_t)
 * and v_t = S_t k_t + noise(r_t).  Each token predicts, then writes the
 * residual v_t - a_t S_{t-1} k_t with the Kalman gain g_t, then reads
 * o_t = S_t q_t.  The uncertainty is one variance per head (Isotropic KDN)
 * or per key dimension (Diagonal KDN); both follow the Mobius map
 *     p_t = (r a^2 p_{t-1} + r w) / (c a^2 p_{t-1} + r + c w)
 * with c = info_scale * ||k_t||^2 (iso) or c = k_{t,i}^2 (diag).
 *
 * Conventions for every call:
 *   - Pointers are caller-owned.  Device pointers unless stated otherwise
 *     (CUDA device memory of the current device, e.g. PyTorch tensors).  The
 *     library never allocates device memory; calls that need scratch take a
 *     caller-provided workspace whose size the matching *_workspace_size()
 *     returns.
 *   - All arrays are dense, row-major, with the last index fastest.
 *   - stream is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     Every call only enqueues work on it and never synchronises the host,
 *     except kdn_read_workspace_status().
 *   - Arguments are checked before anything is enqueued.  A call that returns
 *     anything but KDN_OK has enqueued nothing.  No C++ exception crosses
 *     this interface.
 *   - Floating-point state (a, w, r, S, p, o) is always fp32.  q, k, v are
 *     fp32 or bf16 (in_dtype).  The output o is fp32: the bf16 rounding of an
 *     exact output alone exceeds the layer's error bound (max-abs / RMS
 *     <= 2e-2) for outputs whose max is ~10x their RMS.
 */
#ifndef KDN_H_
#define KDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kdn_status {
  KDN_OK = 0,
  KDN_ERR_INVALID_ARG = 1,  /* null / misaligned pointer, bad size or enum  */
  KDN_ERR_UNSUPPORTED = 2,  /* valid but not implemented (shape, path)      */
  KDN_ERR_WORKSPACE = 3,    /* workspace missing or smaller than required   */
  KDN_ERR_TIMEOUT = 4,      /* a bounded on-device wait gave up             */
  KDN_ERR_CUDA = 5          /* the CUDA runtime reported an error           */
} kdn_status;

/* KDN_E4M3 (8 bits, with fp32 scales: see kdn_fp8_quantize) is an output type
 * of kdn_rmsnorm_forward only; every other dtype argument takes the first two. */
typedef enum kdn_dtype { KDN_F32 = 0, KDN_BF16 = 1, KDN_E4M3 = 2 } kdn_dtype;
typedef enum kdn_variant { KDN_ISO = 0, KDN_DIAG = 1 } kdn_variant;

/* Forward-path selector (the `chunk` argument of the forward calls). */
enum {
  KDN_CHUNK_AUTO = 0,       /* chunked engine when supported, else recurrent */
  KDN_CHUNK_RECURRENT = 1,  /* token-by-token kernel, any supported shape    */
  KDN_CHUNK_64 = 64         /* chunkwise tensor-core engine, 64-token chunks */
};

/* Human-readable name of a status code (static storage, never NULL). */
const char* kdn_status_string(kdn_status status);

/* Library version, major*10000 + minor*100 + patch (0.2.0: adds the packed,
 * host-buffer, backward, dense-filter and KLA entry points; 0.3.0: the gated
 * linear recurrence, the residual RMS norm and the 8-bit projections). */
int kdn_version(void);

/* ------------------------------------------------------------------------
 * kdn_mobius_scan -- the uncertainty recursion alone, over N independent
 * lanes of length T ("Kalman Delta Networks: Uncertainty-aware Associative
 * Memory", abstract: the variance recursions are Mobius maps composed by an
 * associative scan; "Kalman Linear Attention ...", 方法论 §2 prints the
 * fractional-linear form).  For every lane i and step t:
 *     c          = info_scale * n[i,t]
 *     prior[i,t] = a^2 lambda[i,t-1] + w
 *     lambda[i,t]= (r a^2 lambda[i,t-1] + r w) / (c a^2 lambda[i,t-1] + r + c w)
 *     gain[i,t]  = prior / (prior * n + r)     (the isotropic write strength)
 * with lambda[i,-1] = lambda0[i] (or 1 when lambda0 is NULL).
 *
 * a, w, r, n     [N, T] fp32 device; n is the squared key norm (or k_i^2)
 * lambda0        [N] fp32 device, or NULL for all ones
 * info_scale     c = info_scale * n; must be finite and >= 0
 * lambda_out     [N, T] fp32 device, posterior variances (required)
 * prior_out      [N, T] fp32 device or NULL
 * gain_out       [N, T] fp32 device or NULL
 * workspace      device scratch of >= kdn_mobius_scan_workspace_size(N, T)
 *                bytes, 256-byte aligned; its contents are overwritten
 *                (the call clears what it needs on the stream first)
 * Requires a, w, r, n, lambda_out (and prior_out / gain_out when given) to be
 * 16-byte aligned; any T >= 1 and N >= 1 with N*T < 2^40.
 * Errors: KDN_ERR_INVALID_ARG, KDN_ERR_WORKSPACE, KDN_ERR_CUDA.  A look-back
 * wait that gives up (it cannot in correct use) is recorded in the workspace
 * and reported by kdn_read_workspace_status().
 * ---------------------------------------------------------------------- */
size_t kdn_mobius_scan_workspace_size(int64_t N, int64_t T);
kdn_status kdn_mobius_scan(const float* a, const float* w, const float* r,
                           const float* n, const float* lambda0,
                           float info_scale, float* lambda_out,
                           float* prior_out, float* gain_out, int64_t N,
                           int64_t T, void* workspace, size_t workspace_bytes,
                           void* stream);

/* ------------------------------------------------------------------------
 * kdn_mobius_scan_noalloc -- kdn_mobius_scan without a workspace argument,
 * for callers that cannot allocate device memory where they call the scan
 * (for example a host program that gives all device memory to its own pool
 * at start-up and permits no cudaMalloc afterwards, or a plug-in that such a
 * host hands only its input and output buffers).  The pages have no
 * counterpart of this entry point; it only changes where scratch lives.
 *
 * The scratch is a fixed array of about 7.9 MiB inside the library's device
 * code.  Every GPU that loads the library holds it until the process exits.
 * Limit: N * ceil(T / 2048) <= KDN_SCAN_NOALLOC_MAX_TILES (e.g. 4096 lanes
 * up to T = 114688); larger calls return KDN_ERR_WORKSPACE without enqueuing
 * anything.  The call allocates nothing.  Every call looks up the array's
 * device address in the caller's current device and context (the lookup
 * allocates nothing), so the address stays right across context switches
 * and device resets.  The first call in a context also loads the library's
 * device code there: make that first call before any stream capture.  Every
 * call clears the part of the array that must start at zero on `stream`
 * before its kernel.  All calls share the one array: calls whose work
 * overlaps on the GPU (for example on two streams without ordering between
 * them) race and give wrong results, so order them.  A look-back wait that
 * gives up (after 1 s, which only a stalled GPU reaches) is recorded only in
 * that internal array and is not reported by this entry point; callers that
 * must detect it use kdn_mobius_scan with a workspace and
 * kdn_read_workspace_status.  Otherwise the arguments, results and errors
 * are those of kdn_mobius_scan.
 * ---------------------------------------------------------------------- */
#define KDN_SCAN_NOALLOC_MAX_TILES 229376
kdn_status kdn_mobius_scan_noalloc(const float* a, const float* w,
                                   const float* r, const float* n,
                                   const float* lambda0, float info_scale,
                                   float* lambda_out, float* prior_out,
                                   float* gain_out, int64_t N, int64_t T,
                                   void* stream);

/* ------------------------------------------------------------------------
 * kdn_iso_forward -- Isotropic KDN layer forward ("Kalman Delta Networks:
 * Uncertainty-aware Associative Memory", abstract: one uncertainty scalar
 * per head; "Kalman Delta Networks: 不确定性感知的联想记忆", 方法 — 关键模块
 * steps 1-3 and 输出与差异点).  Per (b, h) and token t:
 *     n = ||k_t||^2;  p- = a^2 p + w;  beta = p- / (p- n + r)
 *     p = 1 / (1/p- + info_scale * n / r)
 *     S = a S + (v_t - a S k_t) (beta k_t)';   o_t = S q_t
 *
 * q, k     [B, T, H, dk] in_dtype device
 * v        [B, T, H, dv] in_dtype device
 * a, w, r  [B, T, H] fp32 device (decay in (0,1], process-noise variance
 *          >= 0, observation-noise variance > 0)
 * S0       [B, H, dv, dk] fp32 device initial memory, or NULL for zeros
 * p0       [B, H] fp32 device initial variance, or NULL for ones
 * o        [B, T, H, dv] fp32 device output
 * S_out    [B, H, dv, dk] fp32 device final memory (may alias S0)
 * p_out    [B, H] fp32 device final variance (may alias p0)
 * info_scale  kappa; <= 0 selects 1/dk
 * chunk    KDN_CHUNK_AUTO, KDN_CHUNK_RECURRENT or KDN_CHUNK_64
 * workspace   device scratch of >= kdn_forward_workspace_size(...) bytes,
 *             256-byte aligned (NULL allowed when that size is 0).  The
 *             chunked path keeps its device error word and a copy of p0
 *             there; kdn_read_workspace_status() reads the error word.
 *             The size depends on B, T, H and the current device: few heads
 *             over a long sequence take the segmented forward below, whose
 *             scratch (per segment: a state transition, a state and the
 *             start variances) is much larger, so query the size with the
 *             device that will run the call current.
 * Segmented forward: with dk = dv = 128 on the chunked path, when B H is at
 * most a quarter of the SM count and T is a multiple of 2048 (the segment
 * count S, a power of two >= 4 with B H S <= SMs and 512 S dividing T, is
 * chosen by the library), the sequence is cut into S segments run as extra
 * heads of the engine: the variance at each segment start from the composed
 * Mobius maps, each segment's state transition from a run with V = 0 and
 * S0 = I and its zero-start state and outputs from a run with S0 = 0, the
 * segment starts chained, and the outputs corrected by the segment start
 * state times the transition run's outputs (a tf32 tensor-core product).
 * The memory recursion is affine in the state, so the result is the same up
 * to rounding; it takes two engine passes over T / S tokens each instead of
 * one over T, and a workspace the size of o.
 * Supported: T >= 1; dk in {32, 64, 128}; 1 <= dv <= 128.  KDN_CHUNK_64
 * additionally needs in_dtype == KDN_BF16, dk == 128 and dv in {64, 128}.
 * All pointers 16-byte aligned.  o must not alias the inputs.
 * Errors: KDN_ERR_INVALID_ARG, KDN_ERR_UNSUPPORTED, KDN_ERR_WORKSPACE,
 * KDN_ERR_CUDA.
 * ---------------------------------------------------------------------- */
size_t kdn_forward_workspace_size(kdn_variant variant, int B, int T, int H,
                                  int dk, int dv, int chunk);
kdn_status kdn_iso_forward(const void* q, const void* k, const void* v,
                           kdn_dtype in_dtype, const float* a, const float* w,
                           const float* r, const float* S0, const float* p0,
                           float* o, float* S_out, float* p_out, int B, int T,
                           int H, int dk, int dv, float info_scale, int chunk,
                           void* workspace, size_t workspace_bytes,
                           void* stream);

/* ------------------------------------------------------------------------
 * kdn_diag_forward -- Diagonal KDN layer forward ("Kalman Delta Networks:
 * Uncertainty-aware Associative Memory", abstract: online mean-field
 * variational projection onto diagonal Gaussians).  Per (b, h), token t and
 * key dimension i:
 *     p-_i = a^2 p_i + w_i;   s = sum_i p-_i k_i^2 + r;   g = p- * k / s
 *     p_i  = 1 / (1/p-_i + k_i^2 / r)
 *     S = a S + (v_t - a S k_t) g';   o_t = S q_t
 * Arguments as kdn_iso_forward except:
 * w        [B, T, H, dk] fp32 device (per-dimension process noise)
 * p0, p_out  [B, H, dk] fp32 device (NULL p0 = ones)
 * (no info_scale: the diagonal projection has none)
 * ---------------------------------------------------------------------- */
kdn_status kdn_diag_forward(const void* q, const void* k, const void* v,
                            kdn_dtype in_dtype, const float* a, const float* w,
                            const float* r, const float* S0, const float* p0,
                            float* o, float* S_out, float* p_out, int B, int T,
                            int H, int dk, int dv, int chunk, void* workspace,
                            size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * kdn_forward_varlen -- kdn_iso_forward / kdn_diag_forward (variant) over N
 * packed sequences of different lengths: sequence s is tokens
 * [cu_seqlens[s], cu_seqlens[s+1]) of tensors laid out [total, H, ...]
 * (that is [1, total, H, ...]), and it starts from its own S0[s], p0[s] and
 * ends in its own S_out[s], p_out[s] (the prefill -> decode handoff:
 * kdn_decode_step continues from them; "Kalman Delta Networks: ..."
 * abstract, constant-memory decoding).  A sequence may be empty; it then
 * hands S0, p0 (or zeros, ones) through.  On the chunked engine, when the
 * N x H (sequence, head) problems outnumber the SMs, a one-block kernel first
 * orders the sequences longest first (by chunk count) into the workspace and
 * the engine starts them in that order; results do not depend on the order.
 *
 * q, k     [total, H, dk] in_dtype device;  v [total, H, dv]
 * a, r     [total, H] fp32 device;  w [total, H] (iso) or [total, H, dk]
 * cu_seqlens  [N + 1] int32 device, cu_seqlens[0] = 0, non-decreasing,
 *          cu_seqlens[N] = total.  Offsets out of order or out of range are
 *          clamped and reported through the workspace (KDN_ERR_INVALID_ARG
 *          from kdn_read_workspace_status).
 * S0, S_out  [N, H, dv, dk];  p0, p_out  [N, H] (iso) or [N, H, dk] (diag)
 * o        [total, H, dv] fp32 device
 * info_scale  iso only, as kdn_iso_forward
 * chunk    as kdn_iso_forward; the chunked engine serves d_v = 128 here (at
 *          d_v = 64, KDN_CHUNK_AUTO takes the token-recurrent kernel and
 *          KDN_CHUNK_64 returns KDN_ERR_UNSUPPORTED)
 * workspace   device scratch of >= kdn_forward_varlen_workspace_size(...)
 *             bytes (at least 256), 256-byte aligned: the error word, then
 *             (chunked engine) the sequence order
 * total >= 0, N >= 1.  Other arguments and errors as kdn_iso_forward.
 * ---------------------------------------------------------------------- */
size_t kdn_forward_varlen_workspace_size(kdn_variant variant, int N, int H,
                                         int dk, int dv, int chunk);
kdn_status kdn_forward_varlen(kdn_variant variant, const void* q,
                              const void* k, const void* v, kdn_dtype in_dtype,
                              const float* a, const float* w, const float* r,
                              const int32_t* cu_seqlens, const float* S0,
                              const float* p0, float* o, float* S_out,
                              float* p_out, int N, int total, int H, int dk,
                              int dv, float info_scale, int chunk,
                              void* workspace, size_t workspace_bytes,
                              void* stream);

/* ------------------------------------------------------------------------
 * kdn_forward_host -- kdn_iso_forward / kdn_diag_forward (variant) with every
 * tensor in host memory, for callers whose data is not on the device yet.
 * The batch goes through the device in slices of slice_b entries (<= 0
 * selects 1): a slice's inputs are copied in, the forward runs on them and
 * its o, S_out and p_out are copied back, on two internal streams that
 * alternate between slices, so that the copies of one slice overlap the
 * copies of the next and the kernels.  Results equal those of the device
 * calls on the same data.  The pages have no counterpart of this entry point.
 *
 * q, k, v, a, w, r, S0, p0, o, S_out, p_out  as in kdn_iso_forward /
 *          kdn_diag_forward, but host pointers; pinned (page-locked) memory
 *          is needed for the copies to overlap.  S0, p0 may be NULL.
 * info_scale  iso only (as kdn_iso_forward); ignored for KDN_DIAG
 * workspace   device scratch of >= kdn_forward_host_workspace_size(...)
 *             bytes, 256-byte aligned: an error word, then two slots of
 *             one slice's device buffers.  kdn_read_workspace_status() on it
 *             reports a bounded wait that gave up in any slice.
 * stream   the work is ordered after earlier work on `stream`, and later
 *          work on `stream` waits for all of it; synchronise `stream` before
 *          reading the outputs.  Calls on one device are enqueued one at a
 *          time (an internal lock); the host buffers must stay valid until
 *          `stream` has passed the call.
 * Errors: as kdn_iso_forward.  All checks run before anything is enqueued;
 * a KDN_ERR_CUDA from a runtime call part-way still leaves `stream` waiting
 * for what was enqueued.
 * ---------------------------------------------------------------------- */
size_t kdn_forward_host_workspace_size(kdn_variant variant, int B, int T,
                                       int H, int dk, int dv,
                                       kdn_dtype in_dtype, int chunk,
                                       int slice_b);
kdn_status kdn_forward_host(kdn_variant variant, const void* q, const void* k,
                            const void* v, kdn_dtype in_dtype, const float* a,
                            const float* w, const float* r, const float* S0,
                            const float* p0, float* o, float* S_out,
                            float* p_out, int B, int T, int H, int dk, int dv,
                            float info_scale, int chunk, int slice_b,
                            void* workspace, size_t workspace_bytes,
                            void* stream);

/* ------------------------------------------------------------------------
 * kdn_decode_step -- one recurrent decoding step for B x H heads, updating
 * the state in place (the constant-memory decoding of "Kalman Delta
 * Networks: Uncertainty-aware Associative Memory", abstract).  The same
 * update as one token of kdn_iso_forward / kdn_diag_forward.
 *
 * variant  KDN_ISO or KDN_DIAG
 * q, k     [B, H, dk] in_dtype device;  v [B, H, dv] in_dtype device
 * a, r     [B, H] fp32 device
 * w        [B, H] (iso) or [B, H, dk] (diag) fp32 device
 * S        [B, H, dv, dk] fp32 device, read and overwritten
 * p        [B, H] (iso) or [B, H, dk] (diag) fp32 device, read and overwritten
 * o        [B, H, dv] fp32 device output
 * info_scale  iso only; <= 0 selects 1/dk
 * Supported: dk in {32, 64, 128}; 1 <= dv <= 128; pointers 16-byte aligned.
 * ---------------------------------------------------------------------- */
kdn_status kdn_decode_step(kdn_variant variant, const void* q, const void* k,
                           const void* v, kdn_dtype in_dtype, const float* a,
                           const float* w, const float* r, float* S, float* p,
                           float* o, int B, int H, int dk, int dv,
                           float info_scale, void* stream);

/* ------------------------------------------------------------------------
 * kdn_exact_forward -- the dense (full-covariance) Kalman filter of the same
 * memory model, for small d_k: every row of S shares one d_k x d_k covariance
 * P, carried exactly by the Riccati recursion instead of being projected to a
 * scalar or a diagonal.  The pages name this exact filter as what the KDN
 * projection approximates ("Kalman Delta Networks: Uncertainty-aware
 * Associative Memory", abstract; "Kalman Delta Networks: 不确定性感知的联想
 * 记忆", 局限), so this call measures the projection's error.  Per token:
 *   P- = a^2 P + W,  u = P- k,  s = k.u + r,  g = u / s,
 *   S <- a S + (v - a S k) g^T,  o = S q,  P = P- - u u^T / s
 * with W = w I (variant KDN_ISO) or diag(w) (KDN_DIAG).  There is no
 * information scale: nothing is projected.
 *
 * q, k     [B, T, H, dk] in_dtype device;  v [B, T, H, dv] in_dtype device
 * a, r     [B, T, H] fp32 device
 * w        [B, T, H] (iso) or [B, T, H, dk] (diag) fp32 device
 * S0       [B, H, dv, dk] fp32 device, or NULL for zeros
 * P0       [B, H, dk, dk] fp32 device, or NULL for the identity; only its
 *          symmetric part (P0 + P0^T) / 2 is used
 * o        [B, T, H, dv] fp32 device output
 * S_out    [B, H, dv, dk];  P_out [B, H, dk, dk] fp32 device outputs; they
 *          may alias S0 and P0 (each head reads its state before writing)
 * Supported: dk in {32, 64}; 8 <= dv <= 128 with dv a multiple of 8; every
 * pointer 16-byte aligned.  KDN_ERR_UNSUPPORTED for other sizes.  One CTA
 * per (b, h) runs the T tokens in order; no workspace, no on-device waits.
 * Errors: KDN_ERR_INVALID_ARG (NULL, shape, alignment, variant or dtype),
 * KDN_ERR_CUDA (launch).
 * ---------------------------------------------------------------------- */
kdn_status kdn_exact_forward(kdn_variant variant, const void* q, const void* k,
                             const void* v, kdn_dtype in_dtype, const float* a,
                             const float* w, const float* r, const float* S0,
                             const float* P0, float* o, float* S_out,
                             float* P_out, int B, int T, int H, int dk, int dv,
                             void* stream);

/* ------------------------------------------------------------------------
 * kdn_backward -- the backward pass of kdn_iso_forward / kdn_diag_forward
 * (variant): the gradients of a loss L with respect to every input, given
 * dL/do, dL/dS_T and dL/dp_T ("Kalman Delta Networks: 不确定性感知的联想记忆",
 * 实验: the layers are trained in language models).  It runs the forward
 * again on the token-recurrent kernel, saving the variance before every
 * token and the state before every 16th token in the workspace, then the
 * adjoint recursion from the last token to the first (dS, dp carried
 * backwards), block by block of 16 tokens: each block's states are rebuilt
 * from its checkpoint, with the forward's arithmetic, before its adjoint.
 *
 * q, k, v, a, w, r, S0, p0, info_scale, in_dtype: as the forward call
 * dO       [B, T, H, dv] fp32 device: dL/do
 * dS_T     [B, H, dv, dk], dp_T [B, H] (iso) or [B, H, dk] (diag) fp32
 *          device, or NULL for zero
 * dq, dk   [B, T, H, dk];  dv [B, T, H, dv];  da, dr [B, T, H];
 * dw       [B, T, H] (iso) or [B, T, H, dk] (diag);  dS0 [B, H, dv, dk];
 * dp0      [B, H] (iso) or [B, H, dk] (diag): fp32 device outputs
 * workspace   device scratch of >= kdn_backward_workspace_size(...) bytes,
 *          256-byte aligned: B H ceil(T / 16) dv dk floats of checkpoints,
 *          B H T (1 or dk) floats of variances, B H 16 dv dk floats of
 *          rebuilt states, plus the forward's outputs
 * Supported: dk in {32, 64, 128}; 1 <= dv <= 128; every pointer 16-byte
 * aligned.
 * Errors: KDN_ERR_INVALID_ARG, KDN_ERR_UNSUPPORTED, KDN_ERR_WORKSPACE,
 * KDN_ERR_CUDA, all before anything is enqueued except KDN_ERR_CUDA.
 * ---------------------------------------------------------------------- */
size_t kdn_backward_workspace_size(kdn_variant variant, int B, int T, int H,
                                   int dk, int dv);
kdn_status kdn_backward(kdn_variant variant, const void* q, const void* k,
                        const void* v, kdn_dtype in_dtype, const float* a,
                        const float* w, const float* r, const float* S0,
                        const float* p0, const float* dO, const float* dS_T,
                        const float* dp_T, float* dq, float* dk, float* dv,
                        float* da, float* dw, float* dr, float* dS0,
                        float* dp0, int B, int T, int H, int dk_dim,
                        int dv_dim, float info_scale, void* workspace,
                        size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * kdn_kla_forward -- the diagonal Kalman filter in information form ("Kalman
 * Linear Attention: Parallel Bayesian Filtering ...", 方法论 §1-§3): a
 * precision per key dimension, updated by a Mobius map of the previous one,
 * and an information mean that is an affine recursion given the precisions,
 * read out with the query.  It runs on the Diagonal KDN's inputs (decay a,
 * process noise w per key dimension, value precision 1 / r) with every
 * element of the memory filtered on its own, so per token and dimension i:
 *   lambda-_i = 1 / (a^2 / lambda_i + w_i),  lambda_i = lambda-_i + k_i^2 / r
 *   S <- S diag(f) + v u^T,  f = a lambda- / lambda,  u = (k / r) / lambda
 *   o = S q
 * (forget gate f and write gate u: ratios of precisions).
 *
 * q, k     [B, T, H, dk] in_dtype device;  v [B, T, H, dv] in_dtype device
 * a, r     [B, T, H] fp32 device;  w [B, T, H, dk] fp32 device
 * S0       [B, H, dv, dk] fp32 device posterior mean, or NULL for zeros
 * lam0     [B, H, dk] fp32 device precision, or NULL for ones
 * o        [B, T, H, dv] fp32 device output
 * S_out    [B, H, dv, dk];  lam_out [B, H, dk] fp32 device outputs; they may
 *          alias S0 and lam0
 * Supported: dk in {32, 64, 128}; 8 <= dv <= 128 with dv a multiple of 8;
 * every pointer 16-byte aligned.  One CTA per (b, h); no workspace and no
 * on-device waits.  Errors: KDN_ERR_INVALID_ARG (NULL, shape, alignment,
 * dtype), KDN_ERR_UNSUPPORTED (sizes), KDN_ERR_CUDA (launch).
 * ---------------------------------------------------------------------- */
kdn_status kdn_kla_forward(const void* q, const void* k, const void* v,
                           kdn_dtype in_dtype, const float* a, const float* w,
                           const float* r, const float* S0, const float* lam0,
                           float* o, float* S_out, float* lam_out, int B, int T,
                           int H, int dk, int dv, void* stream);

/* ------------------------------------------------------------------------
 * kdn_kla_forward_ws -- the same filter and arguments as kdn_kla_forward, plus
 * a workspace.  For dk = dv = 128 with bf16 q, k, v it runs the chunked
 * tensor-core engine ("Kalman Linear Attention: ...", 方法论 §2: given the
 * precisions the mean recursion is affine, so a stretch of tokens is a few
 * dense products).  Per 64-token chunk, with G the running product of the
 * forget gates and Q~ = Q . G, U~ = U / G:
 *   A = (Q~ U~^T) masked causal,  O = S0 Q~^T + A V,
 *   S_C = (S0 + V^T U~) diag(G_C),
 * on tcgen05 tensor cores with every fp32 operand split into bf16 hi + lo
 * and fp32 accumulation; the precision recursion runs in fp32 per key
 * dimension.  A chunk whose gates would drive G below 2^-100 is cut into
 * shorter pieces (down to single tokens), so every input is served.  Other
 * shapes and fp32 inputs run kdn_kla_forward's token-recurrent kernel.
 * workspace   device memory of kdn_kla_workspace_size bytes (16-byte
 *             aligned): the call's error word; kdn_read_workspace_status
 *             reports KDN_ERR_TIMEOUT if a bounded on-device wait gave up
 * Results match kdn_kla_forward's to the engine's operand precision (the
 * bf16 hi/lo split keeps 16 significant bits of each fp32 operand).
 * Errors: as kdn_kla_forward, plus KDN_ERR_WORKSPACE (NULL, misaligned or
 * too small).
 * ---------------------------------------------------------------------- */
size_t kdn_kla_workspace_size(int B, int T, int H, int dk, int dv);
kdn_status kdn_kla_forward_ws(const void* q, const void* k, const void* v,
                              kdn_dtype in_dtype, const float* a,
                              const float* w, const float* r, const float* S0,
                              const float* lam0, float* o, float* S_out,
                              float* lam_out, int B, int T, int H, int dk,
                              int dv, void* workspace, size_t workspace_bytes,
                              void* stream);

/* ------------------------------------------------------------------------
 * kdn_linear_scan_forward -- the gated linear recurrence, per channel:
 *     h_t = a_t h_{t-1} + b_t x_t,   y_t = h_t
 * (forget gate a, write gate b), in fp32, over B sequences of T steps, or over
 * packed sequences of mixed length.  It is the affine mean recursion that the
 * information-form filter runs given its gates ("Kalman Linear Attention:
 * Parallel Bayesian Filtering ...", 方法论 §2), as a layer of its own with one
 * state per channel; the steps compose by an associative scan, one pass over
 * the data.
 *
 * a        [B, T, D] gate_dtype device: a forget gate is in [0, 1]; other values
 *          do as long as products of up to 128 consecutive ones stay finite
 * b        [B, T, D] gate_dtype device, or NULL for ones
 * x        [B, T, D] in_dtype device
 * h0       [B, D] fp32 device initial states, or NULL for zeros
 * cu_seqlens  NULL, or [B + 1] int32 device: then B sequences are packed in T
 *          steps, all arrays [B, T, D] are [T, D], and sequence s is steps
 *          [cu_seqlens[s], cu_seqlens[s + 1]); cu_seqlens[0] = 0,
 *          non-decreasing, cu_seqlens[B] <= T.  Steps from cu_seqlens[B] on
 *          are padding: their outputs are left as they were.  Sequences may be
 *          empty.  Offsets out of order or out of range touch no memory
 *          outside the arrays; they give unspecified values and
 *          KDN_ERR_INVALID_ARG from kdn_read_workspace_status.
 * y        [B, T, D] in_dtype device output (fp32 states, rounded once)
 * h_out    [B, D] fp32 device final states (an empty sequence's is its initial
 *          one); may alias h0
 * workspace   device scratch of >= kdn_linear_scan_workspace_size(B, T, D)
 *          bytes (packed: B = 1), 256-byte aligned; the call clears what it
 *          needs first.  Calls that may overlap need a workspace each.
 * B, D >= 1; T >= 0; every other pointer 16-byte aligned; y must not overlap
 * the inputs.
 * Errors: KDN_ERR_INVALID_ARG, KDN_ERR_UNSUPPORTED (more than 2^31 tiles),
 * KDN_ERR_WORKSPACE, KDN_ERR_CUDA; kdn_read_workspace_status() reports a
 * bounded wait that gave up, or bad offsets.
 * ---------------------------------------------------------------------- */
size_t kdn_linear_scan_workspace_size(int B, int T, int D);
kdn_status kdn_linear_scan_forward(const void* a, const void* b,
                                   kdn_dtype gate_dtype, const void* x,
                                   kdn_dtype in_dtype, const float* h0,
                                   const int32_t* cu_seqlens, void* y,
                                   float* h_out, int B, int T, int D,
                                   void* workspace, size_t workspace_bytes,
                                   void* stream);

/* ------------------------------------------------------------------------
 * kdn_linear_scan_backward -- the gradients of kdn_linear_scan_forward.  With
 * c the gradient that reaches the state after step t from later steps (dh_T
 * behind the last step of a sequence), from the last step to the first:
 *     g = dy_t + c;  dx_t = b_t g;  db_t = x_t g;  da_t = g h_{t-1};  c = a_t g
 * and dh0 = c before the first step.  h_{t-1} is read from y as it is stored
 * (h0 before the first step), so with bf16 y it is the rounded state.
 *
 * a, b, x, h0, cu_seqlens, B, T, D, workspace: as the forward call (x is read
 *          only when b is given, and may be NULL otherwise)
 * y        [B, T, D] in_dtype device: the forward's output
 * dy       [B, T, D] in_dtype device: dL/dy
 * dh_T     [B, D] fp32 device: dL/dh_out, or NULL for zeros
 * da, db   [B, T, D] gate_dtype device outputs (db only with b)
 * dx       [B, T, D] in_dtype device output
 * dh0      [B, D] fp32 device output; may alias dh_T
 * The outputs must not overlap the inputs.  Padding steps are left as they
 * were.  Errors: as the forward call.
 * ---------------------------------------------------------------------- */
kdn_status kdn_linear_scan_backward(const void* a, const void* b,
                                    kdn_dtype gate_dtype, const void* x,
                                    const void* y, const void* dy,
                                    kdn_dtype in_dtype, const float* h0,
                                    const float* dh_T,
                                    const int32_t* cu_seqlens, void* da,
                                    void* db, void* dx, float* dh0, int B,
                                    int T, int D, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * kdn_linear_scan_step -- one step for B x D channels, the state updated in
 * place: h <- a h + b x, y = h (the same update as one step of the forward).
 * a, b     [B, D] gate_dtype device (b or NULL);  x, y [B, D] in_dtype device
 * h        [B, D] fp32 device, read and overwritten
 * B, D >= 1; pointers 16-byte aligned.  Errors: KDN_ERR_INVALID_ARG,
 * KDN_ERR_CUDA.
 * ---------------------------------------------------------------------- */
kdn_status kdn_linear_scan_step(const void* a, const void* b,
                                kdn_dtype gate_dtype, const void* x,
                                kdn_dtype in_dtype, float* h, void* y, int B,
                                int D, void* stream);

/* ------------------------------------------------------------------------
 * kdn_rmsnorm_forward -- the residual addition and root-mean-square norm
 * around a mixing layer, over rows of D:
 *     h = x + residual (rounded to residual_dtype; h = x without a residual)
 *     y = h / sqrt(mean(h^2) + eps) * weight
 * x takes the fp32 output of the mixing calls as it is; y is bf16 or fp32, or
 * e4m3 codes with a scale for each 128 of a row, as kdn_fp8_quantize gives and
 * kdn_fp8_matmul takes.  The norm reads h as it is stored.
 *
 * x        [rows, D] x_dtype device
 * residual [rows, D] residual_dtype device, or NULL
 * weight   [D] fp32 device
 * h        [rows, D] residual_dtype device output with a residual (may alias
 *          residual); NULL without
 * y        [rows, D] y_dtype device output; e4m3: rows ldy bytes apart, ldy a
 *          multiple of 16 and at least D (the bytes behind D are left as they
 *          were).  ldy is not read otherwise.
 * scale    [rows, ceil(D / 128)] fp32 device output, e4m3 only
 * eps      >= 0, finite
 * Sums in fp32: |h| up to about 1e18, and where eps is zero or smaller than
 * mean(h^2), from about 1e-18.  No output may overlap an input but as said.
 * rows >= 0 (0: nothing is done);
 * 1 <= D <= 16384; pointers 16-byte aligned.  Errors: KDN_ERR_INVALID_ARG,
 * KDN_ERR_UNSUPPORTED, KDN_ERR_CUDA.
 * ---------------------------------------------------------------------- */
kdn_status kdn_rmsnorm_forward(const void* x, kdn_dtype x_dtype,
                               const void* residual, kdn_dtype residual_dtype,
                               const float* weight, void* h, void* y,
                               kdn_dtype y_dtype, int64_t ldy, float* scale,
                               int64_t rows, int D, float eps, void* stream);

/* ------------------------------------------------------------------------
 * kdn_rmsnorm_backward -- the gradients of kdn_rmsnorm_forward.  With
 * rs = 1 / sqrt(mean(h^2) + eps) and dh what reaches h from its other use:
 *     d = dh + rs (dy weight - h rs^2 mean(dy weight h))
 *     dx = d,  dresidual = d,  dweight = sum over rows of dy h rs
 * dx in fp32 is the dO that kdn_backward takes.  For e4m3 outputs dy is the
 * gradient with respect to the values that codes and scales stand for (the
 * rounding itself is passed straight through).
 *
 * h        [rows, D] h_dtype device: the forward's h (x without a residual)
 * dy       [rows, D] dy_dtype device
 * dh       [rows, D] h_dtype device, or NULL for zeros
 * dx       [rows, D] dx_dtype device output
 * dresidual  [rows, D] h_dtype device output, or NULL; may alias dh
 * dweight  [D] fp32 device output (zeros when rows = 0)
 * workspace   device scratch of >= kdn_rmsnorm_backward_workspace_size(...)
 *          bytes, 256-byte aligned: the blocks' parts of dweight, added in a
 *          fixed order.  Calls that may overlap need a workspace each.
 * Other conditions and errors as the forward, plus KDN_ERR_WORKSPACE.
 * ---------------------------------------------------------------------- */
size_t kdn_rmsnorm_backward_workspace_size(int64_t rows, int D);
kdn_status kdn_rmsnorm_backward(const void* h, kdn_dtype h_dtype,
                                const float* weight, const void* dy,
                                kdn_dtype dy_dtype, const void* dh, void* dx,
                                kdn_dtype dx_dtype, void* dresidual,
                                float* dweight, int64_t rows, int D, float eps,
                                void* workspace, size_t workspace_bytes,
                                void* stream);

/* ------------------------------------------------------------------------
 * kdn_fp8_quantize -- a matrix into e4m3 codes with fp32 scales:
 *     scale = max(largest magnitude of the block, 2^-100) / 448
 *     code  = e4m3(value / scale), to nearest, ties to even
 * of the exact quotient 448 value / magnitude.
 * A block is 128 values along a row of the output (the last one may be
 * shorter), or with `tile` a 128 x 128 tile of it.  `transpose` quantises the
 * transpose of x.  An infinity or NaN in a block makes its scale infinite or
 * NaN, and so every product with the block NaN.
 *
 * x        [rows, cols] x_dtype device
 * q        e4m3 codes, device output: R rows of C bytes, ldq bytes apart, with
 *          (R, C) = (rows, cols), or (cols, rows) with transpose; ldq a
 *          multiple of 16 and at least C (the bytes between C and the next
 *          multiple of 16 may be overwritten, but not behind the last row)
 * scale    [R, ceil(C / 128)] fp32 device output; with tile
 *          [ceil(R / 128), ceil(C / 128)]
 * rows >= 0 (0: nothing is done), cols >= 1; x and q 16-byte aligned.
 * Errors: KDN_ERR_INVALID_ARG, KDN_ERR_UNSUPPORTED (2^31 blocks),
 * KDN_ERR_CUDA.
 * ---------------------------------------------------------------------- */
kdn_status kdn_fp8_quantize(const void* x, kdn_dtype x_dtype, int64_t rows,
                            int64_t cols, int tile, int transpose, void* q,
                            int64_t ldq, float* scale, void* stream);

/* ------------------------------------------------------------------------
 * kdn_fp8_matmul -- the 8-bit projection out = x w^T: x [M, K] and w [N, K] in
 * e4m3, with a scale for each block of 128 along K,
 *     out[m, n] = sum_b x_scale[m, b] w_scale[n', b] sum_{k in b} x[m, k] w[n, k]
 * with n' = n / 128 (w_tile, a weight's 128 x 128 tiles) or n.  It makes the
 * q, k, v (bf16) and gate inputs (fp32) of the mixing calls from
 * kdn_rmsnorm_forward's 8-bit output.  With quantised transposes it is also
 * the backward pass: dx = dy w is the product of dy and w^T (tiles), and
 * dw = dy^T x the product of dy^T and x^T (rows of 128 tokens, w_tile = 0).
 * Block products on the tensor cores, exact products, fp32 sums; the sum over
 * blocks in fp32, in an order that depends only on the sizes and the device.
 *
 * x        e4m3 codes, M rows of K bytes, ldx bytes apart
 * x_scale  [M, ceil(K / 128)] fp32 device
 * w        e4m3 codes, N rows of K bytes, ldw bytes apart
 * w_scale  [ceil(N / 128), ceil(K / 128)] (w_tile) or [N, ceil(K / 128)] fp32
 * out      [M, N] out_dtype device output; must not overlap the inputs
 * status   one device word or NULL.  Not cleared: a bounded on-device wait
 *          that gives up (it cannot in correct use) sets it, and
 *          kdn_read_workspace_status(status, 4, stream) reports it, so zero it
 *          once before the first call
 * M >= 0 (0: nothing is done), N, K >= 1; ldx, ldw multiples of 16 and at
 * least K; x, w, out 16-byte aligned.  Bytes behind K are not read as values.
 * Errors: KDN_ERR_INVALID_ARG, KDN_ERR_UNSUPPORTED (2^31 tiles), KDN_ERR_CUDA.
 * ---------------------------------------------------------------------- */
kdn_status kdn_fp8_matmul(const void* x, int64_t ldx, const float* x_scale,
                          const void* w, int64_t ldw, const float* w_scale,
                          int w_tile, void* out, kdn_dtype out_dtype, int M,
                          int N, int K, uint32_t* status, void* stream);

/* ------------------------------------------------------------------------
 * kdn_read_workspace_status -- synchronise `stream`, then report the device
 * error word a previous call left in `workspace`: KDN_OK, KDN_ERR_TIMEOUT
 * if a bounded on-device wait gave up, or KDN_ERR_INVALID_ARG if packed-
 * sequence offsets were out of order or out of range.  Also returns
 * KDN_ERR_CUDA if the stream reports an error.  This is the only call that
 * blocks the host.
 * ---------------------------------------------------------------------- */
kdn_status kdn_read_workspace_status(const void* workspace,
                                     size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDN_H_ */
