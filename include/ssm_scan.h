/*
 * ssm_scan.h — C ABI of the MI355X (gfx950) selective-scan library.
 *
 * The library computes the Mamba selective scan (S6) forward pass, its
 * backward, its one-token decode step, the Mamba-2 SSD layer, the gated delta
 * rule (forward, backward, decode step), the norms around such a mixer, the gated
 * linear recurrence (forward, backward, decode step), the projections around these
 * (with bias, activation and residual) and the clipping of a model's gradients with
 * hand-written HIP kernels. Every pointer that
 * names tensor data is a DEVICE pointer owned by the caller; the library
 * allocates and frees nothing. Work is enqueued asynchronously on the given
 * HIP stream: buffers must stay alive until the stream has finished with
 * them. No function prints, throws or exits; each returns an ssm_status.
 *
 * Operation (for every batch row b, channel d and state n; each channel is
 * an independent single-input single-output SSM, itwiki "상태 공간 모델",
 * section "제어 이론의 상태 공간 표현과의 관계"):
 *
 *   Abar_t = exp(delta_t * A[d,n])                 discretised decay
 *   Bu_t   = delta_t * B_t[n] * u_t                default: simplified rule
 *          = (exp(delta_t A) - 1)/A * B_t[n] * u_t zero-order hold (SSM_DISC_ZOH)
 *   h_t    = Abar_t * h_{t-1} + Bu_t               h_{-1} = h0 (or 0)
 *   y_t    = sum_n C_t[n] h_t[n] + D[d] u_t        readout after the update
 *   y_t   *= z_t * sigmoid(z_t)                    optional SiLU gate
 *
 * Passages: eommydocs "State Space Models (SSM)" §3.2 "Selective Scan
 * Algorithm" (shapes of u, delta, A, B, C and the deltaA / deltaB_u
 * discretisation); youngju.dev "Mamba와 State Space Model 논문 심층 분석",
 * SelectiveSSM.selective_scan and MambaBlock.forward (recurrence, readout,
 * y + D*x skip, y * silu(z) gate); itwiki "상태 공간 모델", "동작 원리 › 이산화"
 * (zero-order hold); doyouknow.kr "Mamba와 상태 공간 모델(SSM)의 부상 완벽
 * 가이드" §3-1 (h_t = exp(delta_t A) h_{t-1} + delta_t B_t x_t).
 *
 * Numerics: state and arithmetic in fp32; bf16 inputs are widened exactly;
 * bf16 outputs are rounded to nearest-even. NaN and Inf propagate unchecked.
 */
#ifndef SSM_SCAN_H
#define SSM_SCAN_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. Every error is detected on the host before any work is
 * enqueued, except SSM_ERR_HIP, which reports a failed kernel launch. */
typedef enum {
    SSM_OK = 0,
    SSM_ERR_NULL = -1,        /* a required pointer is NULL */
    SSM_ERR_SHAPE = -2,       /* a negative size, or sizes whose byte count overflows */
    SSM_ERR_DTYPE = -3,       /* unknown element type */
    SSM_ERR_UNSUPPORTED = -4, /* dstate outside 1..64, unknown discretisation or flag, conv_width
                                 outside 0..4, bad tuning */
    SSM_ERR_ALIAS = -5,       /* an output overlaps an input or another output */
    SSM_ERR_WORKSPACE = -6,   /* workspace missing or smaller than ssm_scan_workspace_size() */
    SSM_ERR_HIP = -7,         /* the HIP runtime refused a launch (e.g. not a gfx950 device) */
    SSM_ERR_ALIGN = -8,       /* a pointer is not aligned to its element size */
    SSM_ERR_SCRATCH = -9      /* ssm_scan_fwd_noalloc: the problem needs more than
                                 SSM_NOALLOC_SCRATCH_BYTES of scratch */
} ssm_status;

/* Element type of the per-token tensors u, delta, z, B, C and of the output y.
 * A, D and all states are always fp32. */
typedef enum { SSM_F32 = 0, SSM_BF16 = 1 } ssm_dtype;

/* Discretisation of B (A is always exp(delta*A)). */
typedef enum { SSM_DISC_EULER = 0, SSM_DISC_ZOH = 1 } ssm_disc;

/* Sizes and types of one scan, and how the step size is formed.
 * The step used by the recurrence is delta[b,t,d] (+ delta_bias[d] when the
 * bias is given), passed through softplus(x) = log(1 + exp(x)) when
 * delta_softplus is nonzero: the projection output becomes a positive step
 * inside the kernel (youngju.dev SelectiveSSM.forward, dt = softplus(...)).
 * With conv_width W > 0 the Mamba block's prologue runs in the kernel (youngju.dev
 * MambaBlock.forward, x_conv = silu(conv1d(x)), a causal depthwise convolution
 * with left padding W-1): the buffer passed as u holds x, and the scan input is
 *     u[b,t,d] = silu(conv_bias[d] + sum_{k<W} conv_weight[d,k] * x[b,t-(W-1)+k,d]),
 * x before t = 0 being zero; the D skip uses this u. Forward and backward
 * form u in a pass of their own and keep it in fp32, whatever the tensors'
 * type (a bf16 rounding of u can show in y far beyond one rounding of y where
 * the scan's sums cancel).
 * Zero-initialise the struct for "delta used as given, no convolution". */
typedef struct {
    int64_t batch;   /* b  >= 0 */
    int64_t seqlen;  /* L  >= 0 */
    int64_t dim;     /* d  in 0..2^26 (channels, d_inner) */
    int64_t dstate;  /* N  in 1..64 */
    int32_t dtype;   /* ssm_dtype */
    int32_t disc;    /* ssm_disc */
    int32_t delta_softplus;   /* 0 or 1 */
    int32_t conv_width;       /* 0 (u used as given) or W in 1..4: see below */
    const float *delta_bias;  /* (dim) fp32 device pointer, or NULL */
    const float *conv_weight; /* (dim, W) fp32 device pointer when conv_width > 0 */
    const float *conv_bias;   /* (dim) fp32 device pointer, or NULL */
} ssm_scan_desc;

/* Optional launch shape, for tuning and for tests of every kernel variant.
 * Zero fields are chosen by the library. state_groups: waves that share one
 * 64-channel tile, each owning dstate/state_groups states (1,2,4,8,16);
 * segments: independent pieces of the sequence, joined by an affine carry
 * (1..64). */
typedef struct {
    int32_t state_groups;
    int32_t segments;
} ssm_scan_tuning;

/* Bytes of device workspace ssm_scan_fwd needs for `desc`: B and C widened
 * to fp32 (about 2 * batch * seqlen * dstate * 4 bytes) plus, when the
 * sequence is split into segments, three (batch, segments, dim, dstate) fp32
 * arrays, plus, with the convolution prologue, u (batch, seqlen, dim) in
 * fp32. 0 when there is nothing to compute; 0 for an invalid descriptor. */
size_t ssm_scan_workspace_size(const ssm_scan_desc *desc);

/*
 * Selective scan forward (the pages' selective_scan(u, delta, A, B, C) with
 * the D skip and SiLU gate of the Mamba block fused in).
 *
 *   u, delta  (batch, seqlen, dim)   dtype, row-major, channel fastest
 *   A         (dim, dstate)          fp32 (negative for a decaying state)
 *   B, C      (batch, seqlen, dstate) dtype, shared by all channels of a row
 *   D         (dim) fp32, or NULL for no skip term
 *   z         (batch, seqlen, dim)   dtype, or NULL for no gate
 *   h0        (batch, dim, dstate)   fp32 initial state, or NULL for zeros
 *   y         (batch, seqlen, dim)   dtype, written
 *   h_last    (batch, dim, dstate)   fp32 final state, written; may be NULL.
 *             h_last may equal h0 exactly (resume in place).
 *   workspace device scratch of at least ssm_scan_workspace_size(desc) bytes,
 *             256-byte aligned (may be NULL when that size is 0); its
 *             contents on entry do not matter and are clobbered.
 * delta is used as given (the caller applies softplus). Outputs must not
 * overlap any input, each other or the workspace. Pointers must be aligned to
 * their element size. seqlen == 0 writes h_last = h0 (or zeros) and no y.
 */
int ssm_scan_fwd(const ssm_scan_desc *desc,
                 const void *u, const void *delta, const float *A,
                 const void *B, const void *C, const float *D, const void *z,
                 const float *h0, void *y, float *h_last,
                 void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * ssm_scan_fwd for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc. It takes
 * no workspace; the library keeps one fixed scratch buffer of
 * SSM_NOALLOC_SCRATCH_BYTES per GPU (a static device array, held from the
 * module's load on that GPU until the process ends) and runs the same kernels
 * as ssm_scan_fwd on it, so its results equal ssm_scan_fwd's bit for bit.
 *
 *   Arguments, shapes, conditions and errors: those of ssm_scan_fwd, without
 *   workspace and workspace_bytes.
 *   SSM_ERR_SCRATCH when ssm_scan_workspace_size(desc) exceeds
 *   SSM_NOALLOC_SCRATCH_BYTES (checked on the host before anything else is
 *   done; e.g. the 1.4B-shaped layer b8 L8192 d4096 N16 needs 8.4 MB, the
 *   131072-token d5120 layer about 33 MB, and the convolution prologue adds
 *   4*b*L*d bytes of fp32 u).
 *   The buffer's device address is looked up once per GPU, on the first call
 *   whose stream belongs to that GPU; that first call is best made outside
 *   graph capture. The call itself allocates nothing and frees nothing.
 *   Calls on one GPU share its buffer: calls that overlap in time on that GPU
 *   (two streams, or two host threads) race and give wrong results. Calls
 *   ordered on one stream are safe. Nothing in the buffer needs to start at
 *   zero: every pass writes what the next one reads.
 */
#define SSM_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
int ssm_scan_fwd_noalloc(const ssm_scan_desc *desc,
                         const void *u, const void *delta, const float *A,
                         const void *B, const void *C, const float *D, const void *z,
                         const float *h0, void *y, float *h_last, hipStream_t stream);

/* ssm_scan_workspace_size / ssm_scan_fwd with an explicit launch shape
 * (tuning == NULL is the same as the plain calls). */
size_t ssm_scan_workspace_size_tuned(const ssm_scan_desc *desc, const ssm_scan_tuning *tuning);
int ssm_scan_fwd_tuned(const ssm_scan_desc *desc,
                       const void *u, const void *delta, const float *A,
                       const void *B, const void *C, const float *D, const void *z,
                       const float *h0, void *y, float *h_last,
                       void *workspace, size_t workspace_bytes,
                       const ssm_scan_tuning *tuning, hipStream_t stream);

/* The launch shape ssm_scan_fwd would use for `desc` (written to *out). */
int ssm_scan_plan(const ssm_scan_desc *desc, ssm_scan_tuning *out);

/*
 * Backward of ssm_scan_fwd: the gradients of
 *     loss = sum_{b,t,d} dy[b,t,d] * y[b,t,d] + sum_{b,d,n} dh_last[b,d,n] * h_last[b,d,n]
 * with respect to u, delta, A, B, C, D, z and h0, for the same inputs and
 * discretisation as the forward call. The states are recomputed on the GPU
 * (a checkpoint every 16 tokens, or 8 for dstate > 16, then a reverse pass
 * per chunk) instead of being stored by the forward (doyouknow.kr "Mamba와
 * 상태 공간 모델(SSM)의 부상 완벽 가이드" §3-3: the backward recomputes the
 * intermediate states). With lam_t = dloss/dh_t:
 *     lam_t = C_t * dy_t g(z_t) + exp(delta_{t+1} A) lam_{t+1}
 * and every gradient follows by the chain rule through the recurrence,
 * readout, skip and gate stated above.
 *
 *   u .. h0       as for ssm_scan_fwd (same shapes, types, layouts)
 *   dy            (batch, seqlen, dim) dtype: gradient of y
 *   dh_last       (batch, dim, dstate) fp32 gradient of the final state, or NULL (0)
 *   du, ddelta    (batch, seqlen, dim) dtype, written
 *   dz            (batch, seqlen, dim) dtype, written; required when z is given, unused otherwise
 *   dA            (dim, dstate) fp32, written (summed over batch and time)
 *   dB, dC        (batch, seqlen, dstate) fp32, written (summed over channels)
 *   dD            (dim) fp32, written; required when D is given, unused otherwise
 *   dh0           (batch, dim, dstate) fp32, written, or NULL (not wanted)
 *   ddelta_bias   (dim) fp32, written when desc->delta_bias is given (else unused)
 *   dconv_weight  (dim, W) fp32, written; required when desc->conv_width W > 0 (else unused)
 *   dconv_bias    (dim) fp32, written when given and W > 0 (else unused); NULL: not wanted
 * With a delta bias or softplus in the descriptor, ddelta is the gradient of
 * the raw delta (the chain rule through the bias and softplus). With the
 * convolution prologue (W > 0), u holds x as for ssm_scan_fwd and du receives
 * the gradient of x: with pre_t = conv_bias + sum_k w[k] x_{t-(W-1)+k} and
 * g_t the gradient of the scan input u_t = silu(pre_t),
 *     dpre_t = g_t silu'(pre_t),  dx_s = sum_k w[k] dpre_{s+(W-1)-k},
 *     dconv_weight[k] = sum_{b,t} dpre_t x_{t-(W-1)+k},  dconv_bias = sum_{b,t} dpre_t
 * (the chain rule through youngju.dev MambaBlock.forward's x_conv =
 * silu(conv1d(x))). u is formed from x once, in fp32 in the workspace; the
 * recomputation reads it (or, when the sequence is split into segments, forms
 * it from x again as the forward does), and the reverse pass writes its
 * gradient in fp32 in the workspace.
 *   workspace     at least ssm_scan_bwd_workspace_size(desc) bytes, 256-byte
 *                 aligned; contents on entry do not matter.
 * Results do not depend on timing: every sum over channels, batch rows or
 * tiles is taken in a fixed order. Outputs must not overlap each other, any
 * input or the workspace. seqlen == 0 writes dA = 0, dD = 0, dh0 = dh_last.
 */
size_t ssm_scan_bwd_workspace_size(const ssm_scan_desc *desc);
int ssm_scan_bwd(const ssm_scan_desc *desc,
                 const void *u, const void *delta, const float *A,
                 const void *B, const void *C, const float *D, const void *z,
                 const float *h0, const void *dy, const float *dh_last,
                 void *du, void *ddelta, float *dA, float *dB, float *dC, float *dD,
                 void *dz, float *dh0, float *ddelta_bias, float *dconv_weight, float *dconv_bias,
                 void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * The forward and backward of one training step, sharing the recomputation
 * the backward starts with. ssm_scan_fwd_save is ssm_scan_fwd (same arguments
 * and results) run in the backward's launch shape, which also leaves in
 * `workspace` what the backward would first recompute: the state
 * at the start of every chunk of the sequence and the regrouped B and C (the
 * intermediate states of doyouknow.kr "Mamba와 상태 공간 모델(SSM)의 부상 완벽
 * 가이드" §3-3, kept at chunk granularity).
 * ssm_scan_bwd_saved is ssm_scan_bwd without that recomputation; it reads
 * them from the same workspace instead. Its gradients equal ssm_scan_bwd's
 * (the checkpoints are the states the forward passes through). h_last equals
 * ssm_scan_fwd's bit for bit; y may differ from it in the last bit where the
 * backward's launch shape splits the states over another number of waves
 * and so sums the readout in another order. With the convolution prologue the
 * saving forward leaves its fp32 u where the backward then reads it.
 *
 *   workspace  at least ssm_scan_bwd_workspace_size(desc) bytes, 256-byte
 *              aligned, for both calls. ssm_scan_bwd_saved must receive the
 *              workspace of an ssm_scan_fwd_save call with the same descriptor
 *              and the same u, delta, A, B, C, h0 (and delta bias, convolution
 *              taps), unmodified in between; nothing checks this, and other
 *              contents give wrong gradients.
 * Every other argument, condition and error is that of ssm_scan_fwd and
 * ssm_scan_bwd. The caller owns the workspace and keeps it alive from the
 * forward call until the backward call has completed on its stream.
 */
int ssm_scan_fwd_save(const ssm_scan_desc *desc,
                      const void *u, const void *delta, const float *A,
                      const void *B, const void *C, const float *D, const void *z,
                      const float *h0, void *y, float *h_last,
                      void *workspace, size_t workspace_bytes, hipStream_t stream);
int ssm_scan_bwd_saved(const ssm_scan_desc *desc,
                       const void *u, const void *delta, const float *A,
                       const void *B, const void *C, const float *D, const void *z,
                       const float *h0, const void *dy, const float *dh_last,
                       void *du, void *ddelta, float *dA, float *dB, float *dC, float *dD,
                       void *dz, float *dh0, float *ddelta_bias, float *dconv_weight, float *dconv_bias,
                       void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * One decode step: the recurrence for a single new token per sequence, with
 * the fixed-size state updated in place (itwiki "상태 공간 모델", "순환 형태와
 * 합성곱 형태": generation only updates h_t; ricepunchb "Mamba" §4.2: only the
 * last hidden state is needed to produce the next token).
 *
 *   x, delta, z  (batch, dim)          dtype; z may be NULL (no gate)
 *   delta_bias   (dim) fp32 or NULL; delta_softplus 0 or 1: the step is
 *                softplus(delta + bias) as for the scan descriptor
 *   A            (dim, dstate)         fp32
 *   B, C         (batch, dstate)       dtype
 *   D            (dim) fp32 or NULL
 *   h            (batch, dim, dstate)  fp32, read and overwritten
 *   y            (batch, dim)          dtype, written; must not overlap h or an input
 * Equal to ssm_scan_fwd with seqlen 1, h0 = h and h_last = h.
 */
int ssm_state_update(int64_t batch, int64_t dim, int64_t dstate, int32_t dtype, int32_t disc,
                     const void *x, const void *delta, const float *delta_bias, int32_t delta_softplus,
                     const float *A,
                     const void *B, const void *C, const float *D, const void *z,
                     float *h, void *y, hipStream_t stream);

/*
 * Mamba-2 SSD layer (structured state-space duality). Each head h has a
 * scalar decay rate A[h] (the state matrix restricted to a scalar times the
 * identity: itwiki "상태 공간 모델", section "Mamba-2와 상태 공간 쌍대성";
 * eommydocs "State Space Models (SSM)", §2.4) and a (headdim x dstate) state;
 * the heads of a group share B and C. Per batch row b, head h, p < headdim:
 *
 *   dt_t    = dt[b,t,h] (+ dt_bias[h]), through softplus when dt_softplus
 *   H_t     = exp(dt_t A[h]) H_{t-1} + wbar_t x[b,t,h,:] B[b,t,g,:]^T     H_{-1} = h0 (or 0)
 *   wbar_t  = dt_t (SSM_DISC_EULER) or (exp(dt_t A[h]) - 1)/A[h] (SSM_DISC_ZOH)
 *   y[b,t,h,p] = sum_n C[b,t,g,n] H_t[p,n] + D[h] x[b,t,h,p],  times silu(z[b,t,h,p]) with a gate
 *
 * with g = h / (nheads / ngroups). The library evaluates it chunk by chunk
 * in the attention-like form of youngju.dev "mamba-state-space-model-
 * selective-ssm", SSDBlock._chunk_scan (scores C_i . B_j times the causal
 * decay exp(A (cum dt_i - cum dt_j)), applied to wbar x), with the state
 * carried from chunk to chunk, on bf16 matrix cores with fp32 accumulation;
 * the state is kept in fp32 and rounded to bf16 only as a matrix operand.
 */
typedef struct {
    int64_t batch;     /* >= 0 */
    int64_t seqlen;    /* >= 0 */
    int32_t nheads;    /* H >= 1 */
    int32_t headdim;   /* P: 64, 96 or 128 */
    int32_t ngroups;   /* G >= 1, dividing nheads */
    int32_t dstate;    /* N: 64 or 128 */
    int32_t dtype;     /* SSM_BF16 (SSM_F32 is reported as SSM_ERR_UNSUPPORTED) */
    int32_t disc;      /* ssm_disc */
    int32_t dt_softplus;    /* 0 or 1 */
    int32_t reserved;       /* 0 */
    const float *dt_bias;   /* (nheads) fp32 device pointer, or NULL */
} ssm_ssd_desc;

/*
 *   x, z      (batch, seqlen, nheads, headdim)  bf16, row-major; z may be NULL (no gate)
 *   dt        (batch, seqlen, nheads)           bf16
 *   A         (nheads) fp32 (negative for a decaying state); D (nheads) fp32 or NULL
 *   B, C      (batch, seqlen, ngroups, dstate)  bf16
 *   h0        (batch, nheads, headdim, dstate)  fp32, or NULL for zeros
 *   y         (batch, seqlen, nheads, headdim)  bf16, written
 *   h_last    (batch, nheads, headdim, dstate)  fp32, written, or NULL; may equal h0 exactly
 * x, z, y, B, C, h0 and h_last must be 16-byte aligned (dt 2-byte, A, D,
 * dt_bias 4-byte): SSM_ERR_ALIGN otherwise. Outputs must not overlap inputs
 * or each other (SSM_ERR_ALIAS). No workspace. seqlen == 0 writes h_last = h0
 * (or zeros) and no y.
 */
int ssm_ssd_fwd(const ssm_ssd_desc *desc, const void *x, const void *dt, const float *A,
                const void *B, const void *C, const float *D, const void *z, const float *h0,
                void *y, float *h_last, hipStream_t stream);

/*
 * One decode step of the SSD layer: the recurrence above for a single new
 * token per sequence, with each head's (headdim x dstate) state updated in
 * place (itwiki "상태 공간 모델", "순환 형태와 합성곱 형태": generation only
 * updates the state; the SSD layer's state as above). desc->seqlen must be 1.
 *
 *   x, z      (batch, nheads, headdim)   bf16; z may be NULL (no gate)
 *   dt        (batch, nheads)            bf16 (desc->dt_bias, dt_softplus and disc as for ssm_ssd_fwd)
 *   A, D      (nheads) fp32; D may be NULL
 *   B, C      (batch, ngroups, dstate)   bf16, 8-byte aligned
 *   h         (batch, nheads, headdim, dstate) fp32, 16-byte aligned, read and overwritten
 *   y         (batch, nheads, headdim)   bf16, written; must not overlap h or an input
 * Equal to ssm_ssd_fwd with seqlen 1, h0 = h and h_last = h, computed
 * directly in fp32 (no matrix cores: one token is a rank-1 update).
 */
int ssm_ssd_state_update(const ssm_ssd_desc *desc, const void *x, const void *dt, const float *A,
                         const void *B, const void *C, const float *D, const void *z, float *h,
                         void *y, hipStream_t stream);

/*
 * The gated delta rule: a linear-recurrence mixer whose (headdim x dstate)
 * state per head is decayed like the SSD layer's and then corrected along the
 * token's key instead of added to. Per batch row b and head h, with
 * g = h / (nheads / ngroups):
 *
 *   step_t = dt[b,t,h] (+ dt_bias[h]), through softplus when dt_softplus
 *   w_t    = beta[b,t,h], through the logistic sigmoid when beta_sigmoid
 *   k_t, q_t = k[b,t,g,:], q[b,t,g,:]; with qk_norm each divided by
 *            sqrt(its sum of squares + qk_eps)
 *   H_t    = a_t H_{t-1} + w_t (v[b,t,h,:] - a_t H_{t-1} k_t) k_t^T,
 *            a_t = exp(step_t A[h]),  H_{-1} = h0 (or 0)
 *   y[b,t,h,:] = scale * H_t q_t
 *
 * The sequence is evaluated in chunks of 64 tokens on bf16 matrix cores. Every
 * fp32 operand is split into three bf16 parts, so states and fp32 gradients
 * are as exact as fp32 arithmetic makes them, and y is such a value rounded once
 * to bf16. The matrix inverse of a chunk is that of a unit lower
 * triangular matrix, by substitution, and needs no bound on the keys; but the
 * recurrence itself grows without bound unless w_t |k_t|^2 <= 2. A step that
 * decays the state to nothing (also an infinite one with A < 0) is a reset. Any
 * other NaN or infinity among step_t, A, w_t, k_t, q_t, v, the states and the
 * incoming gradients makes whatever depends on it by the formulas NaN or infinite:
 * step, A, w and k of a head its y and state from that token on, a value of v or
 * h0 those of its row p, q_t its own y. Tokens of the same chunk of 64 that do not
 * depend on it (the earlier ones, in a backward the later ones) may become NaN
 * too; chunks that do not, other heads and other batch rows keep their values.
 */
typedef struct {
    int64_t batch;     /* >= 0 */
    int64_t seqlen;    /* >= 0 */
    int32_t nheads;    /* H >= 1: heads of v, dt, beta, y */
    int32_t headdim;   /* P: a multiple of 16 in 16..256 */
    int32_t ngroups;   /* G >= 1, dividing nheads: heads of q and k */
    int32_t dstate;    /* N: 64 or 128 */
    int32_t dtype;     /* SSM_BF16 (SSM_F32 is reported as SSM_ERR_UNSUPPORTED) */
    int32_t dt_softplus;    /* 0 or 1 */
    int32_t beta_sigmoid;   /* 0 or 1 */
    int32_t qk_norm;        /* 0 or 1 */
    float scale;            /* of the readout; finite */
    float qk_eps;           /* > 0 with qk_norm, else unused */
    /* elements from one token's row to the next of q, k, v, dt, beta (of one
     * batch row to the next: seqlen times that); 0 for densely packed rows. A
     * row itself is dense. Strides of q, k, v are multiples of 8; over a
     * sequence (not for the one-token step) none is over 2^24 - 1. */
    int64_t q_stride, k_stride, v_stride, dt_stride, beta_stride;
    const float *dt_bias;   /* (nheads) fp32 device pointer, or NULL */
} ssm_gdr_desc;

/* Bytes of device workspace of the forward, and of the backward and the
 * training pair; 0 when there is nothing to compute and for an invalid
 * descriptor. */
size_t ssm_gdr_workspace_size(const ssm_gdr_desc *desc);
size_t ssm_gdr_bwd_workspace_size(const ssm_gdr_desc *desc);

/*
 *   q, k      (batch, seqlen, ngroups, dstate)  bf16
 *   v         (batch, seqlen, nheads, headdim)  bf16
 *   dt, beta  (batch, seqlen, nheads)           bf16
 *   A         (nheads) fp32 (negative for a decaying state)
 *   h0        (batch, nheads, headdim, dstate)  fp32, or NULL for zeros
 *   y         (batch, seqlen, nheads, headdim)  bf16, dense, written
 *   h_last    (batch, nheads, headdim, dstate)  fp32, written, or NULL; may equal h0 exactly
 *   workspace ssm_gdr_workspace_size(desc) bytes, 256-byte aligned; its
 *             contents on entry do not matter and are clobbered
 * q, k, v, y, h0 and h_last must be 16-byte aligned (dt, beta 2-byte, A,
 * dt_bias 4-byte). Outputs must not overlap inputs, each other or the
 * workspace. seqlen == 0 writes h_last = h0 (or zeros) and no y. Sizes that need
 * 2^32 work items in a launch are refused (SSM_ERR_SHAPE) before the first: from 2^24
 * chunks of 64 tokens, counted over batch rows and heads, from 2^22 heads of 256
 * columns, and in a backward from 2^32 / (4 dstate) chunks counted over groups.
 */
int ssm_gdr_fwd(const ssm_gdr_desc *desc, const void *q, const void *k, const void *v, const void *dt,
                const void *beta, const float *A, const float *h0, void *y, float *h_last,
                void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Gradients of  sum dy . y + sum dh_last . h_last  with respect to everything
 * ssm_gdr_fwd reads (dt, beta, q and k as given, before softplus, sigmoid and
 * the unit lengths).
 *   dy        (batch, seqlen, nheads, headdim)  bf16, dense, 16-byte aligned
 *   dh_last   (batch, nheads, headdim, dstate)  fp32, or NULL (0)
 *   dq, dk    (batch, seqlen, ngroups, dstate)  bf16, dense, written (summed over a group's heads)
 *   dv        (batch, seqlen, nheads, headdim)  bf16, dense, written
 *   ddt, dbeta (batch, seqlen, nheads)          bf16, dense, written
 *   dA        (nheads) fp32, written (summed over batch and time)
 *   ddt_bias  (nheads) fp32, written; required when desc->dt_bias is given, unused otherwise
 *   dh0       (batch, nheads, headdim, dstate)  fp32, written, or NULL (not wanted); may equal dh_last exactly
 *   workspace ssm_gdr_bwd_workspace_size(desc) bytes, 256-byte aligned
 * ssm_gdr_fwd_save is ssm_gdr_fwd (same results) that leaves in `workspace`
 * (ssm_gdr_bwd_workspace_size bytes) what the backward would first recompute;
 * ssm_gdr_bwd_saved is ssm_gdr_bwd reading it there. It must receive the
 * workspace of an ssm_gdr_fwd_save call with the same descriptor and inputs,
 * unmodified; nothing checks this. It clobbers the workspace's other parts
 * only, so it may run again on the same saved contents.
 * Every sum is taken in a fixed order: results do not depend on timing. Each term
 * of ddt, dA and ddt_bias has the token's own decay as a factor, so that strong
 * decays keep their digits.
 * seqlen == 0 writes dA = 0, ddt_bias = 0, dh0 = dh_last (or zeros).
 */
int ssm_gdr_bwd(const ssm_gdr_desc *desc, const void *q, const void *k, const void *v, const void *dt,
                const void *beta, const float *A, const float *h0, const void *dy, const float *dh_last,
                void *dq, void *dk, void *dv, void *ddt, void *dbeta, float *dA, float *ddt_bias, float *dh0,
                void *workspace, size_t workspace_bytes, hipStream_t stream);
int ssm_gdr_fwd_save(const ssm_gdr_desc *desc, const void *q, const void *k, const void *v, const void *dt,
                     const void *beta, const float *A, const float *h0, void *y, float *h_last,
                     void *workspace, size_t workspace_bytes, hipStream_t stream);
int ssm_gdr_bwd_saved(const ssm_gdr_desc *desc, const void *q, const void *k, const void *v, const void *dt,
                      const void *beta, const float *A, const float *h0, const void *dy, const float *dh_last,
                      void *dq, void *dk, void *dv, void *ddt, void *dbeta, float *dA, float *ddt_bias,
                      float *dh0, void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * One decode step of the gated delta rule: desc->seqlen must be 1 (the strides
 * are then those from one batch row to the next).
 *   q, k      (batch, ngroups, dstate)  bf16, 8-byte aligned, strides multiples of 4
 *   v         (batch, nheads, headdim)  bf16;  dt, beta (batch, nheads) bf16
 *   h         (batch, nheads, headdim, dstate) fp32, 16-byte aligned, read
 *   h_out     the same shape, written; h itself for an update in place
 *   y         (batch, nheads, headdim)  bf16, written
 * Computed in fp32 without matrix cores. y must not overlap anything else,
 * h_out nothing but h, and that exactly. A workgroup takes a head's 64 rows of 64
 * or 32 of 128; 2^24 workgroups are refused (SSM_ERR_SHAPE).
 */
int ssm_gdr_state_update(const ssm_gdr_desc *desc, const void *q, const void *k, const void *v, const void *dt,
                         const void *beta, const float *A, const float *h, float *h_out, void *y,
                         hipStream_t stream);

/*
 * The residual add and RMS norm before a block. Per row (token) of `dim`
 * channels, all arithmetic in fp32:
 *
 *   r = residual + scale * x      (scale (dim): a learned scale per channel; NULL: 1; residual NULL: 0)
 *   y = r / sqrt(mean(r^2) + eps) * weight
 *
 * r is first rounded to residual_dtype, and y is that of the rounded r: what
 * the next layer adds to is what was normed.
 *
 * A row takes a part of a workgroup up to 2048 channels of 16 bits (1024 of 32;
 * 256 when rows or pointers are not 16-byte aligned) and a workgroup of 256 work
 * items beyond. Sizes that need 2^32 work items are refused (SSM_ERR_SHAPE): from
 * 2^24 such long rows.
 */
typedef struct {
    int64_t rows;            /* >= 0 */
    int64_t dim;             /* 1..2^20 */
    int32_t dtype;           /* of x, y, dy, dx */
    int32_t residual_dtype;  /* of residual, r, dr, dresidual: dtype, or SSM_F32 */
    float eps;               /* >= 0 */
    int32_t reserved;        /* 0 */
    int64_t x_stride;        /* elements from row to row of x; 0: dim */
} ssm_prenorm_desc;

/*
 *   x         (rows, dim)  dtype
 *   residual  (rows, dim)  residual_dtype, or NULL
 *   scale     (dim) fp32, or NULL
 *   weight    (dim) fp32
 *   r         (rows, dim)  residual_dtype, written; may equal residual
 *             exactly; or NULL (not wanted)
 *   y         (rows, dim)  dtype, written
 * Pointers need their element's alignment only (16-byte aligned rows move
 * faster). Other overlaps of outputs are refused.
 */
int ssm_prenorm_fwd(const ssm_prenorm_desc *desc, const void *x, const void *residual, const float *scale,
                    const float *weight, void *r, void *y, hipStream_t stream);

/*
 * Gradients of  sum dy . y + sum dr . r.
 *   r         (rows, dim)  residual_dtype: what the forward wrote
 *   dr        (rows, dim)  residual_dtype, or NULL (0)
 *   x, scale  as the forward's; x is read only with a scale
 *   dx        (rows, dim)  dtype, dense, written
 *   dresidual (rows, dim)  residual_dtype, written, or NULL (not wanted); may equal dr exactly
 *   dweight   (dim) fp32, written
 *   dscale    (dim) fp32, written; required with a scale, unused otherwise
 *   workspace ssm_prenorm_bwd_workspace_size(desc) bytes, 256-byte aligned
 * Sums over rows are taken in a fixed order.
 */
size_t ssm_prenorm_bwd_workspace_size(const ssm_prenorm_desc *desc);
int ssm_prenorm_bwd(const ssm_prenorm_desc *desc, const void *dy, const void *r, const void *dr, const void *x,
                    const float *scale, const float *weight, void *dx, void *dresidual, float *dweight,
                    float *dscale, void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * The gated RMS norm behind a mixer. Per row (token) and group of `dim`
 * channels, in fp32:
 *
 *   gate_first 0:  y = x / sqrt(mean(x^2) + eps) * weight * silu(z)
 *   gate_first 1:  f = x * silu(z),  y = f / sqrt(mean(f^2) + eps) * weight
 *
 * z NULL: no gate. weight is (groups, dim), or (dim) for every group with
 * weight_shared (a norm per head with one weight for all heads). Sizes that need
 * 2^32 work items are refused as above, a group counting as a row; so is the
 * backward of 2^26 weights.
 */
typedef struct {
    int64_t rows;            /* >= 0 */
    int64_t groups;          /* >= 1 */
    int64_t dim;             /* channels of a group, 1..2^20 */
    int32_t dtype;           /* of x, z, y and their gradients */
    int32_t gate_first;      /* 0 or 1 */
    int32_t weight_shared;   /* 0 or 1 */
    float eps;               /* >= 0 */
    int64_t x_stride, z_stride;   /* elements from row to row; 0: groups * dim */
} ssm_gated_norm_desc;

/*
 *   x, z      (rows, groups, dim)  dtype; z may be NULL
 *   y         (rows, groups, dim)  dtype, dense, written
 * Backward: dy, dx, dz (rows, groups, dim) dtype, dense; dz is required with
 * z, unused otherwise; dweight fp32 in weight's shape. Outputs must not
 * overlap inputs, each other or the workspace (ssm_gated_norm_bwd_workspace_size
 * bytes, 256-byte aligned).
 */
int ssm_gated_norm_fwd(const ssm_gated_norm_desc *desc, const void *x, const void *z, const float *weight,
                       void *y, hipStream_t stream);
size_t ssm_gated_norm_bwd_workspace_size(const ssm_gated_norm_desc *desc);
int ssm_gated_norm_bwd(const ssm_gated_norm_desc *desc, const void *dy, const void *x, const void *z,
                       const float *weight, void *dx, void *dz, float *dweight,
                       void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * The gated linear recurrence. Per batch row and channel, in fp32, with
 * r = sigmoid(rgate), i = sigmoid(igate):
 *
 *   a_t = exp(-rate * softplus(lam) * r_t)          0 where reset_t is set
 *   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t     h_{-1} = h0 (or 0)
 *   y_t = h_t * gate_t                              gate NULL: h_t
 *
 * A reset starts a sequence inside a row: nothing before it reaches what follows,
 * were it NaN or infinite. rgate of minus infinity (a = 1) leaves the state as it
 * is, for tokens that pad a row (x, igate finite); a gate of 0 in its place zeroes
 * y. Any other NaN or infinity makes NaN or infinite what depends on it by the
 * formulas; tokens of the same run of 8 or 16 behind which it stands, other channels
 * and other batch rows keep their values.
 * A row takes one workgroup per 64 channels (32 where channels or addresses do not
 * allow two at a time) and chunk: of 512 work items for 128 or 256 tokens forward, of
 * 256 for 64 tokens backward. Sizes that need 2^32 work items in a launch, counted for
 * the smaller pieces, are refused (SSM_ERR_SHAPE) before the first.
 * Workgroups wait for one another through the workspace: it serves one call at a time,
 * and calls on two streams need one each.
 */
typedef struct {
    int64_t batch;     /* >= 0 */
    int64_t seqlen;    /* >= 0 */
    int64_t dim;       /* 1..2^24 - 1 */
    int32_t dtype;     /* of x, rgate, igate, gate, y and their gradients */
    float rate;        /* >= 0, finite */
    /* elements from one token's row to the next (of one batch row to the next:
     * seqlen times that), up to 2^24 - 1; 0: dim. A row itself is dense. */
    int64_t x_stride, rgate_stride, igate_stride, gate_stride;
} ssm_glr_desc;

/* Bytes of device workspace of the forward (0 for one chunk), and of the backward
 * and the training pair; 0 for an invalid descriptor. */
size_t ssm_glr_workspace_size(const ssm_glr_desc *desc);
size_t ssm_glr_bwd_workspace_size(const ssm_glr_desc *desc);

/*
 *   x, rgate, igate, gate  (batch, seqlen, dim)  dtype; gate may be NULL
 *   lam       (dim) fp32
 *   h0        (batch, dim) fp32, or NULL for zeros
 *   reset     (batch, seqlen) bytes, not 0 at a sequence's first token; or NULL
 *   y         (batch, seqlen, dim)  dtype, dense, written
 *   h_last    (batch, dim) fp32, written, or NULL; may equal h0 exactly
 *   workspace ssm_glr_workspace_size(desc) bytes, 256-byte aligned; its contents on
 *             entry do not matter and are clobbered
 * Pointers need their element's alignment only (pairs of channels move faster).
 * Outputs must not overlap inputs, each other or the workspace. seqlen == 0 writes
 * h_last = h0 (or zeros). Results do not depend on timing.
 */
int ssm_glr_fwd(const ssm_glr_desc *desc, const void *x, const void *rgate, const void *igate, const float *lam,
                const float *h0, const void *gate, const uint8_t *reset, void *y, float *h_last,
                void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Gradients of  sum dy . y + sum dh_last . h_last.
 *   dy        (batch, seqlen, dim)  dtype, dense
 *   dh_last   (batch, dim) fp32, or NULL (0)
 *   dx, drgate, digate  (batch, seqlen, dim)  dtype, dense, written
 *   dgate     the same; required with a gate, unused otherwise
 *   dlam      (dim) fp32, written (summed over batch and time in a fixed order)
 *   dh0       (batch, dim) fp32, written, or NULL (not wanted); may equal dh_last exactly
 *   workspace ssm_glr_bwd_workspace_size(desc) bytes, 256-byte aligned
 * ssm_glr_fwd_save is ssm_glr_fwd (same results) that leaves in `workspace`
 * (ssm_glr_bwd_workspace_size bytes) the state before every 64 tokens, which
 * ssm_glr_bwd would first recompute; ssm_glr_bwd_saved is ssm_glr_bwd reading them
 * there. It must receive the workspace of an ssm_glr_fwd_save call with the same
 * descriptor and inputs; nothing checks this. It clobbers the workspace's other
 * parts only, so it may run again on the same saved contents.
 * seqlen == 0 writes dlam = 0, dh0 = dh_last (or zeros).
 */
int ssm_glr_bwd(const ssm_glr_desc *desc, const void *x, const void *rgate, const void *igate, const float *lam,
                const float *h0, const void *gate, const uint8_t *reset, const void *dy, const float *dh_last,
                void *dx, void *drgate, void *digate, void *dgate, float *dlam, float *dh0,
                void *workspace, size_t workspace_bytes, hipStream_t stream);
int ssm_glr_fwd_save(const ssm_glr_desc *desc, const void *x, const void *rgate, const void *igate, const float *lam,
                     const float *h0, const void *gate, const uint8_t *reset, void *y, float *h_last,
                     void *workspace, size_t workspace_bytes, hipStream_t stream);
int ssm_glr_bwd_saved(const ssm_glr_desc *desc, const void *x, const void *rgate, const void *igate, const float *lam,
                      const float *h0, const void *gate, const uint8_t *reset, const void *dy, const float *dh_last,
                      void *dx, void *drgate, void *digate, void *dgate, float *dlam, float *dh0,
                      void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * One token: desc->seqlen must be 1 (the strides are then those from one batch row
 * to the next).
 *   x, rgate, igate, gate  (batch, dim)  dtype; gate may be NULL
 *   reset     (batch) bytes, or NULL
 *   h         (batch, dim) fp32, read;  h_out the same shape, written: h itself for
 *             an update in place, or apart from everything else
 *   y         (batch, dim)  dtype, dense, written
 */
int ssm_glr_state_update(const ssm_glr_desc *desc, const void *x, const void *rgate, const void *igate,
                         const float *lam, const void *gate, const uint8_t *reset, const float *h, float *h_out,
                         void *y, hipStream_t stream);

/*
 * A projection: a matrix product with what follows it. Per row (token) and group,
 *
 *   pre = x W^T + bias,   y = act(pre) + residual
 *
 * groups 1 is a linear layer, more a block-diagonal one (the gates of a recurrence).
 * bf16 products are summed in fp32 on the matrix cores, fp32 ones are full fp32; bias,
 * activation and residual are applied to the fp32 sums, and y and pre are rounded once.
 * gelu is the form z sigmoid(2 sqrt(2 / pi) (z + 0.044715 z^3)).
 *
 * Up to 16 rows the forward reads the weight once without tiles, unless its rows are
 * long. Results do not depend on timing, nor on other rows' values; they may differ by
 * rounding between numbers of rows. Sizes that need 2^32 work items in a launch are refused (SSM_ERR_SHAPE).
 */
typedef enum { SSM_ACT_NONE = 0, SSM_ACT_SILU = 1, SSM_ACT_GELU = 2, SSM_ACT_SIGMOID = 3 } ssm_activation;

typedef struct {
    int64_t rows;            /* 0..2^31 - 1 */
    int64_t groups;          /* >= 1 */
    int64_t in, out;         /* values of a group in x and in y, >= 1; groups times either < 2^22 */
    int32_t dtype;           /* of x, weight, pre and their gradients */
    int32_t y_dtype;         /* of residual, y, dy: dtype, or SSM_F32 */
    int32_t activation;      /* ssm_activation */
    int32_t reserved;        /* 0 */
    int64_t x_stride;        /* elements from row to row of x, < 2^22; 0: groups * in */
} ssm_proj_desc;

/*
 *   x         (rows, groups, in)        dtype
 *   weight    (groups, out, in)         dtype
 *   bias      (groups, out) fp32, or NULL
 *   residual  (rows, groups, out)       y_dtype, or NULL
 *   pre       (rows, groups, out)       dtype, written, or NULL (not wanted)
 *   y         (rows, groups, out)       y_dtype, written; may equal residual exactly
 *   workspace ssm_proj_workspace_size(desc) bytes, 256-byte aligned; its contents on
 *             entry do not matter. The size goes with x_stride too, and fewer rows may
 *             need more (a product of few tiles is split): one workspace for several
 *             descriptors, here or in the backward, has the largest of their sizes
 * Pointers need their element's alignment only (rows of whole 4-byte words move faster).
 * Other overlaps of outputs are refused.
 */
size_t ssm_proj_workspace_size(const ssm_proj_desc *desc);
int ssm_proj_fwd(const ssm_proj_desc *desc, const void *x, const void *weight, const float *bias,
                 const void *residual, void *pre, void *y, void *workspace, size_t workspace_bytes,
                 hipStream_t stream);

/*
 * Gradients of sum dy . y (that of the residual is dy).
 *   dy        (rows, groups, out)  y_dtype, dense
 *   pre       what the forward wrote; read with an activation only
 *   dpre      (rows, groups, out)  dtype, written: dy act'(pre), rounded; required with an
 *             activation and where dy is not of dtype, else unused (dy serves)
 *   dx        (rows, groups, in)   dtype, dense, written, or NULL (not wanted): that of dpre as stored
 *   dweight   (groups, out, in)    dtype, written, or NULL: that of dpre as stored
 *   dbias     (groups, out) fp32, written, or NULL: the sum of dpre before its rounding
 *   x is read for dweight, weight for dx; each may be NULL without
 *   workspace ssm_proj_bwd_workspace_size(desc) bytes, 256-byte aligned
 * Sums over rows are taken in a fixed order. rows == 0 writes dweight = 0, dbias = 0.
 */
size_t ssm_proj_bwd_workspace_size(const ssm_proj_desc *desc);
int ssm_proj_bwd(const ssm_proj_desc *desc, const void *dy, const void *x, const void *weight, const void *pre,
                 void *dpre, void *dx, void *dweight, float *dbias, void *workspace, size_t workspace_bytes,
                 hipStream_t stream);

/*
 * The norm over all gradients of a model, and their clipping by it:
 *
 *   norm = sqrt(sum over tensors and elements of g^2)   squares and sums in 64 bits
 *   g   <- g * min(1, max_norm / (norm + eps))          factor and product in fp32, rounded once
 *
 * A norm of infinity, which one beyond fp32's range is too, makes finite gradients 0, one
 * of NaN makes all of them NaN; one of 0 leaves them, also without eps. ssm_grad_clip's factor
 * comes from the norm in 64 bits, ssm_grad_scale's from the one in fp32 that it is given: they
 * may differ by its rounding.
 *   count     tensors, 0..2^20; every array below is a HOST array of so many values
 *   grads     device pointers of dense tensors, their element's alignment
 *   out       the same for what is written: grads[k] itself, or apart from everything
 *   sizes     elements, 0..2^35; pointers of empty tensors are not looked at
 *   dtypes    SSM_F32 or SSM_BF16, one for each
 *   norm      one fp32 on the device, written; ssm_grad_scale reads it, for a norm
 *             over more tensors than these (those of other GPUs)
 *   workspace ssm_grad_workspace_size(count) bytes, 256-byte aligned
 * What is written overlaps nothing else; the same gradient twice in one list is
 * refused (SSM_ERR_ALIAS) where it is written and counts twice in ssm_grad_norm. The
 * host arrays are not read after the call returns. Results do not depend on timing;
 * tensors go 128 to a launch.
 */
size_t ssm_grad_workspace_size(int64_t count);
int ssm_grad_norm(int64_t count, const void *const *grads, const int64_t *sizes, const int32_t *dtypes,
                  float *norm, void *workspace, size_t workspace_bytes, hipStream_t stream);
int ssm_grad_clip(int64_t count, const void *const *grads, void *const *out, const int64_t *sizes,
                  const int32_t *dtypes, float max_norm, float eps, float *norm,
                  void *workspace, size_t workspace_bytes, hipStream_t stream);
int ssm_grad_scale(int64_t count, const void *const *grads, void *const *out, const int64_t *sizes,
                   const int32_t *dtypes, const float *norm, float max_norm, float eps, hipStream_t stream);

/* Static, NUL-terminated description of a status code. */
const char *ssm_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* SSM_SCAN_H */
