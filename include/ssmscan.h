/*
 * ssmscan.h -- C ABI of libssmscan.so: the Mamba selective-scan forward
 * operator and its width-4 causal depthwise conv prologue, for AMD MI355X
 * (gfx950).
 *
 * Operation (PaddleNLP Kernel operator-library guide, section 4.1
 * "selective_scan": selective_scan_fn(u, delta, A, B, C, D, z, delta_bias,
 * delta_softplus, return_last_state)).  For every batch b, channel d and
 * state s, with delta' = softplus(delta + delta_bias) when delta_softplus is
 * set (otherwise delta + delta_bias):
 *
 *     x_t[s] = exp(delta'_t * A[d,s]) * x_{t-1}[s] + delta'_t * B_t[s] * u_t
 *     y_t    = sum_s C_t[s] * x_t[s]
 *     out_t  = (y_t + D[d] * u_t) * silu(z_t)          (D, z optional)
 *     last_state[b,d,s] = x_{seqlen-1}[s]              (optional)
 *
 * with x_{-1} = initial_state (zero when not given).  The recurrence is not
 * printed on the pages; it is the standard zero-order-hold discretisation.
 *
 * Shapes (same section): u, delta, z, out: (batch, dim, seqlen); A: (dim,
 * dstate), real; B and C each either fixed (dim, dstate) or time-varying
 * grouped (batch, ngroups, dstate, seqlen) -- the page's 3-D (batch, dstate,
 * seqlen) form is ngroups = 1; D, delta_bias: (dim,); last_state and
 * initial_state: (batch, dim, dstate).  Grouped channel d uses group
 * d / (dim / ngroups).
 *
 * Conventions for every entry point:
 *  - Pointers are DEVICE pointers to dense row-major tensors (innermost
 *    stride 1).  The caller owns and allocates every buffer, including the
 *    outputs.  `out` must not alias an input.
 *  - "io" tensors (u, delta, z, B, C, out, conv x) all have the dtype
 *    io_dtype: SSM_F32 (IEEE binary32), SSM_BF16 (bfloat16, stored as the
 *    upper 16 bits of a binary32) or SSM_F16 (IEEE binary16).  A, D, delta_bias, conv weight and bias,
 *    initial_state and last_state are always binary32; the state is binary32.
 *    bf16 and fp16 outputs are rounded to nearest, ties to even.
 *  - Work is enqueued asynchronously on `hip_stream` (a hipStream_t; NULL is
 *    the default stream).  Nothing synchronises.
 *  - Errors: arguments are checked on the host before anything is enqueued.
 *    Status 1-3 and 5 leave all memory untouched.  Status 4 means a HIP call
 *    failed while enqueueing (ssm_last_hip_error() gives the hipError_t).
 *  - The library allocates no memory and reads no environment variables: the
 *    caller passes every buffer, scratch included (the *_workspace_size
 *    queries give the size).  It keeps no state between calls except a
 *    cached device property query; calls from several host threads are safe.
 */
#ifndef SSMSCAN_H
#define SSMSCAN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_ABI_VERSION 13
#define SSM_CKPT_INTERVAL 32  /* timesteps between saved states (checkpoints) */
#define SSM_MAX_DSTATE 16   /* largest dstate the kernels are built for */
#define SSM_CONV_WIDTH 4    /* the one conv width the kernels are built for */
#define SSM_NOALLOC_SCRATCH_BYTES (8u << 20)   /* built-in scratch of ssm_scan_fwd_noalloc, per device */

/* io dtype.  SSM_F16 (IEEE binary16) is taken by every entry point except
 * ssd_scan_fwd (bf16 only), which returns SSM_ERR_UNSUPPORTED for it. */
enum { SSM_F32 = 0, SSM_BF16 = 1, SSM_F16 = 2 };
/* layout of B and C (one kind per tensor) */
enum { SSM_BC_FIXED = 0,    /* (dim, dstate) */
       SSM_BC_VARYING = 1   /* (batch, ngroups, dstate, seqlen) */ };
/* conv activation ("swish" on the page is silu) */
enum { SSM_ACT_NONE = 0, SSM_ACT_SILU = 1 };
/* status codes */
enum {
  SSM_OK = 0,
  SSM_ERR_NULL = 1,         /* a required pointer is NULL */
  SSM_ERR_SHAPE = 2,        /* a size <= 0, dim % ngroups != 0, or overflow */
  SSM_ERR_UNSUPPORTED = 3,  /* dtype, dstate > 16, conv width != 4, bad enum */
  SSM_ERR_HIP = 4,          /* a HIP runtime call failed */
  SSM_ERR_WORKSPACE = 5,    /* scratch needed but workspace NULL or too small */
  SSM_ERR_SCRATCH = 6       /* ssm_scan_fwd_noalloc: the plan needs more than its scratch */
};

/* Arguments of ssm_scan_fwd.  Every pointer is a device pointer. */
typedef struct ssm_scan_args {
  int64_t batch, dim, seqlen, dstate, ngroups;  /* ngroups: 1 unless grouped */
  int32_t io_dtype;                             /* SSM_F32 or SSM_BF16 */
  const void *u;                                /* (b,d,l) io; ignored with conv */
  const void *delta;                            /* (b,d,l) io, required */
  const float *A;                               /* (d,n) fp32, required */
  const void *B; int32_t B_kind;                /* io, SSM_BC_* */
  const void *C; int32_t C_kind;                /* io, SSM_BC_* */
  const float *D;                               /* (d) fp32 or NULL */
  const float *delta_bias;                      /* (d) fp32 or NULL */
  const void *z;                                /* (b,d,l) io or NULL */
  int32_t delta_softplus;                       /* 0 or 1 */
  void *out;                                    /* (b,d,l) io, required */
  float *last_state;                            /* (b,d,n) fp32 or NULL */
  const float *initial_state;                   /* (b,d,n) fp32 or NULL (zero) */
  /* Optional fused conv prologue (same page, section 4.2 causal_conv1d):
   * when conv_weight != NULL, u is not read and is replaced by
   *   u = round_io(act(conv_bias[d] + sum_k conv_weight[d,k] * conv_x[b,d,t-3+k]))
   * with conv_x[t<0] = 0 -- exactly what causal_conv1d_fwd stores. */
  const void *conv_x;                           /* (b,d,l) io */
  const float *conv_weight;                     /* (d, conv_width) fp32 */
  const float *conv_bias;                       /* (d) fp32 or NULL */
  int32_t conv_width;                           /* must be 4 */
  int32_t conv_act;                             /* SSM_ACT_* */
  /* Scratch for the sequence-split plan (see ssm_scan_workspace_size),
   * caller-allocated device memory of workspace_bytes bytes.  The library
   * allocates nothing: when the plan needs scratch and workspace is NULL or
   * smaller than ssm_scan_workspace_size reports, the call returns
   * SSM_ERR_WORKSPACE before anything is enqueued.  It is not read before it
   * is written, so it needs no clearing, and it may be reused once the call's
   * work on hip_stream has finished. */
  void *workspace;
  size_t workspace_bytes;
  /* Optional output for the backward (ssm_scan_bwd): the state before every
   * SSM_CKPT_INTERVAL-th timestep, (batch, dim, nck, dstate) fp32 with
   * nck = ceil(seqlen / SSM_CKPT_INTERVAL); entry k is x_{k*32-1}, so entry 0
   * is initial_state (zero when not given).  NULL: not written. */
  float *checkpoints;
  /* Sequence split: 0 lets the library choose its plan (it splits the
   * sequence only when the channels alone leave the GPU short of waves, and
   * at dstate 13..16 may run leftover channels with eight lanes per channel
   * to even out the load per SIMD); k >= 1 asks for k segments (equal
   * lengths of whole chunks, so possibly fewer) of the four-lane kernel.
   * The plan changes the results only by rounding order.  Negative values
   * return SSM_ERR_SHAPE. */
  int32_t seq_segments;
} ssm_scan_args_t;

/* Selective-scan forward.  Enqueues the scan on hip_stream and returns a
 * status code (SSM_OK on success). */
int ssm_scan_fwd(const ssm_scan_args_t *args, void *hip_stream);

/* ssm_scan_fwd for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments, results and status codes as ssm_scan_fwd, except that
 * args->workspace and workspace_bytes are ignored: the scratch of the plan
 * (the sequence segments' end states) lives in a buffer built into the
 * library, SSM_NOALLOC_SCRATCH_BYTES per device, held until the process
 * ends.  A plan that needs more scratch than that returns SSM_ERR_SCRATCH
 * before anything is enqueued (ssm_scan_workspace_size gives the need; the
 * Mamba-shaped layers need at most 6.6 MiB).  The caller still allocates
 * every input and output.  The call allocates nothing: the first call on a
 * device looks the buffer's address up once (hipGetSymbolAddress).  Every
 * call on one device shares that device's buffer and leaves its contents
 * behind, so calls that overlap on one device -- different streams, or
 * different threads -- race and give wrong results; calls ordered on one
 * stream are safe. */
int ssm_scan_fwd_noalloc(const ssm_scan_args_t *args, void *hip_stream);

/* Host-only argument check of ssm_scan_fwd: the same status the call would
 * return before enqueueing anything.  Touches no device memory and makes no
 * HIP call, so it is usable on a machine without a GPU. */
int ssm_scan_validate(const ssm_scan_args_t *args);

/* Scratch bytes ssm_scan_fwd needs for these arguments (0 when the plan keeps
 * the whole sequence in one pass).  Host-only: no HIP call except cached
 * queries of the device's compute-unit count and of how many workgroups of
 * a kernel one compute unit holds (on a machine without a GPU those fail and
 * the plan assumes 256 compute units and no mixed plan). */
int ssm_scan_workspace_size(const ssm_scan_args_t *args, size_t *bytes);

/* The launch plan ssm_scan_fwd takes for these arguments (same queries as
 * ssm_scan_workspace_size).  Every wave runs lanes_per_channel lanes per
 * channel over 64 / lanes_per_channel channels; at dstate 13..16 the mixed
 * plan runs the channel blocks left over after whole waves fill the SIMDs
 * evenly as eight_lane_waves waves of eight lanes per channel (8 channels,
 * about half the work each). */
typedef struct {
  int32_t segments;            /* sequence segments (1: one pass) */
  int32_t waves;               /* waves of lanes_per_channel lanes, per segment */
  int32_t lanes_per_channel;
  int32_t eight_lane_waves;    /* mixed plan's extra waves (0: not mixed) */
  size_t workspace_bytes;      /* as ssm_scan_workspace_size */
} ssm_scan_plan_t;
int ssm_scan_plan(const ssm_scan_args_t *args, ssm_scan_plan_t *plan);

/* Selective-scan forward with complex A (the same page, section 4.1: A
 * (dim, dstate) may be real or complex; nothing more is printed about the
 * complex case).  Read as the recurrence above over the complex numbers, with
 * B and C complex too (a real B or C is the case of zero imaginary parts),
 * and the output the real part of the contraction:
 *
 *     x_t[s] = exp(delta'_t A[d,s]) x_{t-1}[s] + delta'_t B_t[s] u_t   (complex)
 *     y_t    = Re(sum_s C_t[s] x_t[s]),   out_t = (y_t + D[d] u_t) silu(z_t)
 *
 * delta', u, z, D, delta_bias and out are real as in ssm_scan_fwd.  The
 * arguments are those of ssm_scan_fwd with these layouts, every complex value
 * a (real, imaginary) pair with the pair innermost:
 *   A: (dim, dstate, 2) fp32;
 *   B, C: io, fixed (dim, dstate, 2) or varying (batch, ngroups, dstate,
 *         seqlen, 2);
 *   initial_state, last_state: (batch, dim, dstate, 2) fp32 or NULL;
 *   checkpoints: (batch, dim, nck, dstate, 2) fp32 or NULL, the state before
 *         every SSM_CKPT_INTERVAL-th timestep, for ssm_scan_bwd_complex.
 * Not taken (SSM_ERR_UNSUPPORTED): the fused conv prologue (conv_weight must
 * be NULL; run causal_conv1d_fwd first).  u is required; workspace is ignored
 * (the sequence is walked in one pass).  The decay's phase uses the
 * hardware sine and cosine on the fractional part of delta' Im(A) / (2 pi),
 * and delta' is the softplus without the cancellation of 1 + e^v (a large
 * |Im A| magnifies an error in delta').  Same conventions and status codes
 * as ssm_scan_fwd. */
int ssm_scan_fwd_complex(const ssm_scan_args_t *args, void *hip_stream);

/* Host-only argument check of ssm_scan_fwd_complex (no HIP call). */
int ssm_scan_complex_validate(const ssm_scan_args_t *args);

/* Arguments of ssm_scan_bwd.  Every pointer is a device pointer.  The inputs
 * are those of the forward call (same shapes, dtypes and layout kinds);
 * checkpoints are the ones that forward call wrote. */
typedef struct ssm_scan_bwd_args {
  int64_t batch, dim, seqlen, dstate, ngroups;
  int32_t io_dtype;
  const void *u;                                /* (b,d,l) io, required */
  const void *delta;                            /* (b,d,l) io, required */
  const float *A;                               /* (d,n) fp32, required */
  const void *B; int32_t B_kind;                /* io, SSM_BC_* */
  const void *C; int32_t C_kind;                /* io, SSM_BC_* */
  const float *D;                               /* (d) fp32 or NULL */
  const float *delta_bias;                      /* (d) fp32 or NULL */
  const void *z;                                /* (b,d,l) io or NULL */
  int32_t delta_softplus;                       /* 0 or 1 */
  const float *checkpoints;                     /* (b,d,nck,n) fp32 from ssm_scan_fwd, required */
  const void *dout;                             /* (b,d,l) io: dL/d out, required */
  /* gradients, caller-allocated and fully overwritten */
  void *du;                                     /* (b,d,l) io, required */
  void *ddelta;                                 /* (b,d,l) io, required */
  void *dz;                                     /* (b,d,l) io, required iff z */
  float *dA;                                    /* (d,n) fp32, required */
  float *dB;                                    /* fp32, B's layout ((d,n) or (b,g,n,l)), required */
  float *dC;                                    /* fp32, C's layout, required */
  float *dD;                                    /* (d) fp32, required iff D */
  float *ddelta_bias;                           /* (d) fp32, required iff delta_bias */
  float *dinitial_state;                        /* (b,d,n) fp32 or NULL */
  /* Scratch for the per-workgroup partial sums (ssm_scan_bwd_workspace_size),
   * caller-allocated device memory; the library allocates nothing, and a NULL
   * or too small workspace returns SSM_ERR_WORKSPACE before anything is
   * enqueued.  Every partial is written before it is read. */
  void *workspace;
  size_t workspace_bytes;
  /* Sequence split: 0 lets the library choose how many segments of whole
   * SSM_CKPT_INTERVAL chunks the sequence is cut into (it splits when the
   * channels alone leave compute units idle); k >= 1 asks for at most k
   * segments (equal whole-chunk lengths, so possibly fewer).  Segments after
   * the first first get their adjoint carry from a pass of their own; the
   * results differ from the unsplit ones only by rounding order.  Negative
   * values return SSM_ERR_SHAPE. */
  int32_t seq_segments;
} ssm_scan_bwd_args_t;

/* Selective-scan backward (the same page, section 4.1: the operator's
 * backward is the extension's bwd entry; last_state carries no gradient).
 * Given dout = dL/d out, writes the gradient of L with respect to every input
 * of the forward:  with h_t = dL/dx_t, the adjoint of the recurrence,
 *
 *     g_t     = dout_t * silu(z_t)                     (dL/d(y_t + D u_t))
 *     h_t[s]  = g_t * C_t[s] + exp(delta'_{t+1} A[d,s]) * h_{t+1}[s],  h_l = 0
 *     du_t    = g_t D[d] + delta'_t sum_s h_t[s] B_t[s]
 *     ddelta_t = softplus'(delta_t + delta_bias[d]) *
 *                sum_s h_t[s] (A[d,s] exp(delta'_t A[d,s]) x_{t-1}[s] + B_t[s] u_t)
 *     dA[d,s] = sum_{b,t} h_t[s] delta'_t exp(delta'_t A[d,s]) x_{t-1}[s]
 *     dB_t[s] = sum over the group's channels of h_t[s] delta'_t u_t   (fixed: summed over b, t)
 *     dC_t[s] = sum over the group's channels of g_t x_t[s]           (fixed: summed over b, t)
 *     dD[d]   = sum_{b,t} g_t u_t,   ddelta_bias[d] = sum_{b,t} ddelta_t
 *     dz_t    = dout_t (y_t + D u_t) silu'(z_t),  dinitial_state = exp(delta'_0 A) h_0
 *
 * (softplus' = 1 without delta_softplus).  Every chunk of SSM_CKPT_INTERVAL
 * timesteps is re-run forward from its checkpoint, then walked in reverse.
 * Every sum over channels, batches and timesteps is taken in a fixed order,
 * so results are bit-for-bit repeatable.  Same conventions and status codes
 * as ssm_scan_fwd. */
int ssm_scan_bwd(const ssm_scan_bwd_args_t *args, void *hip_stream);

/* Gradients of the complex-A forward (ssm_scan_fwd_complex; the same page,
 * section 4.1: A may be complex, and the operator has a backward).  The
 * arguments are those of ssm_scan_bwd read with the complex forward's
 * layouts: A (d,n,2) fp32; B/C io pairs, (d,n,2) fixed or (b,g,n,l,2)
 * varying; checkpoints (b,d,nck,n,2) fp32 written by ssm_scan_fwd_complex;
 * dA (d,n,2), dB/dC in B's/C's pair layout and dinitial_state (b,d,n,2),
 * all fp32, each the gradient of the real and of the imaginary part
 * (G_v = dL/dRe v + i dL/dIm v).  With a_t = exp(delta'_t A):
 *
 *     h_t     = dy_t conj(C_t) + conj(a_{t+1}) h_{t+1},  h_l = 0
 *     dC_t    = dy_t conj(x_t),   G_a = h_t conj(x_{t-1})
 *     dA     += conj(delta'_t a_t) G_a,   dB_t = delta'_t u_t h_t
 *     du_t    = D dy_t + delta'_t sum_s Re(h_t conj(B_t))
 *     ddelta_t = softplus'(.) (sum_s Re(G_a conj(A a_t)) + u_t sum_s Re(h_t conj(B_t)))
 *
 * with dy, dz, dD and d(delta_bias) as in ssm_scan_bwd.  delta'_t is formed
 * as in ssm_scan_fwd_complex, and the phase of a_t to about one rounding
 * (Im(A) / (2 pi) held as two floats, the product's rounding error
 * recovered with an fma): ddelta weighs a phase error by |A|^2 delta'.
 * seq_segments splits the sequence as in ssm_scan_bwd (0: the library's
 * choice, k >= 1: at most k segments of whole chunks): a carry pass walks
 * every segment after the first from a zero carry, and each segment starts
 * from the carry of the later ones, the same recurrence reassociated (the
 * decay over a segment is the product of its a_t, multiplied up step by
 * step).  The
 * workspace (ssm_scan_bwd_complex_workspace_size) holds the partial sums and
 * the carries and is required.  Asynchronous on hip_stream; returns a status
 * code. */
int ssm_scan_bwd_complex(const ssm_scan_bwd_args_t *args, void *hip_stream);

/* Host-only argument check of ssm_scan_bwd_complex (no HIP call). */
int ssm_scan_bwd_complex_validate(const ssm_scan_bwd_args_t *args);

/* Scratch bytes ssm_scan_bwd_complex needs (no HIP call). */
int ssm_scan_bwd_complex_workspace_size(const ssm_scan_bwd_args_t *args, size_t *bytes);

/* Host-only argument check of ssm_scan_bwd (no HIP call). */
int ssm_scan_bwd_validate(const ssm_scan_bwd_args_t *args);

/* Scratch bytes ssm_scan_bwd needs for these arguments.  Host-only, no HIP
 * call except a cached query of the device's compute-unit count. */
int ssm_scan_bwd_workspace_size(const ssm_scan_bwd_args_t *args, size_t *bytes);

/* Causal depthwise conv forward (PaddleNLP Kernel operator-library guide,
 * section 4.2 "causal_conv1d": causal_conv1d_fn(x, weight, bias, ...,
 * activation)).  x, out: (batch, dim, seqlen) io, device pointers; weight:
 * (dim, width) fp32; bias: (dim) fp32 or NULL; act: SSM_ACT_NONE or
 * SSM_ACT_SILU.
 *   out[b,d,t] = round_io(act(bias[d] + sum_k weight[d,k] * x[b,d,t-(width-1)+k]))
 * with x[t<0] = 0 (cross-correlation with left zero padding).  width must be
 * 4.  Asynchronous on hip_stream; returns a status code. */
int causal_conv1d_fwd(const void *x, const float *weight, const float *bias, void *out,
                      int64_t batch, int64_t dim, int64_t seqlen, int32_t width,
                      int32_t io_dtype, int32_t act, void *hip_stream);

/* causal_conv1d_fwd with the optional inputs of causal_conv1d_fn (same page
 * section 4.2: seq_idx, initial_states, return_final_states /
 * final_states_out).  Every pointer is a device pointer.
 *  - initial_states (batch, dim, width-1) io: the inputs before t = 0, oldest
 *    first (replacing the zero padding);
 *  - final_states (batch, dim, width-1) io, written: the last width-1 inputs
 *    of the row (with initial_states / zeros in front when seqlen < width-1),
 *    copied bit for bit -- the conv cache for continuing the sequence;
 *  - seq_idx (batch, seqlen) int32: packed sequences; a tap contributes only
 *    when its position carries the output's id, so each sequence restarts
 *    from zero.  Ids are expected to be contiguous per sequence.  seq_idx
 *    with initial_states or final_states returns SSM_ERR_UNSUPPORTED (the
 *    page: they cannot be used together).
 * width must be 4.  Same status codes as causal_conv1d_fwd. */
typedef struct causal_conv1d_args {
  int64_t batch, dim, seqlen;
  int32_t width, io_dtype, act;
  const void *x;                                /* (b,d,l) io, required */
  const float *weight;                          /* (d, width) fp32, required */
  const float *bias;                            /* (d) fp32 or NULL */
  const int32_t *seq_idx;                       /* (b,l) int32 or NULL */
  const void *initial_states;                   /* (b,d,width-1) io or NULL */
  void *out;                                    /* (b,d,l) io, required */
  void *final_states;                           /* (b,d,width-1) io or NULL */
} causal_conv1d_args_t;
int causal_conv1d_fwd_ex(const causal_conv1d_args_t *args, void *hip_stream);

/* Host-only argument check of causal_conv1d_fwd_ex (no HIP call). */
int causal_conv1d_ex_validate(const causal_conv1d_args_t *args);

/* Host-only argument check of causal_conv1d_fwd (no HIP call). */
int causal_conv1d_validate(const void *x, const float *weight, const void *out,
                           int64_t batch, int64_t dim, int64_t seqlen, int32_t width,
                           int32_t io_dtype, int32_t act);

/* ---------------------------------------------------------------------------
 * Single-step decode.
 * ------------------------------------------------------------------------- */

#define SSM_MAX_CONV_STATE 256  /* largest conv cache length causal_conv1d_update takes */

/* Arguments of ssm_state_update.  Every pointer is a device pointer. */
typedef struct ssm_state_update_args {
  int64_t batch, dim, dstate, ngroups;          /* ngroups: 1 unless grouped */
  int32_t io_dtype;                             /* SSM_F32 or SSM_BF16 */
  float *state;                                 /* (b,d,n) fp32: read, then overwritten */
  const void *x;                                /* (b,d) io, required */
  const void *dt;                               /* (b,d) io, required */
  const float *A;                               /* (d,n) fp32, required */
  const void *B;                                /* (b,g,n) io, required */
  const void *C;                                /* (b,g,n) io, required */
  const float *D;                               /* (d) fp32 or NULL */
  const float *dt_bias;                         /* (d) fp32 or NULL */
  const void *z;                                /* (b,d) io or NULL */
  int32_t dt_softplus;                          /* 0 or 1 */
  void *out;                                    /* (b,d) io, required */
} ssm_state_update_args_t;

/* selective_state_update: one decode step of the recurrence above against a
 * cached state (the PaddleNLP Kernel operator-library guide lists
 * selective_state_update among its mamba operators, section 4.4; it is not
 * printed there, and is read as one timestep of section 4.1's scan applied
 * to a cache).  For every (b, d), with dt' = softplus(dt + dt_bias) when
 * dt_softplus is set (otherwise dt + dt_bias) and g = d / (dim / ngroups):
 *
 *     state[b,d,s] <- exp(dt' * A[d,s]) * state[b,d,s] + dt' * B[b,g,s] * x[b,d]
 *     out[b,d]      = (sum_s C[b,g,s] * state[b,d,s] + D[d] * x[b,d]) * silu(z[b,d])
 *
 * (the contraction uses the updated state).  A Mamba-2 style state
 * (batch, nheads, headdim, dstate) is this call with dim = nheads * headdim
 * and every per-head tensor expanded over headdim.  The state is updated in
 * place and must not overlap any other argument; `out` must not alias an
 * input.  dstate <= SSM_MAX_DSTATE.  Same conventions and status codes as
 * ssm_scan_fwd; the update is a pure function of its inputs, so calls on one
 * stream compose into a sequence of decode steps. */
int ssm_state_update(const ssm_state_update_args_t *args, void *hip_stream);

/* Host-only argument check of ssm_state_update (no HIP call). */
int ssm_state_update_validate(const ssm_state_update_args_t *args);

/* causal_conv1d_update: the causal conv of causal_conv1d_fwd continued from a
 * cache of earlier inputs (same guide, section 4.2: single-step incremental
 * inference over a conv_state cache, with an optional ring buffer indexed by
 * cache_seqlens).  x: (batch, dim, seqlen) io, the new tokens; conv_state:
 * (batch, dim, state_len) io, state_len >= width - 1, read and updated in
 * place; weight: (dim, width) fp32; bias: (dim) fp32 or NULL; out: (batch,
 * dim, seqlen) io.  For every new token t,
 *
 *     out[b,d,t] = round_io(act(bias[d] + sum_k weight[d,k] * h[t - (width-1) + k]))
 *
 * where h is the input history: the inputs before the first new token come
 * from the cache, the rest are x.
 *  - cache_seqlens == NULL: the cache is ordered oldest first (its last
 *    width-1 entries precede x[.,.,0]); afterwards it holds the last state_len
 *    inputs of (cache, x).
 *  - cache_seqlens != NULL (device pointer, one int32 >= 0 per batch): the
 *    cache is a ring buffer; token t is written at slot
 *    (cache_seqlens[b] + t) % state_len and the inputs before it are the
 *    width-1 slots before that one, circularly.  Other slots are untouched
 *    and cache_seqlens is not advanced (the caller adds seqlen).
 * 2 <= width <= SSM_CONV_WIDTH, state_len <= SSM_MAX_CONV_STATE.  x, out and
 * conv_state must not overlap.  Asynchronous on hip_stream; returns a status
 * code. */
int causal_conv1d_update(const void *x, void *conv_state, const float *weight,
                         const float *bias, const int32_t *cache_seqlens, void *out,
                         int64_t batch, int64_t dim, int64_t seqlen, int64_t state_len,
                         int32_t width, int32_t io_dtype, int32_t act, void *hip_stream);

/* Host-only argument check of causal_conv1d_update (no HIP call). */
int causal_conv1d_update_validate(const void *x, const void *conv_state, const float *weight,
                                  const void *out, int64_t batch, int64_t dim, int64_t seqlen,
                                  int64_t state_len, int32_t width, int32_t io_dtype,
                                  int32_t act);

/* ---------------------------------------------------------------------------
 * Mamba-2 chunked scan (state-space duality form).
 * ------------------------------------------------------------------------- */

#define SSD_HEADDIM 64     /* the head width the kernel is built for */
#define SSD_CHUNK 64       /* tokens per chunk of the chunked evaluation */

/* Arguments of ssd_scan_fwd.  Every pointer is a device pointer; x, z, out,
 * B and C must be 16-byte aligned. */
typedef struct ssd_scan_args {
  int64_t batch, seqlen, nheads, headdim, dstate, ngroups;
  int32_t io_dtype;               /* SSM_BF16 */
  const void *x;                  /* (b,l,h,p) io, required */
  const void *dt;                 /* (b,l,h) io, required */
  const float *A;                 /* (h) fp32, required */
  const void *B;                  /* (b,l,g,n) io, required */
  const void *C;                  /* (b,l,g,n) io, required */
  const float *D;                 /* (h) or (h,p) fp32, or NULL */
  int32_t D_per_channel;          /* 1: D is (h,p) */
  const void *z;                  /* (b,l,h,p) io or NULL */
  const float *dt_bias;           /* (h) fp32 or NULL */
  int32_t dt_softplus;            /* 0 or 1 */
  const float *initial_states;    /* (b,h,p,n) fp32 or NULL (zero) */
  void *out;                      /* (b,l,h,p) io, required */
  float *final_states;            /* (b,h,p,n) fp32 or NULL */
  /* Step range (the operators' dt_limit): when dt_limit is 1 the step is
   * clamped, dt' = min(max(dt', dt_min), dt_max), after softplus; 0: no
   * clamp.  dt_min > dt_max returns SSM_ERR_SHAPE. */
  int32_t dt_limit;
  float dt_min, dt_max;
  /* Packed sequences (the operators' seq_idx): (b,l) int32 sequence ids, or
   * NULL.  Ids must not decrease along l (each sequence is one contiguous
   * run); where the id changes the state restarts from zero, so no token
   * sees a token of another sequence.  initial_states is the state before
   * the first sequence of each row, final_states the state after the last.
   * Ids that decrease give unspecified results (never a fault). */
  const int32_t *seq_idx;
  /* Scratch for the sequence split (see ssd_scan_workspace_size): caller-
   * allocated device memory; the library allocates nothing and returns
   * SSM_ERR_WORKSPACE when the plan needs more than workspace_bytes.  Not
   * read before written; reusable once the call's work has finished. */
  void *workspace;
  size_t workspace_bytes;
  /* Sequence split: 0 lets the library choose (its segments may differ in
   * length); k >= 1 asks for k segments of ceil(chunks / k) whole chunks,
   * the last one taking the rest (possibly fewer segments).  Negative values
   * return SSM_ERR_SHAPE.  The split changes the results only by rounding
   * order. */
  int32_t seq_segments;
} ssd_scan_args_t;

/* ssd_scan_fwd: the Mamba-2 chunked scan (the guide's section 4.4 lists
 * mamba_chunk_scan_combined, chunk_state and state_passing among its mamba
 * operators without printing them; they are read as the selective-scan
 * recurrence with a scalar decay per head, evaluated chunk by chunk).  For
 * every (b, h), head h in group g = h / (nheads / ngroups), and token t:
 *
 *     dt'          = softplus(dt[b,t,h] + dt_bias[h])   (or without softplus;
 *                    then clamped to [dt_min, dt_max] with dt_limit)
 *     H[p][n]     <- 0 first where seq_idx[b,t] != seq_idx[b,t-1]
 *     H[p][n]     <- exp(dt' * A[h]) * H[p][n] + dt' * B[b,t,g,n] * x[b,t,h,p]
 *     out[b,t,h,p] = (sum_n C[b,t,g,n] * H[p][n] + D * x[b,t,h,p]) * silu(z[b,t,h,p])
 *
 * with H starting at initial_states and its last value stored to
 * final_states.  The kernel evaluates each chunk of SSD_CHUNK tokens in the
 * quadratic (dual) form on the matrix cores -- products of bf16 operands
 * accumulated in fp32 -- and carries the fp32 state from chunk to chunk.
 * When batch * nheads alone leaves the GPU short of workgroups, the chunks
 * are cut into segments: a first launch finds each segment's end state
 * from zero and its total decay (chunk_state), the second starts every
 * segment from the state carried over the ones before it (state_passing)
 * and computes the outputs (chunk_scan).
 * Supported: io_dtype SSM_BF16, headdim SSD_HEADDIM, dstate 32, 64 or 128;
 * other values return SSM_ERR_UNSUPPORTED.  Same conventions and status
 * codes as ssm_scan_fwd. */
int ssd_scan_fwd(const ssd_scan_args_t *args, void *hip_stream);

/* Host-only argument check of ssd_scan_fwd (no HIP call). */
int ssd_scan_validate(const ssd_scan_args_t *args);

/* Scratch bytes ssd_scan_fwd needs for these arguments (0 without a
 * sequence split).  Host-only apart from cached queries of the device's
 * compute-unit count and the kernels' occupancy. */
int ssd_scan_workspace_size(const ssd_scan_args_t *args, size_t *bytes);

/* The three parts of mamba_chunk_scan_combined as section 4.4 of the guide
 * names them (chunk_state, state_passing, the chunk scan), over chunks of
 * chunk_size tokens (a positive multiple of SSD_CHUNK; the last chunk may be
 * shorter); nchunks = ceil(seqlen / chunk_size).  Per (b, h) the scan of
 * chunk c maps the state entering it affinely, H_end = P_c H_start + E_c,
 * and the three calls composed give ssd_scan_fwd's out and final_states:
 *
 *   ssd_chunk_state:   E_c, the chunk's end state from a zero state, into
 *                      states (nchunks,b,h,p,n) fp32, and P_c into decays
 *                      (nchunks,b,h) fp32: exp(A[h] * the chunk's summed
 *                      steps), or 0 where seq_idx changes at one of the
 *                      chunk's tokens (t > 0), the first included.  Reads
 *                      x, dt, A, B, dt_bias, dt_softplus, dt_limit and
 *                      seq_idx of args (C, D, z, out, the states, workspace
 *                      and seq_segments are ignored and may be NULL).
 *   ssd_state_passing: carried[c] = S_c with S_0 = initial_states (zero
 *                      when NULL) and S_{c+1} = decays[c] S_c + states[c],
 *                      each step one fp32 fma; final_states (b,h,p,n), if
 *                      not NULL, gets S_nchunks.  Plain device arrays of
 *                      the layouts above; carried (nchunks,b,h,p,n) fp32.
 *   ssd_chunk_scan:    out of every chunk from the state carried[c] (the
 *                      whole of args but initial_states, which carried[0]
 *                      replaces, and workspace / seq_segments, which are
 *                      ignored), and the state after the last chunk into
 *                      final_states when given.
 *
 * Same supported sizes, alignment, conventions and status codes as
 * ssd_scan_fwd; a chunk_size that is not a positive multiple of SSD_CHUNK
 * returns SSM_ERR_UNSUPPORTED.  None of them needs scratch.  The *_validate
 * calls are the host-only checks (no HIP call). */
int ssd_chunk_state(const ssd_scan_args_t *args, int64_t chunk_size, float *states, float *decays,
                    void *hip_stream);
int ssd_chunk_state_validate(const ssd_scan_args_t *args, int64_t chunk_size, const float *states,
                             const float *decays);
int ssd_state_passing(int64_t nchunks, int64_t batch, int64_t nheads, int64_t headdim, int64_t dstate,
                      const float *states, const float *decays, const float *initial_states,
                      float *carried, float *final_states, void *hip_stream);
int ssd_state_passing_validate(int64_t nchunks, int64_t batch, int64_t nheads, int64_t headdim,
                               int64_t dstate, const float *states, const float *decays,
                               const float *carried);
int ssd_chunk_scan(const ssd_scan_args_t *args, int64_t chunk_size, const float *carried, void *hip_stream);
int ssd_chunk_scan_validate(const ssd_scan_args_t *args, int64_t chunk_size, const float *carried);

/* ---------------------------------------------------------------------------
 * Packed tokens: a Mamba-2 mixer's short convolution, scan and step, for
 * prompts of several lengths in one call, for single tokens, and in training.
 *
 * The tokens of nseq sequences lie one after another, (total, ...), and
 * cu_seqlens (nseq + 1) int32 on the device holds each sequence's first
 * token, cu_seqlens[nseq] = total; a sequence may be empty.  Edges out of
 * order or outside [0, total] give unspecified results, never an access
 * outside the tensors.  Rows of equal length are the case cu_seqlens[s] = s l.
 *
 * A *_stride is the number of elements from a token to the next; what a token
 * holds is dense.  x, B and C may so be parts of one row, as the input
 * projection and the convolution leave them.
 *
 * Caches hold one entry per request.  Sequence s uses entry slots[s] (s itself
 * when slots is NULL); an entry outside the cache is neither read nor
 * written, and the sequence starts from nothing.  Two sequences of a call must
 * not share an entry.  cache_seqlens[s] (int32, device) is the number of
 * tokens that the request has seen before the call: where it is 0, or
 * cache_seqlens is NULL, the entry is not read, so a new request needs no
 * clearing.  The caller advances cache_seqlens.
 *   conv_state (state_slots, channels, state_len) io: the last inputs as a
 *     ring, position p (from 0) at p % state_len; positions before 0 are zero;
 *   ssm_state (state_slots, nheads, headdim, dstate) fp32.
 * ------------------------------------------------------------------------- */

/* Arguments of causal_conv1d_varlen_fwd and causal_conv1d_varlen_bwd. */
typedef struct causal_conv1d_varlen_args {
  int64_t total, nseq, channels;
  int32_t width, io_dtype, act;                 /* width: SSM_CONV_WIDTH */
  const void *x; int64_t x_stride;              /* (total, channels) io */
  const float *weight;                          /* (channels, width) fp32 */
  const float *bias;                            /* (channels) fp32 or NULL */
  const int32_t *cu_seqlens;                    /* (nseq + 1) */
  /* forward */
  void *out; int64_t out_stride;                /* (total, channels) io */
  void *conv_state;                             /* ring cache or NULL */
  int64_t state_slots, state_len;               /* width <= state_len <= SSM_MAX_CONV_STATE */
  const int32_t *cache_seqlens, *slots;         /* (nseq) or NULL */
  /* backward */
  const void *dout; int64_t dout_stride;        /* (total, channels) io */
  void *dx; int64_t dx_stride;                  /* (total, channels) io */
  float *dweight;                               /* (channels, width) fp32 */
  float *dbias;                                 /* (channels) fp32, required iff bias */
  void *workspace; size_t workspace_bytes;      /* causal_conv1d_varlen_bwd_workspace_size */
} causal_conv1d_varlen_args_t;

/* The causal depthwise conv of causal_conv1d_fwd over packed tokens:
 *   out[t,c] = round_io(act(bias[c] + sum_k weight[c,k] x[t-(width-1)+k,c]))
 * where the inputs before a sequence's first token come from its ring (zero
 * without one).  Afterwards the ring holds the sequence's last inputs.  `out`
 * and conv_state must not overlap x. */
int causal_conv1d_varlen_fwd(const causal_conv1d_varlen_args_t *args, void *hip_stream);
int causal_conv1d_varlen_fwd_validate(const causal_conv1d_varlen_args_t *args);

/* Its gradient, for sequences that start from nothing (no cache is read):
 * with da = dout act'(pre),
 *   dx[t,c] = sum_k weight[c,k] da[t+(width-1)-k,c]   (inside the sequence)
 *   dweight[c,k] = sum_t da[t,c] x[t-(width-1)+k,c],  dbias[c] = sum_t da[t,c]
 * summed in a fixed order (bit-for-bit repeatable). */
int causal_conv1d_varlen_bwd(const causal_conv1d_varlen_args_t *args, void *hip_stream);
int causal_conv1d_varlen_bwd_validate(const causal_conv1d_varlen_args_t *args);
int causal_conv1d_varlen_bwd_workspace_size(const causal_conv1d_varlen_args_t *args, size_t *bytes);

/* Arguments of ssd_varlen_fwd.  x, B, C, z and out must be 16-byte aligned,
 * their strides multiples of 8; those of x, B, C and the backward's dout at
 * most 2^24 elements.  ssm_state, checkpoints and workspace must be 16-byte
 * aligned too. */
typedef struct ssd_varlen_args {
  int64_t total, nseq, max_seqlen;              /* max_seqlen: at least the longest sequence */
  int64_t nheads, headdim, dstate, ngroups;
  int32_t io_dtype;                             /* SSM_BF16 */
  const void *x; int64_t x_stride;              /* (total, h, p) io */
  const void *dt; int64_t dt_stride;            /* (total, h) io */
  const float *A;                               /* (h) fp32 */
  const void *B; int64_t B_stride;              /* (total, g, n) io */
  const void *C; int64_t C_stride;              /* (total, g, n) io */
  const float *D; int32_t D_per_channel;        /* (h) or (h,p) fp32, or NULL */
  const void *z; int64_t z_stride;              /* (total, h, p) io or NULL (forward only) */
  const float *dt_bias;                         /* (h) fp32 or NULL */
  int32_t dt_softplus, dt_limit;                /* as ssd_scan_args_t */
  float dt_min, dt_max;
  const int32_t *cu_seqlens;                    /* (nseq + 1) */
  void *out; int64_t out_stride;                /* (total, h, p) io */
  float *ssm_state; int64_t state_slots;        /* cache or NULL: read and written */
  const int32_t *cache_seqlens, *slots;         /* (nseq) or NULL */
  /* The state entering every chunk of SSD_CHUNK tokens, in 8 bits, for
   * ssd_varlen_bwd (NULL: not kept).  Chunk c of sequence s is entry
   * floor(cu_seqlens[s] / SSD_CHUNK) + s + c of ssd_checkpoint_slots entries;
   * entries of no chunk are not written.  A state is code * scale with one
   * scale per channel, the smallest power of two for which the channel's
   * states are within +-127 scale (at least 2^-100; NaN where one of them is
   * not finite). */
  int8_t *checkpoints;                          /* (entries, h, p, n) */
  float *checkpoint_scales;                     /* (entries, h, p) */
  void *workspace; size_t workspace_bytes;      /* ssd_varlen_fwd_workspace_size */
  int32_t seq_segments;                         /* as ssd_scan_args_t */
} ssd_varlen_args_t;

/* ssd_scan_fwd over packed tokens: the same recurrence for every sequence,
 * from the cached state (or zero) to the cached state.
 *
 * Values that are not finite stay in their sequence.  Here they reach no token
 * before their own, except that one in x can make its channel's outputs NaN for
 * up to 31 tokens before it; in ssd_varlen_bwd they can reach every token of
 * their chunk and of the chunks before. */
int ssd_varlen_fwd(const ssd_varlen_args_t *args, void *hip_stream);
int ssd_varlen_fwd_validate(const ssd_varlen_args_t *args);
int ssd_varlen_fwd_workspace_size(const ssd_varlen_args_t *args, size_t *bytes);

/* Checkpoint entries of packed tokens: floor(total / SSD_CHUNK) + nseq. */
int64_t ssd_checkpoint_slots(int64_t total, int64_t nseq);

/* Arguments of ssd_varlen_bwd: the forward's (fwd.z must be NULL: with the
 * gate outside the scan, as where a gated norm follows, its gradient belongs
 * there; fwd.out, ssm_state, cache_seqlens, slots and workspace are ignored;
 * fwd.checkpoints and scales are those that the forward wrote, or the same
 * values laid out with other strides from entry to entry and head to head),
 * and the gradients, caller-allocated and fully overwritten. */
typedef struct ssd_varlen_bwd_args {
  ssd_varlen_args_t fwd;
  /* (dout, dx, dB, dC and the states' gradients as x: 16-byte aligned) */
  int64_t code_entry_stride, code_head_stride;  /* multiples of 16; as the forward writes: h p n, p n */
  int64_t scale_entry_stride, scale_head_stride;  /* h p, p */
  const void *dout; int64_t dout_stride;        /* (total, h, p) io */
  const float *dfinal_states;                   /* (nseq, h, p, n) fp32 or NULL (zero) */
  void *dx; int64_t dx_stride;                  /* (total, h, p) io */
  void *ddt; int64_t ddt_stride;                /* (total, h) io */
  void *dB; int64_t dB_stride;                  /* (total, g, n) io */
  void *dC; int64_t dC_stride;                  /* (total, g, n) io */
  float *dA;                                    /* (h) fp32 */
  float *dD;                                    /* as D, required iff D */
  float *ddt_bias;                              /* (h) fp32, required iff dt_bias */
  float *dinitial_states;                       /* (nseq, h, p, n) fp32 or NULL */
  void *workspace; size_t workspace_bytes;      /* ssd_varlen_bwd_workspace_size */
} ssd_varlen_bwd_args_t;

/* Gradients of ssd_varlen_fwd.  Every chunk is re-evaluated from its 8-bit
 * state; the adjoint of the state goes backwards in 32 bits.  With dt' the
 * step, cs its running sum times A inside the chunk, H the chunk's entering
 * state, dH the adjoint of its leaving state, g = dout, and for i >= j
 * L_ij = exp(cs_i - cs_j), S_ij = C_i . B_j, M_ij = g_i . x_j:
 *   dx_j  = dt'_j (sum_i S_ij L_ij g_i + exp(cs_end - cs_j) dH B_j) + D g_j
 *   dB_j  = dt'_j (sum_i M_ij L_ij C_i + exp(cs_end - cs_j) dH^T x_j)  (summed over the group's heads)
 *   dC_i  = sum_j M_ij L_ij dt'_j B_j + exp(cs_i) H^T g_i              (summed over the group's heads)
 *   dH   <- exp(cs_end) dH + sum_i exp(cs_i) g_i C_i^T
 * and ddt, dA through the weights and every decay.  Where dt_limit clamps a
 * step its gradient is zero.  Sums are taken in a fixed order (bit-for-bit
 * repeatable). */
int ssd_varlen_bwd(const ssd_varlen_bwd_args_t *args, void *hip_stream);
int ssd_varlen_bwd_validate(const ssd_varlen_bwd_args_t *args);
int ssd_varlen_bwd_workspace_size(const ssd_varlen_bwd_args_t *args, size_t *bytes);

/* Arguments of conv1d_ssd_update. */
typedef struct conv1d_ssd_update_args {
  int64_t batch, nheads, headdim, dstate, ngroups;
  int32_t io_dtype, act, width;                 /* width: SSM_CONV_WIDTH */
  const void *xBC; int64_t xBC_stride;          /* (batch, h p + 2 g n) io: x | B | C before the conv */
  const void *dt; int64_t dt_stride;            /* (batch, h) io */
  const float *A;                               /* (h) fp32 */
  const float *conv_weight;                     /* (h p + 2 g n, width) fp32 */
  const float *conv_bias;                       /* (h p + 2 g n) fp32 or NULL */
  const float *D; int32_t D_per_channel;        /* (h) or (h,p) fp32, or NULL */
  const void *z; int64_t z_stride;              /* (batch, h p) io or NULL */
  const float *dt_bias;                         /* (h) fp32 or NULL */
  int32_t dt_softplus, dt_limit;
  float dt_min, dt_max;
  void *conv_state; int64_t state_len;          /* ring cache, width <= state_len <= SSM_MAX_CONV_STATE */
  float *ssm_state;                             /* cache, 16-byte aligned */
  int64_t state_slots;                          /* entries of both caches */
  const int32_t *cache_seqlens;                 /* (batch) or NULL (every request is new) */
  const int32_t *slots;                         /* (batch) or NULL */
  void *out; int64_t out_stride;                /* (batch, h p) io */
} conv1d_ssd_update_args_t;

/* One token of every request, in one launch: u = act(conv(xBC)) against the
 * ring (kept in fp32, not rounded to io), then ssd_varlen_fwd's recurrence for
 * that token against the cached state, both caches updated.  An entry outside
 * the cache (a padding row) gives the output of a new request and writes
 * nothing.  headdim SSD_HEADDIM, dstate 32, 64 or 128; io fp32, bf16 or fp16. */
int conv1d_ssd_update(const conv1d_ssd_update_args_t *args, void *hip_stream);
int conv1d_ssd_update_validate(const conv1d_ssd_update_args_t *args);

/* ---------------------------------------------------------------------------
 * A gated recurrent block: its recurrence over packed tokens, in serving and
 * in training, and its norm.  Packed tokens, strides, cu_seqlens, caches, slots
 * and cache_seqlens as above, except that tokens before cu_seqlens[0] and from
 * cu_seqlens[nseq] on (a padded batch) belong to no sequence: their outputs are
 * left as they were, and their gradients are 0.
 * The scans' workspaces are aligned to 16 bytes (SSM_ERR_UNSUPPORTED), and
 * serve one call at a time.  A scan's workgroups wait there for what workgroups
 * of the same call that started before them leave.  The wait is bounded, by some
 * 10^6 polls: a call that comes to its end, as where another one writes to its
 * workspace meanwhile, has returned SSM_OK, and the states, outputs and gradients
 * from there on are NaN.
 * ------------------------------------------------------------------------- */

#define GATED_CHUNK 64   /* packed tokens from one kept state to the next */

/* Arguments of gated_scan_varlen_fwd.  Strides of at most 2^24 elements. */
typedef struct gated_scan_varlen_args {
  int64_t total, nseq, channels;
  int32_t io_dtype;
  const void *x; int64_t x_stride;              /* (total, channels) io */
  const void *r; int64_t r_stride;              /* (total, channels) io: recurrence gate before its sigmoid */
  const void *i; int64_t i_stride;              /* (total, channels) io: input gate before its sigmoid */
  const float *A;                               /* (channels) fp32, <= 0: log of the decay at an open gate */
  const float *r_bias, *i_bias;                 /* (channels) fp32 or NULL */
  const int32_t *cu_seqlens;                    /* (nseq + 1) */
  void *out; int64_t out_stride;                /* (total, channels) io */
  float *state; int64_t state_slots;            /* (state_slots, channels) cache or NULL: read and written */
  const int32_t *cache_seqlens, *slots;         /* (nseq) or NULL */
  /* The state before every GATED_CHUNK-th packed token, for
   * gated_scan_varlen_bwd (NULL: not kept); rows of tokens of no sequence are
   * 0. */
  float *checkpoints;                           /* (gated_checkpoint_slots(total), channels) */
  void *workspace; size_t workspace_bytes;      /* gated_scan_varlen_fwd_workspace_size */
} gated_scan_varlen_args_t;

/* A gated linear recurrence over packed tokens.  For every token t of a
 * sequence and channel c, with sigma the logistic function,
 *
 *     rho  = sigma(r[t,c] + r_bias[c]),   iota = sigma(i[t,c] + i_bias[c])
 *     a    = exp(A[c] rho)
 *     h   <- a h + sqrt(1 - a^2) iota x[t,c]
 *     out[t,c] = h
 *
 * with h starting at the sequence's cached state (or zero) and its last value
 * stored there; an empty sequence leaves its entry as it is.  Every token's input
 * has the weight sqrt(1 - a^2), a sequence's first one too (there are models whose
 * first token has the weight 1: their weights do not fit this recurrence).  The
 * state is fp32; sigma and a are formed in fp32, to (3 |v| + 5) 2^-24 of sigma for
 * a gate's sum v, and a sigma below 2^-126 counts as 0.  Where A[c] > 0 the weight
 * sqrt(1 - a^2) is taken as 0, and a state other than 0 may be infinite up to 128
 * tokens before its own value is (a tile's decay is formed before the state is
 * known).  `out` must not overlap an input.  Values that are not finite stay in
 * their sequence and channel and reach no earlier token.  Results are bit-for-bit
 * repeatable. */
int gated_scan_varlen_fwd(const gated_scan_varlen_args_t *args, void *hip_stream);
int gated_scan_varlen_fwd_validate(const gated_scan_varlen_args_t *args);
int gated_scan_varlen_fwd_workspace_size(const gated_scan_varlen_args_t *args, size_t *bytes);

/* Kept states of packed tokens: ceil(total / GATED_CHUNK). */
int64_t gated_checkpoint_slots(int64_t total);

/* Arguments of gated_scan_varlen_bwd, strides as there: the forward's (fwd.checkpoints are those
 * that the forward wrote; fwd.out, state, state_slots, cache_seqlens, slots and
 * workspace are ignored), and the gradients, caller-allocated and fully
 * overwritten. */
typedef struct gated_scan_varlen_bwd_args {
  gated_scan_varlen_args_t fwd;
  const float *initial_states;                  /* (nseq, channels) fp32: the states that the sequences started from, or NULL (zero) */
  const void *dout; int64_t dout_stride;        /* (total, channels) io */
  const float *dfinal_states;                   /* (nseq, channels) fp32: gradient of the last states, or NULL (zero) */
  void *dx; int64_t dx_stride;                  /* (total, channels) io */
  void *dr; int64_t dr_stride;                  /* (total, channels) io */
  void *di; int64_t di_stride;                  /* (total, channels) io */
  float *dA;                                    /* (channels) fp32 */
  float *dr_bias, *di_bias;                     /* (channels) fp32, required iff r_bias, i_bias */
  float *dinitial_states;                       /* (nseq, channels) fp32 or NULL */
  void *workspace; size_t workspace_bytes;      /* gated_scan_varlen_bwd_workspace_size */
} gated_scan_varlen_bwd_args_t;

/* Gradients of gated_scan_varlen_fwd.  With G the adjoint of the state,
 *   G_t = dout_t + a_{t+1} G_{t+1}   (dfinal_states behind the last token),
 * and m = sqrt(1 - a^2):
 *   q   = G rho (a h_{t-1} - (a^2 / m) iota x)   (rho / m taken as 0 where m = 0)
 *   dA  = sum_t q,   dr = A (1 - rho) q,   dr_bias = sum_t dr
 *   dx  = G m iota,  di = G m x iota (1 - iota),   di_bias = sum_t di
 * An empty sequence passes dfinal_states on to dinitial_states.  Gradients must
 * not overlap inputs.  Sums over the tokens are fp32 over at most 128 of them, then
 * 64 bits, in a fixed order (bit-for-bit repeatable).  Values that are not finite
 * stay in their sequence and channel (apart from the sums over the tokens). */
int gated_scan_varlen_bwd(const gated_scan_varlen_bwd_args_t *args, void *hip_stream);
int gated_scan_varlen_bwd_validate(const gated_scan_varlen_bwd_args_t *args);
int gated_scan_varlen_bwd_workspace_size(const gated_scan_varlen_bwd_args_t *args, size_t *bytes);

/* Arguments of gated_scan_update. */
typedef struct gated_scan_update_args {
  int64_t batch, channels;
  int32_t io_dtype;
  const void *x; int64_t x_stride;              /* (batch, channels) io, and so r, i and out */
  const void *r; int64_t r_stride;
  const void *i; int64_t i_stride;
  const float *A;                               /* (channels) fp32 */
  const float *r_bias, *i_bias;                 /* (channels) fp32 or NULL */
  float *state; int64_t state_slots;            /* (state_slots, channels) cache */
  const int32_t *cache_seqlens;                 /* (batch) or NULL (every request is new) */
  const int32_t *slots;                         /* (batch) or NULL */
  void *out; int64_t out_stride;
} gated_scan_update_args_t;

/* One token of every request through gated_scan_varlen_fwd's recurrence
 * against the cached states, which are updated.  An entry outside the cache (a
 * padding row) gives the output of a new request and writes nothing. */
int gated_scan_update(const gated_scan_update_args_t *args, void *hip_stream);
int gated_scan_update_validate(const gated_scan_update_args_t *args);

#define RMS_SCALE_BLOCK 128     /* columns that share a scale in 8 bits */
#define RMS_MAX_GROUP 16384     /* largest group_size */

/* Arguments of rms_norm_fwd.  A *_stride is the number of elements from a row to
 * the next; a row's columns are dense. */
typedef struct rms_norm_args {
  int64_t rows, cols, group_size;               /* group_size divides cols */
  int32_t io_dtype, residual_dtype;             /* residual_dtype: io_dtype or SSM_F32 */
  float eps;
  const void *x; int64_t x_stride;              /* (rows, cols) io */
  const void *z; int64_t z_stride;              /* (rows, cols) io gate, or NULL */
  const void *residual; int64_t residual_stride;  /* (rows, cols) residual_dtype, or NULL; not with z */
  const float *weight;                          /* (cols) fp32 */
  void *residual_out; int64_t residual_out_stride;  /* as residual, required iff residual; may be residual itself */
  /* either */
  void *out; int64_t out_stride;                /* (rows, cols) io */
  /* or */
  void *codes; int64_t codes_stride;            /* (rows, cols) e4m3 */
  float *scales;                                /* (rows, ceil(cols / RMS_SCALE_BLOCK)) fp32 */
} rms_norm_args_t;

/* Root-mean-square norm of every group of group_size neighbouring columns of a
 * row, after the residual's addition or behind a gate:
 *
 *     v = x,  or  residual_out = round(x + residual) and v = residual_out,
 *         or  v = x silu(z)
 *     y = v / sqrt(mean(v^2) + eps) weight
 *
 * (of what the residual stream holds, so that rms_norm_bwd, which reads it, is
 * the gradient of what was computed).  The squares and their sum are fp32, as the
 * values are: where the sum is more than fp32 holds, y is 0; with eps = 0 a group
 * of zeros gives NaN (0 / 0).  y goes to `out`, or in 8 bits to `codes`: y is
 * code * scale, the code rounded to nearest (ties to even) and the scale, one for
 * RMS_SCALE_BLOCK columns of a row, the smallest power of two with which none of
 * them is over 448 (at least 2^-100; NaN where one of them is not finite).  8 bits need one group a row, or a group_size that is a multiple of
 * RMS_SCALE_BLOCK. */
int rms_norm_fwd(const rms_norm_args_t *args, void *hip_stream);
int rms_norm_fwd_validate(const rms_norm_args_t *args);

/* Arguments of rms_norm_bwd. */
typedef struct rms_norm_bwd_args {
  int64_t rows, cols, group_size;
  int32_t io_dtype, x_dtype;                    /* x_dtype: io_dtype or SSM_F32 */
  float eps;
  const void *x; int64_t x_stride;              /* (rows, cols) x_dtype: the forward's x, or its residual_out */
  const void *z; int64_t z_stride;              /* (rows, cols) io, or NULL; not with ds, and x_dtype is io_dtype */
  const float *weight;                          /* (cols) fp32 */
  const void *dy; int64_t dy_stride;            /* (rows, cols) io */
  const void *ds; int64_t ds_stride;            /* (rows, cols) x_dtype: the gradient that reaches residual_out, or NULL */
  void *dx; int64_t dx_stride;                  /* (rows, cols) io */
  void *dresidual; int64_t dresidual_stride;    /* (rows, cols) x_dtype: dx before its rounding to io, or NULL */
  void *dz; int64_t dz_stride;                  /* (rows, cols) io, required iff z */
  float *dweight;                               /* (cols) fp32 */
  void *workspace; size_t workspace_bytes;      /* rms_norm_bwd_workspace_size; aligned to 4 bytes */
} rms_norm_bwd_args_t;

/* Gradients of rms_norm_fwd.  With rstd = 1 / sqrt(mean(v^2) + eps), hat = v rstd
 * and g = dy weight:
 *   dv = rstd (g - hat mean(g hat)),  dweight = sum over rows of dy hat
 *   dx = dv + ds   (the residual's gradient as well),  or with a gate
 *   dx = dv silu(z),  dz = dv x silu'(z)
 * dweight's terms are added in fp32 over at most 256 rows, then in 64 bits, in a
 * fixed order (bit-for-bit repeatable).  Outputs must not overlap inputs.  At most
 * 65535 groups a row. */
int rms_norm_bwd(const rms_norm_bwd_args_t *args, void *hip_stream);
int rms_norm_bwd_validate(const rms_norm_bwd_args_t *args);
int rms_norm_bwd_workspace_size(const rms_norm_bwd_args_t *args, size_t *bytes);

/* Static text for a status code. */
const char *ssm_status_str(int status);

/* The hipError_t of the last SSM_ERR_HIP returned on this thread (0 if none). */
int ssm_last_hip_error(void);

/* SSM_ABI_VERSION of the loaded library. */
int ssm_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SSMSCAN_H */
