/*
 * lapl_ops.h -- C ABI of the operators beside the attention of lapl_attn.h, in the same library:
 *
 *   lapl_scan_*  gated linear recurrence over the tokens (forward, backward, single tokens): the
 *                other linear-time token mixer, one that has a direction;
 *   lapl_norm_*  residual addition + root-mean-square norm of the attention's output, with its
 *                backward, which writes the dout that lapl_attn_backward takes;
 *   lapl_clip_*  global norm of many gradient tensors, and clipping to a largest norm.
 *
 * Conventions are those of lapl_attn.h: lapl_status codes, argument errors detected on the host
 * before any launch, every buffer owned by the caller, handles that hold host state only,
 * stream-ordered asynchronous calls that allocate nothing, never synchronise and may be captured
 * into a graph, and results that are the same bit for bit from call to call.  A handle may be used
 * by one host thread at a time; a workspace by one call at a time (two captured graphs that may
 * run at once need one each).  Buffers must not overlap unless a comment says so.  Calls must be
 * made with the device current on which the handle was created (LAPL_ERR_INVALID_ARG otherwise).
 * Pointers need the alignment of their elements only; the fast paths want 16 bytes (see each
 * operator).
 */
#ifndef LAPL_OPS_H
#define LAPL_OPS_H

#include "lapl_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* An output type of the norm alone: 8 bits, 4 of exponent and 3 of mantissa, largest value 448. */
enum { LAPL_F8E4M3 = 2 };

/* ---- gated linear recurrence ---------------------------------------------------------------
 *
 * For each sequence and channel, over the tokens in processing order i = 0 .. len-1:
 *   LAPL_GATE_DECAY:    h_i = a_i h_{i-1} + x_i,              a_i = g_i, which must be in [-1, 1]
 *   LAPL_GATE_SIGMOID:  h_i = a_i h_{i-1} + (1 - a_i) x_i,    a_i = 1 / (1 + exp(-g_i))
 * with h_{-1} = h0 (zeros if NULL).  The processing order is the tokens' order, or with reverse
 * the opposite one, from token len-1 down to token 0.  Arithmetic and states are fp32; with the
 * sigmoid gate an a or a 1 - a below 2^-126 counts as zero.  A state that is not finite leaves the
 * later ones of its sequence and channel, the final one among them, not finite: infinite or NaN.
 */
typedef enum { LAPL_GATE_DECAY = 0, LAPL_GATE_SIGMOID = 1 } lapl_gate;

/* Tokens from one kept state to the next (see states below). */
#define LAPL_SCAN_CHUNK 16

typedef struct {
  int sequences;  /* S >= 0: B*H for [B,H,N,d], B for [B,N,C] (S == 0: calls are no-ops)       */
  int tokens;     /* N >= 1 (1: a step from h0 to the final state)                             */
  int channels;   /* C >= 1: d for [B,H,N,d]                                                   */
  int gate;       /* lapl_gate                                                                 */
  int reverse;    /* 0, or 1: from the last token to the first                                 */
  int in_dtype;   /* lapl_dtype of x and g                                                     */
  int out_dtype;  /* lapl_dtype of out                                                         */
  int grad_dtype; /* lapl_dtype of dout, dx and dg                                             */
  int x_stride;   /* elements from one token's x (and dx) to the next's, >= C; 0: C            */
  int g_stride;   /* the same for g (and dg)                                                   */
} lapl_scan_config;

typedef struct lapl_scan_plan* lapl_scan_handle;

/* Launch choices of a plan's forward (fixed at create), where pointers allow its fastest kernel. */
typedef struct {
  int cluster;  /* CTAs (one thread-block cluster) that share a sequence's tokens               */
  int lanes;    /* threads across the channels of one token                                     */
  int threads;  /* threads of a CTA                                                             */
  int teams;    /* teams of warps that take the tokens in turn, copied ahead (the kernels for long
                   sequences: 768 tokens or more, backward of bf16 512, and an even number of bf16
                   channels), or 0                                                                */
} lapl_scan_plan_info;

lapl_status lapl_scan_create(const lapl_scan_config* cfg, lapl_scan_handle* out);

/*
 * x, g: device [S,N,C] rows of x_stride / g_stride elements; h0: device [S,C] fp32 or NULL;
 * lengths: device [S] int32 or NULL (all N): tokens at lengths[s] and beyond are padding, neither
 *   read nor part of the recurrence (values below 0 count as 0, above N as N);
 * out: device [S,N,C] contiguous, zeros where padding;
 * states: device [S, ceil(N/16), C] fp32 or NULL: h_{i-1} at i = 0, 16, 32, ... of the processing
 *   order, which the backward wants;
 * final_state: device [S,C] fp32 or NULL: h_{len-1} (h0 for a length of zero); may be h0 itself.
 */
lapl_status lapl_scan_forward(lapl_scan_handle h, const void* x, const void* g, const float* h0,
                              const int* lengths, void* out, float* states, float* final_state,
                              void* stream);

/*
 * Gradients for dout = dLoss/dout and dfinal = dLoss/dfinal_state (device [S,C] fp32 or NULL:
 * zeros).  x, g, lengths: the forward's; states: what that forward wrote.  dx, dg: device [S,N,C]
 * rows of x_stride / g_stride elements, zeros where padding (elements between rows are left as
 * they were); dh0: device [S,C] fp32 or NULL; may be dfinal itself.
 */
lapl_status lapl_scan_backward(lapl_scan_handle h, const void* x, const void* g,
                               const float* states, const int* lengths, const void* dout,
                               const float* dfinal, void* dx, void* dg, float* dh0,
                               void* stream);

lapl_status lapl_scan_plan_info_get(lapl_scan_handle h, lapl_scan_plan_info* info);

/*
 * Device-side failure report, as lapl_attn_device_errors (the same word, one per device, read and
 * cleared; synchronises `stream`): the kernels for long sequences exchange maps between CTAs and
 * bound every wait for them (one second); one that gives up sets bit 8, the kernel ends, and its
 * outputs are undefined.  LAPL_ERR_DEVICE_TIMEOUT when a flag was set.
 */
lapl_status lapl_scan_device_errors(lapl_scan_handle h, void* stream, unsigned* flags);

/*
 * Fault injection, for testing that report: wait_ns: the bound of the waits of this plan's calls
 * from now on (0: one second); skip_last = n > 0: the maps of the n-th last round (or of the first,
 * where there are fewer) are never sent, so that the waits for them run out (kernels for long
 * sequences only: plan_info teams > 0); 0: normal.
 */
lapl_status lapl_scan_set_fault_injection(lapl_scan_handle h, unsigned long long wait_ns,
                                          int skip_last);

const char* lapl_scan_last_error(lapl_scan_handle h);
lapl_status lapl_scan_destroy(lapl_scan_handle h);

/* ---- residual addition + root-mean-square norm ---------------------------------------------
 *
 * For each of the B*N tokens, a row of W = H*d values:
 *   s = x + residual,   rstd = 1 / sqrt(mean(s^2) + eps),   y = s * rstd * weight
 * in fp32.  x is [B,H,N,d], as lapl_attn_forward writes it (H = 1: plain rows); everything else is
 * [B,N,W]: the heads are merged on the way.
 */
typedef struct {
  int batch;       /* B >= 0 (B == 0: calls are no-ops, but dweight is written with zeros)      */
  int heads;       /* H >= 1                                                                    */
  int tokens;      /* N >= 1                                                                    */
  int head_dim;    /* d >= 1; W = H*d <= 16384                                                  */
  float eps;       /* >= 0                                                                      */
  int x_dtype;     /* lapl_dtype of x                                                           */
  int res_dtype;   /* lapl_dtype of residual and sum                                            */
  int out_dtype;   /* lapl_dtype of y, or LAPL_F8E4M3                                           */
  int grad_dtype;  /* lapl_dtype of dy, dsum, dx and dres                                       */
  int scale_group; /* LAPL_F8E4M3: values that share a scale: 32, 64 or 128 (W a multiple), or 0
                      for the whole row; 0 otherwise                                            */
} lapl_norm_config;

typedef struct lapl_norm_plan* lapl_norm_handle;

lapl_status lapl_norm_create(const lapl_norm_config* cfg, lapl_norm_handle* out);

/*
 * residual: NULL: none; weight: device [W] fp32 or NULL (ones); sum: device [B,N,W] res_dtype or
 * NULL: s rounded to res_dtype (the norm itself goes by the unrounded s); may be residual itself;
 * rstd: device [B,N] fp32 or NULL; y: device [B,N,W] out_dtype; scales: LAPL_F8E4M3 only: device
 * [B,N, W/scale_group (1 for whole rows)] fp32.  8-bit values are q = round(y / scale) to nearest,
 * ties to even, with scale = max(largest |y| of the group, 2^-100) / 448; y is about q * scale.  A
 * NaN makes its row's values NaN, and their scales.
 */
lapl_status lapl_norm_forward(lapl_norm_handle h, const void* x, const void* residual,
                              const float* weight, void* sum, float* rstd, void* y,
                              float* scales, void* stream);

/* Bytes of device workspace backward() needs for dweight (a multiple of 256). */
lapl_status lapl_norm_workspace_size(lapl_norm_handle h, size_t* bytes);

/*
 * Gradients for dy = dLoss/dy (for an 8-bit y: as if it were not rounded) and dsum = dLoss/dsum
 * from sum's other uses (NULL: none).  sum, rstd: what the forward wrote; weight: the forward's.
 * dx: device [B,H,N,d] or NULL; dres: device [B,N,W] or NULL, the same values as rows (the
 * gradient of x and of residual is one); may be dsum itself; dweight: device [W] fp32 or NULL.
 */
lapl_status lapl_norm_backward(lapl_norm_handle h, const void* sum, const float* rstd,
                               const float* weight, const void* dy, const void* dsum, void* dx,
                               void* dres, float* dweight, void* workspace,
                               size_t workspace_bytes, void* stream);

const char* lapl_norm_last_error(lapl_norm_handle h);
lapl_status lapl_norm_destroy(lapl_norm_handle h);

/* ---- global gradient norm and clipping -----------------------------------------------------
 *
 * norm = sqrt(sum of the squares of every value of every tensor), out = value * scale with
 * scale = max_norm / norm where norm > max_norm, and 1 otherwise.  Squares neither overflow nor
 * vanish: any norm that fp32 holds, down to its smallest values, comes out right.  A norm that is
 * not finite is reported as such and leaves every value as it is.  A scale below 2^-126 has fewer
 * bits than others.
 */
typedef struct {
  int tensors;             /* T >= 0                                                            */
  const long long* counts; /* [T] values of each tensor, >= 0 (host, read by create)            */
  const int* dtypes;       /* [T] lapl_dtype of each (host, read by create)                     */
} lapl_clip_config;

typedef struct lapl_clip_plan* lapl_clip_handle;

lapl_status lapl_clip_create(const lapl_clip_config* cfg, lapl_clip_handle* out);

/* Bytes of device workspace norm() and apply() need (a multiple of 256). */
lapl_status lapl_clip_workspace_size(lapl_clip_handle h, size_t* bytes);

/* norm: device, 1 fp32.  grads: host array of T device pointers (read during the call; NULL where
 * the count is zero). */
lapl_status lapl_clip_norm(lapl_clip_handle h, const void* const* grads, float* norm,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * outs: host array of T device pointers, or NULL: in place.  A tensor may be its own output.
 * Otherwise outputs must overlap neither each other nor any input (LAPL_ERR_INVALID_ARG; in place,
 * the tensors must not overlap each other).  max_norm: finite, >= 0.
 */
lapl_status lapl_clip_apply(lapl_clip_handle h, const void* const* grads, void* const* outs,
                            float max_norm, float* norm, void* workspace, size_t workspace_bytes,
                            void* stream);

const char* lapl_clip_last_error(lapl_clip_handle h);
lapl_status lapl_clip_destroy(lapl_clip_handle h);

#ifdef __cplusplus
}
#endif

#endif /* LAPL_OPS_H */
