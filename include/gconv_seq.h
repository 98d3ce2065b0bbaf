/*
 * gconv_seq.h -- C ABI of the sequence operators: what a recurrent
 * language-model block runs around a depthwise convolution.
 *
 *   gconv_causal_conv1d_*   causal depthwise convolution along a sequence, with
 *                           the carried state that continues it
 *   gconv_gated_scan_*      gated linear recurrence along a sequence
 *   gconv_rms_norm_q8       residual addition + root-mean-square norm, with an
 *                           output in 8 bits and a scale for each row
 *   gconv_quantize_rows_q8  rows to 8 bits with a scale each (weights, activations)
 *   gconv_matmul_q8         product of two 8-bit matrices with their rows' scales
 *
 * Statuses, data types (gconv_dtype), error strings, streams and ownership are
 * those of gconv.h: the caller owns every buffer and the stream, calls are
 * asynchronous and thread-safe, nothing is allocated or copied between host
 * and device, nothing is launched on an error, and every call may be made
 * inside a stream capture.  A NULL stream is the legacy default stream.
 *
 * Sequence tensors are [B, T, D]: element (b, t, d) lies at
 * b * stride[0] + t * stride[1] + d (in elements; channels are contiguous).
 * A stride pair {0, 0} means packed, {T * D, D}.  Batch-major and time-major
 * orders, and column slices of a wider tensor, are all expressed by strides;
 * rows must not overlap one another.  `lens` (device, int32 [B], or NULL for
 * T everywhere) gives the tokens in each sequence, 0 ... T (other values are
 * clamped): what a tensor holds from position lens[b] on has no effect, NaN
 * included, though it may be read; outputs and input gradients there are zero,
 * and the state that comes out is the one after lens[b] tokens (the state that
 * went in, where lens[b] is 0).
 */
#ifndef GCONV_SEQ_H_
#define GCONV_SEQ_H_

#include "gconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest D of a [B, T, D] tensor (2^31 - 128). */
#define GCONV_SEQ_MAX_D 2147483520

/* ---- causal depthwise convolution -------------------------------------- */

#define GCONV_CONV1D_MAX_K 8

/* Layout: 64 bytes, naturally aligned, no implicit padding. */
typedef struct gconv_conv1d_problem {
  int64_t B, T;         /* >= 1                                              */
  int32_t D;            /* channels, 1 ... GCONV_SEQ_MAX_D                   */
  int32_t K;            /* filter taps, 1 ... GCONV_CONV1D_MAX_K             */
  int32_t act;          /* 0 none, 1 SiLU                                    */
  int32_t reserved;     /* must be 0                                         */
  int64_t x_stride[2];  /* of x and dx                                       */
  int64_t y_stride[2];  /* of y and dy                                       */
} gconv_conv1d_problem;

/*
 * gconv_causal_conv1d_fwd -- each channel's own short filter along time:
 *   u[b, t, d] = bias[d] + sum_{j < K} w[d, j] * e[b, t - (K - 1) + j, d]
 *   y = act(u),  SiLU(u) = u / (1 + exp(-u))
 * e is x, and before it the K - 1 rows of state_in (zeros if that is NULL).
 *   x [B, T, D] dt;  w [D, K] dt;  bias [D] dt or NULL
 *   state_in   [B, K - 1, D] dt packed, or NULL
 *   y          [B, T, D] dt (written)
 *   state_out  [B, K - 1, D] dt packed, or NULL: the last K - 1 rows of e
 *              (written); may be state_in itself.  One token at a time, T = 1
 *              with state_out == state_in, continues the sequence.
 * fp32 sums, one round-to-nearest-even cast.  One launch.  With K == 1 there is
 * no state and both state pointers are ignored.
 * Errors: GCONV_ERR_INVALID_ARG (malformed problem, NULL x / w / y, an output
 * that overlaps an input or another output), GCONV_ERR_UNSUPPORTED (dtype),
 * GCONV_ERR_CUDA.
 */
gconv_status gconv_causal_conv1d_fwd(const void *x, const void *w, const void *bias, const void *state_in,
                                     const int32_t *lens, void *y, void *state_out, const gconv_conv1d_problem *p,
                                     gconv_dtype dt, struct CUstream_st *stream);

/*
 * gconv_causal_conv1d_bwd -- the gradients, given dy (of y) and dstate_out (of
 * state_out; NULL for none), recomputing u from the forward call's inputs:
 *   du = dy * act'(u);  dw[d, j] = sum_{b, t} du[b, t, d] * e[b, t - (K-1) + j, d]
 *   dbias[d] = sum du;  de[b, s, d] = sum_j w[d, j] * du[b, s + (K-1) - j, d]
 *   (+ dstate_out on the last K - 1 rows of e);  dx and dstate_in are de's parts.
 *   dx [B, T, D] dt, dw [D, K] dt (written);  dbias [D] dt, dstate_in
 *   [B, K - 1, D] dt: written, or NULL when not wanted
 *   workspace  gconv_causal_conv1d_bwd_workspace_size() bytes, 16-byte aligned
 * The sums over tokens run in fp32 in an order that depends on the problem
 * only: the result is deterministic.  Two launches.
 */
gconv_status gconv_causal_conv1d_bwd(const void *dy, const void *dstate_out, const void *x, const void *w,
                                     const void *bias, const void *state_in, const int32_t *lens, void *dx, void *dw,
                                     void *dbias, void *dstate_in, const gconv_conv1d_problem *p, gconv_dtype dt,
                                     void *workspace, int64_t workspace_bytes, struct CUstream_st *stream);

/* Device workspace bytes gconv_causal_conv1d_bwd needs.  Host only, no GPU needed. */
gconv_status gconv_causal_conv1d_bwd_workspace_size(const gconv_conv1d_problem *p, gconv_dtype dt, int64_t *bytes);

/* ---- gated linear recurrence -------------------------------------------- */

/* Tokens between two saved states (gconv_gated_scan_saved_size). */
#define GCONV_SCAN_CHUNK 8

/* Layout: 88 bytes, naturally aligned, no implicit padding. */
typedef struct gconv_scan_problem {
  int64_t B, T;         /* >= 1                                              */
  int32_t D;            /* channels, 1 ... GCONV_SEQ_MAX_D                   */
  float decay;          /* c, > 0 and finite                                 */
  int64_t x_stride[2];  /* of x and dx                                       */
  int64_t r_stride[2];  /* of r and dr                                       */
  int64_t i_stride[2];  /* of i and di                                       */
  int64_t y_stride[2];  /* of y and dy                                       */
} gconv_scan_problem;

/*
 * gconv_gated_scan_fwd -- with sig the logistic function,
 *   l[b, t, d] = -c * softplus(lam[d]) * sig(r[b, t, d])          (log decay)
 *   h[b, t, d] = exp(l) * h[b, t - 1, d] + sqrt(1 - exp(2 l)) * sig(i[b, t, d]) * x[b, t, d]
 *   y = h
 *   x, r, i  [B, T, D] dt;  lam [D] fp32
 *   h0       [B, D] fp32 packed: the state before the first token, or NULL (zeros)
 *   y        [B, T, D] dt (written)
 *   hT       [B, D] fp32 packed, or NULL: the state after the last token
 *            (written); may be h0 itself, so T = 1 with hT == h0 decodes a token
 *   saved    NULL, or gconv_gated_scan_saved_size() bytes, 16-byte aligned: the
 *            state before every GCONV_SCAN_CHUNK-th token, for the backward pass
 * c softplus(lam) is taken as at most 3.4e38 (lam of infinity: a = 0, s = 1).
 * The state is held in fp32, 1 - exp(2 l) is computed without cancellation,
 * and y is rounded once.  A factor sqrt(...) sig(i) may come out up to 1e-18 less
 * than it is, and smaller ones as 0, over several tokens; a single token (T = 1) and
 * the backward pass keep them, down to sig(i) of 1e-38.  One launch.  A bounded wait
 * inside it that runs out is reported through the device's status word
 * (gconv_device_status), as in gconv.h; the outputs are then incomplete.  The same
 * holds for the backward pass and gconv_matmul_q8.
 */
gconv_status gconv_gated_scan_fwd(const void *x, const void *r, const void *i, const float *lam, const float *h0,
                                  const int32_t *lens, void *y, float *hT, void *saved, const gconv_scan_problem *p,
                                  gconv_dtype dt, struct CUstream_st *stream);

/*
 * gconv_gated_scan_bwd -- the gradients, given dy (of y) and dhT (of hT, NULL
 * for none), from the forward call's inputs and `saved`.  With a = exp(l),
 * s = sqrt(1 - a^2):
 *   g[t] = dy[t] + a[t + 1] * g[t + 1]  (+ dhT at the last token)
 *   dx = g s sig(i);  di = g s x sig(i) (1 - sig(i))
 *   dl = a g h[t - 1] - a^2 / s * g sig(i) x;  dr = dl * l * (1 - sig(r))
 *   dlam = sum_{b, t} dl * -c sig(r) * sig(lam);  dh0 = a[0] g[0]
 * Where 1 - a^2 is 0 (a gate that is shut altogether) the second term of dl is
 * taken as 0, which is the limit of its share of dr and dlam.
 *   dx, dr, di  [B, T, D] dt (written);  dlam [D] fp32 (written)
 *   dh0         [B, D] fp32 (written), or NULL when not wanted
 *   workspace   gconv_gated_scan_bwd_workspace_size() bytes, 16-byte aligned
 * Deterministic.  Two launches.
 */
gconv_status gconv_gated_scan_bwd(const void *dy, const float *dhT, const void *x, const void *r, const void *i,
                                  const float *lam, const int32_t *lens, const void *saved, void *dx, void *dr,
                                  void *di, float *dlam, float *dh0, const gconv_scan_problem *p, gconv_dtype dt,
                                  void *workspace, int64_t workspace_bytes, struct CUstream_st *stream);

/* Bytes of the forward pass's `saved` / of the backward pass's workspace.  Host only. */
gconv_status gconv_gated_scan_saved_size(const gconv_scan_problem *p, gconv_dtype dt, int64_t *bytes);
gconv_status gconv_gated_scan_bwd_workspace_size(const gconv_scan_problem *p, gconv_dtype dt, int64_t *bytes);

/* ---- norm and 8-bit rows -------------------------------------------------- */

#define GCONV_NORM_MAX_D 32768

/* Layout: 48 bytes, naturally aligned, no implicit padding.  Row strides in
 * elements, at least D; 0 means D. */
typedef struct gconv_norm_problem {
  int64_t rows;            /* >= 0; nothing is done for 0                     */
  int32_t D;               /* 1 ... GCONV_NORM_MAX_D                          */
  float eps;               /* >= 0 and finite                                 */
  int64_t x_stride;        /* of x                                            */
  int64_t residual_stride; /* of residual and residual_out                    */
  int64_t y_stride;        /* of y                                            */
  int64_t reserved;        /* must be 0                                       */
} gconv_norm_problem;

/*
 * gconv_rms_norm_q8 -- for each row
 *   h = round_dt(x + residual)   (h = x when residual is NULL)
 *   v = h / sqrt(mean(h^2) + eps) * weight
 *   scale = max|v| / 127;  q = v / scale, to the nearest integer (ties to even;
 *                          where h weight takes more than 16 bits, within 2^-24 of
 *                          a tie either side)
 * so that v is about q * scale.  The norm reads h as it is stored, so a pass
 * that starts from residual_out computes the same v.  A row of zeros has v 0,
 * scale 0 and q 0; a row whose sum of squares is not finite (it holds a NaN, an
 * infinity, or values whose squares pass fp32) has scale NaN and q 0.
 *   x, residual [rows, D] dt;  weight [D] dt or NULL (ones)
 *   residual_out [rows, D] dt or NULL: h (written); may be x or residual itself
 *   y      [rows, D] dt or NULL: v rounded (written)
 *   q      int8 [rows, D] packed, and scale fp32 [rows]: both or neither (NULL);
 *          at least one of y and q is given
 * fp32 sums and statistics.  One launch.
 */
gconv_status gconv_rms_norm_q8(const void *x, const void *residual, const void *weight, void *residual_out, void *y,
                               int8_t *q, float *scale, const gconv_norm_problem *p, gconv_dtype dt,
                               struct CUstream_st *stream);

/* gconv_quantize_rows_q8 -- q and scale of the rows of x themselves (v = x in
 * the terms of gconv_rms_norm_q8; NaN and q 0 where max|x| is not finite).
 * p->rows, p->D and p->x_stride are read. */
gconv_status gconv_quantize_rows_q8(const void *x, int8_t *q, float *scale, const gconv_norm_problem *p, gconv_dtype dt,
                                    struct CUstream_st *stream);

/* ---- 8-bit matrix product -------------------------------------------------- */

#define GCONV_MATMUL_Q8_MAX_K 65536
#define GCONV_MATMUL_Q8_MAX_N (1 << 21)

/* Layout: 32 bytes, naturally aligned, no implicit padding. */
typedef struct gconv_matmul_q8_problem {
  int64_t M;         /* rows of xq, >= 0; nothing is done for 0               */
  int32_t N;         /* rows of wq, 1 ... GCONV_MATMUL_Q8_MAX_N               */
  int32_t K;         /* 1 ... GCONV_MATMUL_Q8_MAX_K                           */
  int64_t y_stride;  /* elements between rows of y, at least N; 0 means N     */
  int64_t reserved;  /* must be 0                                             */
} gconv_matmul_q8_problem;

/*
 * gconv_matmul_q8 -- y[m, n] = x_scale[m] * w_scale[n] * sum_k xq[m, k] * wq[n, k] (+ bias[n])
 *   xq int8 [M, K], wq int8 [N, K] packed;  x_scale fp32 [M], w_scale fp32 [N]
 *   bias [N] dt or NULL;  y [M, N] dt (written)
 * Products are exact and summed in 32 bits: as integers for up to 8 rows with K and
 * both operands on 16 bytes, else as fp32 on the tensor cores.  The two agree to the
 * bit while a sum and its parts stay below 2^24 (K up to 1024 whatever the values);
 * past that the fp32 sum is rounded, so a row's last bits can depend on how many rows
 * the call has, and with them on the order of its sum.  Scales and bias are applied in
 * fp32 before one rounding.  One launch.
 */
gconv_status gconv_matmul_q8(const int8_t *xq, const float *x_scale, const int8_t *wq, const float *w_scale,
                             const void *bias, void *y, const gconv_matmul_q8_problem *p, gconv_dtype dt,
                             struct CUstream_st *stream);

#ifdef __cplusplus
}
#endif

#endif /* GCONV_SEQ_H_ */
