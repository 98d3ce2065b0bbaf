/*
 * gconv_ssm.h -- C ABI of the selective-block operators: what a selective
 * state-space block runs around a depthwise convolution (gconv_causal_conv1d_*
 * in gconv_seq.h), with its matrix products in 8-bit floating point.
 *
 *   gconv_selective_scan_*  selective state space scan along a sequence, with the
 *                           carried state that continues it, and its gradients
 *   gconv_matmul_f8         product of two 8-bit floating-point matrices with a
 *                           scale for each block of 128
 *   gconv_quantize_f8       rows, columns or both to that form
 *   gconv_rms_norm_f8       residual addition + root-mean-square norm with an
 *                           output in that form
 *
 * Statuses, data types, error strings, streams, ownership, [B, T, D] strides and
 * `lens` are those of gconv.h and gconv_seq.h: the caller owns every buffer and the
 * stream, calls are asynchronous and thread-safe, nothing is allocated or copied
 * between host and device, nothing is launched on an error, and every call may be
 * made inside a stream capture.  Calls that may run at the same time (two streams,
 * two captured graphs) need a workspace each.  Of a tensor with gaps between its rows
 * the 16-bit neighbours of a row's ends may be read, without effect on any result;
 * nothing before a tensor's first element or after its last one is, and nothing but its
 * elements is written.
 */
#ifndef GCONV_SSM_H_
#define GCONV_SSM_H_

#include "gconv_seq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- selective state space scan ------------------------------------------ */

#define GCONV_SSM_MAX_N 64
/* Tokens between two saved states (gconv_selective_scan_saved_size). */
#define GCONV_SSM_CHUNK 16

/* Layout: 128 bytes, naturally aligned, no implicit padding. */
typedef struct gconv_ssm_problem {
  int64_t B, T;             /* >= 1                                          */
  int32_t D;                /* channels, 1 ... GCONV_SEQ_MAX_D               */
  int32_t N;                /* states of a channel, 1 ... GCONV_SSM_MAX_N    */
  int32_t groups;           /* G >= 1, a divisor of D: channels g D / G ...
                               share the g-th Bm and Cm                      */
  int32_t softplus;         /* 0 or 1                                        */
  int64_t x_stride[2];      /* of x and dx                                   */
  int64_t delta_stride[2];  /* of delta and ddelta                           */
  int64_t z_stride[2];      /* of z and dz                                   */
  int64_t b_stride[2];      /* of Bm and dBm, [B, T, G N]                    */
  int64_t c_stride[2];      /* of Cm and dCm, [B, T, G N]                    */
  int64_t y_stride[2];      /* of y and dy                                   */
} gconv_ssm_problem;

/*
 * gconv_selective_scan_fwd -- with channel d's group g, for each state n < N,
 *   v[b, t, d] = delta[b, t, d] + delta_bias[d]
 *   s[b, t, d] = softplus(v), or v where p->softplus is 0         (the step)
 *   h[b, t, d, n] = exp(s A[d, n]) h[b, t - 1, d, n] + s x[b, t, d] Bm[b, t, g, n]
 *   o[b, t, d] = sum_n h[b, t, d, n] Cm[b, t, g, n] + skip[d] x[b, t, d]
 *   y = o, or o z / (1 + exp(-z)) where z is given
 *   x, delta    [B, T, D] dt;  A [D, N] fp32, finite
 *   Bm, Cm      [B, T, G N] dt
 *   skip        [D] fp32 or NULL (0);  delta_bias [D] fp32 or NULL (0)
 *   z           [B, T, D] dt or NULL
 *   h0          [B, D, N] fp32 packed: the state before the first token, or NULL (zeros)
 *   y           [B, T, D] dt (written)
 *   hT          [B, D, N] fp32 packed, or NULL: the state after the last token
 *               (written); may be h0 itself, so T = 1 with hT == h0 decodes a token
 *   saved       NULL, or gconv_selective_scan_saved_size() bytes, 16-byte aligned: the
 *               state before every GCONV_SSM_CHUNK-th token, for the backward pass
 *   workspace   gconv_selective_scan_fwd_workspace_size() bytes, 16-byte aligned
 *               (may be NULL where that is 0)
 * States, steps and sums are fp32; y is rounded once.  A NaN or an infinity in x, delta or z reaches its own
 * channel only (where an infinity may come out as a NaN), one in Bm or Cm its group's.  One launch, or two where the
 * channels are too few to fill the GPU: the walk over time is then split (by a rule on the
 * sizes alone), each part from a state of 0 first.
 * Errors: GCONV_ERR_INVALID_ARG (malformed problem, a NULL that is not allowed, an
 * output that overlaps another buffer, a workspace that is too small), GCONV_ERR_UNSUPPORTED
 * (dtype), GCONV_ERR_CUDA.
 */
gconv_status gconv_selective_scan_fwd(const void *x, const void *delta, const float *A, const void *Bm, const void *Cm,
                                      const float *skip, const void *z, const float *delta_bias, const float *h0,
                                      const int32_t *lens, void *y, float *hT, void *saved, const gconv_ssm_problem *p,
                                      gconv_dtype dt, void *workspace, int64_t workspace_bytes,
                                      struct CUstream_st *stream);

/*
 * gconv_selective_scan_bwd -- the gradients, given dy (of y) and dhT (of hT, NULL for
 * none), from the forward call's inputs and `saved`; o and h are computed anew.  With
 * a = exp(s A) and do = dy z / (1 + exp(-z)) (dy where there is no z):
 *   g[t] = Cm[t] do[t] + a[t + 1] g[t + 1]  (+ dhT at the last token)
 *   dCm = sum over the group's channels of h[t] do[t];  dBm likewise of g[t] s x
 *   dx = s sum_n g Bm + skip do;  dz = dy o sig(z) (1 + z (1 - sig(z)))
 *   dv = (sum_n g h[t - 1] a A + x sum_n g Bm) * (sig(v), or 1 without softplus)
 *   ddelta = dv;  ddelta_bias = sum_{b, t} dv;  dskip = sum_{b, t} do x
 *   dA = sum_{b, t} g h[t - 1] a s;  dh0 = a[0] g[0]
 *   dx, ddelta [B, T, D] dt, dBm, dCm [B, T, G N] dt, dA [D, N] fp32 (written)
 *   dskip, ddelta_bias [D] fp32, dz [B, T, D] dt, dh0 [B, D, N] fp32: written, or NULL
 *               when not wanted (dz is given only with z)
 *   workspace   gconv_selective_scan_bwd_workspace_size() bytes, 16-byte aligned
 * fp32 sums in an order that depends on the problem only: deterministic.  Two or three
 * launches.  The workspace holds each block of channels' share of dBm and dCm, for a token and
 * channel half a byte with up to 8 states, and 2, 8 and 32 bytes with up to 16, 32 and 64.
 */
gconv_status gconv_selective_scan_bwd(const void *dy, const float *dhT, const void *x, const void *delta,
                                      const float *A, const void *Bm, const void *Cm, const float *skip, const void *z,
                                      const float *delta_bias, const int32_t *lens, const void *saved, void *dx,
                                      void *ddelta, float *dA, void *dBm, void *dCm, float *dskip, void *dz,
                                      float *ddelta_bias, float *dh0, const gconv_ssm_problem *p, gconv_dtype dt,
                                      void *workspace, int64_t workspace_bytes, struct CUstream_st *stream);

/* Bytes of the forward pass's `saved` and of the two workspaces.  Host only, no GPU needed. */
gconv_status gconv_selective_scan_saved_size(const gconv_ssm_problem *p, gconv_dtype dt, int64_t *bytes);
gconv_status gconv_selective_scan_fwd_workspace_size(const gconv_ssm_problem *p, gconv_dtype dt, int64_t *bytes);
gconv_status gconv_selective_scan_bwd_workspace_size(const gconv_ssm_problem *p, gconv_dtype dt, int64_t *bytes);

/* ---- 8-bit floating-point matrices with block scales ---------------------- */

/* Formats: 4 exponent and 3 fraction bits, largest value 448; 5 and 2, 57344. */
typedef enum gconv_f8_format { GCONV_E4M3 = 0, GCONV_E5M2 = 1 } gconv_f8_format;

#define GCONV_F8_BLOCK 128

/*
 * A matrix of R rows and C columns in this form is two buffers:
 *   q      one byte a value; a row starts every `pitch` bytes, a multiple of 16, at least
 *          C (by default C rounded up to 16); the buffer is 16-byte aligned.  Bytes from
 *          C on are neither read nor written.
 *   scale  fp32; block k (columns 128 k ...) of row group j at k * scale_stride + j.  A
 *          row group is one row, or 128 rows (the last one fewer); scale_stride is at least
 *          their number, which it is by default.
 * A value is q times its block's scale.
 */

/* Layout: 72 bytes, naturally aligned, no implicit padding.  0 in a stride means the default. */
typedef struct gconv_matmul_f8_problem {
  int64_t M;               /* rows of xq, 0 ... 2^31 - 512; nothing is done for 0 */
  int32_t N;               /* rows of wq, 1 ... 2^21                          */
  int32_t K;               /* 1 ... 2^20                                      */
  int32_t x_format;        /* gconv_f8_format of xq                           */
  int32_t w_format;        /* and of wq                                       */
  int32_t w_rows;          /* rows of wq with one scale: 1 or 128             */
  int32_t reserved;        /* must be 0                                       */
  int64_t x_pitch, x_scale_stride;
  int64_t w_pitch, w_scale_stride;
  int64_t y_stride;        /* elements between rows of y, at least N          */
} gconv_matmul_f8_problem;

/*
 * gconv_matmul_f8 -- with k's block kb,
 *   y[m, n] = sum_kb x_scale[kb, m] w_scale[kb, n / w_rows] sum_{k in kb} xq[m, k] wq[n, k] (+ bias[n])
 *   xq [M, K] with a scale a row and block, wq [N, K];  bias [N] dt or NULL;  y [M, N] dt (written)
 * A block's products are exact and summed by the tensor cores in fp32, blocks are scaled and
 * summed in fp32, and y is rounded once.  A block's sum times one of its scales, and the two
 * scales' product, have to be within fp32's range: one that is not gives an infinity or a NaN,
 * one below 2^-126 loses places.  One launch.  A bounded wait inside it that runs out is
 * reported through the device's status word (gconv_device_status), as in gconv.h; the output is
 * then incomplete.  The order of a row's sums depends on the sizes of the call and on the
 * device's number of SMs.
 */
gconv_status gconv_matmul_f8(const uint8_t *xq, const float *x_scale, const uint8_t *wq, const float *w_scale,
                             const void *bias, void *y, const gconv_matmul_f8_problem *p, gconv_dtype dt,
                             struct CUstream_st *stream);

/* Layout: 56 bytes, naturally aligned, no implicit padding.  0 in a stride means the default. */
typedef struct gconv_quant_f8_problem {
  int64_t rows;            /* 0 ... 2^31 - 512; nothing is done for 0; blocks of
                              128 x 128 number 2^31 - 1 at most               */
  int32_t D;               /* columns, 1 ... 2^20                             */
  int32_t format;          /* gconv_f8_format                                 */
  int32_t block_rows;      /* rows of a block: 1 or 128                       */
  int32_t reserved;        /* must be 0                                       */
  int64_t x_stride;        /* elements between rows of x, at least D          */
  int64_t q_pitch, scale_stride;    /* of q [rows, D]                         */
  int64_t qt_pitch;        /* of qt [D, rows]; its scale_stride is the default */
} gconv_quant_f8_problem;

/*
 * gconv_quantize_f8 -- for each block, with top = 448 or 57344,
 *   m = max(max|x|, 2^-110);  scale = m / top
 *   q = x * f to the nearest number of the format (ties to even), f = top / m rounded to fp32
 * A block that holds a NaN or an infinity has scale NaN and q 0.
 *   x [rows, D] dt
 *   q, scale      x in blocks of block_rows x 128; both or neither (NULL)
 *   qt, scale_t   x transposed, [D, rows], in blocks of block_rows x 128 of its own (those
 *                 of 128 x 128 are the same ones); both or neither
 * at least one of the two.  One launch, x is read once.
 */
gconv_status gconv_quantize_f8(const void *x, uint8_t *q, float *scale, uint8_t *qt, float *scale_t,
                               const gconv_quant_f8_problem *p, gconv_dtype dt, struct CUstream_st *stream);

/*
 * gconv_rms_norm_f8 -- gconv_rms_norm_q8 (whose record it takes) with an output in blocks of
 * 1 x 128: for each row
 *   h = round_dt(x + residual)   (h = x when residual is NULL)
 *   r = 1 / sqrt(mean(h^2) + eps);  u = h * weight  (rounded to fp32)
 *   y = u * r;  for each block: m = max(max|u|, 2^-110), scale = m r / top,
 *   q = u * f to the nearest number of `format` (ties to even), f = top / m rounded to fp32
 * so that y is about q * scale.  A row whose sum of squares is not finite has scales NaN and q 0;
 * a block whose u is not finite, likewise.
 *   x, residual [rows, D] dt;  weight [D] dt or NULL (ones)
 *   residual_out [rows, D] dt or NULL: h (written); may be x or residual itself
 *   y      [rows, D] dt or NULL: rounded (written)
 *   q, scale   default pitch and stride; both or neither (NULL); at least one of y and q is given
 * fp32 sums and statistics.  One launch.
 */
gconv_status gconv_rms_norm_f8(const void *x, const void *residual, const void *weight, void *residual_out, void *y,
                               uint8_t *q, float *scale, int32_t format, const gconv_norm_problem *p, gconv_dtype dt,
                               struct CUstream_st *stream);

#ifdef __cplusplus
}
#endif

#endif /* GCONV_SSM_H_ */
