/*
 * eg_prompt.h -- C ABI of the operators that take in a prompt (sm_103a): the
 * residual stream's addition and norm with an output in 8 bits.  Conventions as in eg_decoder.h:
 * every call returns an eg_status, argument errors are found before any device
 * work is queued, eg_last_error_detail() describes the last failure of this
 * thread, the caller owns every tensor and keeps it alive until the stream has
 * passed it, calls are queued on `stream` of the current device and do not
 * synchronise.  Strides are in ELEMENTS; the innermost dimension is
 * contiguous.  Sums and softmax statistics are float32; each output is rounded
 * once, to its own type, nearest even.
 */
#ifndef EG_PROMPT_H
#define EG_PROMPT_H

#include "eg_decoder.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ----------------------- addition to the residual stream, norm, 8 bits ----
 *
 * For each row, with s = x + residual rounded to the type (s = x without a
 * residual):
 *
 *   h   = s * weight / sqrt(mean(s^2) + eps)
 *   sum = s,  out = h rounded to the type
 *
 * and, with a quant mode, codes and scales of h (from float32, not from out)
 * as the linear plans take them for A and s_a:
 *
 *   EG_NORM_E4M3, EG_NORM_INT8: a = max |h| of the row
 *   EG_NORM_E4M3_BLOCK: a = max |h| of each block of 128 columns
 *   scale = a / 448 (INT8: a / 127), 1 where that is 0; code = h / scale,
 *   nearest even, saturated (+-448; +-127)
 *
 * A row (block) with a NaN has a NaN scale.  sum may be x or residual, out may
 * be x, residual or sum where that is not wanted (same strides); otherwise
 * outputs must not overlap inputs or each other. */
enum { EG_NORM_PLAIN = 0, EG_NORM_E4M3 = 1, EG_NORM_INT8 = 2, EG_NORM_E4M3_BLOCK = 3 };

typedef struct {
  int64_t rows, width;          /* up to 2^24 rows of 1..65536 (blocks: a multiple of 128) */
  int32_t dtype;                /* eg_el_dtype of x, residual, weight, sum and out */
  int32_t quant;                /* EG_NORM_* */
  float eps;
  const void *x, *residual;     /* [rows][width] by the strides; residual: NULL for none */
  const void* weight;           /* [width] */
  int64_t x_row, residual_row;
  void *sum, *out;              /* sum: with a residual; out: may be NULL with a quant mode */
  int64_t sum_row, out_row;
  void* codes;                  /* [rows][width] bytes */
  int64_t codes_row;
  float* scales;                /* [rows] or [rows][width / 128], contiguous */
} eg_norm_args;

EG_API eg_status eg_add_rms_norm(const eg_norm_args* args, void* stream);

/* Gradients, from the given gradient of out (or of what the codes stand for)
 * and, where not NULL, that of sum.  With z = s and g = d_out * weight:
 *
 *   r = 1 / sqrt(mean(z^2) + eps)
 *   dx = d_sum + r g - z r^3 mean(g z)   (the gradient of x and of residual)
 *   d_weight = sum over rows of d_out z r
 *
 * dx may be d_out or d_sum (same stride).  d_weight is float32, summed in a
 * fixed order, NULL: not wanted.  `workspace`: at least
 * eg_add_rms_norm_workspace_bytes() of device memory with d_weight, 16-byte
 * aligned, not shared by calls that overlap. */
typedef struct {
  int64_t rows, width;
  int32_t dtype;                /* eg_el_dtype of d_out, sum, weight, d_sum and dx */
  float eps;
  const void *d_out, *sum, *weight, *d_sum;
  int64_t d_out_row, sum_row, d_sum_row;
  void* dx;
  int64_t dx_row;
  float* d_weight;
  void* workspace;
  size_t workspace_bytes;
} eg_norm_grads;

EG_API eg_status eg_add_rms_norm_backward(const eg_norm_grads* args, void* stream);
EG_API eg_status eg_add_rms_norm_workspace_bytes(const eg_norm_grads* args, size_t* out);

#ifdef __cplusplus
}
#endif
#endif /* EG_PROMPT_H */
