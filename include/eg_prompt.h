/*
 * eg_prompt.h -- C ABI of the operators that take in a prompt (sm_103a): the
 * residual stream's addition and norm with an output in 8 bits, low-rank
 * adapters of many requests beside a shared projection, and attention of
 * chunks of new tokens over a paged cache.  Conventions as in eg_decoder.h:
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
 *   scale = a / 448 (INT8: a / 127), 1 where that is 0; code = h times the
 *   float32 reciprocal of scale (h / scale where scale is below 2^-126),
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

/* --------------------------------- low-rank adapters of many requests -----
 *
 * Sequence b is rows seq_start[b] .. seq_start[b + 1] of x and has adapter
 * a = adapter[b].  For each of its rows, with A_a [rank][inputs] and
 * B_a [outputs][rank]:
 *
 *   out = base + scales[a] * (x A_a^T) B_a^T
 *
 * (base 0 where NULL; scales 1 where NULL; nothing is added where a is outside
 * [0, adapters)).  x A_a^T is kept to float32 sums and enters the second
 * product as two 16-bit parts, some 2^-16 of its row's largest value off.
 * seq_start and adapter are read on the device, so a captured graph replays
 * with new ones; seq_start rises, and is cut to the rows there are.  Rows that
 * no sequence has are not written.  An adapter of a lower rank than the bank's
 * is padded with zeros.  out may be base (same stride). */
typedef struct {
  int32_t rows, sequences;      /* of x; up to 2^24 rows, 65536 sequences */
  int32_t adapters;
  int32_t inputs, outputs;      /* multiples of 8, 8..2^20 */
  int32_t rank;                 /* a multiple of 8, 8..128 */
  int32_t dtype;                /* EG_EL_BF16 or EG_EL_F16 of x, a, b, base and out */
  const void* x;                /* [rows][inputs] by the stride */
  int64_t x_row;
  const void *a, *b;            /* [adapters][rank][inputs], [adapters][outputs][rank], contiguous */
  const float* scales;          /* [adapters] */
  const int32_t* seq_start;     /* [sequences + 1] */
  const int32_t* adapter;       /* [sequences] */
  const void* base;             /* [rows][outputs] by the stride */
  int64_t base_row;
  void* out;
  int64_t out_row;              /* x, a, b, base, out and their rows: multiples of 16 bytes */
  void* workspace;              /* at least eg_lora_workspace_bytes(), 16-byte aligned, not shared by calls that overlap */
  size_t workspace_bytes;
} eg_lora_args;

EG_API eg_status eg_lora(const eg_lora_args* args, void* stream);
EG_API eg_status eg_lora_workspace_bytes(const eg_lora_args* args, size_t* out);
/* Synchronise the current device and report a wait of eg_lora on it that ran
 * past its limit since the last report (EG_ERR_DEVICE_TIMEOUT, then cleared):
 * what the calls since then wrote is not to be used. */
EG_API eg_status eg_lora_device_status(void);
/* Testing hook for failure detection, as eg_token_logprobs_set_test_stall. */
EG_API eg_status eg_lora_set_test_stall(uint64_t wait_limit_ns, int32_t stall_loader);

/* ---------------------- attention of chunks of new tokens over the cache --
 *
 * Sequence b has context_lens[b] cached tokens and n_b = q_start[b + 1] -
 * q_start[b] new ones (0 or more; 1 for ordinary decoding), whose keys and
 * values follow the context in the same cache: place j of the sequence is in
 * page block_table[b][j / page_size], place j % page_size.  New token t
 * (packed row q_start[b] + t of q) stands at place i = context_lens[b] + t and
 * attends to the places j <= i with i - j < window or j < sinks; to all j <= i
 * where window is 0.  For query head h, with the cached head
 * h / (q_heads / kv_heads):
 *
 *   o = sum_j softmax_j(scale q . k_j) v_j,  lse = log sum_j exp(scale q . k_j)
 *
 * Places that a token does not attend to, slots of the cache past a sequence's
 * end and table entries past its pages have no part, whatever they hold.
 * Sequence lengths are read on the device, so a captured graph replays with
 * new ones; lengths beyond the plan's limits, the table or the packed rows are
 * cut to them, and table entries outside [0, num_pages) read as zero keys and
 * values.  Rows of o and lse that are no sequence's (before q_start[0], from
 * q_start[batch] on, and a sequence's past max_chunk) are not written.
 *
 * A plan owns the partial results of sequences that it splits over the GPU;
 * runs of one plan must not overlap on the GPU.  It belongs to the device that
 * is current when it is made, as an eg_tree_plan does. */
typedef struct {
  int32_t q_heads, kv_heads;    /* as in eg_tree_problem */
  int32_t head_dim;             /* a multiple of 8, 8..128 */
  int32_t dtype;                /* EG_EL_BF16 or EG_EL_F16 (q, cache and o) */
  int32_t page_size;            /* a multiple of 8 */
  int32_t max_batch;            /* sequences of a run, 1..65536 */
  int32_t max_chunk;            /* new tokens of a sequence, 1..2^20 */
} eg_chunk_problem;

typedef struct {
  int32_t batch;
  int32_t tokens;               /* rows of q and o */
  const void* q;                /* [tokens][q_heads][head_dim] by the strides, 16-byte aligned rows */
  void* o;
  int64_t q_token, q_head, o_token, o_head;
  const int32_t* block_table;   /* [batch][table_stride], table_stride entries of each may be read */
  int64_t table_stride;
  const int32_t* context_lens;  /* [batch] */
  const int32_t* q_start;       /* [batch + 1], rising */
  int32_t window, sinks;        /* 0 or more; sinks only with a window */
  float scale;                  /* positive */
  float* lse;                   /* [tokens][q_heads], or NULL */
} eg_chunk_args;

typedef struct eg_chunk_plan eg_chunk_plan;

EG_API eg_status eg_chunk_plan_create(const eg_chunk_problem* problem, eg_chunk_plan** out);
EG_API eg_status eg_chunk_plan_workspace_bytes(const eg_chunk_plan* plan, size_t* out);
EG_API eg_status eg_chunk_plan_run(eg_chunk_plan* plan, const eg_chunk_args* args,
                                   const eg_kv_cache* cache, void* stream);
/* As eg_tree_plan_device_status and eg_tree_plan_set_test_stall. */
EG_API eg_status eg_chunk_plan_device_status(eg_chunk_plan* plan);
EG_API eg_status eg_chunk_plan_set_test_stall(eg_chunk_plan* plan, uint64_t wait_limit_ns,
                                              int32_t stall_producer);
EG_API eg_status eg_chunk_plan_destroy(eg_chunk_plan* plan);

#ifdef __cplusplus
}
#endif
#endif /* EG_PROMPT_H */
