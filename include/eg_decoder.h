/*
 * eg_decoder.h -- C ABI of the operators that stand between the fused linear
 * layers of a decoder (sm_103a): per-head norm of queries and keys with the
 * position rotation, appending to a paged key/value cache, attention of
 * drafted token trees over that cache, and the log probabilities of given
 * tokens.  Same conventions as eg.h: every call returns an eg_status,
 * argument errors are found before any device work is queued,
 * eg_last_error_detail() describes the last failure of this thread, the
 * caller owns every tensor and keeps it alive until the stream has passed it,
 * calls are queued on `stream` (a cudaStream_t, NULL: the legacy default
 * stream) of the current device and do not synchronise.
 *
 * Strides are in ELEMENTS; the innermost dimension (head_dim, vocabulary) is
 * contiguous.  Sums, softmax statistics and gradients of weights are float32;
 * each output is rounded once, to its own type, nearest even.
 */
#ifndef EG_DECODER_H
#define EG_DECODER_H

#include "eg.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { EG_EL_BF16 = 0, EG_EL_F16 = 1, EG_EL_F32 = 2 } eg_el_dtype;

/* ------------------------------------ head norm and position rotation ----
 *
 * For each token t and head h, with x the head's head_dim values:
 *
 *   z = x * w / sqrt(mean(x^2) + eps)     (z = x where the weight is NULL)
 *   for each pair i < rot_dim / 2, at position p = positions[t]:
 *     y_a = z_a c - z_b s,  y_b = z_b c + z_a s,
 *     c = cos_sin[p][i],    s = cos_sin[p][rot_dim / 2 + i]
 *   values past rot_dim are z.
 *
 * `pairs` 0: pair i is (i, i + rot_dim / 2); 1: (2 i, 2 i + 1).  A token whose
 * position is outside [0, max_positions) gets NaN in its rotated values (the
 * table is not read there).  Outputs may be their own inputs (same strides);
 * they must not overlap them in another way.
 */
typedef struct {
  int64_t tokens;
  int32_t q_heads, kv_heads;    /* either may be 0 */
  int32_t head_dim;             /* 2..256, even */
  int32_t rot_dim;              /* even, 0..head_dim; 0: no rotation */
  int32_t dtype;                /* eg_el_dtype of q, k, v, weights, outputs, cache */
  int32_t pairs;
  float eps;
  int32_t page_size;            /* eg_kv_append: tokens of a page */
  const float* cos_sin;         /* [max_positions][rot_dim], contiguous */
  int64_t max_positions;
  const int64_t* positions;     /* [tokens]; NULL: 0, 1, 2, ... */
  const void* q_weight;         /* [head_dim]; NULL: queries are not normed */
  const void* k_weight;
  const void *q, *k, *v;        /* [tokens][heads][head_dim] by the strides; v: eg_kv_append */
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  void *q_out, *k_out;          /* k_out: eg_qk_norm_rope and its backward pass */
  int64_t qo_token, qo_head, ko_token, ko_head;
} eg_rope_args;

/* q_out, k_out of the formula above. */
EG_API eg_status eg_qk_norm_rope(const eg_rope_args* args, void* stream);

/* Gradients of eg_qk_norm_rope.  `fwd` holds the forward call's q, k, weights,
 * positions and table; its q_out / k_out (with their strides) are the GIVEN
 * gradients of the outputs and are only read.  Writes dq, dk and, where the
 * weight is not NULL, dq_weight / dk_weight (float32 [head_dim], NULL: not
 * wanted), summed over tokens and heads in a fixed order.  dq / dk may be the
 * given gradients themselves (same strides).  The rotation's table gets no
 * gradient.  `workspace`: at least eg_qk_norm_rope_workspace_bytes() of
 * device memory, 16-byte aligned, not shared by calls that overlap. */
typedef struct {
  void *dq, *dk;
  int64_t dq_token, dq_head, dk_token, dk_head;
  float *dq_weight, *dk_weight;
  void* workspace;
  size_t workspace_bytes;
} eg_rope_grads;

EG_API eg_status eg_qk_norm_rope_backward(const eg_rope_args* fwd, const eg_rope_grads* grads,
                                          void* stream);
EG_API eg_status eg_qk_norm_rope_workspace_bytes(const eg_rope_args* fwd, size_t* out);

/* ------------------------------------------------- paged key/value cache --
 *
 * k and v: [num_pages][page_size][kv_heads][head_dim] by the strides (shared
 * by both), so pages may be stored tokens-first or heads-first. */
typedef struct {
  void *k, *v;
  int64_t num_pages;
  int64_t page_stride, token_stride, head_stride;
} eg_kv_cache;

/* Append: for each token t with 0 <= slots[t] < num_pages * page_size, the
 * normed and rotated key and the value go to page slots[t] / page_size, place
 * slots[t] % page_size; other slots append nothing (a padded token).  Slots
 * of one call differ from each other.  With q and q_out the queries are
 * normed and rotated in the same launch, for every token. */
EG_API eg_status eg_kv_append(const eg_rope_args* args, const eg_kv_cache* cache,
                              const int64_t* slots, void* stream);

/* ------------------------------ attention of drafted trees over the cache --
 *
 * Sequence b has context_lens[b] cached tokens and n_b = q_start[b + 1] -
 * q_start[b] drafted ones (0 or more; 1 for ordinary decoding), whose keys and
 * values follow the context in the same cache: place j of the sequence is in
 * page block_table[b][j / page_size], place j % page_size.  Token t of the
 * tree (packed row q_start[b] + t of q) attends to the whole context and to
 * the drafted tokens u whose bit u is set in its mask words (bit u % 32 of
 * mask[row][u / 32]); without a mask to u <= t.  For query head h, with the
 * cached head h / (q_heads / kv_heads):
 *
 *   o = sum_j softmax_j(scale q . k_j) v_j      over the places j it attends to
 *   lse = log sum_j exp(scale q . k_j)
 *
 * A token that attends to nothing has o = 0 and lse = -infinity.  Places that
 * a token does not attend to, slots of the cache past a sequence's end and
 * table entries past its pages have no part, whatever they hold.  Sequence
 * lengths are read on the device, so a captured graph replays with new ones;
 * lengths beyond the plan's limits, the table or the packed rows are cut to
 * them, and table entries outside [0, num_pages) read as zero keys and values.
 * Rows of o and lse that are no sequence's (before q_start[0], from
 * q_start[batch] on, and a sequence's past max_tree) are not written.
 *
 * A plan owns the partial results of sequences that it splits over the GPU;
 * runs of one plan must not overlap on the GPU.  It belongs to the device that
 * is current when it is made: runs and status calls with another one current
 * are refused (EG_ERR_INVALID_ARG); destroying it is not. */
typedef struct {
  int32_t q_heads, kv_heads;    /* q_heads a multiple of kv_heads: 1..16 times as many, or another
                                   number whose least common multiple with 8 is at most 128 */
  int32_t head_dim;             /* a multiple of 8, 8..128 */
  int32_t dtype;                /* EG_EL_BF16 or EG_EL_F16 (q, cache and o) */
  int32_t page_size;            /* a multiple of 8 */
  int32_t max_batch;            /* sequences of a run, 1..65536 */
  int32_t max_tree;             /* drafted tokens of a sequence, 1..256 */
} eg_tree_problem;

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
  const uint32_t* mask;         /* [tokens][mask_stride] words, or NULL */
  int64_t mask_stride;          /* at least max_tree / 32, rounded up */
  float scale;                  /* positive */
  float* lse;                   /* [tokens][q_heads], or NULL */
} eg_tree_args;

typedef struct eg_tree_plan eg_tree_plan;

EG_API eg_status eg_tree_plan_create(const eg_tree_problem* problem, eg_tree_plan** out);
EG_API eg_status eg_tree_plan_workspace_bytes(const eg_tree_plan* plan, size_t* out);
EG_API eg_status eg_tree_plan_run(eg_tree_plan* plan, const eg_tree_args* args,
                                  const eg_kv_cache* cache, void* stream);
/* Synchronise the plan's device and report a wait in its kernels that ran past
 * its limit (EG_ERR_DEVICE_TIMEOUT, then cleared; what the plan's runs wrote
 * since the wait is not to be used). */
EG_API eg_status eg_tree_plan_device_status(eg_tree_plan* plan);
/* Testing hook for failure detection, as eg_plan_set_test_stall: limit the
 * kernels' waits to `wait_limit_ns` (0: the default) and, with
 * `stall_producer` 1, have no keys loaded, so that the first wait runs out. */
EG_API eg_status eg_tree_plan_set_test_stall(eg_tree_plan* plan, uint64_t wait_limit_ns,
                                             int32_t stall_producer);
/* Free everything the plan owns, after synchronising its device. */
EG_API eg_status eg_tree_plan_destroy(eg_tree_plan* plan);

/* ------------------------------------------- log probabilities of tokens --
 *
 * For each row of logits x[0..vocab):
 *
 *   lse     = log sum_v exp(x_v)
 *   logprob = x[token] - lse                    (0 where the token is outside
 *                                                [0, vocab): none is given)
 *   entropy = -sum_v p_v log p_v, p = exp(x - lse)
 *   top_ids, top_logprobs: the `top` largest logits, of equal ones the lowest
 *             id first, and their x - lse.
 *
 * Logits of -infinity have probability 0.  A row of nothing else has lse and
 * log probabilities of -infinity and entropy 0.  A row with +infinity has lse
 * +infinity and NaN elsewhere; one with a NaN has NaN everywhere and ids -1.
 * Each output may be NULL (not wanted). */
typedef struct {
  int64_t rows, vocab;
  int32_t dtype;                /* eg_el_dtype of the logits (and of d_logits) */
  int32_t top;                  /* 0..32, at most vocab */
  const void* logits;
  int64_t row_stride;           /* at least vocab */
  const int64_t* tokens;        /* [rows]; NULL: none is given */
  float *logprob, *lse, *entropy; /* [rows] */
  int64_t* top_ids;             /* [rows][top] */
  float* top_logprobs;          /* [rows][top] */
} eg_score_args;

EG_API eg_status eg_token_logprobs(const eg_score_args* args, void* stream);
/* Synchronise the current device and report a wait of eg_token_logprobs on it
 * that ran past its limit since the last report (EG_ERR_DEVICE_TIMEOUT, then
 * cleared).  A row whose logits never came has NaN everywhere and ids -1, as
 * one with a NaN among its logits: this call tells them apart. */
EG_API eg_status eg_token_logprobs_device_status(void);
/* Testing hook for failure detection, for the calls that follow in this
 * process: limit the kernel's waits to `wait_limit_ns` (0: the default) and,
 * with `stall_loader` 1, have no logits loaded, so that the first wait for
 * some runs out. */
EG_API eg_status eg_token_logprobs_set_test_stall(uint64_t wait_limit_ns, int32_t stall_loader);

/* The gradient to the logits, from the rows' lse and entropy (as
 * eg_token_logprobs gave them) and the given gradients of logprob and entropy
 * (NULL: zero):
 *
 *   d_x[v] = d_logprob (1[v = token] - p_v) - d_entropy p_v (log p_v + entropy)
 *
 * (no d_logprob where no token is given; 0 for a row whose lse is -infinity).
 * `args` gives rows, vocab, dtype, logits and tokens; its outputs are not
 * used.  d_logits may be the logits (same stride). */
typedef struct {
  const float *lse, *entropy;   /* [rows]; entropy only with d_entropy */
  const float *d_logprob, *d_entropy;
  void* d_logits;
  int64_t d_row_stride;         /* at least vocab */
} eg_score_grads;

EG_API eg_status eg_token_logprobs_backward(const eg_score_args* args, const eg_score_grads* grads,
                                            void* stream);

#ifdef __cplusplus
}
#endif
#endif /* EG_DECODER_H */
