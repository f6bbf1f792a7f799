// eg_tree.h -- launch description of the tree attention kernels.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace eg {

struct TreeParams {
  // the problem
  int32_t q_heads, kv_heads, group, head_dim, page_size, max_batch, max_tree;
  // the run
  int32_t batch, tokens;
  const void* q;
  void* o;
  int64_t q_token, q_head, o_token, o_head;
  const int32_t* block_table;
  int64_t table_stride;
  const int32_t* context_lens;
  const int32_t* q_start;
  const uint32_t* mask;
  int64_t mask_stride;
  float scale;
  float* lse;
  // the cache
  const void *k, *v;
  int64_t num_pages, page_stride, token_stride, head_stride;
};

}  // namespace eg
