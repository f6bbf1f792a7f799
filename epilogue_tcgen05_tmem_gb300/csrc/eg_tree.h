// eg_tree.h -- launch description of the tree attention kernels, shared by
// the host side (eg_tree.cu) and the kernels (eg_tree_kernel.cuh).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace eg {

// What a CTA of the main kernel tells the joining kernel: where its range of
// work units starts and which item (sequence, cached head, row group) that
// unit belongs to.
struct TreeMeta {
  int64_t from;         // the CTA's first unit
  int64_t begin;        // the first unit of the item that holds it,
  int64_t lead, last;   // and the first units of that item's first and last tile
  int64_t total;        // units of the run
  int32_t ctas;         // CTAs that have units
  int32_t start, rows, row0, head;  // the item's first packed row, rows, first row in the sequence, cached head
  int32_t pad;
};

struct TreeParams {
  // the problem
  int32_t q_heads, kv_heads, group, head_dim, page_size, max_tree;
  int32_t box_rows;     // keys of one TMA box: the power of two that divides page_size, at most 128
  int32_t heads_inner;  // the tensor maps' second dimension is the head, not the token
  int32_t q_tiles;      // tiles of 128 rows that one item has room for: 1 or 2
  int32_t box_tokens;   // tokens of one TMA box of queries: with their heads a multiple of 8 rows
  int32_t tile_rows;    // rows of a tile that are used: whole boxes, at most 128
  int32_t item_rows;    // tile_rows * q_tiles
  int32_t stages;
  // the run
  int32_t batch, tokens;
  void* o;
  int64_t o_token, o_head;
  const int32_t* block_table;
  int64_t table_stride;
  const int32_t* context_lens;
  const int32_t* q_start;
  const uint32_t* mask;
  int64_t mask_stride;
  float scale_log2;     // scale * log2(e)
  float* lse;
  // the values again, for the rows that attend to a value that is not finite
  const void* v;
  int64_t num_pages, page_stride, token_stride, head_stride;
  // the plan's
  float* partial;       // [CTAs][2][128 q_tiles][HD] sums, then
  float* partial_ml;    // [CTAs][2][128 q_tiles][2] their maximum (log2) and weight
  TreeMeta* meta;       // [CTAs]
  int32_t* arrivals;    // [CTAs] parts left of the item whose first part that CTA has; NULL: a second kernel joins
  int32_t* status;
  uint64_t wait_limit_ns;
  int32_t stall;        // test hook: the producer issues nothing
};

// Shared memory of the main kernel for a head of HD columns.
template <int HD>
struct TreeSmem {
  static constexpr uint32_t kTileBytes = 128u * HD * 2u;  // 128 rows of queries, keys or values
  static constexpr uint32_t kExtra = 3072u;               // barriers, schedule, exchange of row statistics
};

}  // namespace eg
