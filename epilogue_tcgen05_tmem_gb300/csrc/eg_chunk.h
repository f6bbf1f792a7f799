// eg_chunk.h -- launch description of the chunk attention kernels, shared by
// the host side (eg_chunk.cu) and the kernels (eg_chunk_kernel.cuh).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace eg {

// What a CTA of the main kernel tells the joining kernel: the item (sequence,
// cached head, row group) whose first cut is the start of its range of work
// units, where there is one that CTAs share.
struct __align__(16) ChunkMeta {
  int32_t rows;               // of the item; 0: there is none
  int32_t lead, last, team;   // CTAs lead, lead + team, ... last have parts of it
  int32_t start, row0, head;  // its first packed row, first row in the sequence, cached head
  int32_t pad;
};

struct ChunkParams {
  // the problem
  int32_t q_heads, kv_heads, group, head_dim, page_size, max_chunk;
  int32_t box_rows;     // keys of one TMA box: the power of two that divides page_size, at most 128
  int32_t heads_inner;  // the tensor maps' second dimension is the head, not the token
  int32_t grouped;      // boxes hold both halves of the columns, 8 keys of each in turn: 1 with the heads' halves
                        // in one dimension, 2 with the pages' heads in one; 0: a box for each half
  int32_t q_tiles;      // tiles of 128 rows that one item has room for: 1 or 2
  int32_t box_tokens;   // tokens of one TMA box of queries: with their heads a multiple of 8 rows
  int32_t tile_rows;    // rows of a tile that are used: whole boxes, at most 128
  int32_t item_rows;    // tile_rows * q_tiles
  int32_t item_tokens;  // item_rows / group
  int32_t stages;
  int32_t teams;        // the run's tables can hold more keys and values than the L2 keeps
  // the run
  int32_t batch, tokens;
  int32_t window, sinks;  // window: 0 for none
  void* o;
  int64_t o_token, o_head;
  const int32_t* block_table;
  int64_t table_stride;
  const int32_t* context_lens;
  const int32_t* q_start;
  float scale_log2;     // scale * log2(e)
  float* lse;
  // the values again, for the rows that attend to a value that is not finite
  const void* v;
  int64_t num_pages, page_stride, token_stride, head_stride;
  // the plan's
  float* partial;       // [CTAs][2][128 q_tiles][HD] sums, then
  float* partial_ml;    // [CTAs][2][128 q_tiles][2] their maximum (log2) and weight
  ChunkMeta* meta;      // [CTAs], for the second kernel
  int32_t* arrivals;    // [CTAs] parts left of the item whose first part that CTA has; NULL: a second kernel joins
  int32_t* status;
  uint64_t wait_limit_ns;
  int32_t stall;        // test hook: the producer issues nothing
};

// Shared memory of the main kernel for a head of HD columns.
template <int HD>
struct ChunkSmem {
  static constexpr uint32_t kTileBytes = 128u * HD * 2u;  // 128 rows of queries, keys or values
  static constexpr uint32_t kExtra = 3 * 1024u;              // barriers, schedule, exchange of row statistics
};

}  // namespace eg
