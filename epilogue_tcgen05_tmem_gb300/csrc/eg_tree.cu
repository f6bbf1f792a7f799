// eg_tree.cu -- host side of tree attention over a paged cache
// (include/eg_decoder.h has the formulas, eg_tree_kernel.cuh the kernels):
// plans, argument checks, tensor maps and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <new>

#include "../../include/eg_decoder.h"
#include "eg_host.h"
#include "eg_tree_kernel.cuh"

namespace eg {

namespace {

// Rows of one box of queries: the fewest tokens whose heads (`group` each) make
// a multiple of 8 rows, the unit of the shared-memory swizzle.
int row_box(int group) {
  int box = group;
  while (box % 8) box += group;
  return box;
}

bool multiple16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace eg

using namespace eg;

struct eg_tree_plan {
  eg_tree_problem prob{};
  int device = -1;
  int hd = 0, tile_rows = 0, q_tiles = 0, stages = 0, grid = 0;
  uint32_t smem = 0;
  size_t ws_bytes = 0;
  uint8_t* ws = nullptr;  // partial sums, their statistics, the CTAs' ranges, the status word
  size_t ml_at = 0, meta_at = 0, arrivals_at = 0, status_at = 0;
  bool joins_itself = false;  // the CTA that leaves an item's last part joins it; else a second kernel
  uint64_t wait_limit_ns = 0;
  int stall = 0;
};

namespace {

eg_status check_problem(const eg_tree_problem* p) {
  if (!p) return host_fail(EG_ERR_INVALID_ARG, "problem is NULL");
  if (p->dtype != EG_EL_BF16 && p->dtype != EG_EL_F16)
    return host_fail(p->dtype == EG_EL_F32 ? EG_ERR_UNSUPPORTED : EG_ERR_INVALID_ARG, "dtype must be bf16 or fp16 (got %d)", p->dtype);
  if (p->q_heads < 1 || p->kv_heads < 1 || p->q_heads % p->kv_heads)
    return host_fail(EG_ERR_INVALID_ARG, "q_heads=%d must be a positive multiple of kv_heads=%d", p->q_heads, p->kv_heads);
  if (p->q_heads > 1024) return host_fail(EG_ERR_UNSUPPORTED, "at most 1024 query heads (got %d)", p->q_heads);
  if (row_box(p->q_heads / p->kv_heads) > 128)
    return host_fail(EG_ERR_UNSUPPORTED, "%d query heads for each cached head do not fit a tile of 128 rows in groups of 8 rows", p->q_heads / p->kv_heads);
  if (p->head_dim < 8 || p->head_dim > 128 || p->head_dim % 8)
    return host_fail(EG_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 in 8..128 (got %d)", p->head_dim);
  if (p->page_size < 8 || p->page_size % 8 || p->page_size > 65536)
    return host_fail(EG_ERR_UNSUPPORTED, "page_size must be a multiple of 8 in 8..65536 (got %d)", p->page_size);
  if (p->max_batch < 1 || p->max_batch > 65536)
    return host_fail(EG_ERR_UNSUPPORTED, "max_batch must be in 1..65536 (got %d)", p->max_batch);
  if (p->max_tree < 1 || p->max_tree > 256)
    return host_fail(EG_ERR_UNSUPPORTED, "max_tree must be in 1..256 (got %d)", p->max_tree);
  return EG_OK;
}

eg_status check_run(const eg_tree_plan* plan, const eg_tree_args* a, const eg_kv_cache* c) {
  const eg_tree_problem& p = plan->prob;
  if (!a) return host_fail(EG_ERR_INVALID_ARG, "args is NULL");
  if (!c) return host_fail(EG_ERR_INVALID_ARG, "cache is NULL");
  if (a->batch < 0 || a->tokens < 0) return host_fail(EG_ERR_INVALID_ARG, "negative size (batch=%d tokens=%d)", a->batch, a->tokens);
  if (a->batch > p.max_batch) return host_fail(EG_ERR_INVALID_ARG, "batch=%d exceeds the plan's max_batch=%d", a->batch, p.max_batch);
  if (a->batch == 0 || a->tokens == 0) return EG_OK;
  if (!a->q || !a->o || !multiple16(a->q) || !multiple16(a->o))
    return host_fail(EG_ERR_INVALID_ARG, "q or o is NULL or not 16-byte aligned");
  // the stride of a dimension of one is not used
  for (int64_t s : {a->tokens > 1 ? a->q_token : 8, p.q_heads > 1 ? a->q_head : 8, a->tokens > 1 ? a->o_token : 8, p.q_heads > 1 ? a->o_head : 8})
    if (s < 8 || s % 8) return host_fail(EG_ERR_INVALID_ARG, "the strides of q and o must be positive multiples of 8 elements");
  if (!a->block_table || !a->context_lens || !a->q_start) return host_fail(EG_ERR_INVALID_ARG, "block_table, context_lens or q_start is NULL");
  for (const void* x : {static_cast<const void*>(a->block_table), static_cast<const void*>(a->context_lens),
                        static_cast<const void*>(a->q_start), static_cast<const void*>(a->mask), static_cast<const void*>(a->lse)})
    if (reinterpret_cast<uintptr_t>(x) % 4) return host_fail(EG_ERR_INVALID_ARG, "a side tensor is not aligned to its elements");
  if (a->table_stride < 1 || a->table_stride * p.page_size > INT32_MAX - 1024)
    return host_fail(EG_ERR_UNSUPPORTED, "a sequence's table must cover between 1 page and 2^31 tokens (table_stride=%lld)", (long long)a->table_stride);
  if (a->mask && a->mask_stride < (p.max_tree + 31) / 32)
    return host_fail(EG_ERR_INVALID_ARG, "mask_stride=%lld is less than the words of max_tree=%d", (long long)a->mask_stride, p.max_tree);
  if (!(a->scale > 0.0f && a->scale < 1e30f)) return host_fail(EG_ERR_INVALID_ARG, "scale must be positive and finite");
  if (!c->k || !c->v || !multiple16(c->k) || !multiple16(c->v))
    return host_fail(EG_ERR_INVALID_ARG, "the cache is NULL or not 16-byte aligned");
  if (c->num_pages < 1 || c->num_pages > INT32_MAX) return host_fail(EG_ERR_INVALID_ARG, "num_pages=%lld", (long long)c->num_pages);
  // the stride of a dimension of one is not used
  const int64_t strides[3] = {c->num_pages > 1 ? c->page_stride : 8, c->token_stride, p.kv_heads > 1 ? c->head_stride : 8};
  for (int64_t s : strides)
    if (s < 8 || s % 8) return host_fail(EG_ERR_INVALID_ARG, "the cache's strides must be positive multiples of 8 elements");
  return EG_OK;
}

// The tensor map of keys or values: columns, then token and head in the order
// of their strides, then pages; boxes of 64 columns by `box_rows` tokens.
eg_status encode_cache(const eg_tree_problem& p, const eg_kv_cache& c, const void* base, int box_rows, bool heads_inner, CUtensorMap* map) {
  EncodeTiledFn fn = host_encode_tiled();
  if (!fn) return host_fail(EG_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t heads = static_cast<cuuint64_t>(p.kv_heads), places = static_cast<cuuint64_t>(p.page_size);
  const cuuint64_t head_bytes = p.kv_heads > 1 ? static_cast<cuuint64_t>(c.head_stride) * 2 : 16;
  const cuuint64_t place_bytes = static_cast<cuuint64_t>(c.token_stride) * 2;
  const cuuint64_t page_bytes = c.num_pages > 1 ? static_cast<cuuint64_t>(c.page_stride) * 2 : 16;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(p.head_dim), heads_inner ? heads : places, heads_inner ? places : heads,
                              static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[3] = {heads_inner ? head_bytes : place_bytes, heads_inner ? place_bytes : head_bytes, page_bytes};
  const cuuint32_t rows = static_cast<cuuint32_t>(box_rows);
  const cuuint32_t box[4] = {64, heads_inner ? 1u : rows, heads_inner ? rows : 1u, 1};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, p.dtype == EG_EL_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                        const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return host_fail(EG_ERR_INVALID_ARG, "cuTensorMapEncodeTiled failed (%d) for the cache", static_cast<int>(r));
  return EG_OK;
}

// The tensor map of queries: columns, heads, packed tokens; boxes of 64
// columns by the heads of one cached head by `box_tokens` tokens.
eg_status encode_queries(const eg_tree_problem& p, const eg_tree_args& a, int box_tokens, CUtensorMap* map) {
  EncodeTiledFn fn = host_encode_tiled();
  if (!fn) return host_fail(EG_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.head_dim), static_cast<cuuint64_t>(p.q_heads), static_cast<cuuint64_t>(a.tokens)};
  const cuuint64_t strides[2] = {p.q_heads > 1 ? static_cast<cuuint64_t>(a.q_head) * 2 : 16, a.tokens > 1 ? static_cast<cuuint64_t>(a.q_token) * 2 : 16};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.q_heads / p.kv_heads), static_cast<cuuint32_t>(box_tokens)};
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUresult r = fn(map, p.dtype == EG_EL_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                        const_cast<void*>(a.q), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return host_fail(EG_ERR_INVALID_ARG, "cuTensorMapEncodeTiled failed (%d) for the queries", static_cast<int>(r));
  return EG_OK;
}

using TreeKernel = void (*)(TreeParams, CUtensorMap, CUtensorMap, CUtensorMap);
using JoinKernel = void (*)(TreeParams);

TreeKernel main_kernel(const eg_tree_plan& pl) {
  if (pl.prob.dtype == EG_EL_BF16) return pl.hd == 64 ? tree_kernel<__nv_bfloat16, 64> : tree_kernel<__nv_bfloat16, 128>;
  return pl.hd == 64 ? tree_kernel<__half, 64> : tree_kernel<__half, 128>;
}
JoinKernel join_kernel(const eg_tree_plan& pl) {
  if (pl.prob.dtype == EG_EL_BF16) return pl.hd == 64 ? tree_join_kernel<__nv_bfloat16, 64> : tree_join_kernel<__nv_bfloat16, 128>;
  return pl.hd == 64 ? tree_join_kernel<__half, 64> : tree_join_kernel<__half, 128>;
}

int rows_of(const eg_tree_plan& pl) {
  return std::min(pl.tile_rows * pl.q_tiles, pl.prob.max_tree * (pl.prob.q_heads / pl.prob.kv_heads));
}

// A plan's memory and its kernels' settings are on the device that it was made on.
eg_status check_current(const eg_tree_plan* plan) {
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return host_cuda_fail(e, "cudaGetDevice");
  if (dev != plan->device)
    return host_fail(EG_ERR_INVALID_ARG, "the plan was made on device %d, and device %d is the current one", plan->device, dev);
  return EG_OK;
}

// Clear the plan's words from `at` on, and wait for it: the clear is queued on
// the legacy stream, which a run on a non-blocking stream does not wait for.
eg_status clear_words(eg_tree_plan* pl, size_t at, const char* what) {
  cudaError_t e = cudaMemset(pl->ws + at, 0, pl->ws_bytes - at);
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
  return e == cudaSuccess ? EG_OK : host_cuda_fail(e, what);
}

eg_status set_up(eg_tree_plan* pl) {
  int sms = 0;
  eg_status s = host_check_device(&pl->device, &sms);
  if (s != EG_OK) return s;
  cudaError_t e = cudaSuccess;
  const eg_tree_problem& p = pl->prob;
  pl->hd = p.head_dim <= 64 ? 64 : 128;
  const int group = p.q_heads / p.kv_heads;
  pl->tile_rows = 128 / row_box(group) * row_box(group);
  // two tiles of rows share each key tile where a tree can have more than one;
  // with one the second tile's shared memory is a stage of the ring (16
  // sequences of 32 to 64 tokens of 64 heads over 8 cached: two 163 us, one at a
  // time 197 us)
  pl->q_tiles = p.max_tree * group > pl->tile_rows ? 2 : 1;
  const uint32_t tile = pl->hd == 64 ? TreeSmem<64>::kTileBytes : TreeSmem<128>::kTileBytes;
  const uint32_t extra = TreeSmem<64>::kExtra;
  pl->stages = std::min<int>(12, static_cast<int>((232448u - extra) / tile) - pl->q_tiles);
  pl->smem = (pl->q_tiles + pl->stages) * tile + extra;
  pl->grid = sms;
  const size_t rows = static_cast<size_t>(pl->grid) * 2 * 128 * pl->q_tiles;
  pl->ml_at = rows * pl->hd * 4;
  pl->meta_at = pl->ml_at + rows * 8;
  pl->arrivals_at = pl->meta_at + pl->grid * sizeof(TreeMeta);
  pl->status_at = pl->arrivals_at + (pl->grid * 4 + 15) / 16 * 16;
  pl->ws_bytes = pl->status_at + 16;
  if ((e = cudaMalloc(&pl->ws, pl->ws_bytes)) != cudaSuccess) return host_cuda_fail(e, "allocating the plan's workspace");
  if ((s = clear_words(pl, pl->meta_at, "clearing the plan's workspace")) != EG_OK) return s;
  if ((e = cudaFuncSetAttribute(reinterpret_cast<const void*>(main_kernel(*pl)), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(pl->smem))) != cudaSuccess)
    return host_cuda_fail(e, "cudaFuncSetAttribute");
  pl->wait_limit_ns = host_wait_limit_ns();
  // One CTA reads at most the parts of the most CTAs that share an item (those
  // of a single sequence: the grid over the cached heads).  Up to 256 KB are
  // joined by the last of them, which spares a second kernel (32 query heads
  // over 8 cached ones, one token after 517 and after 8000, cold L2: 19.1 and
  // 27.3 us, with the second kernel 21.1 and 32.4 us); above, the second kernel
  // joins with the whole GPU (32 tokens after 8000: 33.4 us, 76 us by the last;
  // 16 sequences of 32 to 64 tokens of 64 heads: 163 and 189 us).
  const int64_t parts = pl->grid / p.kv_heads + 2;
  pl->joins_itself = parts * rows_of(*pl) * pl->hd * 4 <= 256 * 1024;
  return EG_OK;
}

}  // namespace

extern "C" {

eg_status eg_tree_plan_create(const eg_tree_problem* problem, eg_tree_plan** out) {
  if (!out) return host_fail(EG_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  eg_status s = check_problem(problem);
  if (s != EG_OK) return s;
  int dev = 0;
  if ((s = host_check_device(&dev)) != EG_OK) return s;
  eg_tree_plan* pl = new (std::nothrow) eg_tree_plan;
  if (!pl) return host_fail(EG_ERR_NO_MEMORY, "no host memory for a plan");
  pl->prob = *problem;
  pl->device = dev;
  if ((s = set_up(pl)) != EG_OK) {
    if (pl->ws) cudaFree(pl->ws);
    delete pl;
    return s;
  }
  *out = pl;
  return EG_OK;
}

eg_status eg_tree_plan_workspace_bytes(const eg_tree_plan* plan, size_t* out) {
  if (!plan || !out) return host_fail(EG_ERR_INVALID_ARG, "plan or out is NULL");
  *out = plan->ws_bytes;
  return EG_OK;
}

eg_status eg_tree_plan_run(eg_tree_plan* plan, const eg_tree_args* args, const eg_kv_cache* cache, void* stream) {
  if (!plan) return host_fail(EG_ERR_INVALID_ARG, "plan is NULL");
  eg_status s = check_run(plan, args, cache);
  if (s == EG_OK) s = check_current(plan);
  if (s != EG_OK) return s;
  const eg_tree_problem& b = plan->prob;
  const eg_tree_args& a = *args;
  if (a.batch == 0 || a.tokens == 0) return EG_OK;
  TreeParams p{};
  p.q_heads = b.q_heads, p.kv_heads = b.kv_heads, p.group = b.q_heads / b.kv_heads, p.head_dim = b.head_dim;
  p.page_size = b.page_size, p.max_tree = b.max_tree;
  p.box_rows = std::min(128, b.page_size & -b.page_size);
  p.heads_inner = b.kv_heads > 1 && cache->head_stride < cache->token_stride ? 1 : 0;
  p.q_tiles = plan->q_tiles, p.stages = plan->stages;
  p.box_tokens = row_box(p.group) / p.group, p.tile_rows = plan->tile_rows, p.item_rows = plan->tile_rows * plan->q_tiles;
  p.batch = a.batch, p.tokens = a.tokens;
  p.o = a.o, p.o_token = a.o_token, p.o_head = a.o_head;
  p.block_table = a.block_table, p.table_stride = a.table_stride, p.context_lens = a.context_lens, p.q_start = a.q_start;
  p.mask = a.mask, p.mask_stride = a.mask_stride, p.scale_log2 = a.scale * 1.4426950408889634f, p.lse = a.lse;
  p.v = cache->v, p.num_pages = cache->num_pages;
  p.page_stride = cache->page_stride, p.token_stride = cache->token_stride, p.head_stride = cache->head_stride;
  p.partial = reinterpret_cast<float*>(plan->ws);
  p.partial_ml = reinterpret_cast<float*>(plan->ws + plan->ml_at);
  p.meta = reinterpret_cast<TreeMeta*>(plan->ws + plan->meta_at);
  p.arrivals = plan->joins_itself ? reinterpret_cast<int32_t*>(plan->ws + plan->arrivals_at) : nullptr;
  p.status = reinterpret_cast<int32_t*>(plan->ws + plan->status_at);
  p.wait_limit_ns = plan->wait_limit_ns, p.stall = plan->stall;
  CUtensorMap map_q, map_k, map_v;
  if ((s = encode_queries(b, a, p.box_tokens, &map_q)) != EG_OK) return s;
  if ((s = encode_cache(b, *cache, cache->k, p.box_rows, p.heads_inner != 0, &map_k)) != EG_OK) return s;
  if ((s = encode_cache(b, *cache, cache->v, p.box_rows, p.heads_inner != 0, &map_v)) != EG_OK) return s;

  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(plan->grid));
  cfg.blockDim = dim3(kTreeThreads);
  cfg.dynamicSmemBytes = plan->smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaLaunchKernelEx(&cfg, main_kernel(*plan), p, map_q, map_k, map_v);
  if (e != cudaSuccess) return host_cuda_fail(e, "launching tree attention");
  if (plan->joins_itself) return EG_OK;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(plan->grid - 1), static_cast<unsigned>((rows_of(*plan) + 7) / 8));
  cfg.blockDim = dim3(static_cast<unsigned>(plan->hd * 2));
  cfg.dynamicSmemBytes = 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, join_kernel(*plan), p);
  return e == cudaSuccess ? EG_OK : host_cuda_fail(e, "launching the join of tree attention");
}

eg_status eg_tree_plan_device_status(eg_tree_plan* plan) {
  if (!plan) return host_fail(EG_ERR_INVALID_ARG, "plan is NULL");
  eg_status s = check_current(plan);
  if (s != EG_OK) return s;
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return host_cuda_fail(e, "synchronising the plan's device");
  int32_t status = 0;
  if ((e = cudaMemcpy(&status, plan->ws + plan->status_at, 4, cudaMemcpyDeviceToHost)) != cudaSuccess)
    return host_cuda_fail(e, "reading the plan's status");
  if (status == 0) return EG_OK;
  // a CTA that gave up leaves items half counted
  if ((s = clear_words(plan, plan->arrivals_at, "clearing the plan's status")) != EG_OK) return s;
  return host_fail(EG_ERR_DEVICE_TIMEOUT, "a wait of the tree attention kernel ran past its limit");
}

eg_status eg_tree_plan_set_test_stall(eg_tree_plan* plan, uint64_t wait_limit_ns, int32_t stall_producer) {
  if (!plan) return host_fail(EG_ERR_INVALID_ARG, "plan is NULL");
  if (stall_producer != 0 && stall_producer != 1) return host_fail(EG_ERR_INVALID_ARG, "stall_producer must be 0 or 1");
  plan->wait_limit_ns = wait_limit_ns ? wait_limit_ns : host_wait_limit_ns();
  plan->stall = stall_producer;
  return EG_OK;
}

eg_status eg_tree_plan_destroy(eg_tree_plan* plan) {
  if (!plan) return EG_OK;
  int dev = plan->device;
  cudaGetDevice(&dev);
  if (dev != plan->device) cudaSetDevice(plan->device);
  cudaDeviceSynchronize();
  cudaFree(plan->ws);
  if (dev != plan->device) cudaSetDevice(dev);
  delete plan;
  return EG_OK;
}

}  // extern "C"
