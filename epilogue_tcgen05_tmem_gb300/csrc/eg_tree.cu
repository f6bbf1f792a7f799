// eg_tree.cu -- attention of drafted token trees over a paged cache
// (include/eg_decoder.h has the formulas), the plain form: one CTA for each
// token and query head, its warps take every fourth key and join at the end.
#include <cuda_runtime.h>
#include <math_constants.h>

#include <new>

#include "../../include/eg_decoder.h"
#include "eg_el.cuh"
#include "eg_host.h"
#include "eg_ptx.cuh"
#include "eg_tree.h"

namespace eg {

namespace {

constexpr int kWarps = 4;

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) tree_simple_kernel(const TreeParams p) {
  const int row = blockIdx.x, head = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the last sequence that starts at or before the row
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (p.q_start[mid] <= row) lo = mid;
    else hi = mid;
  }
  const int start = p.q_start[lo];
  const int t = row - start;
  const int n = min(min(p.q_start[lo + 1], p.tokens) - start, p.max_tree);
  if (t < 0 || t >= n) return;
  const int64_t room = p.table_stride * p.page_size;
  const int64_t ctx = min(static_cast<int64_t>(max(p.context_lens[lo], 0)), room);
  const int64_t keys = min(ctx + n, room);
  const int32_t* table = p.block_table + lo * p.table_stride;
  const int64_t at_head = static_cast<int64_t>(head / p.group) * p.head_stride;
  float q[4], o[4] = {0, 0, 0, 0}, m = -CUDART_INF_F, l = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane * 4 + i;
    q[i] = e < p.head_dim ? El<T>::to_float(static_cast<const T*>(p.q)[row * p.q_token + head * p.q_head + e]) : 0.0f;
  }
  for (int64_t j = warp; j < keys; j += kWarps) {
    if (j >= ctx) {
      const int u = static_cast<int>(j - ctx);
      const bool sees = p.mask ? (p.mask[row * p.mask_stride + (u >> 5)] >> (u & 31)) & 1u : u <= t;
      if (!sees) continue;
    }
    const int page = table[j / p.page_size];
    const bool ok = page >= 0 && page < p.num_pages;
    const int64_t at = (ok ? page : 0) * p.page_stride + (j % p.page_size) * p.token_stride + at_head;
    float k[4], v[4], s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = lane * 4 + i;
      const bool in = ok && e < p.head_dim;
      k[i] = in ? El<T>::to_float(static_cast<const T*>(p.k)[at + e]) : 0.0f;
      v[i] = in ? El<T>::to_float(static_cast<const T*>(p.v)[at + e]) : 0.0f;
      s += q[i] * k[i];
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale;
    const float next = fmaxf(m, s);
    const float ref = next == -CUDART_INF_F ? 0.0f : next;
    const float f = expf(m - ref), e = expf(s - ref);
    l = l * f + e;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = o[i] * f + e * v[i];
    m = next;
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][128];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int i = 0; i < 4; ++i) so[warp][lane * 4 + i] = o[i];
  __syncthreads();
  float top = -CUDART_INF_F;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  const float ref = top == -CUDART_INF_F ? 0.0f : top;
  float total = 0.0f, y = 0.0f;
  for (int w = 0; w < kWarps; ++w) {
    const float f = expf(sm[w] - ref);
    total += sl[w] * f;
    y += so[w][threadIdx.x] * f;
  }
  if (threadIdx.x < p.head_dim)
    static_cast<T*>(p.o)[row * p.o_token + head * p.o_head + threadIdx.x] = El<T>::from_float(total == 0.0f ? 0.0f : y / total);
  if (p.lse && threadIdx.x == 0) p.lse[static_cast<int64_t>(row) * p.q_heads + head] = total == 0.0f ? -CUDART_INF_F : top + logf(total);
}

bool multiple16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace eg

using namespace eg;

struct eg_tree_plan {
  eg_tree_problem prob{};
  int device = -1;
  size_t ws_bytes = 0;
};

namespace {

eg_status check_problem(const eg_tree_problem* p) {
  if (!p) return host_fail(EG_ERR_INVALID_ARG, "problem is NULL");
  if (p->dtype != EG_EL_BF16 && p->dtype != EG_EL_F16)
    return host_fail(p->dtype == EG_EL_F32 ? EG_ERR_UNSUPPORTED : EG_ERR_INVALID_ARG, "dtype must be bf16 or fp16 (got %d)", p->dtype);
  if (p->q_heads < 1 || p->kv_heads < 1 || p->q_heads % p->kv_heads)
    return host_fail(EG_ERR_INVALID_ARG, "q_heads=%d must be a positive multiple of kv_heads=%d", p->q_heads, p->kv_heads);
  if (p->q_heads > 1024) return host_fail(EG_ERR_UNSUPPORTED, "at most 1024 query heads (got %d)", p->q_heads);
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
  for (int64_t s : {a->q_token, a->q_head, a->o_token, a->o_head})
    if (s < 0 || s % 8) return host_fail(EG_ERR_INVALID_ARG, "the strides of q and o must be multiples of 8 elements");
  if (!a->block_table || !a->context_lens || !a->q_start) return host_fail(EG_ERR_INVALID_ARG, "block_table, context_lens or q_start is NULL");
  for (const void* x : {static_cast<const void*>(a->block_table), static_cast<const void*>(a->context_lens),
                        static_cast<const void*>(a->q_start), static_cast<const void*>(a->mask), static_cast<const void*>(a->lse)})
    if (reinterpret_cast<uintptr_t>(x) % 4) return host_fail(EG_ERR_INVALID_ARG, "a side tensor is not aligned to its elements");
  if (a->table_stride < 1 || a->table_stride * p.page_size > INT32_MAX - 1024)
    return host_fail(EG_ERR_UNSUPPORTED, "a sequence's table must cover between 1 page and 2^31 tokens (table_stride=%lld)", (long long)a->table_stride);
  if (a->mask && a->mask_stride < (p.max_tree + 31) / 32)
    return host_fail(EG_ERR_INVALID_ARG, "mask_stride=%lld is less than the words of max_tree=%d", (long long)a->mask_stride, p.max_tree);
  if (!(a->scale == a->scale)) return host_fail(EG_ERR_INVALID_ARG, "scale is not a number");
  if (!c->k || !c->v || !multiple16(c->k) || !multiple16(c->v))
    return host_fail(EG_ERR_INVALID_ARG, "the cache is NULL or not 16-byte aligned");
  if (c->num_pages < 1 || c->num_pages > INT32_MAX) return host_fail(EG_ERR_INVALID_ARG, "num_pages=%lld", (long long)c->num_pages);
  for (int64_t s : {c->page_stride, c->token_stride, c->head_stride})
    if (s < 0 || s % 8) return host_fail(EG_ERR_INVALID_ARG, "the cache's strides must be multiples of 8 elements");
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
  if (s != EG_OK) return s;
  const eg_tree_problem& b = plan->prob;
  const eg_tree_args& a = *args;
  if (a.batch == 0 || a.tokens == 0) return EG_OK;
  TreeParams p{};
  p.q_heads = b.q_heads, p.kv_heads = b.kv_heads, p.group = b.q_heads / b.kv_heads, p.head_dim = b.head_dim;
  p.page_size = b.page_size, p.max_batch = b.max_batch, p.max_tree = b.max_tree;
  p.batch = a.batch, p.tokens = a.tokens;
  p.q = a.q, p.o = a.o, p.q_token = a.q_token, p.q_head = a.q_head, p.o_token = a.o_token, p.o_head = a.o_head;
  p.block_table = a.block_table, p.table_stride = a.table_stride, p.context_lens = a.context_lens, p.q_start = a.q_start;
  p.mask = a.mask, p.mask_stride = a.mask_stride, p.scale = a.scale, p.lse = a.lse;
  p.k = cache->k, p.v = cache->v, p.num_pages = cache->num_pages;
  p.page_stride = cache->page_stride, p.token_stride = cache->token_stride, p.head_stride = cache->head_stride;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(a.tokens), static_cast<unsigned>(b.q_heads));
  if (b.dtype == EG_EL_BF16) tree_simple_kernel<__nv_bfloat16><<<grid, kWarps * 32, 0, st>>>(p);
  else tree_simple_kernel<__half><<<grid, kWarps * 32, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? EG_OK : host_cuda_fail(e, "launching tree attention");
}

eg_status eg_tree_plan_device_status(eg_tree_plan* plan) {
  if (!plan) return host_fail(EG_ERR_INVALID_ARG, "plan is NULL");
  const cudaError_t e = cudaDeviceSynchronize();
  return e == cudaSuccess ? EG_OK : host_cuda_fail(e, "synchronising the plan's device");
}

eg_status eg_tree_plan_destroy(eg_tree_plan* plan) {
  if (!plan) return EG_OK;
  delete plan;
  return EG_OK;
}

}  // extern "C"
