// eg_score.cu -- log probabilities of given tokens with entropy and the top
// alternatives, and their gradient (include/eg_decoder.h has the formulas).
//
// Both are bound by memory: the logits are read once (and their gradient
// written once).  Forward: a CTA, or a cluster of CTAs where there are few
// rows, takes one row.  A thread keeps the maximum m of what it saw and, to
// that reference, s = sum 2^y and t = sum 2^y y with y = (x - m) log2 e; then
// lse = (m log2 e + log2 s) ln 2 and entropy = (log2 s - t / s) ln 2.  The top
// alternatives come from the same pass: a value is looked at again only where
// it reaches the smallest of the best ones so far, which after the first few
// thousand values few do.
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/eg_decoder.h"
#include <math_constants.h>

#include "eg_el.cuh"
#include "eg_host.h"
#include "eg_ptx.cuh"

namespace eg {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;        // 16-byte loads of a thread in flight
constexpr int kMostTop = 32;
constexpr int kKept = 1024;       // room for candidates between two selections
constexpr int kSelectAt = 256;    // select once this many candidates wait
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct ScoreParams {
  int64_t rows, vocab, row_stride;
  const void* logits;
  const int64_t* tokens;
  float *logprob, *lse, *entropy, *top_logprobs;
  int64_t* top_ids;
  int32_t top;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Values below this count as this: 2^y is 0 for them unless nothing in the
// row is far above it, and then the row is done again (see `plain_row`).
// Its size keeps the rounding of m log2 e, which every y of a thread shares,
// far below one.
constexpr float kLowest = -65504.0f;

// The reference that a maximum stands for: rounded once, the same everywhere.
__device__ __forceinline__ float reference(float m) { return __fmul_rn(m, kLog2e); }

// A 32-bit word of -infinities.
template <typename T>
constexpr uint32_t kNothing = 0xFF800000u;
template <>
constexpr uint32_t kNothing<__nv_bfloat16> = 0xFF80FF80u;
template <>
constexpr uint32_t kNothing<__half> = 0xFC00FC00u;

// A candidate: larger for a larger value, then for a lower id; 0 for none.
__device__ __forceinline__ uint64_t candidate(float x, uint32_t id) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 counts as 0
  const uint32_t o = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return x == x ? (static_cast<uint64_t>(o) << 32) | (0xFFFFFFFFu - id) : 0ull;
}
__device__ __forceinline__ float candidate_value(uint64_t c) {
  const uint32_t o = static_cast<uint32_t>(c >> 32);
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint32_t candidate_id(uint64_t c) { return 0xFFFFFFFFu - static_cast<uint32_t>(c); }

struct Sums {
  float m, s, t;
};

// Both sums to the reference of the larger maximum.
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
  Sums r;
  r.m = max_nan(a.m, b.m);
  const float ref = reference(r.m);
  const float da = reference(a.m) - ref, db = reference(b.m) - ref;
  const float fa = ex2(da), fb = ex2(db);
  r.s = a.s * fa + b.s * fb;
  r.t = (a.t + a.s * da) * fa + (b.t + b.s * db) * fb;
  return r;
}

struct TopShared {
  uint64_t kept[kMostTop];   // the best so far, in order
  uint64_t waiting[kKept];   // candidates not yet selected from
  uint64_t least;            // a value has to reach this to be a candidate
  int count;                 // candidates that asked for a place
  float groups[kMostTop];
};

struct RowShared {
  Sums warps[kWarps];
  Sums cta;
  TopShared top;
};

// The best `top` of kept and waiting into kept, in order; the next candidate
// has to be better than the last of them.  All threads.
__device__ __forceinline__ void select_top(TopShared& sh, int top) {
  __syncthreads();
  const int waiting = min(sh.count, kKept);
  const int total = waiting + top;
  uint64_t mine[(kKept + kMostTop + kThreads - 1) / kThreads];
  int rank[(kKept + kMostTop + kThreads - 1) / kThreads];
#pragma unroll
  for (int i = 0; i < (kKept + kMostTop + kThreads - 1) / kThreads; ++i) {
    const int at = threadIdx.x + i * kThreads;
    rank[i] = kMostTop;
    if (at >= total) continue;
    mine[i] = at < top ? sh.kept[at] : sh.waiting[at - top];
    if (mine[i] == 0) continue;
    int better = 0;
    for (int j = 0; j < top; ++j) better += sh.kept[j] > mine[i];
    for (int j = 0; j < waiting; ++j) better += sh.waiting[j] > mine[i];
    rank[i] = better;
  }
  __syncthreads();
  if (threadIdx.x < top) sh.kept[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < (kKept + kMostTop + kThreads - 1) / kThreads; ++i)
    if (rank[i] < top) sh.kept[rank[i]] = mine[i];
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint64_t last = sh.kept[top - 1];
    if (last) sh.least = last + 1;
    sh.count = 0;
  }
  __syncthreads();
}

// The outputs of one row by one thread group of the CTA that holds the sums.
__device__ __forceinline__ void write_row(const ScoreParams& p, int64_t row, float lse, float entropy, float token_logit,
                                          bool given, bool nan_row, const TopShared* top) {
  const float nan = __int_as_float(0x7FC00000);
  const bool nothing = lse == -CUDART_INF_F;
  if (threadIdx.x == 0) {
    if (p.lse) p.lse[row] = lse;
    if (p.entropy) p.entropy[row] = entropy;
    if (p.logprob) p.logprob[row] = !given ? 0.0f : nothing ? -CUDART_INF_F : lse == CUDART_INF_F ? nan : token_logit - lse;
  }
  if (top && threadIdx.x < p.top) {
    const uint64_t c = top->kept[threadIdx.x];
    const int64_t at = row * p.top + threadIdx.x;
    if (p.top_ids) p.top_ids[at] = nan_row ? -1 : static_cast<int64_t>(candidate_id(c));
    if (p.top_logprobs)
      p.top_logprobs[at] = nan_row || lse == CUDART_INF_F ? nan : nothing ? -CUDART_INF_F : candidate_value(c) - lse;
  }
}

__device__ __forceinline__ Sums block_join(Sums v, RowShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sums b;
    b.m = __shfl_xor_sync(0xffffffffu, v.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, v.s, o);
    b.t = __shfl_xor_sync(0xffffffffu, v.t, o);
    v = join(v, b);
  }
  __syncthreads();
  if (lane == 0) sh.warps[warp] = v;
  __syncthreads();
  if (warp == 0) {
    v = sh.warps[lane < kWarps ? lane : 0];
    if (lane >= kWarps) v.s = 0.0f, v.t = 0.0f;
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) {
      Sums b;
      b.m = __shfl_xor_sync(0xffffffffu, v.m, o);
      b.s = __shfl_xor_sync(0xffffffffu, v.s, o);
      b.t = __shfl_xor_sync(0xffffffffu, v.t, o);
      v = join(v, b);
    }
    if (lane == 0) sh.cta = v;
  }
  __syncthreads();
  return sh.cta;
}

// A row whose maximum is so low, so high or so infinite that the pass above
// does not hold: its statistics from the definition, by one CTA.
template <typename T>
__device__ __noinline__ void plain_row(const T* x, int64_t vocab, float* lse, float* entropy) {
  __shared__ float red[kThreads];
  float m = -CUDART_INF_F;
  for (int64_t i = threadIdx.x; i < vocab; i += kThreads) m = max_nan(m, El<T>::to_float(x[i]));
  red[threadIdx.x] = m;
  __syncthreads();
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    if (threadIdx.x < o) red[threadIdx.x] = max_nan(red[threadIdx.x], red[threadIdx.x + o]);
    __syncthreads();
  }
  m = red[0];
  __syncthreads();
  float s = 0.0f, t = 0.0f;
  if (fabsf(m) < CUDART_INF_F)
    for (int64_t i = threadIdx.x; i < vocab; i += kThreads) {
      const float d = El<T>::to_float(x[i]) - m, e = expf(d);
      if (e > 0.0f) s += e, t += e * d;
    }
  for (int k = 0; k < 2; ++k) {
    red[threadIdx.x] = k ? t : s;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
      if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
      __syncthreads();
    }
    (k ? t : s) = red[0];
    __syncthreads();
  }
  if (m == -CUDART_INF_F) *lse = m, *entropy = 0.0f;
  else if (!(fabsf(m) < CUDART_INF_F)) *lse = m, *entropy = __int_as_float(0x7FC00000);
  else *lse = m + logf(s), *entropy = logf(s) - t / s;
}

// One vector of 16 bytes as floats.
template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, 2) score_kernel(const ScoreParams p) {
  constexpr int V = kVec<T>;
  __shared__ RowShared sh;
  uint32_t ranks, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
  rank = cluster_ctarank();
  const int64_t row = blockIdx.x / ranks;
  const T* x = static_cast<const T*>(p.logits) + row * p.row_stride;
  // values before the first 16-byte boundary, whole vectors, and the rest
  const int64_t head = min(static_cast<int64_t>((16 - reinterpret_cast<uintptr_t>(x) % 16) % 16 / sizeof(T)), p.vocab);
  const int64_t vectors = (p.vocab - head) / V;
  const int tail = static_cast<int>(p.vocab - head - vectors * V);
  const int64_t from = vectors * rank / ranks, to = vectors * (rank + 1) / ranks;
  const T* body = x + head;
  constexpr float low = kLowest;
  Sums acc{low, 0.0f, 0.0f};
  if (TOP) {
    if (threadIdx.x < kMostTop) sh.top.kept[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.top.least = 1, sh.top.count = 0;
  }

  // the values outside whole vectors: the first and the last CTA of a row
  float odd = -CUDART_INF_F;
  int64_t odd_id = -1;
  if (rank == 0 && threadIdx.x < head) odd_id = threadIdx.x;
  if (rank == ranks - 1 && threadIdx.x >= 32 && threadIdx.x < 32 + tail) odd_id = head + vectors * V + threadIdx.x - 32;
  if (odd_id >= 0) {
    odd = El<T>::to_float(x[odd_id]);
    const float c = max_nan(odd, low);
    const float y = fmaf(c, kLog2e, -reference(c));
    acc.m = c, acc.s = ex2(y), acc.t = acc.s * y;
  }

  uint4 next[kUnroll];
  auto load = [&](int64_t at) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t v = at + u * kThreads + threadIdx.x;
      // past the end: -infinity, which adds nothing
      constexpr uint32_t n = kNothing<T>;
      next[u] = v < to ? __ldcs(reinterpret_cast<const uint4*>(body) + v) : make_uint4(n, n, n, n);
    }
  };
  load(from);
  bool first = true;
  for (int64_t at = from; at < to || first; at += kUnroll * kThreads) {
    Chunk<T, V> now[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) now[u].w[0] = next[u].x, now[u].w[1] = next[u].y, now[u].w[2] = next[u].z, now[u].w[3] = next[u].w;
    if (at + kUnroll * kThreads < to) load(at + kUnroll * kThreads);
    float best[kUnroll], most = low;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float f[V];
      now[u].get(f);
      best[u] = f[0];
#pragma unroll
      for (int i = 1; i < V; ++i) best[u] = max_nan(best[u], f[i]);
      most = max_nan(most, best[u]);
    }
    if (!(most <= acc.m)) {  // a new maximum (or not a number)
      const float m = max_nan(acc.m, most);
      const float d = reference(acc.m) - reference(m), f = ex2(d);
      acc.t = (acc.t + acc.s * d) * f;
      acc.s *= f;
      acc.m = m;
    }
    const float ref = -reference(acc.m);
    float s[2] = {0.0f, 0.0f}, t[2] = {0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float f[V];
      now[u].get(f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float y = fmaf(max_nan(f[i], low), kLog2e, ref);
        const float e = ex2(y);
        s[i & 1] += e;
        t[i & 1] = fmaf(e, y, t[i & 1]);
      }
    }
    acc.s += s[0] + s[1];
    acc.t += t[0] + t[1];
    if (TOP) {
      if (first) {
        // a first bound: of 32 groups of threads, the lowest group maximum;
        // at least 32 values reach it
        float g = max_nan(most, odd);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
        if ((threadIdx.x & 15) == 0) sh.top.groups[threadIdx.x >> 4] = g;
        __syncthreads();
        if (threadIdx.x < 32) {
          g = sh.top.groups[threadIdx.x];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) g = fminf(g, __shfl_xor_sync(0xffffffffu, g, o));
          // groups that hold only values below `low` give no bound
          if (threadIdx.x == 0 && g > low) sh.top.least = candidate(g, 0xFFFFFFFFu);
        }
        __syncthreads();
      }
      bool again = false;
      for (;;) {
        const uint64_t least = sh.top.least;
        const float bar = candidate_value(least);
        bool many = false, lost = false;
        auto offer = [&](float f, int64_t id) {
          const uint64_t c = candidate(f, static_cast<uint32_t>(id));
          if (c < least) return;
          if (again)
            for (int j = 0; j < p.top; ++j)
              if (sh.top.kept[j] == c) return;
          const int place = atomicAdd(&sh.top.count, 1);
          if (place < kKept) sh.top.waiting[place] = c;
          many |= place >= kSelectAt;
          lost |= place >= kKept;
        };
        if (first && odd_id >= 0) offer(odd, odd_id);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int64_t v = at + u * kThreads + threadIdx.x;
          // not below the bar, or no bar yet (or not a number)
          if (v >= to || best[u] < bar) continue;
          float f[V];
          now[u].get(f);
#pragma unroll 1
          for (int i = 0; i < V; ++i) {
            float y = f[0];
#pragma unroll
            for (int j = 1; j < V; ++j) y = i == j ? f[j] : y;
            if (!(y < bar)) offer(y, head + v * V + i);
          }
        }
        if (!__syncthreads_or(many || first)) break;
        const bool more = __syncthreads_or(lost);
        select_top(sh.top, p.top);
        if (!more) break;
        again = true;
      }
    }
    first = false;
  }

  Sums all = block_join(acc, sh);
  if (TOP) select_top(sh.top, p.top);
  if (ranks > 1) {
    cluster_sync_all();
    if (rank == 0) {
      for (uint32_t r = 1; r < ranks; ++r) {
        const uint32_t base = cluster_map(smem_u32(&sh.cta), r);
        Sums b;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(b.m) : "r"(base));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(b.s) : "r"(base + 4));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(b.t) : "r"(base + 8));
        all = join(all, b);
      }
      if (TOP) {
        // at most 7 x 32 candidates of the other CTAs
        const int others = static_cast<int>(ranks - 1) * p.top;
        if (threadIdx.x < others) {
          const uint32_t a = cluster_map(smem_u32(&sh.top.kept[threadIdx.x % p.top]), 1 + threadIdx.x / p.top);
          uint64_t c;
          asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(c) : "r"(a));
          sh.top.waiting[threadIdx.x] = c;
        }
        if (threadIdx.x == 0) sh.top.count = others;
        select_top(sh.top, p.top);
      }
    }
    cluster_sync_all();  // the others' shared memory stays until it was read
    if (rank != 0) return;
  }
  const bool nan_row = all.m != all.m;
  float lse, entropy;
  if (all.m > low + 1024.0f && all.m < -low) {
    const float l = log2f(all.s);
    lse = (reference(all.m) + l) * kLn2;
    entropy = (l - all.t / all.s) * kLn2;
  } else {
    plain_row(x, p.vocab, &lse, &entropy);
  }
  const int64_t token = p.tokens ? p.tokens[row] : -1;
  const bool given = token >= 0 && token < p.vocab;
  const float logit = given && threadIdx.x == 0 ? El<T>::to_float(x[token]) : 0.0f;
  write_row(p, row, lse, entropy, logit, given, nan_row, TOP ? &sh.top : nullptr);
}

// --------------------------------------------------------------- gradient --

struct GradParams {
  int64_t rows, vocab, row_stride, d_row_stride;
  const void* logits;
  void* d_logits;
  const int64_t* tokens;
  const float *lse, *entropy, *d_logprob, *d_entropy;
  int32_t parts;  // CTAs of one row
};

constexpr int kGradThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kGradThreads) score_backward_kernel(const GradParams p) {
  constexpr int V = kVec<T>;
  const int64_t row = blockIdx.x / p.parts;
  const int part = blockIdx.x % p.parts;
  const T* x = static_cast<const T*>(p.logits) + row * p.row_stride;
  T* d = static_cast<T*>(p.d_logits) + row * p.d_row_stride;
  const int64_t token = p.tokens ? p.tokens[row] : -1;
  const bool given = token >= 0 && token < p.vocab;
  const float lse = p.lse[row];
  const float gl = given && p.d_logprob ? p.d_logprob[row] : 0.0f;
  const float ge = p.d_entropy ? p.d_entropy[row] : 0.0f;
  const float a = gl + (p.d_entropy ? ge * p.entropy[row] : 0.0f);
  const bool nothing = lse == -CUDART_INF_F;
  auto grad = [&](float f) {
    const float y = f - lse;
    const float e = ex2(y * kLog2e);
    // a probability of 0 has no part, whatever its logarithm
    const float g = -e * (e > 0.0f ? fmaf(ge, y, a) : a);
    return nothing ? 0.0f : g;
  };
  // vectors where both rows reach a 16-byte boundary together
  const int64_t head = min(static_cast<int64_t>((16 - reinterpret_cast<uintptr_t>(x) % 16) % 16 / sizeof(T)), p.vocab);
  const bool same = reinterpret_cast<uintptr_t>(x) % 16 == reinterpret_cast<uintptr_t>(d) % 16;
  const int64_t vectors = same ? (p.vocab - head) / V : 0;
  const int64_t from = vectors * part / p.parts, to = vectors * (part + 1) / p.parts;
  for (int64_t at = from; at < to; at += kUnroll * kGradThreads) {
    Chunk<T, V> now[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t v = at + u * kGradThreads + threadIdx.x;
      if (v >= to) continue;
      const uint4 w = __ldcs(reinterpret_cast<const uint4*>(x + head) + v);
      now[u].w[0] = w.x, now[u].w[1] = w.y, now[u].w[2] = w.z, now[u].w[3] = w.w;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t v = at + u * kGradThreads + threadIdx.x;
      if (v >= to) continue;
      float f[V];
      now[u].get(f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = grad(f[i]);
      const int64_t off = token - head - v * V;
      if (gl != 0.0f && off >= 0 && off < V && !nothing) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (off == i) f[i] += gl;
      }
      now[u].set(f);
      __stcs(reinterpret_cast<uint4*>(d + head) + v, make_uint4(now[u].w[0], now[u].w[1], now[u].w[2], now[u].w[3]));
    }
  }
  // the rest: before the first vector and after the last
  const int64_t rest = same ? p.vocab - vectors * V : p.vocab;
  for (int64_t i = static_cast<int64_t>(part) * kGradThreads + threadIdx.x; i < rest; i += static_cast<int64_t>(p.parts) * kGradThreads) {
    const int64_t id = same && i >= head ? i + vectors * V : i;
    float g = grad(El<T>::to_float(x[id]));
    if (id == token && !nothing) g += gl;
    d[id] = El<T>::from_float(g);
  }
}

// ------------------------------------------------------------------- host --

int el_bytes(int dtype) { return dtype == EG_EL_F32 ? 4 : 2; }

eg_status check_score(const eg_score_args* a) {
  if (!a) return host_fail(EG_ERR_INVALID_ARG, "args is NULL");
  if (a->rows < 0 || a->vocab < 0)
    return host_fail(EG_ERR_INVALID_ARG, "negative size (rows=%lld vocab=%lld)", (long long)a->rows, (long long)a->vocab);
  if (a->dtype != EG_EL_BF16 && a->dtype != EG_EL_F16 && a->dtype != EG_EL_F32)
    return host_fail(EG_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
  if (a->rows > (1 << 24) || a->vocab > INT32_MAX)
    return host_fail(EG_ERR_UNSUPPORTED, "at most 2^24 rows of fewer than 2^31 logits a call");
  if (a->rows == 0) return EG_OK;
  if (a->vocab == 0) return host_fail(EG_ERR_INVALID_ARG, "rows without logits");
  if (!a->logits || reinterpret_cast<uintptr_t>(a->logits) % el_bytes(a->dtype))
    return host_fail(EG_ERR_INVALID_ARG, "logits is NULL or not aligned to its elements");
  if (a->row_stride < a->vocab) return host_fail(EG_ERR_INVALID_ARG, "row_stride must be at least vocab");
  if (reinterpret_cast<uintptr_t>(a->tokens) % 8)
    return host_fail(EG_ERR_INVALID_ARG, "tokens are not aligned to their elements");
  return EG_OK;
}

int sm_count() {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <typename T>
cudaError_t launch_score(const ScoreParams& p, int ranks, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.top ? cudaLaunchKernelEx(&cfg, score_kernel<T, true>, p) : cudaLaunchKernelEx(&cfg, score_kernel<T, false>, p);
}

}  // namespace
}  // namespace eg

using namespace eg;

extern "C" {

eg_status eg_token_logprobs(const eg_score_args* args, void* stream) {
  eg_status s = check_score(args);
  if (s != EG_OK) return s;
  const eg_score_args& a = *args;
  if (a.top < 0 || a.top > kMostTop) return host_fail(EG_ERR_UNSUPPORTED, "top must be in 0..%d (got %d)", kMostTop, a.top);
  for (const void* o : {static_cast<const void*>(a.logprob), static_cast<const void*>(a.lse), static_cast<const void*>(a.entropy),
                        static_cast<const void*>(a.top_logprobs)})
    if (reinterpret_cast<uintptr_t>(o) % 4) return host_fail(EG_ERR_INVALID_ARG, "an output is not aligned to its elements");
  if (reinterpret_cast<uintptr_t>(a.top_ids) % 8) return host_fail(EG_ERR_INVALID_ARG, "top_ids is not aligned to its elements");
  if (a.rows == 0) return EG_OK;
  if (a.top > a.vocab) return host_fail(EG_ERR_INVALID_ARG, "top=%d of %lld logits", a.top, (long long)a.vocab);
  int dev = 0;
  if ((s = host_check_device(&dev)) != EG_OK) return s;
  ScoreParams p{};
  p.rows = a.rows, p.vocab = a.vocab, p.row_stride = a.row_stride;
  p.logits = a.logits, p.tokens = a.tokens;
  p.logprob = a.logprob, p.lse = a.lse, p.entropy = a.entropy;
  p.top = a.top_ids || a.top_logprobs ? a.top : 0;
  p.top_ids = a.top_ids, p.top_logprobs = a.top_logprobs;
  // a cluster for a row while that still leaves every CTA an SM of its own
  // and 16 KB of logits
  int ranks = 1;
  while (ranks < 8 && a.rows * ranks * 2 <= sm_count() && a.vocab * el_bytes(a.dtype) / (ranks * 2) >= 16384) ranks *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = a.dtype == EG_EL_F32    ? launch_score<float>(p, ranks, st)
                  : a.dtype == EG_EL_BF16 ? launch_score<__nv_bfloat16>(p, ranks, st)
                                          : launch_score<__half>(p, ranks, st);
  return e == cudaSuccess ? EG_OK : host_cuda_fail(e, "launching token_logprobs");
}

eg_status eg_token_logprobs_backward(const eg_score_args* args, const eg_score_grads* grads, void* stream) {
  eg_status s = check_score(args);
  if (s != EG_OK) return s;
  if (!grads) return host_fail(EG_ERR_INVALID_ARG, "grads is NULL");
  const eg_score_args& a = *args;
  const eg_score_grads& g = *grads;
  if (a.rows == 0) return EG_OK;
  if (!g.lse) return host_fail(EG_ERR_INVALID_ARG, "lse is NULL");
  if (g.d_entropy && !g.entropy) return host_fail(EG_ERR_INVALID_ARG, "d_entropy needs entropy");
  for (const float* o : {g.lse, g.entropy, g.d_logprob, g.d_entropy})
    if (reinterpret_cast<uintptr_t>(o) % 4) return host_fail(EG_ERR_INVALID_ARG, "an input is not aligned to its elements");
  if (!g.d_logits || reinterpret_cast<uintptr_t>(g.d_logits) % el_bytes(a.dtype))
    return host_fail(EG_ERR_INVALID_ARG, "d_logits is NULL or not aligned to its elements");
  if (g.d_row_stride < a.vocab) return host_fail(EG_ERR_INVALID_ARG, "d_row_stride must be at least vocab");
  int dev = 0;
  if ((s = host_check_device(&dev)) != EG_OK) return s;
  GradParams p{};
  p.rows = a.rows, p.vocab = a.vocab, p.row_stride = a.row_stride, p.d_row_stride = g.d_row_stride;
  p.logits = a.logits, p.d_logits = g.d_logits, p.tokens = a.tokens;
  p.lse = g.lse, p.entropy = g.entropy, p.d_logprob = g.d_logprob, p.d_entropy = g.d_entropy;
  // a CTA for each 64 KB of a row
  const int64_t parts = std::max<int64_t>(1, a.vocab * el_bytes(a.dtype) / 65536);
  if (a.rows * parts > INT32_MAX) return host_fail(EG_ERR_UNSUPPORTED, "too many logits for one call");
  p.parts = static_cast<int32_t>(parts);
  const unsigned grid = static_cast<unsigned>(a.rows * parts);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.dtype == EG_EL_F32) score_backward_kernel<float><<<grid, kGradThreads, 0, st>>>(p);
  else if (a.dtype == EG_EL_BF16) score_backward_kernel<__nv_bfloat16><<<grid, kGradThreads, 0, st>>>(p);
  else score_backward_kernel<__half><<<grid, kGradThreads, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? EG_OK : host_cuda_fail(e, "launching the gradient of token_logprobs");
}

}  // extern "C"
