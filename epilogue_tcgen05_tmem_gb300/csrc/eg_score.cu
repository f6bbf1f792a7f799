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

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;        // 16-byte loads of a thread in flight
constexpr int kMostTop = 32;
constexpr int kWaiting = 2048;    // room for candidates of one selection
constexpr int kQueue = 1024;      // room for vectors that may hold one
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
template <typename T>
constexpr float kLowest = -65504.0f;
template <>
constexpr float kLowest<__nv_bfloat16> = -65536.0f;

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
  alignas(16) uint64_t waiting[kWaiting];  // candidates not yet selected from
  alignas(16) uint64_t kept[2][kMostTop];  // the best so far, in order; 0: none
  uint64_t least;            // a value has to reach this to be a candidate
  int count, queued;         // candidates and vectors that asked for a place
  int lost;                  // some found none
  uint32_t queue[kQueue];    // vectors with a value above the bar
  uint64_t groups[kMostTop];
};

struct RowShared {
  Sums warps[kWarps];
  Sums cta;
  TopShared top;
};

// The best `top` of kept[cur] and waiting into kept[cur ^ 1], in order; the
// next candidate has to be better than the last of them.  All threads; the
// place of each is the number of better ones.
__device__ __forceinline__ void select_top(TopShared& sh, int top, int& cur) {
  __syncthreads();
  const int waiting = min(sh.count, kWaiting);
  const int total = waiting + top;
  for (int at = threadIdx.x; at < total; at += kThreads) {
    const uint64_t mine = at < top ? sh.kept[cur][at] : sh.waiting[at - top];
    if (mine == 0) continue;
    int better = 0;
    for (int j = 0; j < top; ++j) better += sh.kept[cur][j] > mine;
    int j = 0;
    for (; j + 1 < waiting; j += 2) {
      const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(&sh.waiting[j]);
      better += (two.x > mine) + (two.y > mine);
    }
    if (j < waiting) better += sh.waiting[j] > mine;
    if (better < top) sh.kept[cur ^ 1][better] = mine;
  }
  cur ^= 1;
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint64_t last = sh.kept[cur][top - 1];
    if (last) sh.least = last + 1;
    sh.count = sh.queued = 0;
  }
  __syncthreads();
}

// The outputs of one row by one thread group of the CTA that holds the sums.
__device__ __forceinline__ void write_row(const ScoreParams& p, int64_t row, float lse, float entropy, float token_logit,
                                          bool given, bool nan_row, const uint64_t* top) {
  const float nan = __int_as_float(0x7FC00000);
  const bool nothing = lse == -CUDART_INF_F;
  if (threadIdx.x == 0) {
    if (p.lse) p.lse[row] = lse;
    if (p.entropy) p.entropy[row] = entropy;
    if (p.logprob) p.logprob[row] = !given ? 0.0f : nothing ? -CUDART_INF_F : lse == CUDART_INF_F ? nan : token_logit - lse;
  }
  if (top && threadIdx.x < p.top) {
    const uint64_t c = top[threadIdx.x];
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

__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpair(uint64_t v, float* lo, float* hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Elements of one vector of 16 bytes.
template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

// Larger of two words' elements, or not a number where either is none.
template <typename T>
__device__ __forceinline__ uint32_t word_max(uint32_t a, uint32_t b) {
  if constexpr (sizeof(T) == 4) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
  } else if constexpr (El<T>::kBf16) {
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  } else {
    const __half2 m = __hmax2_nan(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
}
template <typename T>
__device__ __forceinline__ float word_top(uint32_t w) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(w);
  else {
    const float2 f = El<T>::unpack2(w);
    return max_nan(f.x, f.y);
  }
}
template <typename T>
__device__ __forceinline__ uint32_t lowest_word() {
  if constexpr (sizeof(T) == 4) return __float_as_uint(kLowest<T>);
  else return El<T>::pack2(kLowest<T>, kLowest<T>);
}

// The part of a row that one CTA of its cluster has.
template <typename T>
struct Part {
  const T* body;     // the row's first 16-byte boundary
  int64_t head;      // values before it
  int64_t from, to;  // vectors
  float odd;         // a value outside whole vectors that this thread has
  int64_t odd_id;    // -1: none
};

// Take a value for a candidate.
__device__ __forceinline__ void offer_top(TopShared& sh, float f, int64_t id) {
  const uint64_t c = candidate(f, static_cast<uint32_t>(id));
  if (c < sh.least) return;
  const int place = atomicAdd(&sh.count, 1);
  if (place < kWaiting) sh.waiting[place] = c;
  else sh.lost = 1;
}

// Candidates of the noted vectors.  All threads; the result (and whether a
// place was lost) is there for all after it.
template <typename T>
__device__ __forceinline__ void open_queue(const Part<T>& part, TopShared& sh) {
  constexpr int V = kVec<T>;
  __syncthreads();
  const int queued = min(sh.queued, kQueue);
  for (int i = threadIdx.x; i < queued; i += kThreads) {
    const int64_t v = sh.queue[i];
    Chunk<T, V> c;
    c.load(part.body + v * V);
    float f[V];
    c.get(f);
#pragma unroll
    for (int j = 0; j < V; ++j) offer_top(sh, f[j], part.head + v * V + j);
  }
  __syncthreads();
}

// The best of a part, when more candidates came between two selections than
// there is room for (values that rise along the row, many equal ones): batch
// by batch, with a selection whenever one fills the room.
template <typename T>
__device__ __noinline__ void careful_top(const Part<T>& part, TopShared& sh, int top, int* where) {
  constexpr int V = kVec<T>;
  int cur = 0;
  __syncthreads();
  if (threadIdx.x < kMostTop) sh.kept[0][threadIdx.x] = sh.kept[1][threadIdx.x] = 0;
  if (threadIdx.x == 0) sh.least = 1, sh.count = 0;
  __syncthreads();
  for (int64_t at = part.from; at < part.to || at == part.from; at += kThreads) {
    const int64_t v = at + threadIdx.x;
    bool again = false;
    for (;;) {
      const uint64_t least = sh.least;
      bool lost = false;
      auto offer = [&](float f, int64_t id) {
        const uint64_t c = candidate(f, static_cast<uint32_t>(id));
        if (c < least) return;
        if (again)
          for (int j = 0; j < top; ++j)
            if (sh.kept[cur][j] == c) return;
        const int place = atomicAdd(&sh.count, 1);
        if (place < kWaiting) sh.waiting[place] = c;
        else lost = true;
      };
      if (at == part.from && part.odd_id >= 0) offer(part.odd, part.odd_id);
      if (v < part.to)
        for (int i = 0; i < V; ++i) offer(El<T>::to_float(part.body[v * V + i]), part.head + v * V + i);
      const bool more = __syncthreads_or(lost);
      select_top(sh, top, cur);
      if (!more) break;
      again = true;
    }
  }
  *where = cur;
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, 4) score_kernel(const ScoreParams p) {
  constexpr int V = kVec<T>;
  constexpr int W = 4;  // words of a vector
  __shared__ RowShared sh;
  uint32_t ranks, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
  rank = cluster_ctarank();
  const int64_t row = blockIdx.x / ranks;
  const T* x = static_cast<const T*>(p.logits) + row * p.row_stride;
  // values before the first 16-byte boundary, whole vectors, and the rest
  Part<T> part;
  part.head = min(static_cast<int64_t>((16 - reinterpret_cast<uintptr_t>(x) % 16) % 16 / sizeof(T)), p.vocab);
  const int64_t vectors = (p.vocab - part.head) / V;
  const int tail = static_cast<int>(p.vocab - part.head - vectors * V);
  part.from = vectors * rank / ranks, part.to = vectors * (rank + 1) / ranks;
  part.body = x + part.head;
  constexpr float low = kLowest<T>;
  Sums acc{low, 0.0f, 0.0f};
  int cur = 0;
  if (TOP) {
    if (threadIdx.x < kMostTop) sh.top.kept[0][threadIdx.x] = sh.top.kept[1][threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.top.least = 1, sh.top.count = sh.top.queued = sh.top.lost = 0;
  }

  // the values outside whole vectors: the first and the last CTA of a row
  part.odd = -CUDART_INF_F;
  part.odd_id = -1;
  if (rank == 0 && threadIdx.x < part.head) part.odd_id = threadIdx.x;
  if (rank == ranks - 1 && threadIdx.x >= 32 && threadIdx.x < 32 + tail) part.odd_id = part.head + vectors * V + threadIdx.x - 32;
  if (part.odd_id >= 0) {
    part.odd = El<T>::to_float(x[part.odd_id]);
    const float c = max_nan(part.odd, low);
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
      next[u] = v < part.to ? __ldcs(reinterpret_cast<const uint4*>(part.body) + v) : make_uint4(n, n, n, n);
    }
  };
  load(part.from);
  float bar = -CUDART_INF_F;  // a value below this is no candidate
  uint32_t batch = 0;
  for (int64_t at = part.from; at < part.to || batch == 0; at += kUnroll * kThreads, ++batch) {
    uint32_t now[kUnroll][W];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) now[u][0] = next[u].x, now[u][1] = next[u].y, now[u][2] = next[u].z, now[u][3] = next[u].w;
    if (at + kUnroll * kThreads < part.to) load(at + kUnroll * kThreads);
    uint32_t high[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) high[u] = word_max<T>(word_max<T>(now[u][0], now[u][1]), word_max<T>(now[u][2], now[u][3]));
    const float most = word_top<T>(word_max<T>(word_max<T>(high[0], high[1]), word_max<T>(high[2], high[3])));
    if (TOP) {
      if (batch == 0) {
        // a first bar: each of 32 groups of threads has a best candidate, and
        // `top` of those reach the `top`-th of them
        uint64_t best = 0;
#pragma unroll
        for (int u = kUnroll - 1; u >= 0; --u) {
          const int64_t v = at + u * kThreads + threadIdx.x;
          if (v >= part.to) continue;
          const float own = word_top<T>(high[u]);
          int in = -1;
#pragma unroll
          for (int w = W - 1; w >= 0; --w) {
            if constexpr (sizeof(T) == 4) {
              if (__uint_as_float(now[u][w]) == own) in = w;
            } else {
              const float2 f = El<T>::unpack2(now[u][w]);
              if (f.y == own) in = 2 * w + 1;
              if (f.x == own) in = 2 * w;
            }
          }
          const uint64_t c = in >= 0 ? candidate(own, static_cast<uint32_t>(part.head + v * V + in)) : 0;
          best = c > best ? c : best;
        }
        if (part.odd_id >= 0) {
          const uint64_t c = candidate(part.odd, static_cast<uint32_t>(part.odd_id));
          best = c > best ? c : best;
        }
#pragma unroll
        for (int o = kThreads / 64; o > 0; o >>= 1) {
          const uint64_t c = __shfl_xor_sync(0xffffffffu, best, o);
          best = c > best ? c : best;
        }
        if ((threadIdx.x & (kThreads / 32 - 1)) == 0) sh.top.groups[threadIdx.x / (kThreads / 32)] = best;
        __syncthreads();
        if (threadIdx.x < 32) {
          best = sh.top.groups[threadIdx.x];
          int better = 0;
#pragma unroll 8
          for (int j = 0; j < 32; ++j) better += __shfl_sync(0xffffffffu, best, j) > best;
          if (better == p.top - 1 && best) sh.top.least = best;
        }
        __syncthreads();
        bar = candidate_value(sh.top.least);
      }
      // above the bar, or no bar yet, or not a number; later values that equal
      // it come after the ones that set it.  The vector is only noted here: a
      // warp pays for what any of its threads does, so the values are looked
      // at when all threads have one.
      if (batch == 0 ? !(most < bar) : !(most <= bar)) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const float own = word_top<T>(high[u]);
          const int64_t v = at + u * kThreads + threadIdx.x;
          if (v < part.to && (batch == 0 ? !(own < bar) : !(own <= bar))) {
            const int place = atomicAdd(&sh.top.queued, 1);
            if (place < kQueue) sh.top.queue[place] = static_cast<uint32_t>(v);
            else sh.top.lost = 1;
          }
        }
      }
      if (batch == 0 && part.odd_id >= 0) offer_top(sh.top, part.odd, part.odd_id);
      // raise the bar after 4, 16, 64, ... batches
      if (batch && ((batch + 1) & batch) == 0 && ((batch + 1) & 0x55555555u) && at + kUnroll * kThreads < part.to) {
        open_queue(part, sh.top);
        select_top(sh.top, p.top, cur);
        bar = candidate_value(sh.top.least);
      }
    }
    const float m = max_nan(acc.m, most);
    if (!(m <= acc.m)) {  // a new maximum (or not a number)
      const float d = reference(acc.m) - reference(m), f = ex2(d);
      acc.t = (acc.t + acc.s * d) * f;
      acc.s *= f;
      acc.m = m;
    }
    // two values in one instruction where there is one
    const float ref = -reference(acc.m);
    const uint64_t ref2 = pair_of(ref, ref), log2e2 = pair_of(kLog2e, kLog2e);
    uint64_t s2 = 0, t2 = 0;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int w = 0; w < W; w += (sizeof(T) == 4 ? 2 : 1)) {
        float f0, f1;
        const uint32_t c = word_max<T>(now[u][w], lowest_word<T>());
        if constexpr (sizeof(T) == 4) {
          f0 = __uint_as_float(c);
          f1 = __uint_as_float(word_max<T>(now[u][w + 1], lowest_word<T>()));
        } else {
          const float2 two = El<T>::unpack2(c);
          f0 = two.x, f1 = two.y;
        }
        const uint64_t y = fma_pair(pair_of(f0, f1), log2e2, ref2);
        float y0, y1;
        unpair(y, &y0, &y1);
        const uint64_t e = pair_of(ex2(y0), ex2(y1));
        s2 = add_pair(s2, e);
        t2 = fma_pair(e, y, t2);
      }
    float a, b;
    unpair(s2, &a, &b);
    acc.s += a + b;
    unpair(t2, &a, &b);
    acc.t += a + b;
  }

  Sums all = block_join(acc, sh);
  if (TOP) {
    open_queue(part, sh.top);
    if (sh.top.lost) careful_top(part, sh.top, p.top, &cur);
    else select_top(sh.top, p.top, cur);
  }
  if (ranks > 1) {
    if (TOP && cur != 0) {  // where the first CTA of the row looks
      if (threadIdx.x < kMostTop) sh.top.kept[0][threadIdx.x] = sh.top.kept[1][threadIdx.x];
      cur = 0;
    }
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
          const uint32_t a = cluster_map(smem_u32(&sh.top.kept[0][threadIdx.x % p.top]), 1 + threadIdx.x / p.top);
          uint64_t c;
          asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(c) : "r"(a));
          sh.top.waiting[threadIdx.x] = c;
        }
        if (threadIdx.x == 0) sh.top.count = others;
        select_top(sh.top, p.top, cur);
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
  write_row(p, row, lse, entropy, logit, given, nan_row, TOP ? sh.top.kept[cur] : nullptr);
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
