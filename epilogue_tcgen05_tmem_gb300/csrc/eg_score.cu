// eg_score.cu -- log probabilities of given tokens with entropy and the top
// alternatives, and their gradient (include/eg_decoder.h has the formulas).
//
// Both are bound by memory: the logits are read once (and their gradient
// written once).  Single calls with cold L2: 4096 x 131072 in bf16 take 175 us
// (6.1 TB/s of the 6.8 that a copy reaches), with 20 alternatives 217 us (207 us
// in succession), the rest being instructions and the barriers at a row's end;
// the gradient of 2048 x 100003 in float32 246 us (6.6 TB/s; 240 us in
// succession).  Forward: a CTA, or a cluster of CTAs where there are few
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

constexpr int kUnroll = 4;        // 16-byte vectors of a thread and batch
constexpr int kStages = 2;        // batches in flight of a CTA
constexpr int kMostTop = 32;
constexpr int kWaiting = 1024;    // room for candidates of one selection
constexpr int kQueue = 128;       // room of a warp for notes of threads' batches that may hold one
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct ScoreParams {
  int64_t rows, vocab, row_stride;
  const void* logits;
  const int64_t* tokens;
  float *logprob, *lse, *entropy, *top_logprobs;
  int64_t* top_ids;
  int32_t top;
  int32_t stall;           // test hook: the loading warp loads nothing
  uint64_t wait_limit_ns;
};

// Set when a wait of score_kernel ran past its limit (one for each device);
// eg_token_logprobs_device_status reads it.
__device__ int32_t g_score_status;

// N threads of a CTA look at values (one more warp loads them); a barrier of these.
template <int N>
__device__ __forceinline__ void sync_lookers() { asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory"); }

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

template <int N>
struct TopShared {
  alignas(16) uint64_t waiting[kWaiting];  // candidates
  alignas(16) uint64_t bests[N];    // the best one of each thread
  alignas(16) uint64_t kept[kMostTop];     // the best, in order; 0: none
  alignas(16) float groups[2][32];         // maxima of 32 groups of threads
  uint64_t least;            // a value has to reach this to be a candidate
  int count;                 // candidates that asked for a place
  int lost;                  // some candidates or notes found none
  int flood;                 // a warp has more notes than two for a thread
  int2 queue[N / 32][kQueue];  // a thread's batches above the bar: the first vector, and the largest value
};

template <int N>
struct RowShared {
  alignas(16) uint8_t ring[kStages][N * kUnroll * 16];
  uint64_t full[kStages], empty[kStages];
  int abort;
  Sums warps[N / 32];
  Sums cta;
  TopShared<N> top;
};

// How many of list[0, n) are better than `mine`; the list is zero up to the
// next multiple of 16.
__device__ __forceinline__ int better_than(const uint64_t* list, int n, uint64_t mine) {
  int better = 0;
  for (int j = 0; j < n; j += 16) {
    ulonglong2 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = reinterpret_cast<const ulonglong2*>(list + j)[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) better += (v[i].x > mine) + (v[i].y > mine);
  }
  return better;
}

// The best `top` of the candidates into kept, in order.  All threads, after a
// barrier that follows the last candidate (`waiting` is zero behind it); the
// place of each is the number of better ones.  Ends with a barrier; returns
// the number of candidates.
template <int N>
__device__ __forceinline__ int select_top(TopShared<N>& sh, int top) {
  const int n = min(sh.count, kWaiting);
  if (static_cast<int>(threadIdx.x) >= n && threadIdx.x < kMostTop) sh.kept[threadIdx.x] = 0;
  uint64_t least = 0;
  if (n > N) {
    // more than one for a thread: only what reaches the `top`-th of the
    // threads' best is placed
    uint64_t best = 0;
    for (int at = threadIdx.x; at < n; at += N) best = max(best, sh.waiting[at]);
    sh.bests[threadIdx.x] = best;
    if (threadIdx.x == 0) sh.least = 0;
    sync_lookers<N>();
    if (better_than(sh.bests, N, best) == top - 1) sh.least = best;
    sync_lookers<N>();
    least = sh.least;
  }
  for (int at = threadIdx.x; at < n; at += N) {
    const uint64_t mine = sh.waiting[at];
    if (mine < least) continue;
    const int place = better_than(sh.waiting, n, mine);
    if (place < top) sh.kept[place] = mine;
  }
  sync_lookers<N>();
  return n;
}

// Ready for the next row's candidates, of which there were `used`; a barrier has to come before the first.
template <int N>
__device__ __forceinline__ void clear_top(TopShared<N>& sh, int used) {
  for (int i = threadIdx.x; i < used; i += N) sh.waiting[i] = 0;
  if (threadIdx.x == 0) sh.count = sh.lost = sh.flood = 0;
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

// Sums of a warp to the reference of its maximum: the maximum first, then one
// scaling a lane.
__device__ __forceinline__ Sums warp_join(Sums v, int lanes) {
  float m = v.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float d = reference(v.m) - reference(m), f = ex2(d);
  float s = v.s * f, t = (v.t + v.s * d) * f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      t += __shfl_xor_sync(0xffffffffu, t, o);
    }
  return {m, s, t};
}

// A row whose maximum is so low, so high or so infinite that the pass above
// does not hold: its statistics from the definition, by one CTA.
template <typename T, int N>
__device__ __noinline__ void plain_row(const T* x, int64_t vocab, float* red, float* lse, float* entropy) {
  float m = -CUDART_INF_F;
  for (int64_t i = threadIdx.x; i < vocab; i += N) m = max_nan(m, El<T>::to_float(x[i]));
  red[threadIdx.x] = m;
  sync_lookers<N>();
  for (int o = N / 2; o > 0; o >>= 1) {
    if (threadIdx.x < o) red[threadIdx.x] = max_nan(red[threadIdx.x], red[threadIdx.x + o]);
    sync_lookers<N>();
  }
  m = red[0];
  sync_lookers<N>();
  float s = 0.0f, t = 0.0f;
  if (fabsf(m) < CUDART_INF_F)
    for (int64_t i = threadIdx.x; i < vocab; i += N) {
      const float d = El<T>::to_float(x[i]) - m, e = expf(d);
      if (e > 0.0f) s += e, t += e * d;
    }
  for (int k = 0; k < 2; ++k) {
    red[threadIdx.x] = k ? t : s;
    sync_lookers<N>();
    for (int o = N / 2; o > 0; o >>= 1) {
      if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
      sync_lookers<N>();
    }
    (k ? t : s) = red[0];
    sync_lookers<N>();
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
  int32_t head;      // values before it
  int32_t from, to;  // vectors
  float odd;         // a value outside whole vectors that this thread has
  int32_t odd_id;    // -1: none
};

// Take a value for a candidate.
template <int N>
__device__ __forceinline__ void offer_top(TopShared<N>& sh, uint64_t least, float f, int32_t id) {
  const uint64_t c = candidate(f, static_cast<uint32_t>(id));
  if (c < least) return;
  const int place = atomicAdd(&sh.count, 1);
  if (place < kWaiting) sh.waiting[place] = c;
  else sh.lost = 1;
}

// A value that `top` of 32 groups of threads have reached, from each thread's
// largest so far: at least `top` values reach it, and few more do.  One
// barrier, after which every warp finds it by itself; `turn` counts the calls.
template <int N>
__device__ __forceinline__ float group_bar(TopShared<N>& sh, float most, int top, int turn) {
#pragma unroll
  for (int o = N / 64; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  float* groups = sh.groups[turn & 1];
  if (threadIdx.x % (N / 32) == 0) groups[threadIdx.x / (N / 32)] = most;
  sync_lookers<N>();
  const float g = groups[threadIdx.x & 31];
  int better = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float4 f = reinterpret_cast<const float4*>(groups)[j];
    better += (f.x > g) + (f.y > g) + (f.z > g) + (f.w > g);
  }
  // the smallest of those with fewer than `top` better ones
  const uint32_t least = __reduce_min_sync(0xffffffffu, better < top ? static_cast<uint32_t>(candidate(g, 0) >> 32) : 0xFFFFFFFFu);
  return candidate_value(static_cast<uint64_t>(least) << 32);
}

// The candidates among the values of the vectors that this warp noted: those
// that reach the last bar.  Where there is no bar, or many were noted (many
// equal values, a short row), a better bound first: each thread has a best
// candidate, and `top` of those reach the `top`-th of them.
template <typename T, int N>
__device__ __forceinline__ void open_queue(const Part<T>& part, TopShared<N>& sh, int queued, float bar, int top) {
  constexpr int V = kVec<T>;
  const int2* queue = sh.queue[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31;
  queued = min(queued, kQueue);
  uint64_t least = candidate(bar, 0xFFFFFFFFu);
  // the vectors of a note that may matter
  auto open = [&](const int2& note, Chunk<T, V> (&c)[kUnroll]) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int32_t v = note.x + u * N;
      if (v < part.to) c[u].load(part.body + static_cast<int64_t>(v) * V);
      else c[u].w[0] = c[u].w[1] = c[u].w[2] = c[u].w[3] = kNothing<T>;
    }
  };
  if (sh.flood || bar == -CUDART_INF_F) {
    if (threadIdx.x == 0) sh.least = 0;
    uint64_t best = 0;
    for (int i = lane; i < queued; i += 32) {
      Chunk<T, V> c[kUnroll];
      open(queue[i], c);
#pragma unroll 1
      for (int u = 0; u < kUnroll; ++u) {
        float f[V];
        c[0].get(f);
        const int32_t v = queue[i].x + u * N;
        if (v < part.to)
#pragma unroll
          for (int j = 0; j < V; ++j) best = max(best, candidate(f[j], static_cast<uint32_t>(part.head + v * V + j)));
#pragma unroll
        for (int i = 0; i + 1 < kUnroll; ++i) c[i] = c[i + 1];
      }
    }
    sh.bests[threadIdx.x] = best;
    sync_lookers<N>();
    // only the first threads have any in a short row
    const int teams = min(N, (part.to - part.from + 31) & ~31);
    if (best && better_than(sh.bests, teams, best) == top - 1) sh.least = best;
    sync_lookers<N>();
    least = max(least, sh.least);
  }
  for (int i = lane; i < queued; i += 32) {
    const int2 note = queue[i];
    if (__int_as_float(note.y) < bar) continue;
    Chunk<T, V> c[kUnroll];
    open(note, c);
#pragma unroll 1
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t high = word_max<T>(word_max<T>(c[0].w[0], c[0].w[1]), word_max<T>(c[0].w[2], c[0].w[3]));
      const int32_t v = note.x + u * N;
      if (v < part.to && !(word_top<T>(high) < bar)) {
        float f[V];
        c[0].get(f);
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (!(f[j] < bar)) offer_top(sh, least, f[j], part.head + v * V + j);
      }
#pragma unroll
      for (int i = 0; i + 1 < kUnroll; ++i) c[i] = c[i + 1];
    }
  }
}

// The best of a part, when more vectors or candidates came than there is room
// for (values that rise along the row): some vectors at a time, with a
// selection after each lot.
template <typename T, int N>
__device__ __noinline__ int careful_top(const Part<T>& part, TopShared<N>& sh, int top) {
  constexpr int V = kVec<T>;
  constexpr int kLot = (kWaiting - kMostTop - 16) / V < N ? (kWaiting - kMostTop - 16) / V : N;
  sync_lookers<N>();
  int used = 0;
  if (threadIdx.x < kMostTop) sh.kept[threadIdx.x] = 0;
  for (int32_t at = part.from; at < part.to || at == part.from; at += kLot) {
    sync_lookers<N>();
    clear_top(sh, kWaiting);
    sync_lookers<N>();
    const uint64_t last = sh.kept[top - 1];
    if (threadIdx.x < top) sh.waiting[threadIdx.x] = sh.kept[threadIdx.x];
    if (threadIdx.x == 0) sh.count = top;
    sync_lookers<N>();
    // a zero among the kept ones is no candidate: nothing is worse
    const uint64_t least = last + 1;
    const int32_t v = at + static_cast<int32_t>(threadIdx.x);
    if (at == part.from && part.odd_id >= 0) offer_top(sh, least, part.odd, part.odd_id);
    if (static_cast<int>(threadIdx.x) < kLot && v < part.to)
      for (int i = 0; i < V; ++i) offer_top(sh, least, El<T>::to_float(part.body[static_cast<int64_t>(v) * V + i]), part.head + v * V + i);
    sync_lookers<N>();
    used = select_top(sh, top);
  }
  return used;
}

// Where the row's vectors start, and which of them this CTA of `ranks` has.
template <typename T>
__device__ __forceinline__ Part<T> part_of(const T* x, int64_t vocab, uint32_t rank, uint32_t ranks) {
  Part<T> part;
  part.head = static_cast<int32_t>(min(static_cast<int64_t>((16 - reinterpret_cast<uintptr_t>(x) % 16) % 16 / sizeof(T)), vocab));
  const uint32_t vectors = static_cast<uint32_t>(vocab - part.head) / kVec<T>;
  part.from = static_cast<int32_t>(vectors * rank / ranks), part.to = static_cast<int32_t>(vectors * (rank + 1) / ranks);  // 2^29 x 8 fits
  part.body = x + part.head;
  return part;
}

// CTAs of an SM, as many as the ring and the registers allow.
template <int N>
constexpr int kCtas = N == 256 ? 4 : 7;

// Bounded wait; gives up at once after any wait of the CTA has run out.
__device__ __forceinline__ bool wait_batch(uint64_t* bar, uint32_t phase, int* abort, uint64_t limit_ns) {
  if (mbar_try_wait(bar, phase & 1)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 0;; ++it) {
    if (mbar_try_wait(bar, phase & 1)) return true;
    if ((it & 63u) == 0) {
      if (*reinterpret_cast<volatile int*>(abort)) return false;
      if (global_timer_ns() - t0 > limit_ns) {
        *reinterpret_cast<volatile int*>(abort) = 1;
        *reinterpret_cast<volatile int32_t*>(&g_score_status) = 1;
        return false;
      }
    }
  }
}

// A CTA takes rows (or its part of a cluster's row) one after the other.  The
// loading warp streams them into a ring of batches and runs ahead into the
// next row, so the memory stays busy while a row is being finished.
template <typename T, bool TOP, int N>
__global__ void __launch_bounds__(N + 32, kCtas<N>) score_kernel(const ScoreParams p) {
  constexpr int V = kVec<T>;
  constexpr int W = 4;  // words of a vector
  extern __shared__ __align__(128) uint8_t raw[];
  RowShared<N>& sh = *reinterpret_cast<RowShared<N>*>(raw);
  uint32_t ranks, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
  rank = cluster_ctarank();
  const int64_t first_row = blockIdx.x / ranks, row_step = gridDim.x / ranks;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&sh.full[i], 1), mbar_init(&sh.empty[i], N / 32);
    fence_mbar_init();
    sh.abort = 0;
  }
  if (TOP && threadIdx.x < N) clear_top(sh.top, kWaiting);
  __syncthreads();
  if (threadIdx.x >= N) {
    if (threadIdx.x == N && !p.stall) {
      uint32_t n = 0;  // batches so far
      bool ok = true;
      for (int64_t row = first_row; ok && row < p.rows; row += row_step) {
        const Part<T> part = part_of(static_cast<const T*>(p.logits) + row * p.row_stride, p.vocab, rank, ranks);
        for (int32_t at = part.from; at < part.to; at += kUnroll * N) {
          const int slot = n % kStages;
          if (!(ok = wait_batch(&sh.empty[slot], n / kStages + 1, &sh.abort, p.wait_limit_ns))) break;
          const uint32_t bytes = static_cast<uint32_t>(min(part.to - at, kUnroll * N)) * 16u;
          mbar_arrive_expect_tx(&sh.full[slot], bytes);
          asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                           smem_u32(sh.ring[slot])),
                       "l"(reinterpret_cast<uint64_t>(part.body + static_cast<int64_t>(at) * V)), "r"(bytes), "r"(smem_u32(&sh.full[slot]))
                       : "memory");
          ++n;
        }
      }
      // leave no copy in flight behind
      for (uint32_t i = n > kStages ? n - kStages : 0; i < n; ++i) mbar_wait(&sh.full[i % kStages], (i / kStages) & 1, p.wait_limit_ns);
    }
    __syncwarp();
    if (ranks > 1) {  // as often as the other warps below: a cluster has one row
      cluster_sync_all();
      cluster_sync_all();
    }
    return;
  }
  uint32_t slot = 0, turns = 0;  // place in the ring, and how often it was passed
  for (int64_t row = first_row; row < p.rows; row += row_step) {
  const T* x = static_cast<const T*>(p.logits) + row * p.row_stride;
  // values before the first 16-byte boundary, whole vectors, and the rest
  Part<T> part = part_of(x, p.vocab, rank, ranks);
  const int32_t vocab = static_cast<int32_t>(p.vocab), whole = part.head + (vocab - part.head) / V * V;
  constexpr float low = kLowest<T>;
  Sums acc{low, 0.0f, 0.0f};
  // the given token's logit, long before it is needed
  const int64_t token = p.tokens ? p.tokens[row] : -1;
  const bool given = token >= 0 && token < p.vocab;
  const float logit = given && threadIdx.x == 0 ? El<T>::to_float(x[token]) : 0.0f;

  // the values outside whole vectors: the first and the last CTA of a row
  part.odd = -CUDART_INF_F;
  part.odd_id = -1;
  if (rank == 0 && static_cast<int>(threadIdx.x) < part.head) part.odd_id = threadIdx.x;
  if (rank == ranks - 1 && threadIdx.x >= 32 && static_cast<int>(threadIdx.x) - 32 < vocab - whole) part.odd_id = whole + threadIdx.x - 32;
  if (part.odd_id >= 0) {
    part.odd = El<T>::to_float(x[part.odd_id]);
    const float c = max_nan(part.odd, low);
    const float y = fmaf(c, kLog2e, -reference(c));
    acc.m = c, acc.s = ex2(y), acc.t = acc.s * y;
  }

  float bar = -CUDART_INF_F;  // a value below this is no candidate
  float seen = -CUDART_INF_F; // this thread's largest value
  int turn = 0, queued = 0;   // bars so far; vectors this warp has noted
  uint32_t batch = 0;
  bool gave_up = false;  // a load never came
  for (int32_t at = part.from; at < part.to || batch == 0; at += kUnroll * N, ++batch) {
    uint32_t now[kUnroll][W];
    if (part.from < part.to) {
      if (!wait_batch(&sh.full[slot], turns, &sh.abort, p.wait_limit_ns)) gave_up = true;
      const uint4* vec = reinterpret_cast<const uint4*>(sh.ring[slot]);
      const int32_t left = part.to - at - static_cast<int32_t>(threadIdx.x);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const uint4 q = vec[u * N + threadIdx.x];
        now[u][0] = q.x, now[u][1] = q.y, now[u][2] = q.z, now[u][3] = q.w;
      }
      if (part.to - at < kUnroll * N) {
        // past the end: -infinity, which adds nothing
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (u * N >= left) now[u][0] = now[u][1] = now[u][2] = now[u][3] = kNothing<T>;
      }
      // The copy that fills this place again writes through another proxy: the
      // reads above have to be done for it before the place is given back.
      fence_proxy_async_smem();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.empty[slot]);
      if (++slot == kStages) slot = 0, ++turns;
    } else {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) now[u][0] = now[u][1] = now[u][2] = now[u][3] = kNothing<T>;
    }
    uint32_t high[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) high[u] = word_max<T>(word_max<T>(now[u][0], now[u][1]), word_max<T>(now[u][2], now[u][3]));
#pragma unroll
    for (int step = 1; step < kUnroll; step *= 2)
#pragma unroll
      for (int u = 0; u + step < kUnroll; u += 2 * step) high[u] = word_max<T>(high[u], high[u + step]);
    const float most = word_top<T>(high[0]);
    if (TOP) {
      seen = fmaxf(seen, most);
      if (batch == 0) bar = group_bar(sh.top, seen, p.top, turn++);
      // Later values that only equal the bar come after `top` that reach it.
      // The thread's vectors of this batch are only noted: a warp pays for
      // what any of its threads does, so the values are looked at when all
      // threads have some.
      const bool note = (batch == 0 ? !(most < bar) : !(most <= bar)) && at + static_cast<int32_t>(threadIdx.x) < part.to;
      const uint32_t all = __ballot_sync(0xffffffffu, note);
      if (all) {
        const int place = queued + __popc(all & ((1u << (threadIdx.x & 31)) - 1u));
        if (note && place < kQueue) sh.top.queue[threadIdx.x >> 5][place] = make_int2(at + threadIdx.x, __float_as_int(most));
        queued += __popc(all);
      }
      // raise the bar after 4, 16, 64, ... batches
      if (batch && ((batch + 1) & batch) == 0 && ((batch + 1) & 0x55555555u) && at + kUnroll * N < part.to)
        bar = fmaxf(bar, group_bar(sh.top, seen, p.top, turn++));
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

  if (gave_up) acc.m = __int_as_float(0x7FC00000);
  // the warps' sums, and the last bar, over one barrier
  acc = warp_join(acc, 32);
  if ((threadIdx.x & 31) == 0) sh.warps[threadIdx.x >> 5] = acc;
  if (TOP) {
    if (queued > kQueue) sh.top.lost = 1;
    if (queued > 64) sh.top.flood = 1;
    if (batch > 1) bar = fmaxf(bar, group_bar(sh.top, seen, p.top, turn++));
    else sync_lookers<N>();
  } else {
    sync_lookers<N>();
  }
  int used = 0;  // candidates of the row
  Sums all = warp_join(sh.warps[threadIdx.x % (N / 32)], N / 32);
  if (TOP) {
    if (part.odd_id >= 0 && !(part.odd < bar)) offer_top(sh.top, candidate(bar, 0xFFFFFFFFu), part.odd, part.odd_id);
    open_queue(part, sh.top, queued, bar, p.top);
    sync_lookers<N>();
    used = sh.top.lost ? careful_top(part, sh.top, p.top) : select_top(sh.top, p.top);
  }
  if (ranks > 1) {
    if (threadIdx.x == 0) sh.cta = all;
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
        // at most 8 x 32 candidates of the row's CTAs
        clear_top(sh.top, used);
        sync_lookers<N>();
        if (threadIdx.x < ranks * p.top) {
          const uint32_t a = cluster_map(smem_u32(&sh.top.kept[threadIdx.x % p.top]), threadIdx.x / p.top);
          uint64_t c;
          asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(c) : "r"(a));
          sh.top.waiting[threadIdx.x] = c;
        }
        if (threadIdx.x == 0) sh.top.count = static_cast<int>(ranks) * p.top;
        sync_lookers<N>();
        select_top(sh.top, p.top);
      }
    }
    cluster_sync_all();  // the others' shared memory stays until it was read
    if (rank != 0) return;
  }
  const bool nan_row = all.m != all.m;
  float lse, entropy;
  const bool plain = !nan_row && !(all.m > low + 1024.0f && all.m < -low);
  if (plain) plain_row<T, N>(x, p.vocab, reinterpret_cast<float*>(sh.top.bests), &lse, &entropy);
  if (threadIdx.x < 32) {
    if (nan_row) {
      lse = entropy = __int_as_float(0x7FC00000);
    } else if (!plain) {
      const float l = log2f(all.s);
      lse = (reference(all.m) + l) * kLn2;
      entropy = (l - all.t / all.s) * kLn2;
    }
    write_row(p, row, lse, entropy, logit, given, nan_row, TOP ? sh.top.kept : nullptr);
  }
  if (TOP) clear_top(sh.top, used);
  else if (ranks == 1) sync_lookers<N>();  // before the next row's sums
  }
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

// Many rows of up to this many bytes go to CTAs of 128, of which seven share
// an SM: a row's end is barriers and one warp's work, and less stands idle
// meanwhile (20 alternatives, bf16, cold L2, CTAs of 256 and of 128: 8192 x 1000
// 124 and 57 us, 8192 x 32000 179 and 159 us; longer rows need the larger batch:
// 4096 x 131072 217 and 254 us; and rows that all run at once the more threads:
// 300 x 32000 17.0 and 20.8 us).
constexpr int64_t kShortRow = 65536;

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

// What eg_token_logprobs_set_test_stall set: the limit of a wait (0: the default).
std::atomic<uint64_t> g_limit_ns{0};
std::atomic<int32_t> g_stall{0};

template <typename T, bool TOP, int N>
eg_status launch_score(const ScoreParams& p, int ranks, int dev, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  cudaLaunchConfig_t cfg{};
  auto kernel = score_kernel<T, TOP, N>;
  const eg_status s = host_allow_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(sizeof(RowShared<N>)), dev, &done);
  if (s != EG_OK) return s;
  // four CTAs of 256 an SM take rows in turn (4096 x 131072 bf16, 20
  // alternatives: three with a ring of three batches 233 us, four with two
  // 217 us, two with four 253 us); a cluster takes one
  const int64_t clusters = ranks > 1 ? p.rows : std::min<int64_t>(p.rows, kCtas<N> * sms);
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * ranks));
  cfg.blockDim = dim3(N + 32);
  cfg.dynamicSmemBytes = sizeof(RowShared<N>);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e == cudaSuccess ? EG_OK : host_cuda_fail(e, "launching token_logprobs");
}

template <typename T>
eg_status launch_score(const ScoreParams& p, int ranks, int dev, int sms, cudaStream_t st) {
  const bool small = p.rows > kCtas<256> * sms && p.vocab * static_cast<int64_t>(sizeof(T)) <= kShortRow;
  if (p.top) return small ? launch_score<T, true, 128>(p, ranks, dev, sms, st) : launch_score<T, true, 256>(p, ranks, dev, sms, st);
  return small ? launch_score<T, false, 128>(p, ranks, dev, sms, st) : launch_score<T, false, 256>(p, ranks, dev, sms, st);
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
  int dev = 0, sms = 0;
  if ((s = host_check_device(&dev, &sms)) != EG_OK) return s;
  ScoreParams p{};
  p.rows = a.rows, p.vocab = a.vocab, p.row_stride = a.row_stride;
  p.logits = a.logits, p.tokens = a.tokens;
  p.logprob = a.logprob, p.lse = a.lse, p.entropy = a.entropy;
  p.top = a.top_ids || a.top_logprobs ? a.top : 0;
  p.top_ids = a.top_ids, p.top_logprobs = a.top_logprobs;
  p.wait_limit_ns = g_limit_ns.load(std::memory_order_relaxed), p.stall = g_stall.load(std::memory_order_relaxed);
  if (p.wait_limit_ns == 0) p.wait_limit_ns = host_wait_limit_ns();
  // a cluster for a row while that still leaves every CTA an SM of its own
  // and 16 KB of logits (float32, 50021 of them, five alternatives: 5 rows 13.9
  // us, 17.0 us by one CTA each; 32 rows 15.0 and 17.3 us)
  int ranks = 1;
  while (ranks < 8 && a.rows * ranks * 2 <= sms && a.vocab * el_bytes(a.dtype) / (ranks * 2) >= 16384) ranks *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a.dtype == EG_EL_F32    ? launch_score<float>(p, ranks, dev, sms, st)
         : a.dtype == EG_EL_BF16 ? launch_score<__nv_bfloat16>(p, ranks, dev, sms, st)
                                 : launch_score<__half>(p, ranks, dev, sms, st);
}

eg_status eg_token_logprobs_device_status(void) {
  int dev = 0;
  const eg_status s = host_check_device(&dev);
  if (s != EG_OK) return s;
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return host_cuda_fail(e, "synchronising the current device");
  int32_t status = 0;
  if ((e = cudaMemcpyFromSymbol(&status, g_score_status, 4)) != cudaSuccess) return host_cuda_fail(e, "reading the status of token_logprobs");
  if (status == 0) return EG_OK;
  status = 0;
  e = cudaMemcpyToSymbol(g_score_status, &status, 4);
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);  // later calls may be on streams that do not wait for this one
  if (e != cudaSuccess) return host_cuda_fail(e, "clearing the status of token_logprobs");
  return host_fail(EG_ERR_DEVICE_TIMEOUT, "a wait of the token_logprobs kernel ran past its limit");
}

eg_status eg_token_logprobs_set_test_stall(uint64_t wait_limit_ns, int32_t stall_loader) {
  if (stall_loader != 0 && stall_loader != 1) return host_fail(EG_ERR_INVALID_ARG, "stall_loader must be 0 or 1");
  g_limit_ns.store(wait_limit_ns, std::memory_order_relaxed);
  g_stall.store(stall_loader, std::memory_order_relaxed);
  return EG_OK;
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
  int dev = 0, sms = 0;
  if ((s = host_check_device(&dev, &sms)) != EG_OK) return s;
  GradParams p{};
  p.rows = a.rows, p.vocab = a.vocab, p.row_stride = a.row_stride, p.d_row_stride = g.d_row_stride;
  p.logits = a.logits, p.d_logits = g.d_logits, p.tokens = a.tokens;
  p.lse = g.lse, p.entropy = g.entropy, p.d_logprob = g.d_logprob, p.d_entropy = g.d_entropy;
  // A CTA for each 32 KB of a row, or 16 KB, which is one batch of each thread,
  // where that many CTAs run at once or nearly so (float32, 64, 32, 16 and 8
  // KB: 2048 x 100003 259, 246, 255 and 300 us; 4 x 100003 13.0, 10.4, 8.8 and
  // 8.8 us; one CTA for a row 289 and 33 us)
  const int64_t bytes = a.vocab * el_bytes(a.dtype);
  const int64_t parts = std::max<int64_t>(1, bytes / (a.rows * (bytes / 16384) <= 16 * sms ? 16384 : 32768));
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
