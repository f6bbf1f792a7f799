// eg_rope.cu -- per-head norm of queries and keys with the position rotation
// in the same pass, its gradient, and appending keys and values to a paged
// cache (include/eg_decoder.h has the formulas).
//
// Each value is read once and written once.  In succession, bf16, 32 + 8 heads
// of 128: 8191 tokens forward 37 us (4.7 TB/s, much of it in L2), 16384 tokens'
// gradient 96 us (5.3 TB/s); fp16, 24593 tokens appended 96 us (6.4 TB/s of the
// 6.8 that a copy reaches, its bound).  Forward and gradient are bound by
// latency before that: with 16 warps an SM and one token's rows in flight in
// each, neither DRAM (42 and 62 %) nor the issue slots (57 and 64 %; some 330
// instructions for 512 values) are full.
//
// A row (one head of one token) is held in registers by a group of lanes, each
// with two chunks of CH consecutive elements chosen so that both members of
// every rotated pair are in the same lane: with pairs (i, i + rot/2) chunk j
// and the chunk rot/2 elements later, else any two; lanes lie side by side in
// both.  The norm's sum is then the only exchange between lanes.  A warp has
// the same heads of one kind (queries, keys or values) for its whole life and
// walks the tokens: addresses step and weights stay in registers.  The next
// token's rows and angles come in by asynchronous copies to shared memory while
// this one's are worked on; a lane copies what it will read itself, so the rows
// need no barrier.
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/eg_decoder.h"
#include "eg_el.cuh"
#include "eg_host.h"
#include "eg_ptx.cuh"

namespace eg {

namespace {

#define EG_TRY(call)              \
  do {                            \
    eg_status s_ = (call);        \
    if (s_ != EG_OK) return s_;   \
  } while (0)

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// One call of any of the three entry points.
struct RopeParams {
  int32_t tokens, q_heads, kv_heads, head_dim, rot_dim;
  int32_t lanes;        // lanes of a row's group (power of two, 1..32)
  int32_t parts, parts_q, parts_k;  // the warps of one token, of its queries and of its keys
  int32_t wide_table;   // the table can be read in 16-byte vectors
  float eps, inv_dim;
  const float* cos_sin;
  int64_t max_positions;
  const int64_t* positions;
  const void *q_weight, *k_weight;
  const void *q, *k, *v;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  void *q_out, *k_out;  // backward: the given gradients (read only)
  int64_t qo_token, qo_head, ko_token, ko_head;
  // append
  const int64_t* slots;
  void *k_cache, *v_cache;
  int64_t num_slots, page_stride, slot_stride, cache_head;
  int32_t page_size;
  // backward
  void *dq, *dk;
  int64_t dq_token, dq_head, dk_token, dk_head;
  float* partial;       // [CTAs][2][head_dim] sums of the weights' gradients
};

// Cosines and sines of the pairs one lane holds, two in a register.  With pairs
// (i, i + rot/2) they serve both chunks, and both are rotated or neither is;
// with neighbouring pairs the first half serves the first chunk.
template <int CH>
struct Angles {
  pk_t c[CH / 2], s[CH / 2];
};

// 8 or 16 bytes to shared memory, in the background.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  static_assert(BYTES == 8 || BYTES == 16, "one chunk");
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// What one warp has in flight for one token: `N` chunks of every lane, and the
// table's row, cosines then sines.
template <typename T, int CH, int N>
struct Stage {
  static constexpr int kChunk = CH * static_cast<int>(sizeof(T));
  uint8_t* at;
  int lane;

  __device__ __forceinline__ void* chunk(int i) const { return at + (i * 32 + lane) * kChunk; }
  __device__ __forceinline__ float* table() const { return reinterpret_cast<float*>(at + N * 32 * kChunk); }
  __device__ __forceinline__ void copy(int i, const T* from) const { copy_async<kChunk>(chunk(i), from); }
  __device__ __forceinline__ Chunk<T, CH> read(int i) const {
    Chunk<T, CH> c;
    c.load(static_cast<const T*>(chunk(i)));
    return c;
  }
  static __host__ __device__ int bytes(int rot_dim) { return N * 32 * kChunk + (rot_dim * 4 + 15) / 16 * 16; }
};

// Where a lane's angles are in the table's row: CH of them from `a0` on, or
// CH / 2 from `a0` and from `a1`; t0, t1: whether its chunks are rotated.
struct AnglePlace {
  int a0, a1;
  bool t0, t1;
  template <int CH, bool PAIRS>
  static __device__ __forceinline__ AnglePlace of(const RopeParams& p, int slot, int e0, int e1) {
    if constexpr (PAIRS) return {e0 / 2, e1 / 2, e0 < p.rot_dim, e1 < p.rot_dim};
    const bool t = slot * CH < (p.rot_dim >> 1);
    return {slot * CH, slot * CH + CH / 2, t, t};
  }
};

// Ask for the table's row (for a position outside it: of position 0, not used).
// The lanes of the first group copy it for all.
template <int CH>
__device__ __forceinline__ void copy_angles(const RopeParams& p, int64_t pos, const AnglePlace& at, float* to) {
  const bool ok = pos >= 0 && pos < p.max_positions;
  const int half = p.rot_dim >> 1;
  const float* row = p.cos_sin + (ok ? pos : 0) * p.rot_dim;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!(k ? at.t1 : at.t0)) continue;
    const int a = k ? at.a1 : at.a0;
    if (p.wide_table) {  // rows and halves on boundaries of CH / 2 floats
      copy_async<CH * 2>(to + a, row + a), copy_async<CH * 2>(to + half + a, row + half + a);
    } else {
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) to[a + i] = __ldg(row + a + i), to[half + a + i] = __ldg(row + half + a + i);
    }
  }
}

template <int CH>
__device__ __forceinline__ void read_angles(const RopeParams& p, int64_t pos, const AnglePlace& at, const float* from, Angles<CH>& a) {
  const int half = p.rot_dim >> 1;
  if (p.wide_table) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!(k ? at.t1 : at.t0)) continue;
      const float* c = from + (k ? at.a1 : at.a0);
#pragma unroll
      for (int i = 0; i < CH / 2; i += 4) {
        if constexpr (CH == 8) {
          const float4 u = *reinterpret_cast<const float4*>(c), v = *reinterpret_cast<const float4*>(c + half);
          a.c[2 * k] = pk(u.x, u.y), a.c[2 * k + 1] = pk(u.z, u.w);
          a.s[2 * k] = pk(v.x, v.y), a.s[2 * k + 1] = pk(v.z, v.w);
        } else {
          a.c[k] = *reinterpret_cast<const float2*>(c);
          a.s[k] = *reinterpret_cast<const float2*>(c + half);
        }
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!(k ? at.t1 : at.t0)) continue;
      const int e = k ? at.a1 : at.a0;
#pragma unroll
      for (int i = 0; i < CH / 2; i += 2) {
        a.c[k * (CH / 4) + i / 2] = pk(from[e + i], from[e + i + 1]);
        a.s[k * (CH / 4) + i / 2] = pk(from[half + e + i], from[half + e + i + 1]);
      }
    }
  }
  if (pos < 0 || pos >= p.max_positions) {
    const float bad = __int_as_float(0x7FC00000);
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) a.c[i] = a.s[i] = pk(bad, bad);
  }
}
__device__ __forceinline__ int64_t position_of(const RopeParams& p, int token) {
  return p.rot_dim == 0 || !p.positions ? token : __ldg(p.positions + token);
}

// The chunk places of a lane's two chunks.
template <int CH>
__device__ __forceinline__ void chunk_places(const RopeParams& p, bool pairs, int slot, int* e0, int* e1) {
  if (pairs) {
    *e0 = slot * CH, *e1 = (slot + (p.head_dim / CH + 1) / 2) * CH;
    if (*e1 - *e0 <= slot * CH) *e0 = p.head_dim;  // past the lanes that have any
    return;
  }
  const int paired = (p.rot_dim >> 1) / CH;  // chunk pairs half a rotation apart
  *e0 = slot < paired ? slot * CH : 2 * slot * CH;
  *e1 = slot < paired ? slot * CH + (p.rot_dim >> 1) : (2 * slot + 1) * CH;
}

__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Row groups of one work unit: two of 512 elements (8191 tokens of 32 + 8 heads of
// 128 in bf16, cold L2: two 40 us, four 58 us; a third CTA an SM spills, 82 us).
constexpr int kBatch = 2;

// The factors of one lane for one token: y_a = r (x_a ca + x_b sb) and
// y_b = r (x_b cb + x_a sa), the weight and the sine's sign multiplied into
// each.  With
// neighbouring pairs (PAIRS) a register holds both members: y = r (x c + x' s)
// with x' the members exchanged and the sine's sign in s.
template <int CH, bool PAIRS>
struct Turn {
  pk_t c0[CH / 2], c1[CH / 2], s0[CH / 2], s1[CH / 2];

  __device__ __forceinline__ void form(const Angles<CH>& a, const pk_t (&w0)[CH / 2], const pk_t (&w1)[CH / 2], const AnglePlace& at) {
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) c0[i] = w0[i], c1[i] = w1[i];
    if (at.t0) {
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) {
        if constexpr (PAIRS) {
          // the members of pair i of the first chunk
          const float2 c = unpk(a.c[i / 2]), s = unpk(a.s[i / 2]);
          const float c_ = i & 1 ? c.y : c.x, s_ = i & 1 ? s.y : s.x;
          c0[i] = pk_mul(w0[i], pk(c_, c_)), s0[i] = pk_mul(pk_swap(w0[i]), pk(-s_, s_));
        } else {
          c0[i] = pk_mul(w0[i], a.c[i]), s0[i] = pk_mul(w0[i], a.s[i]);
          c1[i] = pk_mul(w1[i], a.c[i]), s1[i] = pk_mul(pk_mul(w1[i], a.s[i]), pk(-1.0f, -1.0f));
        }
      }
    }
    if constexpr (PAIRS) {
      if (at.t1)
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
          const float2 c = unpk(a.c[CH / 4 + i / 2]), s = unpk(a.s[CH / 4 + i / 2]);
          const float c_ = i & 1 ? c.y : c.x, s_ = i & 1 ? s.y : s.x;
          c1[i] = pk_mul(w1[i], pk(c_, c_)), s1[i] = pk_mul(pk_swap(w1[i]), pk(-s_, s_));
        }
    }
  }
  // (x0, x1) of a lane times the weight and turned, without the factor r; a
  // chunk that is not rotated has only its weight in c
  __device__ __forceinline__ void apply(pk_t (&x0)[CH / 2], pk_t (&x1)[CH / 2], const AnglePlace& at) const {
    if constexpr (PAIRS) {
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) {
        if (at.t0) x0[i] = pk_fma(x0[i], c0[i], pk_mul(pk_swap(x0[i]), s0[i]));
        else x0[i] = pk_mul(x0[i], c0[i]);
        if (at.t1) x1[i] = pk_fma(x1[i], c1[i], pk_mul(pk_swap(x1[i]), s1[i]));
        else x1[i] = pk_mul(x1[i], c1[i]);
      }
    } else if (at.t0) {
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) {
        const pk_t a = x0[i], b = x1[i];
        x0[i] = pk_fma(a, c0[i], pk_mul(b, s1[i]));
        x1[i] = pk_fma(b, c1[i], pk_mul(a, s0[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) x0[i] = pk_mul(x0[i], c0[i]), x1[i] = pk_mul(x1[i], c1[i]);
    }
  }
};

// What a warp does for its whole life: a kind of rows (0 queries, 1 keys, 2
// values) and `count` of their row groups from `group0` on, of every `step`-th
// token.
struct Task {
  int kind, group0;
  uint32_t token, step;
  __device__ __forceinline__ Task(const RopeParams& p, uint32_t warp, uint32_t warps, int per_part) {
    step = warps / p.parts;
    token = warp / p.parts;
    const int part = warp % p.parts;
    kind = part < p.parts_q ? 0 : part < p.parts_q + p.parts_k ? 1 : 2;
    group0 = (part - (kind == 0 ? 0 : kind == 1 ? p.parts_q : p.parts_q + p.parts_k)) * per_part;
    if (token >= step) token = 0xFFFFFFFFu;  // no whole token's warps are left
  }
};

template <typename T, int CH, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 2) rope_kernel(const RopeParams p) {
  using St = Stage<T, CH, 2 * kBatch>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = 32 / p.lanes;                   // rows of a warp at a time
  const int slot = lane & (p.lanes - 1), sub = lane / p.lanes;
  int e0, e1;
  chunk_places<CH>(p, PAIRS, slot, &e0, &e1);
  const bool on0 = e0 < p.head_dim, on1 = e1 < p.head_dim;
  Task task(p, blockIdx.x * kWarps + warp, gridDim.x * kWarps, kBatch);
  const int kind = task.kind;
  const uint32_t tokens = p.tokens;
  uint32_t token = task.token;
  const int heads = kind == 0 ? p.q_heads : p.kv_heads, head0 = task.group0 * rows + sub;
  const int64_t src_token = kind == 0 ? p.q_token : kind == 1 ? p.k_token : p.v_token, src_head = kind == 0 ? p.q_head : kind == 1 ? p.k_head : p.v_head;
  const bool cached = kind > 0 && p.slots;
  const int64_t dst_token = kind == 0 ? p.qo_token : p.ko_token, dst_head = kind == 0 ? p.qo_head : cached ? p.cache_head : p.ko_head;
  const T* src = static_cast<const T*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) + head0 * src_head;
  T* dst = static_cast<T*>(kind == 0 ? p.q_out : !p.slots ? p.k_out : kind == 1 ? p.k_cache : p.v_cache) + head0 * dst_head;
  const T* weight = static_cast<const T*>(kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr);
  Chunk<T, CH> w0, w1;
  w0.zero(), w1.zero();
  if (weight && on0) w0.load(weight + e0);
  if (weight && on1) w1.load(weight + e1);
  if (!weight) {
    pk_t one[CH / 2];
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) one[i] = pk(1.0f, 1.0f);
    w0.set(one), w1.set(one);
  }
  AnglePlace place = AnglePlace::of<CH, PAIRS>(p, slot, e0, e1);
  if (kind == 2) place.t0 = place.t1 = false;
  const bool works = kind < 2 && (weight || p.rot_dim > 0);  // else the rows are copied
  const int stage_bytes = St::bytes(p.rot_dim);
  St now{smem + (warp * 2) * stage_bytes, lane}, next{now.at + stage_bytes, lane};
  // ask for one token's rows and its angles
  auto ask = [&](const St& st, uint32_t t, int64_t pos) {
    const T* row = src + static_cast<int64_t>(t) * src_token;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (head0 + b * rows >= heads) continue;
      if (on0) st.copy(2 * b, row + b * rows * src_head + e0);
      if (on1) st.copy(2 * b + 1, row + b * rows * src_head + e1);
    }
    if (sub == 0) copy_angles<CH>(p, pos, place, st.table());
  };
  auto slot_of = [&](uint32_t t) { return cached ? __ldg(p.slots + t) : 0; };
  int64_t pos = 0, next_pos = 0, at = 0, next_at = 0;  // positions and cache slots of this token and the next
  if (token < tokens) {
    pos = kind < 2 ? position_of(p, token) : 0, at = slot_of(token);
    ask(now, token, pos);
  }
  cp_async_commit();
  if (static_cast<uint64_t>(token) + task.step < tokens) next_pos = kind < 2 ? position_of(p, token + task.step) : 0, next_at = slot_of(token + task.step);
  for (; token < tokens; token += task.step) {
    const uint32_t after = token + task.step;
    __syncwarp();  // the other stage's angles have been read
    if (after < tokens) ask(next, after, next_pos);
    cp_async_commit();
    const int64_t its_pos = pos, its_at = at;
    pos = next_pos, at = next_at;
    if (after + task.step < tokens) next_pos = kind < 2 ? position_of(p, after + task.step) : 0, next_at = slot_of(after + task.step);
    cp_async_wait<1>();
    __syncwarp();  // the first group's lanes have the angles for all
    T* to = dst + (cached ? 0 : token * dst_token);
    bool put = true;
    if (cached) {
      put = its_at >= 0 && its_at < p.num_slots;
      const bool small = p.num_slots <= 0x7FFFFFFF;  // a 64-bit division costs a hundred instructions
      const int64_t page = small ? static_cast<int64_t>(static_cast<uint32_t>(its_at) / static_cast<uint32_t>(p.page_size)) : its_at / p.page_size;
      to += page * p.page_stride + (its_at - page * p.page_size) * p.slot_stride;
    }
    Turn<CH, PAIRS> turn;
    if (works) {
      Angles<CH> ang;
      read_angles<CH>(p, its_pos, place, now.table(), ang);
      pk_t f0[CH / 2], f1[CH / 2];
      w0.get(f0), w1.get(f1);
      turn.form(ang, f0, f1, place);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (head0 - sub + b * rows >= heads) continue;  // the warp has no row of this group
      const bool has = head0 + b * rows < heads;
      Chunk<T, CH> x0, x1;
      x0.zero(), x1.zero();
      if (has && on0) x0 = now.read(2 * b);
      if (has && on1) x1 = now.read(2 * b + 1);
      if (works) {
        pk_t lo[CH / 2], hi[CH / 2];
        x0.get(lo), x1.get(hi);
        float r = 1.0f;
        if (weight) {
          pk_t sum = pk(0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < CH / 2; ++i) sum = pk_fma(lo[i], lo[i], sum), sum = pk_fma(hi[i], hi[i], sum);
          r = rsqrtf(group_sum(pk_sum(sum), p.lanes) * p.inv_dim + p.eps);
        }
        turn.apply(lo, hi, place);
        if (weight) {
          const pk_t r2 = pk(r, r);
#pragma unroll
          for (int i = 0; i < CH / 2; ++i) lo[i] = pk_mul(lo[i], r2), hi[i] = pk_mul(hi[i], r2);
        }
        x0.set(lo), x1.set(hi);
      }
      if (put && has && on0) x0.store(to + b * rows * dst_head + e0);
      if (put && has && on1) x1.store(to + b * rows * dst_head + e1);
    }
    const St t = now;
    now = next, next = t;
  }
}

// Any head_dim, rotation, stride and alignment: one warp for each row, one
// element of each 32 a lane; the other member of a pair is read (and normed)
// again, which the L1 cache serves.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_any_kernel(const RopeParams p) {
  const int lane = threadIdx.x & 31;
  const int heads = p.q_heads + p.kv_heads * (p.v_cache ? 2 : 1);
  const int half = p.rot_dim >> 1;
  const bool pairs = p.lanes != 0;  // this kernel's own use of the field
  const int64_t units = static_cast<int64_t>(p.tokens) * heads;
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); unit < units;
       unit += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int token = static_cast<int>(unit / heads);
    int head = static_cast<int>(unit % heads);
    const int kind = head < p.q_heads ? 0 : head < p.q_heads + p.kv_heads ? 1 : 2;
    head -= kind == 0 ? 0 : kind == 1 ? p.q_heads : p.q_heads + p.kv_heads;
    const T* src = static_cast<const T*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
                   token * (kind == 0 ? p.q_token : kind == 1 ? p.k_token : p.v_token) +
                   head * (kind == 0 ? p.q_head : kind == 1 ? p.k_head : p.v_head);
    T* dst;
    if (kind == 0) {
      dst = static_cast<T*>(p.q_out) + token * p.qo_token + head * p.qo_head;
    } else if (p.slots) {
      const int64_t s = p.slots[token];
      if (s < 0 || s >= p.num_slots) continue;
      dst = static_cast<T*>(kind == 1 ? p.k_cache : p.v_cache) + s / p.page_size * p.page_stride +
            s % p.page_size * p.slot_stride + head * p.cache_head;
    } else {
      dst = static_cast<T*>(p.k_out) + token * p.ko_token + head * p.ko_head;
    }
    const T* weight = static_cast<const T*>(kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr);
    float r = 1.0f;
    if (weight) {
      float sum = 0.0f;
      for (int e = lane; e < p.head_dim; e += 32) {
        const float x = El<T>::to_float(src[e]);
        sum += x * x;
      }
      r = rsqrtf(group_sum(sum, 32) * p.inv_dim + p.eps);
    }
    const int64_t pos = p.positions ? p.positions[token] : token;
    const bool ok = pos >= 0 && pos < p.max_positions;
    const float* row = p.cos_sin + (ok ? pos : 0) * p.rot_dim;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      if (e >= p.head_dim) continue;
      float z = El<T>::to_float(src[e]);
      if (weight) z = z * r * El<T>::to_float(weight[e]);
      if (kind < 2 && e < p.rot_dim) {
        const int at = pairs ? e >> 1 : e < half ? e : e - half;
        const bool second = pairs ? (e & 1) != 0 : e >= half;
        const int o = pairs ? e ^ 1 : second ? e - half : e + half;
        float other = El<T>::to_float(src[o]);
        if (weight) other = other * r * El<T>::to_float(weight[o]);
        const float c = ok ? row[at] : __int_as_float(0x7FC00000), s = ok ? row[half + at] : c;
        z = second ? z * c + other * s : z * c - other * s;
      }
      y[i] = z;
    }
    __syncwarp();  // the row is read before it is written in place
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      if (e < p.head_dim) dst[e] = El<T>::from_float(y[i]);
    }
  }
}

// --------------------------------------------------------------- gradient --
//
// With dy the gradient of the output, dz = dy turned back, h = x r, g = dz w:
//   dx = r (g - h mean(g h)),  dw = sum over tokens and heads of dz h.
// A lane keeps the sums of its own elements in registers over all its rows;
// they are joined over the warp's lane groups, over the CTA's warps, and (by
// the second kernel) over the CTAs, each in a fixed order.

constexpr int kGradRows = 2;  // row groups of one work unit, each with its gradient

// A lane's gradients turned back: (a c + b s, b c - a s).
template <int CH, bool PAIRS>
__device__ __forceinline__ void turn_back(pk_t (&x0)[CH / 2], pk_t (&x1)[CH / 2], const Angles<CH>& a, const AnglePlace& at) {
  const pk_t minus = pk(-1.0f, -1.0f);
#pragma unroll
  for (int i = 0; i < CH / 2; ++i) {
    if constexpr (PAIRS) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (!(k ? at.t1 : at.t0)) continue;
        const float2 c = unpk(a.c[k * (CH / 4) + i / 2]), s = unpk(a.s[k * (CH / 4) + i / 2]);
        const float c_ = i & 1 ? c.y : c.x, s_ = i & 1 ? s.y : s.x;
        pk_t& x = k ? x1[i] : x0[i];
        x = pk_fma(x, pk(c_, c_), pk_mul(pk_swap(x), pk(s_, -s_)));
      }
    } else if (at.t0) {
      const pk_t u = x0[i], v = x1[i];
      x0[i] = pk_fma(u, a.c[i], pk_mul(v, a.s[i]));
      x1[i] = pk_fma(v, a.c[i], pk_mul(pk_mul(u, minus), a.s[i]));
    }
  }
}

template <typename T, int CH, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 2) rope_backward_kernel(const RopeParams p) {
  using St = Stage<T, CH, 4 * kGradRows>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = 32 / p.lanes;
  const int slot = lane & (p.lanes - 1), sub = lane / p.lanes;
  int e0, e1;
  chunk_places<CH>(p, PAIRS, slot, &e0, &e1);
  const bool on0 = e0 < p.head_dim, on1 = e1 < p.head_dim;
  Task task(p, blockIdx.x * kWarps + warp, gridDim.x * kWarps, kGradRows);
  const bool keys = task.kind != 0;
  const uint32_t tokens = p.tokens;
  uint32_t token = task.token;
  const int heads = keys ? p.kv_heads : p.q_heads, head0 = task.group0 * rows + sub;
  const T* weight = static_cast<const T*>(keys ? p.k_weight : p.q_weight);
  const int64_t x_token = keys ? p.k_token : p.q_token, x_head = keys ? p.k_head : p.q_head;
  const int64_t y_token = keys ? p.ko_token : p.qo_token, y_head = keys ? p.ko_head : p.qo_head;
  const int64_t d_token = keys ? p.dk_token : p.dq_token, d_head = keys ? p.dk_head : p.dq_head;
  const T* xs = static_cast<const T*>(keys ? p.k : p.q) + head0 * x_head;
  const T* ys = static_cast<const T*>(keys ? p.k_out : p.q_out) + head0 * y_head;
  T* ds = static_cast<T*>(keys ? p.dk : p.dq) + head0 * d_head;
  pk_t sums[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) sums[i] = pk(0.0f, 0.0f);
  Chunk<T, CH> w0, w1;
  w0.zero(), w1.zero();
  if (weight && on0) w0.load(weight + e0);
  if (weight && on1) w1.load(weight + e1);
  const AnglePlace place = AnglePlace::of<CH, PAIRS>(p, slot, e0, e1);
  const int stage_bytes = St::bytes(p.rot_dim);
  St now{smem + (warp * 2) * stage_bytes, lane}, next{now.at + stage_bytes, lane};
  auto ask = [&](const St& st, uint32_t t, int64_t pos) {
    const T* y = ys + static_cast<int64_t>(t) * y_token;
    const T* x = xs + static_cast<int64_t>(t) * x_token;
#pragma unroll
    for (int b = 0; b < kGradRows; ++b) {
      if (head0 + b * rows >= heads) continue;
      if (on0) st.copy(4 * b, y + b * rows * y_head + e0);
      if (on1) st.copy(4 * b + 1, y + b * rows * y_head + e1);
      if (weight && on0) st.copy(4 * b + 2, x + b * rows * x_head + e0);
      if (weight && on1) st.copy(4 * b + 3, x + b * rows * x_head + e1);
    }
    if (sub == 0) copy_angles<CH>(p, pos, place, st.table());
  };
  int64_t pos = 0, next_pos = 0;
  if (token < tokens) {
    pos = position_of(p, token);
    ask(now, token, pos);
  }
  cp_async_commit();
  if (static_cast<uint64_t>(token) + task.step < tokens) next_pos = position_of(p, token + task.step);
  for (; token < tokens; token += task.step) {
    const uint32_t after = token + task.step;
    __syncwarp();  // the other stage's angles have been read
    if (after < tokens) ask(next, after, next_pos);
    cp_async_commit();
    const int64_t its_pos = pos;
    pos = next_pos;
    if (after + task.step < tokens) next_pos = position_of(p, after + task.step);
    cp_async_wait<1>();
    __syncwarp();  // the first group's lanes have the angles for all
    Angles<CH> ang;
    read_angles<CH>(p, its_pos, place, now.table(), ang);
#pragma unroll
    for (int b = 0; b < kGradRows; ++b) {
      if (head0 - sub + b * rows >= heads) continue;  // the warp has no row of this group
      const bool has = head0 + b * rows < heads;
      Chunk<T, CH> y0, y1, x0, x1;
      y0.zero(), y1.zero(), x0.zero(), x1.zero();
      if (has && on0) y0 = now.read(4 * b);
      if (has && on1) y1 = now.read(4 * b + 1);
      pk_t lo[CH / 2], hi[CH / 2];
      y0.get(lo), y1.get(hi);
      turn_back<CH, PAIRS>(lo, hi, ang, place);
      if (weight) {
        if (has && on0) x0 = now.read(4 * b + 2);
        if (has && on1) x1 = now.read(4 * b + 3);
        pk_t h0[CH / 2], h1[CH / 2], f0[CH / 2], f1[CH / 2], sum = pk(0.0f, 0.0f);
        x0.get(h0), x1.get(h1);
        w0.get(f0), w1.get(f1);
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) sum = pk_fma(h0[i], h0[i], sum), sum = pk_fma(h1[i], h1[i], sum);
        float r = rsqrtf(group_sum(pk_sum(sum), p.lanes) * p.inv_dim + p.eps);
        // a lane group past the last head holds zeros and adds none
        if (!has) r = 0.0f;
        const pk_t r2 = pk(r, r);
        pk_t dot = pk(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
          h0[i] = pk_mul(h0[i], r2), h1[i] = pk_mul(h1[i], r2);
          sums[i] = pk_fma(lo[i], h0[i], sums[i]);
          sums[CH / 2 + i] = pk_fma(hi[i], h1[i], sums[CH / 2 + i]);
          lo[i] = pk_mul(lo[i], f0[i]), hi[i] = pk_mul(hi[i], f1[i]);
          dot = pk_fma(lo[i], h0[i], dot), dot = pk_fma(hi[i], h1[i], dot);
        }
        const float mean = -group_sum(pk_sum(dot), p.lanes) * p.inv_dim;
        const pk_t mean2 = pk(mean, mean);
#pragma unroll
        for (int i = 0; i < CH / 2; ++i)
          lo[i] = pk_mul(r2, pk_fma(h0[i], mean2, lo[i])), hi[i] = pk_mul(r2, pk_fma(h1[i], mean2, hi[i]));
      }
      y0.set(lo), y1.set(hi);
      T* d = ds + static_cast<int64_t>(token) * d_token + b * rows * d_head;
      if (has && on0) y0.store(d + e0);
      if (has && on1) y1.store(d + e1);
    }
    const St t = now;
    now = next, next = t;
  }
  if (!p.partial) return;
  // over the warp's lane groups, then over the CTA's warps of either kind
  cp_async_wait<0>();
  __syncthreads();
  float(*shared)[256 + 32] = reinterpret_cast<float(*)[256 + 32]>(smem);
#pragma unroll
  for (int i = 0; i < 2 * CH; ++i) {
    const float2 two = unpk(sums[i / 2]);
    float v = i & 1 ? two.y : two.x;
    for (int o = p.lanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int e = i < CH ? e0 + i : e1 + i - CH;
    if (sub == 0 && e < p.head_dim) shared[warp][e] = v;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.head_dim; i += kThreads) {
    const int kind = i >= p.head_dim, e = i - kind * p.head_dim;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const bool its = static_cast<int>((blockIdx.x * kWarps + w) % p.parts) >= p.parts_q;
      if (its == (kind != 0)) v += shared[w][e];
    }
    p.partial[(static_cast<int64_t>(blockIdx.x) * 2 + kind) * p.head_dim + e] = v;
  }
}

// The gradient for any head_dim, stride and alignment: one warp a row.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_backward_any_kernel(const RopeParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int half = p.rot_dim >> 1;
  const bool pairs = p.lanes != 0;
  const int heads = p.q_heads + p.kv_heads;
  float sums[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[0][i] = sums[1][i] = 0.0f;
  const int64_t units = static_cast<int64_t>(p.tokens) * heads;
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp; unit < units; unit += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int token = static_cast<int>(unit / heads);
    const int at_head = static_cast<int>(unit % heads);
    const bool kind = at_head >= p.q_heads;
    const int head = at_head - (kind ? p.q_heads : 0);
    const T* x = static_cast<const T*>(kind ? p.k : p.q) + token * (kind ? p.k_token : p.q_token) + head * (kind ? p.k_head : p.q_head);
    const T* dy = static_cast<const T*>(kind ? p.k_out : p.q_out) + token * (kind ? p.ko_token : p.qo_token) +
                  head * (kind ? p.ko_head : p.qo_head);
    T* dx = static_cast<T*>(kind ? p.dk : p.dq) + token * (kind ? p.dk_token : p.dq_token) + head * (kind ? p.dk_head : p.dq_head);
    const T* weight = static_cast<const T*>(kind ? p.k_weight : p.q_weight);
    const int64_t pos = p.positions ? p.positions[token] : token;
    const bool ok = pos >= 0 && pos < p.max_positions;
    const float* row = p.cos_sin + (ok ? pos : 0) * p.rot_dim;
    float g[8], h[8], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      g[i] = h[i] = 0.0f;
      if (e >= p.head_dim) continue;
      g[i] = El<T>::to_float(dy[e]);
      if (e < p.rot_dim) {
        const int at = pairs ? e >> 1 : e < half ? e : e - half;
        const bool second = pairs ? (e & 1) != 0 : e >= half;
        const float other = El<T>::to_float(dy[pairs ? e ^ 1 : second ? e - half : e + half]);
        const float c = ok ? row[at] : __int_as_float(0x7FC00000), s = ok ? row[half + at] : c;
        g[i] = second ? g[i] * c - other * s : g[i] * c + other * s;
      }
      if (weight) h[i] = El<T>::to_float(x[e]);
      sum += h[i] * h[i];
    }
    if (weight) {
      const float r = rsqrtf(group_sum(sum, 32) * p.inv_dim + p.eps);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = lane + 32 * i;
        if (e >= p.head_dim) continue;
        h[i] *= r;
        if (kind) sums[1][i] += g[i] * h[i];
        else sums[0][i] += g[i] * h[i];
        g[i] *= El<T>::to_float(weight[e]);
        dot += g[i] * h[i];
      }
      const float mean = group_sum(dot, 32) * p.inv_dim;
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = r * (g[i] - h[i] * mean);
    }
    __syncwarp();  // the row is read before it is written in place
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      if (e < p.head_dim) dx[e] = El<T>::from_float(g[i]);
    }
  }
  if (!p.partial) return;
  __shared__ float shared[kWarps][2][256];
#pragma unroll
  for (int i = 0; i < 8; ++i) shared[warp][0][lane + 32 * i] = sums[0][i], shared[warp][1][lane + 32 * i] = sums[1][i];
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.head_dim; i += kThreads) {
    const int kind = i >= p.head_dim, e = i - kind * p.head_dim;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += shared[w][kind][e];
    p.partial[(static_cast<int64_t>(blockIdx.x) * 2 + kind) * p.head_dim + e] = v;
  }
}

// dw[e] = sum over the CTAs of their sums of one kind: one CTA for 32 elements
// of one weight, each warp a fixed share of the rows.
__global__ void __launch_bounds__(1024) rope_weight_kernel(const float* partial, int ctas, int head_dim, float* dq_weight,
                                                           float* dk_weight) {
  griddep_wait();
  __shared__ float shared[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int column = blockIdx.x * 32 + lane, kind = blockIdx.y;
  float* out = kind ? dk_weight : dq_weight;
  if (!out) return;
  float v = 0.0f;
  if (column < head_dim)
#pragma unroll 8
    for (int c = warp; c < ctas; c += 32) v += partial[(static_cast<int64_t>(c) * 2 + kind) * head_dim + column];
  shared[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && column < head_dim) {
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < 32; ++w) v += shared[w][lane];
    out[column] = v;
  }
}

// ------------------------------------------------------------------- host --

int el_bytes(int dtype) { return dtype == EG_EL_F32 ? 4 : 2; }

eg_status check_rows(const char* name, const void* ptr, int64_t token, int64_t head, int heads, int64_t tokens,
                     const eg_rope_args& a) {
  if (heads == 0 || tokens == 0) return EG_OK;
  if (!ptr) return host_fail(EG_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(ptr) % el_bytes(a.dtype))
    return host_fail(EG_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
  if (token < 0 || head < 0) return host_fail(EG_ERR_INVALID_ARG, "%s has a negative stride", name);
  return EG_OK;
}

eg_status check_args(const eg_rope_args* a) {
  if (!a) return host_fail(EG_ERR_INVALID_ARG, "args is NULL");
  if (a->tokens < 0 || a->q_heads < 0 || a->kv_heads < 0)
    return host_fail(EG_ERR_INVALID_ARG, "negative size (tokens=%lld q_heads=%d kv_heads=%d)", (long long)a->tokens,
                     a->q_heads, a->kv_heads);
  if (a->dtype != EG_EL_BF16 && a->dtype != EG_EL_F16 && a->dtype != EG_EL_F32)
    return host_fail(EG_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
  if (a->head_dim < 2 || a->head_dim > 256 || a->head_dim % 2)
    return host_fail(EG_ERR_UNSUPPORTED, "head_dim must be even and in 2..256 (got %d)", a->head_dim);
  if (a->rot_dim < 0 || a->rot_dim > a->head_dim || a->rot_dim % 2)
    return host_fail(EG_ERR_INVALID_ARG, "rot_dim must be even and in 0..head_dim (got %d)", a->rot_dim);
  if (a->pairs != 0 && a->pairs != 1) return host_fail(EG_ERR_INVALID_ARG, "pairs must be 0 or 1");
  if (a->tokens > (1 << 24) || a->q_heads > 1024 || a->kv_heads > 1024)
    return host_fail(EG_ERR_UNSUPPORTED, "at most 2^24 tokens and 1024 heads a call");
  if (a->rot_dim > 0 && a->tokens > 0) {
    if (!a->cos_sin) return host_fail(EG_ERR_INVALID_ARG, "cos_sin is NULL");
    if (reinterpret_cast<uintptr_t>(a->cos_sin) % 4)
      return host_fail(EG_ERR_INVALID_ARG, "cos_sin is not aligned to its elements");
    if (a->max_positions < 1) return host_fail(EG_ERR_INVALID_ARG, "max_positions must be positive");
  }
  if (reinterpret_cast<uintptr_t>(a->positions) % 8)
    return host_fail(EG_ERR_INVALID_ARG, "positions are not aligned to their elements");
  if ((a->q_weight || a->k_weight) && !(a->eps >= 0.0f))
    return host_fail(EG_ERR_INVALID_ARG, "eps must not be negative");
  for (const void* w : {a->q_weight, a->k_weight})
    if (reinterpret_cast<uintptr_t>(w) % el_bytes(a->dtype))
      return host_fail(EG_ERR_INVALID_ARG, "a weight is not aligned to its elements");
  return EG_OK;
}

RopeParams base_params(const eg_rope_args& a) {
  RopeParams p{};
  p.tokens = static_cast<int32_t>(a.tokens);
  p.q_heads = a.q_heads, p.kv_heads = a.kv_heads, p.head_dim = a.head_dim, p.rot_dim = a.rot_dim;
  p.eps = a.eps, p.inv_dim = 1.0f / static_cast<float>(a.head_dim);
  p.cos_sin = a.cos_sin, p.max_positions = a.max_positions, p.positions = a.positions;
  p.q_weight = a.q_weight, p.k_weight = a.k_weight;
  p.q = a.q, p.k = a.k, p.v = a.v;
  p.q_token = a.q_token, p.q_head = a.q_head, p.k_token = a.k_token, p.k_head = a.k_head;
  p.v_token = a.v_token, p.v_head = a.v_head;
  p.q_out = a.q_out, p.k_out = a.k_out;
  p.qo_token = a.qo_token, p.qo_head = a.qo_head, p.ko_token = a.ko_token, p.ko_head = a.ko_head;
  p.page_size = 1;
  return p;
}

// Whether chunks of `ch` elements serve this call: every address a chunk
// starts at is a multiple of its size, and a lane's pairs are all rotated or
// none.  8 where they do (float32: 4, the same 16 bytes), else 4, else single
// elements: the three take 40, 55 and 244 us for 8191 tokens of 32 + 8 heads of
// 128 in bf16, and 110, 137 and 1103 us for 16384 tokens' gradient (cold L2).
bool chunks_fit(const eg_rope_args& a, int ch, std::initializer_list<const void*> ptrs,
                std::initializer_list<int64_t> strides) {
  if (a.head_dim % ch) return false;
  if ((a.rot_dim / 2) % ch) return false;
  const uintptr_t bytes = static_cast<uintptr_t>(ch * el_bytes(a.dtype));
  for (const void* x : ptrs)
    if (reinterpret_cast<uintptr_t>(x) % bytes) return false;
  for (int64_t s : strides)
    if (s % ch) return false;
  return true;
}

// Lanes of a row's group, and the warps of a token: `per_part` row groups of
// one kind each.
void plan_rows(RopeParams* p, int ch, int per_part, bool append) {
  const int slots = (p->head_dim / ch + 1) / 2;
  p->lanes = 1;
  while (p->lanes < slots) p->lanes *= 2;
  const int rows = per_part * (32 / p->lanes);
  p->parts_q = (p->q_heads + rows - 1) / rows;
  p->parts_k = (p->kv_heads + rows - 1) / rows;
  p->parts = p->parts_q + p->parts_k * (append ? 2 : 1);
  // a lane's angles come in copies of ch / 2 floats
  p->wide_table = (p->rot_dim / 2) % (ch / 2) == 0 && reinterpret_cast<uintptr_t>(p->cos_sin) % (ch * 2) == 0;
}

// CTAs for every warp of every token, at most what the SMs hold at once, at
// least the warps of one token.
int grid_of(const RopeParams& p, int most) {
  const int64_t ctas = (static_cast<int64_t>(p.tokens) * p.parts + kWarps - 1) / kWarps;
  return static_cast<int>(std::max<int64_t>(std::min<int64_t>(ctas, most), (p.parts + kWarps - 1) / kWarps));
}

// Launch with the kernel's dynamic shared memory: two stages a warp.
template <typename Kernel>
eg_status launch_staged(Kernel kernel, const RopeParams& p, int grid, int stage_bytes, std::atomic<uint64_t>* done, cudaStream_t st) {
  const int bytes = std::max(kWarps * 2 * stage_bytes, kWarps * 288 * 4);  // the gradient's sums reuse it
  if (bytes > 48 * 1024) {
    int dev = 0;
    EG_TRY(host_check_device(&dev));
    EG_TRY(host_allow_smem(reinterpret_cast<const void*>(kernel), 2 * kWarps * (8 * 32 * 16 + 1024), dev, done));
  }
  kernel<<<grid, kThreads, bytes, st>>>(p);
  return EG_OK;
}

template <typename T, int CH, bool PAIRS>
eg_status launch_rows(const RopeParams& p, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  return launch_staged(rope_kernel<T, CH, PAIRS>, p, grid, Stage<T, CH, 2 * kBatch>::bytes(p.rot_dim), &done, st);
}
template <typename T, int CH, bool PAIRS>
eg_status launch_backward(const RopeParams& p, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  return launch_staged(rope_backward_kernel<T, CH, PAIRS>, p, grid, Stage<T, CH, 4 * kGradRows>::bytes(p.rot_dim), &done, st);
}
template <typename T, int CH>
eg_status launch_rows(const RopeParams& p, bool pairs, int grid, cudaStream_t st) {
  return pairs ? launch_rows<T, CH, true>(p, grid, st) : launch_rows<T, CH, false>(p, grid, st);
}
template <typename T, int CH>
eg_status launch_backward(const RopeParams& p, bool pairs, int grid, cudaStream_t st) {
  return pairs ? launch_backward<T, CH, true>(p, grid, st) : launch_backward<T, CH, false>(p, grid, st);
}

eg_status forward(const eg_rope_args& a, RopeParams p, int ch, bool append, int sms, cudaStream_t st) {
  if (ch) {
    plan_rows(&p, ch, kBatch, append);
    const int grid = grid_of(p, sms * 2);
    if (a.dtype == EG_EL_F32) EG_TRY((launch_rows<float, 4>(p, a.pairs, grid, st)));
    else if (a.dtype == EG_EL_BF16 && ch == 8) EG_TRY((launch_rows<__nv_bfloat16, 8>(p, a.pairs, grid, st)));
    else if (a.dtype == EG_EL_BF16) EG_TRY((launch_rows<__nv_bfloat16, 4>(p, a.pairs, grid, st)));
    else if (ch == 8) EG_TRY((launch_rows<__half, 8>(p, a.pairs, grid, st)));
    else EG_TRY((launch_rows<__half, 4>(p, a.pairs, grid, st)));
  } else {
    p.lanes = a.pairs;
    const int64_t rows = static_cast<int64_t>(p.tokens) * (p.q_heads + p.kv_heads * (append ? 2 : 1));
    const int grid = static_cast<int>(std::min<int64_t>((rows + kWarps - 1) / kWarps, sms * 8));
    if (a.dtype == EG_EL_F32) rope_any_kernel<float><<<grid, kThreads, 0, st>>>(p);
    else if (a.dtype == EG_EL_BF16) rope_any_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(p);
    else rope_any_kernel<__half><<<grid, kThreads, 0, st>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? EG_OK : host_cuda_fail(e, append ? "launching kv_append" : "launching qk_norm_rope");
}

// Most CTAs of the gradient kernels: each leaves a row of sums of both kinds.
int backward_ctas(int sms) { return sms * 2; }

}  // namespace
}  // namespace eg

using namespace eg;

extern "C" {

eg_status eg_qk_norm_rope(const eg_rope_args* args, void* stream) {
  EG_TRY(check_args(args));
  const eg_rope_args& a = *args;
  EG_TRY(check_rows("q", a.q, a.q_token, a.q_head, a.q_heads, a.tokens, a));
  EG_TRY(check_rows("q_out", a.q_out, a.qo_token, a.qo_head, a.q_heads, a.tokens, a));
  EG_TRY(check_rows("k", a.k, a.k_token, a.k_head, a.kv_heads, a.tokens, a));
  EG_TRY(check_rows("k_out", a.k_out, a.ko_token, a.ko_head, a.kv_heads, a.tokens, a));
  if (a.tokens == 0 || a.q_heads + a.kv_heads == 0) return EG_OK;
  int dev = 0, sms = 0;
  EG_TRY(host_check_device(&dev, &sms));
  int ch = 0;
  for (int c : {8, 4}) {
    if (ch || (c == 8 && a.dtype == EG_EL_F32)) continue;
    const int64_t on = a.q_heads ? 1 : 0, kon = a.kv_heads ? 1 : 0;
    if (chunks_fit(a, c, {on ? a.q : nullptr, on ? a.q_out : nullptr, kon ? a.k : nullptr, kon ? a.k_out : nullptr, a.q_weight, a.k_weight},
                   {on * a.q_token, on * a.q_head, on * a.qo_token, on * a.qo_head, kon * a.k_token, kon * a.k_head,
                    kon * a.ko_token, kon * a.ko_head}))
      ch = c;
  }
  return forward(a, base_params(a), ch, false, sms, static_cast<cudaStream_t>(stream));
}

eg_status eg_kv_append(const eg_rope_args* args, const eg_kv_cache* cache, const int64_t* slots, void* stream) {
  EG_TRY(check_args(args));
  eg_rope_args a = *args;
  if (!cache) return host_fail(EG_ERR_INVALID_ARG, "cache is NULL");
  if (!a.q) a.q_heads = 0;
  EG_TRY(check_rows("q", a.q, a.q_token, a.q_head, a.q_heads, a.tokens, a));
  EG_TRY(check_rows("q_out", a.q_out, a.qo_token, a.qo_head, a.q_heads, a.tokens, a));
  EG_TRY(check_rows("k", a.k, a.k_token, a.k_head, a.kv_heads, a.tokens, a));
  EG_TRY(check_rows("v", a.v, a.v_token, a.v_head, a.kv_heads, a.tokens, a));
  if (a.page_size < 1) return host_fail(EG_ERR_INVALID_ARG, "page_size must be positive");
  if (cache->num_pages < 0 || cache->page_stride < 0 || cache->token_stride < 0 || cache->head_stride < 0)
    return host_fail(EG_ERR_INVALID_ARG, "negative page count or stride of the cache");
  if (a.tokens == 0 || a.q_heads + a.kv_heads == 0) return EG_OK;
  if (a.kv_heads && (!cache->k || !cache->v)) return host_fail(EG_ERR_INVALID_ARG, "the cache is NULL");
  if (a.kv_heads && (reinterpret_cast<uintptr_t>(cache->k) % el_bytes(a.dtype) ||
                     reinterpret_cast<uintptr_t>(cache->v) % el_bytes(a.dtype)))
    return host_fail(EG_ERR_INVALID_ARG, "the cache is not aligned to its elements");
  if (!slots) return host_fail(EG_ERR_INVALID_ARG, "slots is NULL");
  if (reinterpret_cast<uintptr_t>(slots) % 8)
    return host_fail(EG_ERR_INVALID_ARG, "slots are not aligned to their elements");
  int dev = 0, sms = 0;
  EG_TRY(host_check_device(&dev, &sms));
  RopeParams p = base_params(a);
  p.q_heads = a.q_heads;
  p.slots = slots;
  p.k_cache = cache->k, p.v_cache = cache->v;
  p.page_size = a.page_size;
  p.num_slots = cache->num_pages * a.page_size;
  p.page_stride = cache->page_stride, p.slot_stride = cache->token_stride, p.cache_head = cache->head_stride;
  int ch = 0;
  for (int c : {8, 4}) {
    if (ch || (c == 8 && a.dtype == EG_EL_F32)) continue;
    const int64_t on = a.q_heads ? 1 : 0, kon = a.kv_heads ? 1 : 0;
    if (chunks_fit(a, c, {on ? a.q : nullptr, on ? a.q_out : nullptr, kon ? a.k : nullptr, kon ? a.v : nullptr,
                          kon ? cache->k : nullptr, kon ? cache->v : nullptr, a.q_weight, a.k_weight},
                   {on * a.q_token, on * a.q_head, on * a.qo_token, on * a.qo_head, kon * a.k_token, kon * a.k_head,
                    kon * a.v_token, kon * a.v_head, cache->page_stride, cache->token_stride, cache->head_stride}))
      ch = c;
  }
  return forward(a, p, ch, true, sms, static_cast<cudaStream_t>(stream));
}

eg_status eg_qk_norm_rope_workspace_bytes(const eg_rope_args* fwd, size_t* out) {
  EG_TRY(check_args(fwd));
  if (!out) return host_fail(EG_ERR_INVALID_ARG, "out is NULL");
  int dev = 0, sms = 0;
  EG_TRY(host_check_device(&dev, &sms));
  *out = (fwd->q_weight || fwd->k_weight) ? static_cast<size_t>(backward_ctas(sms)) * 2 * fwd->head_dim * 4 : 0;
  return EG_OK;
}

eg_status eg_qk_norm_rope_backward(const eg_rope_args* fwd, const eg_rope_grads* grads, void* stream) {
  EG_TRY(check_args(fwd));
  if (!grads) return host_fail(EG_ERR_INVALID_ARG, "grads is NULL");
  const eg_rope_args& a = *fwd;
  const eg_rope_grads& d = *grads;
  EG_TRY(check_rows("the given gradient of q_out", a.q_out, a.qo_token, a.qo_head, a.q_heads, a.tokens, a));
  EG_TRY(check_rows("the given gradient of k_out", a.k_out, a.ko_token, a.ko_head, a.kv_heads, a.tokens, a));
  if (a.q_weight) EG_TRY(check_rows("q", a.q, a.q_token, a.q_head, a.q_heads, a.tokens, a));
  if (a.k_weight) EG_TRY(check_rows("k", a.k, a.k_token, a.k_head, a.kv_heads, a.tokens, a));
  EG_TRY(check_rows("dq", d.dq, d.dq_token, d.dq_head, a.q_heads, a.tokens, a));
  EG_TRY(check_rows("dk", d.dk, d.dk_token, d.dk_head, a.kv_heads, a.tokens, a));
  for (const float* w : {d.dq_weight, d.dk_weight})
    if (reinterpret_cast<uintptr_t>(w) % 4) return host_fail(EG_ERR_INVALID_ARG, "a weight's gradient is not aligned to its elements");
  float* dqw = a.q_weight ? d.dq_weight : nullptr;
  float* dkw = a.k_weight ? d.dk_weight : nullptr;
  int dev = 0, sms = 0;
  EG_TRY(host_check_device(&dev, &sms));
  int ctas = backward_ctas(sms);
  if (dqw || dkw) {
    if (!d.workspace || reinterpret_cast<uintptr_t>(d.workspace) % 16)
      return host_fail(EG_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned");
    if (d.workspace_bytes < static_cast<size_t>(ctas) * 2 * a.head_dim * 4)
      return host_fail(EG_ERR_INVALID_ARG, "workspace holds %zu bytes of %zu", d.workspace_bytes,
                       static_cast<size_t>(ctas) * 2 * a.head_dim * 4);
  }
  RopeParams p = base_params(a);
  p.dq = d.dq, p.dk = d.dk;
  p.dq_token = d.dq_token, p.dq_head = d.dq_head, p.dk_token = d.dk_token, p.dk_head = d.dk_head;
  p.partial = dqw || dkw ? static_cast<float*>(d.workspace) : nullptr;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t on = a.q_heads ? 1 : 0, kon = a.kv_heads ? 1 : 0;
  int ch = 0;
  for (int c : {8, 4}) {
    if (ch || (c == 8 && a.dtype == EG_EL_F32)) continue;
    const int64_t xq = a.q_weight ? on : 0, xk = a.k_weight ? kon : 0;
    if (chunks_fit(a, c, {xq ? a.q : nullptr, on ? a.q_out : nullptr, on ? d.dq : nullptr, xk ? a.k : nullptr,
                          kon ? a.k_out : nullptr, kon ? d.dk : nullptr, a.q_weight, a.k_weight},
                   {xq * a.q_token, xq * a.q_head, on * a.qo_token, on * a.qo_head, on * d.dq_token, on * d.dq_head,
                    xk * a.k_token, xk * a.k_head, kon * a.ko_token, kon * a.ko_head, kon * d.dk_token, kon * d.dk_head}))
      ch = c;
  }
  if (ch) {
    plan_rows(&p, ch, kGradRows, false);
    if (p.parts == 0) p.parts = 1;  // no heads: the weights' gradients are zero
    ctas = std::min(ctas, grid_of(p, ctas));
    if (a.dtype == EG_EL_F32) EG_TRY((launch_backward<float, 4>(p, a.pairs, ctas, st)));
    else if (a.dtype == EG_EL_BF16 && ch == 8) EG_TRY((launch_backward<__nv_bfloat16, 8>(p, a.pairs, ctas, st)));
    else if (a.dtype == EG_EL_BF16) EG_TRY((launch_backward<__nv_bfloat16, 4>(p, a.pairs, ctas, st)));
    else if (ch == 8) EG_TRY((launch_backward<__half, 8>(p, a.pairs, ctas, st)));
    else EG_TRY((launch_backward<__half, 4>(p, a.pairs, ctas, st)));
  } else {
    p.lanes = a.pairs;
    if (a.dtype == EG_EL_F32) rope_backward_any_kernel<float><<<ctas, kThreads, 0, st>>>(p);
    else if (a.dtype == EG_EL_BF16) rope_backward_any_kernel<__nv_bfloat16><<<ctas, kThreads, 0, st>>>(p);
    else rope_backward_any_kernel<__half><<<ctas, kThreads, 0, st>>>(p);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return host_cuda_fail(e, "launching the gradient of qk_norm_rope");
  if (dqw || dkw) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((a.head_dim + 31) / 32), 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, rope_weight_kernel, static_cast<const float*>(p.partial), ctas, static_cast<int>(a.head_dim), dqw, dkw);
    if (e != cudaSuccess) return host_cuda_fail(e, "launching the sum of the weights' gradients");
  }
  return EG_OK;
}

}  // extern "C"
