// eg_rope.cu -- per-head norm of queries and keys with the position rotation
// in the same pass, its gradient, and appending keys and values to a paged
// cache (include/eg_decoder.h has the formulas).
//
// All of it is bound by memory: each value is read once and written once.  A
// row (one head of one token) is held in registers by a group of lanes, each
// with two chunks of CH consecutive elements chosen so that both members of
// every rotated pair are in the same lane: with pairs (i, i + rot/2) chunk j
// and the chunk rot/2 elements later, else two neighbouring chunks.  The norm's
// sum is then the only exchange between lanes.  A warp walks the heads of one
// token, so the token's cosines and sines and the weights are read once and
// stay in registers, and it has kBatch rows of every lane group in flight.
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/eg_decoder.h"
#include "eg_el.cuh"
#include "eg_host.h"
#include "eg_ptx.cuh"

namespace eg {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// One call of any of the three entry points.
struct RopeParams {
  int32_t tokens, q_heads, kv_heads, head_dim, rot_dim;
  int32_t lanes;        // lanes of a row's group (power of two, 1..32)
  int32_t groups_q, groups_k, groups_v;  // row groups (32 / lanes rows) of each kind
  int32_t per_warp, parts;  // row groups of one work unit; units of one token
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
  float* partial;       // [CTAs][head_dim] sums of a weight's gradient: of keys for the first key_ctas, then of queries
  int32_t key_ctas, per_warp_k;
};

// Cosine and sine of the pairs one lane holds.  Pairs past rot_dim are not
// rotated: `turns` has a bit for each that is.
template <int CH>
struct Angles {
  float c[CH], s[CH];
  uint32_t turns;
};

template <int CH>
__device__ __forceinline__ void load_angles(const RopeParams& p, int64_t pos, int slot, Angles<CH>& a) {
  const int half = p.rot_dim >> 1;
  a.turns = 0u;
  if (slot * CH >= half) return;
  const bool ok = pos >= 0 && pos < p.max_positions;
  const float* row = p.cos_sin + (ok ? pos : 0) * p.rot_dim;
  const float bad = __int_as_float(0x7FC00000);
  if (p.wide_table && slot * CH + CH <= half) {  // rows and halves on 16-byte boundaries
    a.turns = (1u << CH) - 1u;
#pragma unroll
    for (int i = 0; i < CH; i += 4) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + slot * CH + i)), s = __ldg(reinterpret_cast<const float4*>(row + half + slot * CH + i));
      a.c[i] = c.x, a.c[i + 1] = c.y, a.c[i + 2] = c.z, a.c[i + 3] = c.w;
      a.s[i] = s.x, a.s[i + 1] = s.y, a.s[i + 2] = s.z, a.s[i + 3] = s.w;
    }
    if (!ok)
#pragma unroll
      for (int i = 0; i < CH; ++i) a.c[i] = a.s[i] = bad;
    return;
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int at = slot * CH + i;
    if (at < half) {
      a.turns |= 1u << i;
      a.c[i] = ok ? __ldg(row + at) : bad;
      a.s[i] = ok ? __ldg(row + half + at) : bad;
    }
  }
}
__device__ __forceinline__ int64_t position_of(const RopeParams& p, int token) {
  return p.rot_dim == 0 || !p.positions ? token : __ldg(p.positions + token);
}

// The chunk places of a lane's two chunks.
template <int CH>
__device__ __forceinline__ void chunk_places(const RopeParams& p, bool pairs, int slot, int* e0, int* e1) {
  const int paired = pairs ? 0 : (p.rot_dim >> 1) / CH;  // chunk pairs half a rotation apart
  *e0 = slot < paired ? slot * CH : 2 * slot * CH;
  *e1 = slot < paired ? slot * CH + (p.rot_dim >> 1) : (2 * slot + 1) * CH;
}

// Pair i of a lane: (lo[i], hi[i]) when the halves are apart, else
// neighbours in the 2 CH consecutive values (lo, hi).  DIR 1 turns by the
// angle, -1 back.
template <int CH, bool PAIRS, int DIR>
__device__ __forceinline__ void rotate(float (&lo)[CH], float (&hi)[CH], const Angles<CH>& a) {
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if (!(a.turns >> i & 1u)) continue;
    float& x = PAIRS ? (2 * i < CH ? lo[2 * i < CH ? 2 * i : 0] : hi[2 * i < CH ? 0 : 2 * i - CH]) : lo[i];
    float& y = PAIRS ? (2 * i < CH ? lo[2 * i < CH ? 2 * i + 1 : 0] : hi[2 * i < CH ? 0 : 2 * i + 1 - CH]) : hi[i];
    const float s = DIR > 0 ? a.s[i] : -a.s[i];
    const float u = x * a.c[i] - y * s;
    y = y * a.c[i] + x * s;
    x = u;
  }
}

__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Row groups of one work unit, all in flight at once: four rows of 256 bytes a
// lane group.  The rows' loads go out before the position's and the table's,
// which depend on each other, so a unit waits twice and not three times.
constexpr int kBatch = 4;

template <typename T, int CH, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const RopeParams p) {
  const int lane = threadIdx.x & 31;
  const int rows = 32 / p.lanes;                   // rows of a warp at a time
  const int slot = lane & (p.lanes - 1), sub = lane / p.lanes;
  int e0, e1;
  chunk_places<CH>(p, PAIRS, slot, &e0, &e1);
  const bool on0 = e0 < p.head_dim, on1 = e1 < p.head_dim;
  const int groups = p.groups_q + p.groups_k + p.groups_v;
  const uint32_t units = static_cast<uint32_t>(p.tokens) * p.parts;
  for (uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5); unit < units;
       unit += gridDim.x * kWarps) {
    const int token = unit / p.parts;
    const int first = static_cast<int>(unit % p.parts) * p.per_warp;
    const int last = min(first + p.per_warp, groups);
    Chunk<T, CH> x0[kBatch], x1[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int g = first + b;
      x0[b].zero(), x1[b].zero();
      if (g >= last) continue;
      const int kind = g < p.groups_q ? 0 : g < p.groups_q + p.groups_k ? 1 : 2;
      const int head = (g - (kind == 0 ? 0 : kind == 1 ? p.groups_q : p.groups_q + p.groups_k)) * rows + sub;
      if (head >= (kind == 0 ? p.q_heads : p.kv_heads)) continue;
      const T* src = static_cast<const T*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
                     token * (kind == 0 ? p.q_token : kind == 1 ? p.k_token : p.v_token) +
                     head * (kind == 0 ? p.q_head : kind == 1 ? p.k_head : p.v_head);
      if (on0) x0[b].load(src + e0);
      if (on1) x1[b].load(src + e1);
    }
    Angles<CH> ang;
    ang.turns = 0u;
    if (first < p.groups_q + p.groups_k) load_angles<CH>(p, position_of(p, token), slot, ang);
    int64_t cache_at = -1;
    if (p.slots && last > p.groups_q) {
      const int64_t s = __ldg(p.slots + token);
      if (s >= 0 && s < p.num_slots) {
        const bool small = p.num_slots <= 0x7FFFFFFF;  // a 64-bit division costs a hundred instructions
        const int64_t page = small ? static_cast<int64_t>(static_cast<uint32_t>(s) / static_cast<uint32_t>(p.page_size)) : s / p.page_size;
        cache_at = page * p.page_stride + (s - page * p.page_size) * p.slot_stride;
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int g = first + b;
      if (g >= last) continue;
      const int kind = g < p.groups_q ? 0 : g < p.groups_q + p.groups_k ? 1 : 2;
      const int head = (g - (kind == 0 ? 0 : kind == 1 ? p.groups_q : p.groups_q + p.groups_k)) * rows + sub;
      const bool has = head < (kind == 0 ? p.q_heads : p.kv_heads);
      if (kind < 2) {
        float lo[CH], hi[CH];
        x0[b].get(lo), x1[b].get(hi);
        const T* weight = static_cast<const T*>(kind == 0 ? p.q_weight : p.k_weight);
        if (weight) {
          Chunk<T, CH> w0, w1;
          w0.zero(), w1.zero();
          if (on0) w0.load(weight + e0);
          if (on1) w1.load(weight + e1);
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < CH; ++i) sum += lo[i] * lo[i] + hi[i] * hi[i];
          const float r = rsqrtf(group_sum(sum, p.lanes) * p.inv_dim + p.eps);
          float f0[CH], f1[CH];
          w0.get(f0), w1.get(f1);
#pragma unroll
          for (int i = 0; i < CH; ++i) lo[i] = lo[i] * r * f0[i], hi[i] = hi[i] * r * f1[i];
        }
        rotate<CH, PAIRS, 1>(lo, hi, ang);
        x0[b].set(lo), x1[b].set(hi);
      }
      T* dst;
      bool put = has;
      if (kind == 0) {
        dst = static_cast<T*>(p.q_out) + token * p.qo_token + head * p.qo_head;
      } else if (p.slots) {
        put = put && cache_at >= 0;
        dst = static_cast<T*>(kind == 1 ? p.k_cache : p.v_cache) + cache_at + head * p.cache_head;
      } else {
        dst = static_cast<T*>(p.k_out) + token * p.ko_token + head * p.ko_head;
      }
      if (put && on0) x0[b].store(dst + e0);
      if (put && on1) x1[b].store(dst + e1);
    }
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

// A warp has units of queries or of keys for its whole life, so one set of sums.
constexpr int kGradRows = 2;  // rows of a lane group in flight, each with its gradient

template <typename T, int CH, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 2) rope_backward_kernel(const RopeParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = 32 / p.lanes;
  const int slot = lane & (p.lanes - 1), sub = lane / p.lanes;
  int e0, e1;
  chunk_places<CH>(p, PAIRS, slot, &e0, &e1);
  const bool on0 = e0 < p.head_dim, on1 = e1 < p.head_dim;
  // the first key_ctas CTAs have the keys
  const bool keys = static_cast<int>(blockIdx.x) < p.key_ctas;
  const int ctas = keys ? p.key_ctas : gridDim.x - p.key_ctas, cta = keys ? blockIdx.x : blockIdx.x - p.key_ctas;
  const int heads = keys ? p.kv_heads : p.q_heads, groups = keys ? p.groups_k : p.groups_q;
  const T* weight = static_cast<const T*>(keys ? p.k_weight : p.q_weight);
  const T* xs = static_cast<const T*>(keys ? p.k : p.q);
  const T* ys = static_cast<const T*>(keys ? p.k_out : p.q_out);
  T* ds = static_cast<T*>(keys ? p.dk : p.dq);
  const int64_t x_token = keys ? p.k_token : p.q_token, x_head = keys ? p.k_head : p.q_head;
  const int64_t y_token = keys ? p.ko_token : p.qo_token, y_head = keys ? p.ko_head : p.qo_head;
  const int64_t d_token = keys ? p.dk_token : p.dq_token, d_head = keys ? p.dk_head : p.dq_head;
  float sums[2 * CH];
#pragma unroll
  for (int i = 0; i < 2 * CH; ++i) sums[i] = 0.0f;
  // all groups of a token, or for few tokens a part of them
  const int per_unit = keys ? p.per_warp_k : p.per_warp;
  const int parts = (groups + per_unit - 1) / per_unit;
  const uint32_t units = static_cast<uint32_t>(p.tokens) * parts, step = ctas * kWarps;
  uint32_t unit = cta * kWarps + warp;
  int64_t next_pos = unit < units ? position_of(p, unit / parts) : 0;
  for (; unit < units; unit += step) {
    const int token = unit / parts, from = static_cast<int>(unit % parts) * per_unit, to = min(from + per_unit, groups);
    Angles<CH> ang;
    const int64_t pos = next_pos;
    if (unit + step < units) next_pos = position_of(p, (unit + step) / parts);
    for (int g0 = from; g0 < to; g0 += kGradRows) {
      Chunk<T, CH> x0[kGradRows], x1[kGradRows], y0[kGradRows], y1[kGradRows];
#pragma unroll
      for (int b = 0; b < kGradRows; ++b) {
        const int head = (g0 + b) * rows + sub;
        x0[b].zero(), x1[b].zero(), y0[b].zero(), y1[b].zero();
        if (g0 + b >= to || head >= heads) continue;
        const T* y = ys + token * y_token + head * y_head;
        if (on0) y0[b].load(y + e0);
        if (on1) y1[b].load(y + e1);
        if (weight) {
          const T* x = xs + token * x_token + head * x_head;
          if (on0) x0[b].load(x + e0);
          if (on1) x1[b].load(x + e1);
        }
      }
      if (g0 == from) load_angles<CH>(p, pos, slot, ang);
#pragma unroll
      for (int b = 0; b < kGradRows; ++b) {
        if (g0 + b >= to) continue;
        const int head = (g0 + b) * rows + sub;
        float lo[CH], hi[CH];
        y0[b].get(lo), y1[b].get(hi);
        rotate<CH, PAIRS, -1>(lo, hi, ang);
        if (weight) {
          float h0[CH], h1[CH], f0[CH], f1[CH];
          x0[b].get(h0), x1[b].get(h1);
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < CH; ++i) sum += h0[i] * h0[i] + h1[i] * h1[i];
          float r = rsqrtf(group_sum(sum, p.lanes) * p.inv_dim + p.eps);
          // a lane group past the last head holds zeros and adds none
          if (head >= heads) r = 0.0f;
          Chunk<T, CH> w0, w1;
          w0.zero(), w1.zero();
          if (on0) w0.load(weight + e0);
          if (on1) w1.load(weight + e1);
          w0.get(f0), w1.get(f1);
          float dot = 0.0f;
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            h0[i] *= r, h1[i] *= r;
            sums[i] += lo[i] * h0[i];
            sums[CH + i] += hi[i] * h1[i];
            lo[i] *= f0[i], hi[i] *= f1[i];
            dot += lo[i] * h0[i] + hi[i] * h1[i];
          }
          const float mean = group_sum(dot, p.lanes) * p.inv_dim;
#pragma unroll
          for (int i = 0; i < CH; ++i) lo[i] = r * (lo[i] - h0[i] * mean), hi[i] = r * (hi[i] - h1[i] * mean);
        }
        if (head >= heads) continue;
        y0[b].set(lo), y1[b].set(hi);
        T* d = ds + token * d_token + head * d_head;
        if (on0) y0[b].store(d + e0);
        if (on1) y1[b].store(d + e1);
      }
    }
  }
  if (!p.partial) return;
  // over the warp's lane groups, then over the warps
  __shared__ float shared[kWarps][256 + 32];
#pragma unroll
  for (int i = 0; i < 2 * CH; ++i) {
    float v = sums[i];
    for (int o = p.lanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int e = i < CH ? e0 + i : e1 + i - CH;
    if (sub == 0 && e < p.head_dim) shared[warp][e] = v;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.head_dim; e += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += shared[w][e];
    p.partial[static_cast<int64_t>(blockIdx.x) * p.head_dim + e] = v;
  }
}

// The gradient for any head_dim, stride and alignment: one warp a row.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_backward_any_kernel(const RopeParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int half = p.rot_dim >> 1;
  const bool pairs = p.lanes != 0;
  const bool kind = static_cast<int>(blockIdx.x) < p.key_ctas;
  const int ctas = kind ? p.key_ctas : gridDim.x - p.key_ctas, cta = kind ? blockIdx.x : blockIdx.x - p.key_ctas;
  const int heads = kind ? p.kv_heads : p.q_heads;
  float sums[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[i] = 0.0f;
  const int64_t units = static_cast<int64_t>(p.tokens) * heads;
  for (int64_t unit = static_cast<int64_t>(cta) * kWarps + warp; unit < units; unit += static_cast<int64_t>(ctas) * kWarps) {
    const int token = static_cast<int>(unit / heads);
    const int head = static_cast<int>(unit % heads);
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
        sums[i] += g[i] * h[i];
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
  __shared__ float shared[kWarps][256];
#pragma unroll
  for (int i = 0; i < 8; ++i) shared[warp][lane + 32 * i] = sums[i];
  __syncthreads();
  for (int e = threadIdx.x; e < p.head_dim; e += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += shared[w][e];
    p.partial[static_cast<int64_t>(blockIdx.x) * p.head_dim + e] = v;
  }
}

// dw[e] = sum over the CTAs that have queries (or keys) of their sums: one CTA
// for 32 elements of one weight, each warp a fixed share of the rows.
__global__ void __launch_bounds__(1024) rope_weight_kernel(const float* partial, int ctas, int key_ctas, int head_dim,
                                                           float* dq_weight, float* dk_weight) {
  griddep_wait();
  __shared__ float shared[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int column = blockIdx.x * 32 + lane;
  const bool keys = blockIdx.y != 0;
  const int from = keys ? 0 : key_ctas, to = keys ? key_ctas : ctas;
  float* out = keys ? dk_weight : dq_weight;
  if (!out) return;
  float v = 0.0f;
  if (column < head_dim)
#pragma unroll 8
    for (int c = from + warp; c < to; c += 32) v += partial[static_cast<int64_t>(c) * head_dim + column];
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

#define EG_TRY(call)              \
  do {                            \
    eg_status s_ = (call);        \
    if (s_ != EG_OK) return s_;   \
  } while (0)

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
// starts at is a multiple of its size, and pairs do not straddle lanes.
bool chunks_fit(const eg_rope_args& a, int ch, std::initializer_list<const void*> ptrs,
                std::initializer_list<int64_t> strides) {
  if (a.head_dim % ch) return false;
  if (!a.pairs && (a.rot_dim / 2) % ch) return false;
  const uintptr_t bytes = static_cast<uintptr_t>(ch * el_bytes(a.dtype));
  for (const void* x : ptrs)
    if (reinterpret_cast<uintptr_t>(x) % bytes) return false;
  for (int64_t s : strides)
    if (s % ch) return false;
  return true;
}

// Lanes of a row's group, row groups, and the units of a token: `kBatch`
// groups each.
void plan_rows(RopeParams* p, int ch, bool append) {
  const int slots = (p->head_dim / ch + 1) / 2;
  p->lanes = 1;
  while (p->lanes < slots) p->lanes *= 2;
  const int rows = 32 / p->lanes;
  p->groups_q = (p->q_heads + rows - 1) / rows;
  p->groups_k = (p->kv_heads + rows - 1) / rows;
  p->groups_v = append ? p->groups_k : 0;
  const int groups = p->groups_q + p->groups_k + p->groups_v;
  p->parts = std::max(1, (groups + kBatch - 1) / kBatch);
  p->per_warp = std::max(1, (groups + p->parts - 1) / p->parts);
  p->parts = std::max(1, (groups + p->per_warp - 1) / p->per_warp);
  p->wide_table = ch % 4 == 0 && p->rot_dim % 8 == 0 && reinterpret_cast<uintptr_t>(p->cos_sin) % 16 == 0;
}

// The gradient's units: all row groups of a token, or where there are few
// tokens for the warps a part of them (at least what is in flight at once).
int grad_groups(int64_t tokens, int groups, int warps) {
  if (groups == 0) return 1;
  const int64_t parts = tokens ? std::max<int64_t>(1, warps / tokens) : 1;
  return static_cast<int>(std::max<int64_t>(kGradRows, (groups + parts - 1) / parts));
}

template <typename T, int CH>
void launch_rows(const RopeParams& p, bool pairs, int grid, cudaStream_t st) {
  if (pairs) rope_kernel<T, CH, true><<<grid, kThreads, 0, st>>>(p);
  else rope_kernel<T, CH, false><<<grid, kThreads, 0, st>>>(p);
}

template <typename T, int CH>
void launch_backward(const RopeParams& p, bool pairs, int grid, cudaStream_t st) {
  if (pairs) rope_backward_kernel<T, CH, true><<<grid, kThreads, 0, st>>>(p);
  else rope_backward_kernel<T, CH, false><<<grid, kThreads, 0, st>>>(p);
}

eg_status forward(const eg_rope_args& a, RopeParams p, int ch, bool append, int sms, cudaStream_t st) {
  if (ch) {
    plan_rows(&p, ch, append);
    const int64_t ctas = (static_cast<int64_t>(p.tokens) * p.parts + kWarps - 1) / kWarps;
    const int grid = static_cast<int>(std::min<int64_t>(ctas, 1 << 20));
    if (a.dtype == EG_EL_F32) launch_rows<float, 4>(p, a.pairs, grid, st);
    else if (a.dtype == EG_EL_BF16 && ch == 8) launch_rows<__nv_bfloat16, 8>(p, a.pairs, grid, st);
    else if (a.dtype == EG_EL_BF16) launch_rows<__nv_bfloat16, 4>(p, a.pairs, grid, st);
    else if (ch == 8) launch_rows<__half, 8>(p, a.pairs, grid, st);
    else launch_rows<__half, 4>(p, a.pairs, grid, st);
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

// CTAs of the gradient kernels (each leaves one row of partial sums) and how
// many of them have keys: as the heads are divided.
int backward_ctas(const eg_rope_args& a, int sms, int* key_ctas) {
  const int64_t rows = a.tokens * (a.q_heads + a.kv_heads);
  int ctas = static_cast<int>(std::max<int64_t>(2, std::min<int64_t>((rows + kWarps - 1) / kWarps, sms * 2)));
  const int heads = a.q_heads + a.kv_heads;
  int keys = heads ? static_cast<int>((static_cast<int64_t>(ctas) * a.kv_heads + heads / 2) / heads) : 1;
  *key_ctas = std::min(ctas - 1, std::max(1, keys));
  return ctas;
}

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
  int dev = 0, sms = 0, key_ctas = 0;
  EG_TRY(host_check_device(&dev, &sms));
  *out = (fwd->q_weight || fwd->k_weight) ? static_cast<size_t>(backward_ctas(*fwd, sms, &key_ctas)) * fwd->head_dim * 4 : 0;
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
  int key_ctas = 0;
  const int ctas = backward_ctas(a, sms, &key_ctas);
  if (dqw || dkw) {
    if (!d.workspace || reinterpret_cast<uintptr_t>(d.workspace) % 16)
      return host_fail(EG_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned");
    if (d.workspace_bytes < static_cast<size_t>(ctas) * a.head_dim * 4)
      return host_fail(EG_ERR_INVALID_ARG, "workspace holds %zu bytes of %zu", d.workspace_bytes,
                       static_cast<size_t>(ctas) * a.head_dim * 4);
  }
  RopeParams p = base_params(a);
  p.dq = d.dq, p.dk = d.dk;
  p.dq_token = d.dq_token, p.dq_head = d.dq_head, p.dk_token = d.dk_token, p.dk_head = d.dk_head;
  p.key_ctas = key_ctas;
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
    plan_rows(&p, ch, false);
    p.per_warp = grad_groups(a.tokens, p.groups_q, (ctas - key_ctas) * kWarps);
    p.per_warp_k = grad_groups(a.tokens, p.groups_k, key_ctas * kWarps);
    if (a.dtype == EG_EL_F32) launch_backward<float, 4>(p, a.pairs, ctas, st);
    else if (a.dtype == EG_EL_BF16 && ch == 8) launch_backward<__nv_bfloat16, 8>(p, a.pairs, ctas, st);
    else if (a.dtype == EG_EL_BF16) launch_backward<__nv_bfloat16, 4>(p, a.pairs, ctas, st);
    else if (ch == 8) launch_backward<__half, 8>(p, a.pairs, ctas, st);
    else launch_backward<__half, 4>(p, a.pairs, ctas, st);
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
    e = cudaLaunchKernelEx(&cfg, rope_weight_kernel, static_cast<const float*>(p.partial), ctas, key_ctas, static_cast<int>(a.head_dim), dqw, dkw);
    if (e != cudaSuccess) return host_cuda_fail(e, "launching the sum of the weights' gradients");
  }
  return EG_OK;
}

}  // extern "C"
