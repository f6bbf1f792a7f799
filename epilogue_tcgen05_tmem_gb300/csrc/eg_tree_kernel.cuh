// eg_tree_kernel.cuh -- attention of drafted token trees over a paged cache.
//
// Mathematics.  The rows of one item are the n tokens of a sequence's tree
// times the G query heads that share a cached head: for key tiles of 128,
//   S = Q K^T,  P = 2^(c S - m),  O += P V,  l += rowsum P,
// with c = scale log2 e and m a row reference at least the row maximum less 8:
// O and l are only brought to a new reference when the maximum grew by more
// than 2^8, which few tiles do.  Weights are rounded to 16 bits for the second
// product, whose operands are: at most 2^-8 (bf16) or 2^-11 (fp16) of each
// weight, the output type's own rounding, which makes the error against 64 bits
// up to 1.4 times that of weights in float32.  l sums them before that
// rounding, in float32 as S, O and m are.
//
// Work.  Every item has units for its key tiles (see kTreeFixed); all items'
// units in a row are cut into equal ranges, one for each CTA (one CTA an SM),
// on the device from the sequences' lengths.  An item that a cut divides leaves
// float32 partial results that its last CTA or a second small kernel joins in a
// fixed order, so equal inputs give equal bits.
//
// One CTA: a producer warp (TMA boxes of pages into a ring of 128-key tiles,
// K and V alike), one issuing thread (tcgen05.mma), two softmax warpgroups, a
// warp that fetches queries and one that walks the range for the softmax
// warpgroups (who spill registers when they do it: 4 % slower in the wide case below).  S and
// O of both warpgroups fill tensor memory (4 x 128 columns); P overwrites S as
// 16-bit values and feeds the second product from there.  With at most 128 rows
// the warpgroups take turns on the key tiles and are joined at the end of the
// range; with more rows each has 128 of them and K and V tiles are used twice.
// So while one warpgroup forms weights the tensor cores work for the other.
//
// Measured in succession, and what bounds it.  Two sequences of 98304 and
// 131072 places, 32 query heads over 8 cached, one token each: 151 us, 6.2 TB/s
// of the 6.8 that a copy reaches; CTAs get uneven shares of the bandwidth, and
// the last decides.
// 24 sequences of up to 13 tokens and 9001 places: 97 us, 4.3 TB/s; a CTA has
// 2.1 segments, and each costs some 4 us beside its tiles.  16 sequences of 32
// to 64 tokens, 64 query heads, 3800 to 8200 places: 167 us, 812 TFLOP/s of the
// 1954 of a plain product.  There a tile's two products take 1050 cycles of
// the tensor cores and its weights 1480 of their warpgroup (read and maximum
// 380, exponentials 680, store and signal 320), so a warpgroup's turn is 1700
// cycles where two full overlaps would be 1050.  Two warpgroups for each row
// tile, half the keys each, were 17 % slower (104 registers a thread spill), and
// so were a signal after half the weights (2 %) and scores in halves of 64 keys,
// each formed while the other's weights are (25 %: products of 64 columns take
// the tensor cores nearly as long as 128).
#pragma once
#include <math_constants.h>

#include "eg_el.cuh"
#include "eg_ptx.cuh"
#include "eg_tree.h"

namespace eg {

constexpr int kTreeThreads = 384;
constexpr uint32_t kTreeKeys = 128;

// 4-D tiled bulk-tensor load global -> shared.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y, int32_t z,
                                            int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// 3-D tiled bulk-tensor load global -> shared.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Matrix descriptor of an operand whose M or N index is the contiguous one,
// in 128-byte swizzled rows: 64 columns of 8 keys are 1024 bytes, the next 8
// keys follow (stride byte offset), the next 64 columns are `next` bytes on
// (leading byte offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t next) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(next >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
  return p != 0;
}
// The products with an accumulator that is added to (the predicate is a
// constant here: no instruction for it).
__device__ __forceinline__ void umma_f16_add(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, 0, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc)
      : "memory");
}
__device__ __forceinline__ void umma_f16_ts_add(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, 0, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc)
      : "memory");
}

// Two float32 lanes in one instruction.
__device__ __forceinline__ uint64_t pack64(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ void unpack64(uint64_t v, float* lo, float* hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ float tree_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One sequence's lengths, cut to what the table, the packed rows and the plan
// hold.
struct TreeSeq {
  int32_t start, n;    // packed rows
  int32_t ctx, keys;   // cached places, with the drafted tokens
  int32_t tiles;       // key tiles
  int32_t groups;      // row groups: items of a cached head
  int32_t lots;        // costs of those items together
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int32_t start, int32_t n, int32_t ctx) {
  TreeSeq s;
  const int32_t room = static_cast<int32_t>(p.table_stride * p.page_size);
  s.start = start, s.n = n, s.ctx = ctx;
  s.keys = min(ctx + n, room);
  s.tiles = (s.keys + static_cast<int32_t>(kTreeKeys) - 1) >> 7;
  s.groups = (n * p.group + p.item_rows - 1) / p.item_rows;
  s.lots = s.groups * p.q_tiles;
  if (p.q_tiles == 2 && s.groups > 0 && n * p.group - (s.groups - 1) * p.item_rows <= p.tile_rows) --s.lots;
  return s;
}
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b) {
  const int32_t room = static_cast<int32_t>(p.table_stride * p.page_size);
  const int32_t from = __ldg(p.q_start + b), to = __ldg(p.q_start + b + 1), ctx = __ldg(p.context_lens + b);
  const int32_t start = min(max(from, 0), p.tokens);
  return tree_seq(p, start, min(min(max(to, start), p.tokens) - start, p.max_tree), min(max(ctx, 0), room));
}
// Units.  A key tile of an item costs one, or two where the item has two row
// tiles: that takes 1.8 times as long (16 sequences of 24 to 48 tokens, 64
// query heads, 8 cached, 3800 to 8200 places, cold L2: 177 us when both count the
// same, 155 us so; 32 to 64 tokens: 176 and 163 us).  An item has kTreeFixed more
// tiles' units for what it costs beside them: queries, the first and the last
// tile's latency, the result (2, 3, 4 and 6: 168, 164, 163 and 167 us with 32
// to 64 tokens, 98, 100, 101 and 105 us for 24 sequences of 7 to 13 tokens and
// up to 9001 places).  A tile belongs to the CTA that has its first unit.
constexpr int32_t kTreeFixed = 4;
__device__ __forceinline__ int64_t tree_units(const TreeParams& p, const TreeSeq& s) {
  return static_cast<int64_t>(s.tiles + kTreeFixed) * (s.lots * p.kv_heads);
}

// The item that has unit `idx` of a sequence.
struct TreeItem {
  int32_t head, row0, rows;
  int32_t cost;        // units of a tile
  int32_t in, units;   // the unit's place in the item, and how many that has
};
__device__ __forceinline__ TreeItem tree_item(const TreeParams& p, const TreeSeq& s, int64_t idx) {
  TreeItem item;
  const int32_t each = s.tiles + kTreeFixed;
  const int64_t of_head = static_cast<int64_t>(each) * s.lots;
  int32_t g;
  if ((of_head * p.kv_heads) >> 32) {
    item.head = static_cast<int32_t>(idx / of_head);
    const int64_t rest = idx - item.head * of_head, most = static_cast<int64_t>(each) * p.q_tiles;
    g = min(static_cast<int32_t>(rest / most), s.groups - 1);
    item.in = static_cast<int32_t>(rest - g * most);
  } else {
    const uint32_t most = static_cast<uint32_t>(each) * p.q_tiles;
    item.head = static_cast<int32_t>(static_cast<uint32_t>(idx) / static_cast<uint32_t>(of_head));
    const uint32_t rest = static_cast<uint32_t>(idx) - item.head * static_cast<uint32_t>(of_head);
    g = min(static_cast<int32_t>(rest / most), s.groups - 1);
    item.in = static_cast<int32_t>(rest - g * most);
  }
  item.row0 = g * p.item_rows;
  item.rows = min(s.n * p.group - item.row0, p.item_rows);
  item.cost = item.rows > p.tile_rows ? 2 : 1;
  item.units = each * item.cost;
  return item;
}

// The first unit of CTA c, and the CTA that has unit u, when `total` units are
// cut into `ctas` equal ranges.
__device__ __forceinline__ int64_t tree_from(int64_t total, int32_t ctas, int32_t c) {
  if (total < (1 << 20)) return static_cast<uint32_t>(total) * static_cast<uint32_t>(c) / static_cast<uint32_t>(ctas);
  return total * c / ctas;
}
__device__ __forceinline__ int32_t tree_owner(int64_t total, int32_t ctas, int64_t u) {
  if (total < (1 << 20))
    return static_cast<int32_t>((static_cast<uint32_t>(u + 1) * static_cast<uint32_t>(ctas) + static_cast<uint32_t>(total) - 1) / static_cast<uint32_t>(total)) - 1;
  return static_cast<int32_t>(((u + 1) * ctas + total - 1) / total) - 1;
}

constexpr int kTreeNear = 16;  // sequences whose lengths a CTA keeps in shared memory

// Consecutive key tiles of one item.
struct TreeSegment {
  TreeSeq seq;
  int32_t b;
  int32_t head, row0, rows, first, count;
  int32_t cost;
  int32_t more;        // 0: there is none
  int64_t begin;       // the first unit of its item
  __device__ __forceinline__ bool whole() const { return first == 0 && count == seq.tiles; }
};

// A walk over a CTA's range, one segment at a time.
struct TreeWalk : TreeSegment {
  int64_t before;      // units of the sequences before b
  int64_t at, to;
  const int32_t (*near_)[4];  // start, n, ctx of the sequences from near_b on
  int32_t near_b;

  __device__ __forceinline__ void load(const TreeParams& p) {
    const int i = b - near_b;
    seq = i < kTreeNear ? tree_seq(p, near_[i][0], near_[i][1], near_[i][2]) : tree_seq(p, b);
  }
  __device__ __forceinline__ bool next(const TreeParams& p) {
    for (;;) {
      if (at >= to) return false;
      int64_t units = tree_units(p, seq);
      while (at - before >= units) {
        before += units;
        ++b;
        load(p);
        units = tree_units(p, seq);
      }
      const TreeItem item = tree_item(p, seq, at - before);
      const int32_t take = static_cast<int32_t>(min(static_cast<int64_t>(item.units - item.in), to - at));
      begin = at - item.in;
      at += take;
      cost = item.cost;
      // tiles whose first unit is here; the first kTreeFixed stand for none
      first = max((item.in + cost - 1) / cost - kTreeFixed, 0);
      count = (item.in + take + cost - 1) / cost - kTreeFixed - first;
      if (count <= 0) continue;
      head = item.head, row0 = item.row0, rows = item.rows;
      return true;
    }
  }
};

// Shared state after the tiles.
struct TreeShared {
  uint64_t full[12], empty[12];   // ring stages
  uint64_t s_full[2], p_ready[2], o_done[2];
  uint64_t q_full, q_empty, exchange, drained;
  uint64_t told[2], done[2];      // segments for the softmax warpgroups
  uint32_t tmem;
  int32_t abort;
  int32_t poisoned[2];            // the last segment (counted from 1) that found a value that is not finite
  int32_t b;
  int32_t joins;                  // this CTA has the last part of an item
  int64_t before;
  int64_t warps[2][12];
  int32_t near_[kTreeNear][4];
  TreeSegment segments[2];
  float2 stats[2][128];           // a warpgroup's row references and weights
};
static_assert(sizeof(TreeShared) <= TreeSmem<64>::kExtra, "fits the room after the tiles");

// Position of a tile's values in the ring's order: K0, K1, V0, K2, V1, ...
__device__ __forceinline__ uint32_t tree_pos_v(uint32_t i, uint32_t count) { return i + 1 < count ? 2 * i + 2 : 2 * count - 1; }

// Four columns of one row of an item that CTAs lead..last have parts of, joined
// in the order of the CTAs.
template <typename T, int HD>
__device__ __forceinline__ void tree_join_piece(const TreeParams& p, int lead, int last, int r, int col, int64_t packed, int head) {
  constexpr float kShift = El<T>::kBf16 ? 0.0f : 7.0f;
  const int64_t rows = static_cast<int64_t>(128) * p.q_tiles;
  const float2* ml = reinterpret_cast<const float2*>(p.partial_ml) + r;
  const float* part = p.partial + static_cast<int64_t>(col) * rows + r * 4;
  // both to the reference of the largest maximum so far
  float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float top = -CUDART_INF_F, weight = 0.0f;
#pragma unroll 4
  for (int c = lead; c <= last; ++c) {
    const int64_t slot = (static_cast<int64_t>(c) * 2 + (c == lead ? 1 : 0)) * rows;
    const float2 w = __ldcg(ml + slot);
    const float4 x = __ldcg(reinterpret_cast<const float4*>(part + slot * HD));
    const float next = fmaxf(top, w.x);
    const float ref = next == -CUDART_INF_F ? 0.0f : next;
    const float f_old = tree_ex2(top - ref), f = tree_ex2(w.x - ref);
    top = next;
    weight = weight * f_old + w.y * f;
    y.x *= f_old, y.y *= f_old, y.z *= f_old, y.w *= f_old;
    if (w.y != 0.0f) y.x = fmaf(x.x, f, y.x), y.y = fmaf(x.y, f, y.y), y.z = fmaf(x.z, f, y.z), y.w = fmaf(x.w, f, y.w);
  }
  const float scale = weight == 0.0f ? 0.0f : 1.0f / weight;
  if (col < p.head_dim) {
    T* o = static_cast<T*>(p.o) + packed * p.o_token + static_cast<int64_t>(head) * p.o_head + col;
    *reinterpret_cast<uint2*>(o) = make_uint2(El<T>::pack2(y.x * scale, y.y * scale), El<T>::pack2(y.z * scale, y.w * scale));
  }
  if (p.lse && col == 0)
    p.lse[packed * p.q_heads + head] = weight == 0.0f ? -CUDART_INF_F : (top - kShift + __log2f(weight)) * 0.6931471805599453f;
}

template <typename T, int HD>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_kernel(const TreeParams p, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v) {
  constexpr uint32_t kTile = TreeSmem<HD>::kTileBytes;
  constexpr int kChunks = HD / 64;           // 64-column parts of a tile, 16 KB each
  constexpr uint32_t kPart = 128u * 128u;    // bytes of one part
  constexpr uint32_t kFmt = sizeof(T) == 2 && El<T>::kBf16 ? 1u : 0u;
  // the scores' reference lies this far below their maximum, so that small
  // weights keep their bits as fp16 (its normal numbers end at 2^-14)
  constexpr float kShift = El<T>::kBf16 ? 0.0f : 7.0f;
  constexpr float kGrow = 8.0f;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* q_smem = smem;
  uint8_t* ring = smem + p.q_tiles * kTile;
  TreeShared& sh = *reinterpret_cast<TreeShared*>(ring + p.stages * kTile);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t stages = p.stages;

  griddep_launch_dependents();

  // ---- this CTA's range of units.  One pass over the sequences where every
  // thread has one; else a pass for the total and one to find the place.
  const bool once = p.batch <= kTreeThreads;
  int64_t mine = 0;
  TreeSeq seq{};
  for (int b = tid; b < p.batch; b += kTreeThreads) {
    seq = tree_seq(p, b);
    mine += tree_units(p, seq);
  }
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) sh.warps[0][warp] = upto;
  if (tid == 0) {
    for (uint32_t i = 0; i < stages; ++i) mbar_init(&sh.full[i], 1), mbar_init(&sh.empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sh.s_full[i], 1), mbar_init(&sh.p_ready[i], 4), mbar_init(&sh.o_done[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sh.told[i], 1), mbar_init(&sh.done[i], 8);
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    mbar_init(&sh.exchange, 256);
    mbar_init(&sh.drained, 1);
    fence_mbar_init();
    sh.abort = 0;
    sh.poisoned[0] = sh.poisoned[1] = 0;
  }
  __syncthreads();
  int64_t total = 0, base = 0;
#pragma unroll
  for (int w = 0; w < kTreeThreads / 32; ++w) {
    if (w < warp) base += sh.warps[0][w];
    total += sh.warps[0][w];
  }
  // a range is no shorter than a tile's units, so that a CTA between the first
  // and the last of an item has a tile of it
  const int32_t ctas = static_cast<int32_t>(min(static_cast<int64_t>(gridDim.x), p.q_tiles == 2 ? total >> 1 : total));
  if (static_cast<int32_t>(blockIdx.x) >= ctas) {
    if (blockIdx.x == 0 && tid == 0) p.meta[0].ctas = 0;
    return;
  }
  const int64_t from = tree_from(total, ctas, blockIdx.x), to = tree_from(total, ctas, blockIdx.x + 1);
  if (once) {
    if (base + upto - mine <= from && from < base + upto) sh.b = tid, sh.before = base + upto - mine;
  } else {
    int64_t before = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kTreeThreads) {
      const int64_t units = b0 + tid < p.batch ? tree_units(p, tree_seq(p, b0 + tid)) : 0;
      upto = units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      __syncthreads();
      if (lane == 31) sh.warps[1][warp] = upto;
      __syncthreads();
      int64_t chunk = 0;
      base = before;
      for (int w = 0; w < kTreeThreads / 32; ++w) {
        if (w < warp) base += sh.warps[1][w];
        chunk += sh.warps[1][w];
      }
      if (base + upto - units <= from && from < base + upto) sh.b = b0 + tid, sh.before = base + upto - units;
      before += chunk;
      if (before > from) break;  // the same for every thread
    }
  }
  __syncthreads();
  const int near_b = sh.b;
  if (once ? tid >= near_b && tid < min(near_b + kTreeNear, p.batch) : tid < kTreeNear && near_b + tid < p.batch) {
    if (!once) seq = tree_seq(p, near_b + tid);
    int32_t* at = sh.near_[once ? tid - near_b : tid];
    at[0] = seq.start, at[1] = seq.n, at[2] = seq.ctx;
  }
  if (warp == 8) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  // Bounded wait: false once any wait of the CTA has run past its limit.
  volatile int32_t* abort = &sh.abort;
  auto wait = [&](uint64_t* bar, uint32_t phase) {
    if (mbar_try_wait(bar, phase & 1)) return true;
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
      if (mbar_try_wait(bar, phase & 1)) return true;
      if ((it & 63u) == 0) {
        if (*abort) return false;
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > p.wait_limit_ns) {
          *abort = 1;
          *reinterpret_cast<volatile int32_t*>(p.status) = 1;
          return false;
        }
      }
    }
  };

  // The whole warp goes on or gives up.
  auto wait_all = [&](uint64_t* bar, uint32_t phase) { return __all_sync(0xffffffffu, wait(bar, phase)) != 0; };

  // Registers from the four warps that need few to the two warpgroups that
  // hold a row of 128 scores a thread: 4 x 32 x 88 + 8 x 32 x 208 is what the
  // block was launched with (384 x 168).
  if (warp >= 8) {
  setmaxnreg_dec<88>();
  TreeWalk walk;
  walk.b = near_b, walk.before = sh.before, walk.at = from, walk.to = to;
  walk.near_ = sh.near_, walk.near_b = near_b;
  walk.load(p);
  if (warp == 8) {
    // ------------------------------------------------------- producer ----
    uint32_t pos = 0;  // loads so far
    bool ok = true;
    const int boxes = 128 / p.box_rows;
    if (lane == 0) tma_prefetch_desc(&map_k), tma_prefetch_desc(&map_v);
    while (ok && walk.next(p)) {
      const int32_t* table = p.block_table + walk.b * p.table_stride;
      auto place = [&](int tile, int* page, int* off) {
        const int key = (walk.first + tile) * static_cast<int>(kTreeKeys) + lane * p.box_rows;
        *page = -1, *off = 0;
        if (lane < boxes && key < walk.seq.keys) {
          *page = __ldg(table + key / p.page_size);
          *off = key % p.page_size;
        }
        return lane < boxes && key < walk.seq.keys;
      };
      auto issue = [&](const CUtensorMap* map, bool has, int page, int off) {
        const uint32_t slot = pos % stages;
        if (!wait_all(&sh.empty[slot], pos / stages + 1)) return false;
        ++pos;
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, has)) * p.box_rows * 128u * kChunks;
        if (p.stall) return true;
        if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], bytes);
        __syncwarp();
        if (has) {
          const uint32_t dst = smem_u32(ring + slot * kTile) + lane * p.box_rows * 128u;
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            tma_load_4d(dst + c * kPart, map, &sh.full[slot], c * 64, p.heads_inner ? walk.head : off, p.heads_inner ? off : walk.head, page);
        }
        return true;
      };
      int page, off, next_page = -1, next_off = 0;
      bool has = place(0, &page, &off), next_has = false;
      for (int i = 0; ok && i <= walk.count; ++i) {
        // K of tile i, then V of the one before; the next tile's table
        // entries are on their way meanwhile
        const int last_page = page, last_off = off;
        const bool last_has = has;
        if (i > 0) page = next_page, off = next_off, has = next_has;
        if (i + 1 < walk.count) next_has = place(i + 1, &next_page, &next_off);
        if (i < walk.count) ok = issue(&map_k, has, page, off);
        if (ok && i > 0) ok = issue(&map_v, last_has, last_page, last_off);
      }
    }
    if (!p.stall) {
      // the CTA leaves no copy in flight behind
      for (uint32_t i = pos > stages ? pos - stages : 0; i < pos; ++i)
        if (!mbar_wait(&sh.full[i % stages], (i / stages) & 1, p.wait_limit_ns)) break;
    }
  } else if (warp == 9) {
    // --------------------------------------------------------- issuer ----
    // The whole warp walks, so that addresses stay in uniform registers; one
    // elected lane issues.  What the tensor cores wait for most is this
    // warp: positions in the ring are stepped, not divided out.
    constexpr uint32_t kIdescS = idesc_f32acc(kFmt, kFmt, 128, 128);
    constexpr uint32_t kIdescO = idesc_f32acc(kFmt, kFmt, 128, HD) | (1u << 16);  // values: keys are the strided index
    const uint64_t q_desc = sdesc_k_sw128(smem_u32(q_smem)), k_desc = sdesc_k_sw128(smem_u32(ring));
    const uint64_t v_desc = sdesc_mn_sw128(smem_u32(ring), kPart);
    uint32_t segment = 0, used0 = 0, used1 = 0;  // segments, and tiles given to each warpgroup
    uint32_t slot0 = 0, turn0 = 0;               // the segment's first place in the ring, and how often the ring was full
    auto step = [&](uint32_t& slot, uint32_t& turn, uint32_t by) {
      slot += by;
      if (slot >= stages) slot -= stages, ++turn;
    };
    bool ok = true;
    while (ok && walk.next(p)) {
      const uint32_t count = walk.count;
      const bool pair = walk.rows > p.tile_rows;
      const uint32_t jobs = pair ? 2 * count : count;
      uint32_t slot_k = slot0, turn_k = turn0, slot_v = slot0, turn_v = turn0;
      step(slot_v, turn_v, count == 1 ? 1 : 2);
      if (!(ok = wait_all(&sh.q_full, segment))) break;
      // job j is warpgroup j & 1's next tile; the scores of two jobs run
      // ahead of the weighted sums
      for (uint32_t j = 0; j < jobs + 2; ++j) {
        const uint32_t s = j & 1;
        const bool first_use = !pair || s == 0, last_use = !pair || s == 1;
        if (j >= 2) {
          // O += P V of job j - 2
          if (first_use && !(ok = wait_all(&sh.full[slot_v], turn_v))) break;
          if (!(ok = wait_all(&sh.p_ready[s], s ? used1 : used0))) break;
          tc_fence_after();
          const uint64_t v = v_desc + (slot_v * kTile >> 4);
          const uint32_t o = tmem + 256 + s * 128, w = tmem + s * 128;
          if (elect_one()) {
            umma_f16_ts(o, w, v, kIdescO, j >= 4 ? 1 : 0);
#pragma unroll
            for (int k = 1; k < 8; ++k) umma_f16_ts_add(o, w + k * 8, v + k * (2048 >> 4), kIdescO);
            umma_commit(&sh.o_done[s]);
            if (last_use) umma_commit(&sh.empty[slot_v]);
          }
          if (s) ++used1;
          else ++used0;
          // V of tile i is 2 i + 2 places on, the last one directly after the one before
          if (last_use) {
            const uint32_t i = pair ? (j - 2) >> 1 : j - 2;
            step(slot_v, turn_v, i + 2 == count ? 1 : 2);
          }
        }
        if (j < jobs) {
          // S of job j
          if (first_use && !(ok = wait_all(&sh.full[slot_k], turn_k))) break;
          tc_fence_after();
          const uint64_t q = q_desc + (pair && s ? kTile >> 4 : 0), key = k_desc + (slot_k * kTile >> 4);
          const uint32_t d = tmem + s * 128;
          if (elect_one()) {
            umma_f16(d, q, key, kIdescS, 0);
#pragma unroll
            for (int k = 1; k < HD / 16; ++k) {
              const uint32_t at = ((k / 4) * kPart + (k % 4) * 32) >> 4;
              umma_f16_add(d, q + at, key + at, kIdescS);
            }
            umma_commit(&sh.s_full[s]);
            if (last_use) umma_commit(&sh.empty[slot_k]);
            if (j + 1 == jobs) umma_commit(&sh.q_empty);
          }
          if (last_use) step(slot_k, turn_k, j < (pair ? 2 : 1) ? 1 : 2);
        }
      }
      // the segment took 2 count places
      uint32_t places = 2 * count;
      turn0 += places / stages;
      step(slot0, turn0, places % stages);
      ++segment;
    }
    // products in flight have to end before tensor memory is freed
    if (elect_one()) umma_commit(&sh.drained);
    __syncwarp();
    if (!mbar_wait(&sh.drained, 0, p.wait_limit_ns)) mbar_wait(&sh.drained, 0, 8 * p.wait_limit_ns);
  } else {
    // -------------------------------------------------------- queries ----
    if (tid == kTreeThreads - 1) {
      // what the joining kernel has to know of this CTA's first item
      TreeMeta m;
      m.from = from;
      const TreeItem item = tree_item(p, walk.seq, from - sh.before);
      m.begin = from - item.in, m.total = total, m.ctas = ctas;
      m.lead = m.begin + kTreeFixed * item.cost, m.last = m.begin + item.units - item.cost;
      m.start = walk.seq.start, m.row0 = item.row0, m.head = item.head, m.rows = item.rows, m.pad = 0;
      p.meta[blockIdx.x] = m;
    }
    if (warp == 11) {
      // the walk for the warpgroups below, whose registers have no room for it
      bool more = true;
      for (uint32_t n = 0; more; ++n) {
        if (!wait_all(&sh.done[n & 1], (n >> 1) + 1)) break;
        more = walk.next(p);
        walk.more = more;
        if (lane == 0) {
          sh.segments[n & 1] = walk;
          mbar_arrive(&sh.told[n & 1]);
        }
      }
    }
    if (warp == 10) {
      // a box is `box_tokens` tokens by the heads that share a cached one;
      // lane i has box i of each tile
      uint32_t segment = 0;
      const int box = p.box_tokens * p.group, boxes = p.tile_rows / box;
      while (walk.next(p)) {
        if (!wait_all(&sh.q_empty, segment + 1)) break;
        const int all = (walk.rows + box - 1) / box;  // boxes that hold a row
        if (lane == 0) mbar_arrive_expect_tx(&sh.q_full, all * box * 128u * kChunks);
        __syncwarp();
        for (int i = lane; i < all; i += 32) {
          const int tile = i >= boxes ? 1 : 0, in = i - tile * boxes;
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            tma_load_3d(smem_u32(q_smem) + tile * kTile + c * kPart + in * box * 128u, &map_q, &sh.q_full, c * 64, walk.head * p.group,
                        walk.seq.start + walk.row0 / p.group + i * p.box_tokens);
        }
        ++segment;
      }
      if (segment > 0) mbar_wait(&sh.q_full, (segment - 1) & 1, p.wait_limit_ns);  // leaves no copy in flight behind
    }
  }
  } else {
    // -------------------------------------------------------- softmax ----
    setmaxnreg_inc<208>();
    const int s = warp >> 2;            // the warpgroup
    const int row_in = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t t_s = tmem + lanes + s * 128, t_o = tmem + lanes + 256;
    const float c = p.scale_log2;
    uint32_t base = 0, uses = 0, exchanges = 0;
    int32_t segment = 0;
    bool ok = true;
    for (;;) {
      const TreeSegment& walk = sh.segments[segment & 1];
      if (!(ok = wait_all(&sh.told[segment & 1], segment >> 1)) || !walk.more) break;
      ++segment;
      const bool pair = walk.rows > p.tile_rows;
      const int count = walk.count, first = walk.first, ctx = walk.seq.ctx, keys = walk.seq.keys;
      const int r = (pair ? s * p.tile_rows : 0) + row_in;
      const bool valid = row_in < p.tile_rows && r < walk.rows;
      const bool busy = __any_sync(0xffffffffu, valid);  // the warp has a row
      const int t = (walk.row0 + r) / p.group;
      const int64_t packed = walk.seq.start + t;
      const int head = walk.head * p.group + (walk.row0 + r) - t * p.group;
      const int drafted = keys - ctx;  // drafted keys that exist
      // 32 bits of the row's mask from drafted token u on
      auto drafted_bits = [&](int u) -> uint32_t {
        const int left = drafted - u;
        if (left <= 0 || !valid) return 0u;
        uint32_t bits;
        if (p.mask) {
          const int words = (p.max_tree + 31) >> 5, w = u >> 5;
          const uint32_t* m = p.mask + packed * p.mask_stride;
          bits = __funnelshift_r(m[w], w + 1 < words ? m[w + 1] : 0u, u & 31);
        } else {
          const int upto = t - u + 1;
          bits = upto >= 32 ? 0xFFFFFFFFu : upto <= 0 ? 0u : (1u << upto) - 1u;
        }
        return left >= 32 ? bits : bits & ((1u << left) - 1u);
      };
      float m = -CUDART_INF_F, l = 0.0f;  // m: the reference (log2), before the shift
      bool fresh = true;                  // no tile of this segment yet
      for (int i = pair ? 0 : s; ok && i < count; i += pair ? 1 : 2) {
        const int key0 = (first + i) * static_cast<int>(kTreeKeys);
        const bool edge = key0 + static_cast<int>(kTreeKeys) > ctx;
        if (!(ok = wait_all(&sh.s_full[s], uses))) break;
        tc_fence_after();
        if (busy) {
          uint32_t x[128];
#pragma unroll
          for (int j = 0; j < 4; ++j) tmem_ld32p(t_s + j * 32, x + j * 32);
          tmem_ld_wait();
          reg_fence<128>(x);
          if (edge) {
            // a tile with drafted places or past the end: -infinity where the
            // row does not attend to
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int d = ctx - (key0 + 32 * w);  // context places of this word
              const uint32_t bits = d >= 32  ? 0xFFFFFFFFu
                                    : d <= 0 ? drafted_bits(-d)
                                             : ((1u << d) - 1u) | (drafted_bits(0) << d);
              if (__all_sync(0xffffffffu, bits == 0xFFFFFFFFu)) continue;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(bits >> j & 1u)) x[w * 32 + j] = 0xFF800000u;
            }
          }
          float top[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) top[j] = __uint_as_float(x[j]);
#pragma unroll
          for (int j = 4; j < 128; ++j) top[j & 3] = fmaxf(top[j & 3], __uint_as_float(x[j]));
          float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          high = high == -CUDART_INF_F ? high : high * c;
          if (!valid) high = -CUDART_INF_F;
          if (fresh) {
            m = high;
          } else if (__any_sync(0xffffffffu, high > m + kGrow)) {
            // bring this row's sums to its new maximum
            const float next = fmaxf(m, high);
            const float f = next == m ? 1.0f : tree_ex2(m - next);
            if (!(ok = wait_all(&sh.o_done[s], uses - 1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < HD; j += 16) {
              uint32_t y[16];
              tmem_ld16(t_o + s * 128 + j, y);
              tmem_ld_wait();
              reg_fence<16>(y);
#pragma unroll
              for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
              tmem_st16(t_o + s * 128 + j, y);
            }
            l *= f;
            m = next;
          }
          const float ref = m == -CUDART_INF_F ? 0.0f : kShift - m;
          const uint64_t c2 = pack64(__float_as_uint(c), __float_as_uint(c)), ref2 = pack64(__float_as_uint(ref), __float_as_uint(ref));
          uint64_t sum2[2] = {0, 0};
#pragma unroll
          for (int j = 0; j < 64; ++j) {
            float a, b;
            unpack64(fma2(pack64(x[2 * j], x[2 * j + 1]), c2, ref2), &a, &b);
            a = tree_ex2(a), b = tree_ex2(b);
            sum2[j & 1] = add2(sum2[j & 1], pack64(__float_as_uint(a), __float_as_uint(b)));
            x[j] = El<T>::pack2(a, b);
          }
          float sum_a, sum_b;
          unpack64(add2(sum2[0], sum2[1]), &sum_a, &sum_b);
          l += sum_a + sum_b;
          tmem_st32(t_s, x);
          tmem_st32(t_s + 32, x + 32);
          tmem_st_wait();
        }
        fresh = false;
        const bool cut = keys < key0 + static_cast<int>(kTreeKeys), scan = p.mask || drafted > 1;
        if (edge && (cut || scan)) {
          // values of places past the end become zero, and so do drafted
          // values that are not finite: a weight of zero times one would
          // reach rows that do not attend to it (`repair` adds it to those
          // that do)
          const uint32_t at = base + tree_pos_v(i, count), slot = at % stages;
          if (!(ok = wait_all(&sh.full[slot], at / stages))) break;
          const int key = key0 + row_in;
          uint8_t* v_row = ring + slot * kTile + row_in * 128;
          if (key >= keys) {
#pragma unroll 4
            for (int j = 0; j < kChunks * 8; ++j) *reinterpret_cast<uint4*>(v_row + (j >> 3) * kPart + (j & 7) * 16) = make_uint4(0, 0, 0, 0);
          } else if (scan && key >= ctx) {
            constexpr uint32_t kInf = El<T>::kBf16 ? 0x7F80u : 0x7C00u;
            bool found = false;
#pragma unroll 1
            for (int j = 0; j < kChunks * 8; ++j) {
              uint4* at_v = reinterpret_cast<uint4*>(v_row + (j >> 3) * kPart + (j & 7) * 16);
              uint4 v = *at_v;
              uint32_t* word = reinterpret_cast<uint32_t*>(&v);
              bool here = false;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if ((word[k] & kInf) == kInf) word[k] &= 0xFFFF0000u, here = true;
                if ((word[k] & (kInf << 16)) == (kInf << 16)) word[k] &= 0x0000FFFFu, here = true;
              }
              if (here) *at_v = v, found = true;
            }
            if (found) *reinterpret_cast<volatile int32_t*>(&sh.poisoned[s]) = segment;
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_ready[s]);
        ++uses;
      }
      if (!ok) break;
      // ---- the segment's result
      const int tiles0 = pair ? count : (count + 1) / 2, tiles1 = pair ? count : count / 2;
      if ((s ? tiles1 : tiles0) > 0) {
        if (!(ok = wait_all(&sh.o_done[s], uses - 1))) break;
        tc_fence_after();
      }
      float2 own = make_float2(m, l), other = make_float2(-CUDART_INF_F, 0.0f);
      sh.stats[s][row_in] = own;
      tc_fence_before();
      mbar_arrive(&sh.exchange);
      if (!(ok = wait_all(&sh.exchange, exchanges))) break;
      ++exchanges;
      tc_fence_after();
      if (!pair) other = sh.stats[s ^ 1][row_in];
      // either warpgroup may have met the value first
      const bool repair = *reinterpret_cast<volatile int32_t*>(&sh.poisoned[0]) == segment ||
                          *reinterpret_cast<volatile int32_t*>(&sh.poisoned[1]) == segment;
      const float both = fmaxf(own.x, other.x);
      const float ref = both == -CUDART_INF_F ? 0.0f : both;
      const float f_own = tree_ex2(own.x - ref), f_other = tree_ex2(other.x - ref);
      const float weight = own.y * f_own + other.y * f_other;
      const bool whole = walk.whole();
      if (busy) {
        // a pair's warpgroup writes its rows, else each writes half the columns
        constexpr int kCols = HD / 2;  // at a time
        const int from_col = pair ? 0 : s * (HD / 2), to_col = pair ? HD : from_col + HD / 2;
        const float f0 = (pair || s == 0 ? f_own : f_other), f1 = (s == 0 ? f_other : f_own);
        const float scale = whole ? (weight == 0.0f ? 0.0f : 1.0f / weight) : 1.0f;
        const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (walk.first == 0 ? 1 : 0);
        const int64_t at = slot * 128 * p.q_tiles + r;
        const int part_rows = 128 * p.q_tiles;
        T* o = static_cast<T*>(p.o) + packed * p.o_token + static_cast<int64_t>(head) * p.o_head;
        // [slot][4 columns][row][column]: a warp's rows are stored side by side
        float* part = p.partial + slot * part_rows * HD + r * 4;
#pragma unroll 1
        for (int j = from_col; j < to_col; j += kCols) {
          uint32_t a[kCols];
#pragma unroll
          for (int k = 0; k < kCols; k += 32) tmem_ld32p(t_o + (pair ? s * 128 : 0) + j + k, a + k);
          if (!pair && tiles1 > 0) {
            uint32_t b[kCols];
#pragma unroll
            for (int k = 0; k < kCols; k += 32) tmem_ld32p(t_o + 128 + j + k, b + k);
            tmem_ld_wait();
            reg_fence<kCols>(a), reg_fence<kCols>(b);
#pragma unroll
            for (int k = 0; k < kCols; ++k)
              a[k] = __float_as_uint(fmaf(__uint_as_float(b[k]), f1, __uint_as_float(a[k]) * f0));
          } else {
            tmem_ld_wait();
            reg_fence<kCols>(a);
#pragma unroll
            for (int k = 0; k < kCols; ++k) a[k] = __float_as_uint(__uint_as_float(a[k]) * f0);
          }
          if (!valid) continue;
#pragma unroll
          for (int k = 0; k < kCols; k += 8) {
            if (j + k >= p.head_dim) continue;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = weight == 0.0f ? 0.0f : __uint_as_float(a[k + e]) * scale;
            if (whole) {
              Chunk<T, 8> out;
              out.set(y);
              out.store(o + j + k);
            } else {
              *reinterpret_cast<float4*>(part + static_cast<int64_t>(j + k) * part_rows) = make_float4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<float4*>(part + static_cast<int64_t>(j + k + 4) * part_rows) = make_float4(y[4], y[5], y[6], y[7]);
            }
          }
        }
        if (valid && (pair || s == 0)) {
          if (!whole) *reinterpret_cast<float2*>(p.partial_ml + at * 2) = make_float2(both, weight);
          else if (p.lse)
            p.lse[packed * p.q_heads + head] =
                weight == 0.0f ? -CUDART_INF_F : (both - kShift + __log2f(weight)) * 0.6931471805599453f;
        }
        if (repair && valid) {
          // drafted values that are not finite, to the rows that attend to them
          const int last = min(walk.seq.keys, (walk.first + count) * static_cast<int>(kTreeKeys));
          for (int key = max(walk.seq.ctx, walk.first * static_cast<int>(kTreeKeys)); key < last; ++key) {
            if (!(drafted_bits(key - walk.seq.ctx) & 1u)) continue;
            const int page = p.block_table[walk.b * p.table_stride + key / p.page_size];
            if (page < 0 || page >= p.num_pages) continue;
            const T* v = static_cast<const T*>(p.v) + page * p.page_stride + (key % p.page_size) * p.token_stride + walk.head * p.head_stride;
            for (int e = from_col; e < min(to_col, p.head_dim); ++e) {
              const float x = El<T>::to_float(v[e]);
              if (fabsf(x) < CUDART_INF_F) continue;
              if (whole) o[e] = El<T>::from_float(El<T>::to_float(o[e]) + x);
              else part[static_cast<int64_t>(e & ~3) * part_rows + (e & 3)] += x;
            }
          }
        }
      }
      // the other warpgroup's accumulator is read: it may be written again
      if (!whole && p.arrivals) __threadfence();
      tc_fence_before();
      mbar_arrive(&sh.exchange);
      if (!(ok = wait_all(&sh.exchange, exchanges))) break;
      ++exchanges;
      tc_fence_after();
      if (!whole && p.arrivals) {
        // the CTA that leaves the last part of the item joins all of them
        const int32_t lead = tree_owner(total, ctas, walk.begin + kTreeFixed * walk.cost);
        const int32_t last = tree_owner(total, ctas, walk.begin + (walk.seq.tiles + kTreeFixed - 1) * walk.cost);
        if (tid == 0) {
          const int before = atomicAdd(p.arrivals + lead, 1);
          sh.joins = before == last - lead;
          if (before == last - lead) p.arrivals[lead] = 0;
          __threadfence();
        }
        mbar_arrive(&sh.exchange);
        if (!(ok = wait_all(&sh.exchange, exchanges))) break;
        ++exchanges;
        if (sh.joins) {
          const int pieces = walk.rows * (HD / 4);
          for (int i = tid; i < pieces; i += 256) {
            const int r_ = i % walk.rows, t_ = (walk.row0 + r_) / p.group;
            tree_join_piece<T, HD>(p, lead, last, r_, i / walk.rows * 4, walk.seq.start + t_,
                                   walk.head * p.group + (walk.row0 + r_) - t_ * p.group);
          }
        }
      }
      base += 2 * count;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.done[(segment - 1) & 1]);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) {
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partial results of the items that a cut between CTAs divides, where
// the main kernel leaves that to it: the blocks of cut x (between CTAs x - 1
// and x) serve the item whose first cut it is, eight rows each.  A thread has
// four columns of a row; a warp has eight rows of 16 columns, which is how they
// lie side by side.
template <typename T, int HD>
__global__ void __launch_bounds__(HD * 2) tree_join_kernel(const TreeParams p) {
  griddep_wait();
  const int cut = blockIdx.x + 1;
  const int ctas = p.meta[0].ctas;
  const TreeMeta m = p.meta[cut];
  const int64_t from_before = p.meta[cut - 1].from;
  if (cut >= ctas || m.from <= m.begin || from_before > m.begin) return;
  // the CTAs with the item's first tile and with its last: those between them
  // have some too
  const int lead = tree_owner(m.total, ctas, m.lead), last = tree_owner(m.total, ctas, m.last);
  if (lead == last) return;
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.y * 8 + (lane & 7);
  if (r >= m.rows) return;
  const int t = (m.row0 + r) / p.group;
  tree_join_piece<T, HD>(p, lead, last, r, ((threadIdx.x >> 5) * 4 + (lane >> 3)) * 4, m.start + t, m.head * p.group + (m.row0 + r) - t * p.group);
}

}  // namespace eg
