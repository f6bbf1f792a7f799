// eg_tree_kernel.cuh -- attention of drafted token trees over a paged cache.
//
// Mathematics.  The rows of one item are the n tokens of a sequence's tree
// times the G query heads that share a cached head: for key tiles of 128,
//   S = Q K^T,  P = 2^(c S - m),  O += P V,  l += rowsum P,
// with c = scale log2 e and m a row reference at least the row maximum less 8:
// O and l are only brought to a new reference when the maximum grew by more
// than 2^8, which few tiles do.  Weights are rounded to 16 bits for the second
// product (their error, 2^-9 or 2^-12 of each weight, is the output type's own);
// l sums them before that rounding, in float32 as S, O and m are.
//
// Work.  Every item has as many units as key tiles; all items' units in a row
// are cut into equal ranges, one for each CTA (one CTA an SM), on the device
// from the sequences' lengths.  An item that a cut divides leaves float32
// partial results that a second small kernel joins in a fixed order, so equal
// inputs give equal bits.
//
// One CTA: a producer warp (TMA boxes of pages into a ring of 128-key tiles,
// K and V alike), one issuing thread (tcgen05.mma), two softmax warpgroups
// and two warps that fetch queries.  S and O of both warpgroups fill tensor
// memory (4 x 128 columns); P overwrites S as 16-bit values and feeds the
// second product from there.  With at most 128 rows the warpgroups take turns
// on the key tiles and are joined at the end of the range; with more rows
// each has 128 of them and K and V tiles are used twice.  So while one
// warpgroup forms weights the tensor cores work for the other.
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
  int32_t groups;      // row groups
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b) {
  TreeSeq s;
  const int32_t room = static_cast<int32_t>(p.table_stride * p.page_size);
  s.start = min(max(p.q_start[b], 0), p.tokens);
  s.n = min(min(max(p.q_start[b + 1], s.start), p.tokens) - s.start, p.max_tree);
  s.ctx = min(max(p.context_lens[b], 0), room);
  s.keys = min(s.ctx + s.n, room);
  s.tiles = (s.keys + static_cast<int32_t>(kTreeKeys) - 1) / static_cast<int32_t>(kTreeKeys);
  s.groups = (s.n * p.group + 128 * p.q_tiles - 1) / (128 * p.q_tiles);
  return s;
}
__device__ __forceinline__ int64_t tree_units(const TreeParams& p, const TreeSeq& s) {
  return static_cast<int64_t>(s.tiles) * s.groups * p.kv_heads;
}

// A walk over a CTA's range: one segment (consecutive key tiles of one item)
// at a time.
struct TreeWalk {
  TreeSeq seq;
  int32_t b;
  int64_t before;      // units of the sequences before b
  int64_t at, to;
  // the segment
  int32_t head, row0, rows, first, count;

  __device__ __forceinline__ bool next(const TreeParams& p) {
    if (at >= to) return false;
    for (;;) {
      const int64_t units = tree_units(p, seq);
      if (at - before < units) break;
      before += units;
      seq = tree_seq(p, ++b);
    }
    const int64_t idx = at - before;
    const int32_t item = static_cast<int32_t>(idx / seq.tiles);
    first = static_cast<int32_t>(idx - static_cast<int64_t>(item) * seq.tiles);
    head = item / seq.groups;
    row0 = (item - head * seq.groups) * 128 * p.q_tiles;
    rows = min(seq.n * p.group - row0, 128 * p.q_tiles);
    count = static_cast<int32_t>(min(static_cast<int64_t>(seq.tiles - first), to - at));
    at += count;
    return true;
  }
  __device__ __forceinline__ bool whole() const { return first == 0 && count == seq.tiles; }
};

// Shared state after the tiles.
struct TreeShared {
  uint64_t full[12], empty[12];   // ring stages
  uint64_t s_full[2], p_ready[2], o_done[2];
  uint64_t q_full, q_empty, exchange, drained;
  uint32_t tmem;
  int32_t abort;
  int32_t poisoned[2];            // the last segment (counted from 1) that found a value that is not finite
  int32_t b;
  int32_t pad;
  int64_t before, from, to, total;
  int64_t warps[12];
  float2 stats[2][128];           // a warpgroup's row references and weights
};
static_assert(sizeof(TreeShared) <= 2560, "fits the room after the tiles");

// Position of a tile's load in the ring's order: K0, K1, V0, K2, V1, ...
__device__ __forceinline__ uint32_t tree_pos_k(uint32_t i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ uint32_t tree_pos_v(uint32_t i, uint32_t count) { return i + 1 < count ? 2 * i + 2 : 2 * count - 1; }

template <typename T, int HD>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_kernel(const TreeParams p, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
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

  // ---- this CTA's range of units
  int64_t mine = 0;
  for (int b = tid; b < p.batch; b += kTreeThreads) mine += tree_units(p, tree_seq(p, b));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) sh.warps[warp] = mine;
  if (tid == 0) {
    for (uint32_t i = 0; i < stages; ++i) mbar_init(&sh.full[i], 1), mbar_init(&sh.empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sh.s_full[i], 1), mbar_init(&sh.p_ready[i], 4), mbar_init(&sh.o_done[i], 1);
    mbar_init(&sh.q_full, 64);
    mbar_init(&sh.q_empty, 1);
    mbar_init(&sh.exchange, 256);
    mbar_init(&sh.drained, 1);
    fence_mbar_init();
    sh.abort = 0;
    sh.poisoned[0] = sh.poisoned[1] = 0;
  }
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < kTreeThreads / 32; ++w) total += sh.warps[w];
  const int32_t ctas = static_cast<int32_t>(min(static_cast<int64_t>(gridDim.x), total));
  if (static_cast<int32_t>(blockIdx.x) >= ctas) {
    if (blockIdx.x == 0 && tid == 0) p.meta[0].ctas = 0;
    return;
  }
  const int64_t from = total * blockIdx.x / ctas, to = total * (blockIdx.x + 1) / ctas;
  {
    int64_t before = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kTreeThreads) {
      const int64_t units = b0 + tid < p.batch ? tree_units(p, tree_seq(p, b0 + tid)) : 0;
      int64_t upto = units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      __syncthreads();
      if (lane == 31) sh.warps[warp] = upto;
      __syncthreads();
      int64_t chunk = 0, base = before;
      for (int w = 0; w < kTreeThreads / 32; ++w) {
        if (w < warp) base += sh.warps[w];
        chunk += sh.warps[w];
      }
      if (base + upto - units <= from && from < base + upto) sh.b = b0 + tid, sh.before = base + upto - units;
      before += chunk;
      if (before > from) break;  // the same for every thread
    }
  }
  if (warp == 8) tmem_alloc(&sh.tmem, 512);
  if (p.head_dim < HD) {  // columns past head_dim: keys are zero there, so are queries
    for (uint32_t i = tid; i < p.q_tiles * kTile / 16; i += kTreeThreads) reinterpret_cast<uint4*>(q_smem)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  TreeWalk walk;
  walk.b = sh.b, walk.before = sh.before, walk.at = from, walk.to = to;
  walk.seq = tree_seq(p, walk.b);
  if (tid == 0) {
    TreeWalk w = walk;
    w.next(p);
    TreeMeta m;
    m.from = from, m.begin = from - w.first, m.end = m.begin + w.seq.tiles, m.total = total;
    m.ctas = ctas, m.start = w.seq.start, m.rows = w.rows, m.row0 = w.row0, m.head = w.head, m.pad = 0;
    p.meta[blockIdx.x] = m;
  }

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
        if (!__all_sync(0xffffffffu, wait(&sh.empty[slot], pos / stages + 1))) return false;
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
    if (lane == 0) {
      constexpr uint32_t kIdescS = idesc_f32acc(kFmt, kFmt, 128, 128);
      constexpr uint32_t kIdescO = idesc_f32acc(kFmt, kFmt, 128, HD) | (1u << 16);  // values: keys are the strided index
      uint32_t base = 0, segment = 0;
      uint32_t uses[2] = {0, 0};  // tiles given to each warpgroup
      bool ok = true;
      while (ok && walk.next(p)) {
        const uint32_t count = walk.count;
        const bool pair = walk.rows > 128;
        // S of key tile i for warpgroup s
        auto product_s = [&](uint32_t i, int s, bool first_use, bool last_use) {
          const uint32_t at = base + tree_pos_k(i), slot = at % stages;
          if (first_use && !wait(&sh.full[slot], at / stages)) return false;
          tc_fence_after();
          const uint32_t a = smem_u32(q_smem) + (pair ? s : 0) * kTile, b = smem_u32(ring + slot * kTile);
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {
            const uint32_t step = (k / 4) * kPart + (k % 4) * 32;
            umma_f16(tmem + s * 128, sdesc_k_sw128(a + step), sdesc_k_sw128(b + step), kIdescS, k > 0);
          }
          umma_commit(&sh.s_full[s]);
          if (last_use) umma_commit(&sh.empty[slot]);
          return true;
        };
        // O += P V of key tile i for warpgroup s
        auto product_o = [&](uint32_t i, int s, bool first, bool first_use, bool last_use) {
          const uint32_t at = base + tree_pos_v(i, count), slot = at % stages;
          if (first_use && !wait(&sh.full[slot], at / stages)) return false;
          if (!wait(&sh.p_ready[s], uses[s])) return false;
          tc_fence_after();
          const uint32_t b = smem_u32(ring + slot * kTile);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            umma_f16_ts(tmem + 256 + s * 128, tmem + s * 128 + k * 8, sdesc_mn_sw128(b + k * 2048, kPart), kIdescO, k > 0 || !first);
          umma_commit(&sh.o_done[s]);
          if (last_use) umma_commit(&sh.empty[slot]);
          ++uses[s];
          return true;
        };
        ok = wait(&sh.q_full, segment);
        if (!ok) break;
        if (pair) {
          ok = product_s(0, 0, true, false) && product_s(0, 1, false, true);
          if (count == 1) umma_commit(&sh.q_empty);
          for (uint32_t i = 0; ok && i < count; ++i) {
            const bool more = i + 1 < count;
            ok = product_o(i, 0, i == 0, true, false) && (!more || product_s(i + 1, 0, true, false)) &&
                 product_o(i, 1, i == 0, false, true) && (!more || product_s(i + 1, 1, false, true));
            if (i + 2 == count) umma_commit(&sh.q_empty);
          }
        } else {
          ok = product_s(0, 0, true, true);
          if (count == 1) umma_commit(&sh.q_empty);
          for (uint32_t i = 0; ok && i < count; ++i) {
            if (i + 1 < count) ok = product_s(i + 1, (i + 1) & 1, true, true);
            if (i + 2 == count) umma_commit(&sh.q_empty);
            ok = ok && product_o(i, i & 1, i < 2, true, true);
          }
        }
        base += 2 * count;
        ++segment;
      }
      // products in flight have to end before tensor memory is freed
      umma_commit(&sh.drained);
      if (!mbar_wait(&sh.drained, 0, p.wait_limit_ns)) mbar_wait(&sh.drained, 0, 8 * p.wait_limit_ns);
    }
  } else if (warp >= 10) {
    // -------------------------------------------------------- queries ----
    const int at = tid - 320;  // 0..63
    const int vecs = p.head_dim / 8;
    uint32_t segment = 0;
    while (walk.next(p)) {
      if (!wait(&sh.q_empty, segment + 1)) break;
      for (int i = at; i < walk.rows * vecs; i += 64) {
        const int r = i / vecs, c = i - r * vecs;
        const int t = (walk.row0 + r) / p.group, g = (walk.row0 + r) - t * p.group;
        const T* src = static_cast<const T*>(p.q) + static_cast<int64_t>(walk.seq.start + t) * p.q_token +
                       static_cast<int64_t>(walk.head * p.group + g) * p.q_head + c * 8;
        const uint32_t to_ = (r >> 7) * kTile + (c >> 3) * kPart + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4);
        *reinterpret_cast<uint4*>(q_smem + to_) = __ldg(reinterpret_cast<const uint4*>(src));
      }
      fence_proxy_async_smem();
      mbar_arrive(&sh.q_full);
      ++segment;
    }
  } else {
    // -------------------------------------------------------- softmax ----
    const int s = warp >> 2;            // the warpgroup
    const int row_in = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t t_s = tmem + lanes + s * 128, t_o = tmem + lanes + 256;
    const float c = p.scale_log2;
    uint32_t base = 0, uses = 0, exchanges = 0;
    int32_t segment = 0;
    bool ok = true;
    // the whole warp goes on or gives up
    auto wait_all = [&](uint64_t* bar, uint32_t phase) { return __all_sync(0xffffffffu, wait(bar, phase)) != 0; };
    while (ok && walk.next(p)) {
      ++segment;
      const bool pair = walk.rows > 128;
      const int count = walk.count;
      const int r = (pair ? s * 128 : 0) + row_in;
      const bool valid = r < walk.rows;
      const bool busy = (pair ? s * 128 : 0) + (warp & 3) * 32 < walk.rows;  // the warp has a row
      const int t = (walk.row0 + r) / p.group;
      const int64_t packed = walk.seq.start + t;
      const int head = walk.head * p.group + (walk.row0 + r) - t * p.group;
      const int drafted = walk.seq.keys - walk.seq.ctx;  // drafted keys that exist
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
        const int key0 = (walk.first + i) * static_cast<int>(kTreeKeys);
        const bool edge = key0 + static_cast<int>(kTreeKeys) > walk.seq.ctx;
        if (!(ok = wait_all(&sh.s_full[s], uses))) break;
        tc_fence_after();
        if (busy) {
          uint32_t x[128];
#pragma unroll
          for (int j = 0; j < 4; ++j) tmem_ld32p(t_s + j * 32, x + j * 32);
          tmem_ld_wait();
          reg_fence<128>(x);
          if (edge) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int d = walk.seq.ctx - (key0 + 32 * w);  // context places of this word
              const uint32_t bits = d >= 32  ? 0xFFFFFFFFu
                                    : d <= 0 ? drafted_bits(-d)
                                             : ((1u << d) - 1u) | (drafted_bits(0) << d);
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
#pragma unroll
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
          float sum[2] = {0.0f, 0.0f};
#pragma unroll
          for (int j = 0; j < 64; ++j) {
            const float a = tree_ex2(fmaf(__uint_as_float(x[2 * j]), c, ref));
            const float b = tree_ex2(fmaf(__uint_as_float(x[2 * j + 1]), c, ref));
            sum[0] += a, sum[1] += b;
            x[j] = El<T>::pack2(a, b);
          }
          l += sum[0] + sum[1];
          tmem_st32(t_s, x);
          tmem_st32(t_s + 32, x + 32);
          tmem_st_wait();
        }
        fresh = false;
        if (edge && (walk.seq.keys < key0 + static_cast<int>(kTreeKeys) || p.mask || drafted > 1)) {
          // values of places past the end become zero, and so do drafted
          // values that are not finite: a weight of zero times one would
          // reach rows that do not attend to it (`repair` adds it to those
          // that do)
          const uint32_t at = base + tree_pos_v(i, count), slot = at % stages;
          if (!(ok = wait_all(&sh.full[slot], at / stages))) break;
          const int key = key0 + row_in;
          uint8_t* v_row = ring + slot * kTile + row_in * 128;
          if (key >= walk.seq.keys) {
#pragma unroll
            for (int j = 0; j < kChunks * 8; ++j) *reinterpret_cast<uint4*>(v_row + (j >> 3) * kPart + (j & 7) * 16) = make_uint4(0, 0, 0, 0);
          } else if (key >= walk.seq.ctx) {
            constexpr uint32_t kInf = El<T>::kBf16 ? 0x7F80u : 0x7C00u;
            bool found = false;
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
      bool repair;
      if (pair) {
        repair = *reinterpret_cast<volatile int32_t*>(&sh.poisoned[s]) == segment;
      } else {
        other = sh.stats[s ^ 1][row_in];
        repair = *reinterpret_cast<volatile int32_t*>(&sh.poisoned[0]) == segment || *reinterpret_cast<volatile int32_t*>(&sh.poisoned[1]) == segment;
      }
      const float both = fmaxf(own.x, other.x);
      const float ref = both == -CUDART_INF_F ? 0.0f : both;
      const float f_own = tree_ex2(own.x - ref), f_other = tree_ex2(other.x - ref);
      const float weight = own.y * f_own + other.y * f_other;
      const bool whole = walk.whole();
      if (busy) {
        // a pair's warpgroup writes its rows, else each writes half the columns
        const int from_col = pair ? 0 : s * (HD / 2), to_col = pair ? HD : from_col + HD / 2;
        const float f0 = (pair || s == 0 ? f_own : f_other), f1 = (s == 0 ? f_other : f_own);
        const float scale = whole ? (weight == 0.0f ? 0.0f : 1.0f / weight) : 1.0f;
        const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (walk.first == 0 ? 1 : 0);
        const int64_t at = slot * 128 * p.q_tiles + r;
        T* o = static_cast<T*>(p.o) + packed * p.o_token + static_cast<int64_t>(head) * p.o_head;
        float* part = p.partial + at * HD;
        for (int j = from_col; j < to_col; j += 32) {
          uint32_t a[32];
          tmem_ld32p(t_o + (pair ? s * 128 : 0) + j, a);
          tmem_ld_wait();
          reg_fence<32>(a);
#pragma unroll
          for (int k = 0; k < 32; ++k) a[k] = __float_as_uint(__uint_as_float(a[k]) * f0);
          if (!pair && tiles1 > 0) {
            uint32_t b[32];
            tmem_ld32p(t_o + 128 + j, b);
            tmem_ld_wait();
            reg_fence<32>(b);
#pragma unroll
            for (int k = 0; k < 32; ++k) a[k] = __float_as_uint(fmaf(__uint_as_float(b[k]), f1, __uint_as_float(a[k])));
          }
          if (!valid) continue;
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            if (j + k >= p.head_dim) continue;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = weight == 0.0f ? 0.0f : __uint_as_float(a[k + e]) * scale;
            if (whole) {
              Chunk<T, 8> out;
              out.set(y);
              out.store(o + j + k);
            } else {
              *reinterpret_cast<float4*>(part + j + k) = make_float4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<float4*>(part + j + k + 4) = make_float4(y[4], y[5], y[6], y[7]);
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
              else part[e] += x;
            }
          }
        }
      }
      // the other warpgroup's accumulator is read: it may be written again
      tc_fence_before();
      mbar_arrive(&sh.exchange);
      if (!(ok = wait_all(&sh.exchange, exchanges))) break;
      ++exchanges;
      tc_fence_after();
      base += 2 * count;
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

// Joins the partial results of the items that a cut between CTAs divides: the
// blocks of cut x (between CTAs x - 1 and x) serve the item whose first cut it
// is; a warp takes one row.
template <typename T, int HD>
__global__ void __launch_bounds__(256) tree_join_kernel(const TreeParams p) {
  constexpr float kShift = El<T>::kBf16 ? 0.0f : 7.0f;
  constexpr int V = HD / 32;  // columns of a lane
  griddep_wait();
  const int cut = blockIdx.x + 1;
  const int ctas = p.meta[0].ctas;
  if (cut >= ctas) return;
  const TreeMeta m = p.meta[cut];
  if (m.from <= m.begin || p.meta[cut - 1].from > m.begin) return;
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (r >= m.rows) return;
  // the last CTA with a unit of the item
  const int last = static_cast<int>((m.end * ctas + m.total - 1) / m.total) - 1;
  const int64_t stride = static_cast<int64_t>(128) * p.q_tiles;
  auto row_of = [&](int c) { return (static_cast<int64_t>(c) * 2 + (c == cut - 1 ? 1 : 0)) * stride + r; };
  float top = -CUDART_INF_F;
  for (int c = cut - 1 + lane; c <= last; c += 32) top = fmaxf(top, p.partial_ml[row_of(c) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float ref = top == -CUDART_INF_F ? 0.0f : top;
  float y[V], weight = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) y[i] = 0.0f;
#pragma unroll 4
  for (int c = cut - 1; c <= last; ++c) {
    const int64_t row = row_of(c);
    const float2 ml = *reinterpret_cast<const float2*>(p.partial_ml + row * 2);
    const float f = tree_ex2(ml.x - ref);
    float x[V];
    if constexpr (V == 4) {
      const float4 v = *reinterpret_cast<const float4*>(p.partial + row * HD + lane * 4);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(p.partial + row * HD + lane * 2);
      x[0] = v.x, x[1] = v.y;
    }
    weight = fmaf(ml.y, f, weight);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (ml.y != 0.0f) y[i] = fmaf(x[i], f, y[i]);
  }
  const int t = (m.row0 + r) / p.group;
  const int64_t packed = m.start + t;
  const int head = m.head * p.group + (m.row0 + r) - t * p.group;
  const float scale = weight == 0.0f ? 0.0f : 1.0f / weight;
  T* o = static_cast<T*>(p.o) + packed * p.o_token + static_cast<int64_t>(head) * p.o_head;
  if (lane * V < p.head_dim) {
    if constexpr (V == 4) {
      *reinterpret_cast<uint2*>(o + lane * 4) = make_uint2(El<T>::pack2(y[0] * scale, y[1] * scale), El<T>::pack2(y[2] * scale, y[3] * scale));
    } else {
      *reinterpret_cast<uint32_t*>(o + lane * 2) = El<T>::pack2(y[0] * scale, y[1] * scale);
    }
  }
  if (p.lse && lane == 0)
    p.lse[packed * p.q_heads + head] = weight == 0.0f ? -CUDART_INF_F : (top - kShift + __log2f(weight)) * 0.6931471805599453f;
}

}  // namespace eg
