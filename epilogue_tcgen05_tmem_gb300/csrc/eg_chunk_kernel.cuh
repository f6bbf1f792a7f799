// eg_chunk_kernel.cuh -- attention of chunks of new tokens over a paged cache,
// all of it or a sliding window and the first places.
//
// Mathematics.  The rows of one item are a group of a sequence's new tokens
// times the G query heads that share a cached head: for key tiles of 128,
//   S = Q K^T,  P = 2^(c S - m),  O += P V,  l += rowsum P,
// with c = scale log2 e and m a row reference at least the row maximum less 8:
// O and l are only brought to a new reference when the maximum grew by more
// than 2^8, which few tiles do.  So weights are formed against the reference at
// hand while the maximum is formed beside them, and a tile that turns out too
// high is done again.  Weights are rounded to 16 bits for the second product,
// whose operands are: at most 2^-8 (bf16) or 2^-11 (fp16) of each weight, the
// output type's own rounding, which makes the error against 64 bits up to 1.4
// times that of weights in float32.  l sums them before that rounding, in
// float32 as S, O and m are.
//
// Work.  Every item has units for the places that its rows attend to (see
// kChunkFixed); all items' units in a row are cut into equal ranges, one for
// each CTA (one CTA an SM), on the device from the sequences' lengths.  An item
// that a cut divides leaves float32 partial results that its last CTA or a
// second small kernel joins in a fixed order, so equal inputs give equal bits.
// Tiles outside a window are not looked at, and boxes of keys that no row of
// the item attends to are not loaded.
//
// One CTA: a producer warp (TMA boxes of pages into a ring of 128-key tiles, K
// and V alike), two issuing warps (tcgen05.mma), two softmax warpgroups, and a
// warp that walks the range for the warpgroups and fetches queries.  S and O of
// both warpgroups fill tensor memory (4 x 128 columns); P overwrites S as 16-bit
// values and feeds the second product from there.  With at most 128 rows the
// warpgroups take turns on the key tiles and are joined at the end of the range;
// with more rows (a pair) each has 128 of them and K and V tiles are used twice.
//
// Measured in succession, and what bounds it.
// One prompt of 8192 tokens, 32 query heads over 8 cached: 402 to 435 us from
// run to run, 1.26 to 1.37 PFLOP/s of the 1.90 of a plain product; two chunks of
// 512 after 65536 and 98304: 888 to 978 us, 1.41 to 1.55.  There a pair of
// row tiles takes 2800 cycles a key tile where its products take 2060: from a
// warpgroup's weights to its next scores, one after the other, pass 180 cycles
// until the issuer sees them, 1300 of products and their start, 270 until the
// scores are seen, 920 of weights, 220 of storing them.  One issuer for both was
// 483 us for the prompt (each wait of the issuer costs 200 cycles that no
// product hides), two that do not take turns 494 us (the warpgroups fall into
// step), tiles that are masked through the fast path too 436 us.
// Five prompts of 700 to 4001 tokens, 64 query heads over 8 cached, a window of
// 1024: 511 to 541 us; an item has 9.3 tiles, three of them edges, and 7000
// cycles from its last product to the next item's first.
// 64 single tokens with a window of 4096: 176 us, 5.6 TB/s of the 6.8 that a
// copy reaches (without a window 573 us, 6.6 TB/s).
#pragma once
#include "eg_attn.cuh"
#include "eg_chunk.h"

namespace eg {

constexpr int kChunkThreads = 384;
constexpr uint32_t kChunkKeys = 128;
constexpr int64_t kChunkKept = 64 << 20;  // bytes of keys and values that the L2 (of 129 MB) keeps beside the rest

// One sequence's lengths, cut to what the table, the packed rows and the plan
// hold, and its items: row groups (of item_tokens tokens with the heads that
// share a cached one) of each cached head.  `team` neighbouring groups are one
// super: as many neighbouring CTAs (a team) have the same range of supers'
// units, each one group of every super, so that they read the same keys and
// values at the same time.
struct ChunkSeq {
  int32_t start, n;    // packed rows
  int32_t ctx, keys;   // cached places, with the new tokens
  int32_t groups;      // items of a cached head
  int32_t low_groups;  // those of them whose window starts at place 0
  int32_t team, supers;
  int32_t last_cost;   // row tiles of the last super's groups, at most
};

__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams& p, int32_t team, int32_t start, int32_t n, int32_t ctx) {
  ChunkSeq s;
  const int32_t room = static_cast<int32_t>(p.table_stride * p.page_size);
  s.start = start, s.n = n, s.ctx = ctx;
  s.keys = min(ctx + n, room);
  s.groups = (n + p.item_tokens - 1) / p.item_tokens;
  s.low_groups = p.window == 0 ? s.groups : p.window > ctx ? min(s.groups, (p.window - ctx - 1) / p.item_tokens + 1) : 0;
  s.team = team, s.supers = (s.groups + team - 1) / team;
  const bool more = s.groups - (s.supers - 1) * team > 1;
  s.last_cost = p.q_tiles == 2 && (more || (n - (s.groups - 1) * p.item_tokens) * p.group > p.tile_rows) ? 2 : 1;
  return s;
}
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams& p, int32_t team, int b) {
  const int32_t room = static_cast<int32_t>(p.table_stride * p.page_size);
  const int32_t from = __ldg(p.q_start + b), to = __ldg(p.q_start + b + 1), ctx = __ldg(p.context_lens + b);
  const int32_t start = min(max(from, 0), p.tokens);
  return chunk_seq(p, team, start, min(min(max(to, start), p.tokens) - start, p.max_chunk), min(max(ctx, 0), room));
}

// Units are places: a super counts some span of places, an estimate of what the
// rows of its last group attend to, once for each of an item's row tiles, and
// kChunkFixed more for what an item costs beside its tiles.  Spans are linear in
// the super, so that their sums need no loop.  Tile k of an item belongs to the
// CTA that has the super's unit fixed + min(128 k, span - 1), times the row
// tiles.
constexpr int32_t kChunkFixed = 512;

__device__ __forceinline__ int64_t chunk_span(const ChunkParams& p, const ChunkSeq& s, int32_t super) {
  const int32_t g = min((super + 1) * s.team, s.groups) - 1;
  if (g < s.low_groups) return static_cast<int64_t>(s.ctx) + (g + 1) * static_cast<int64_t>(p.item_tokens);
  return static_cast<int64_t>(p.item_tokens) + p.window + min(p.sinks, s.ctx);
}
// Units of the first supers of a cached head, were all of them full.
__device__ __forceinline__ int64_t chunk_before(const ChunkParams& p, const ChunkSeq& s, int32_t super) {
  const int64_t low = min(super, s.low_groups / s.team), rest = super - low, tokens = static_cast<int64_t>(s.team) * p.item_tokens;
  const int64_t places = low * (kChunkFixed + static_cast<int64_t>(s.ctx)) + tokens * (low * (low + 1) / 2) +
                         rest * (kChunkFixed + static_cast<int64_t>(p.item_tokens) + p.window + min(p.sinks, s.ctx));
  return places * p.q_tiles;
}
// Units of a cached head's supers.
__device__ __forceinline__ int64_t chunk_of_head(const ChunkParams& p, const ChunkSeq& s) {
  if (s.supers == 0) return 0;
  return chunk_before(p, s, s.supers - 1) + (kChunkFixed + chunk_span(p, s, s.supers - 1)) * s.last_cost;
}
__device__ __forceinline__ int64_t chunk_units(const ChunkParams& p, const ChunkSeq& s) { return chunk_of_head(p, s) * p.kv_heads; }

// An item: its rows, and the key tiles that any of them attends to: `sink_tiles`
// from the first on, then those from `low_tile` on.
struct ChunkItem {
  int32_t row0, rows;
  int32_t cost;             // row tiles
  int32_t lo, hi;           // places of the window that any row attends to, [lo, hi)
  int32_t sinks;            // first places that rows attend to, window or not
  int32_t sink_tiles, low_tile, tiles;
  int32_t unit_cost;        // of the super's units
  int64_t span;             // units of one row tile, without the fixed ones
  __device__ __forceinline__ int64_t units() const { return (kChunkFixed + span) * unit_cost; }
  // the item's tiles that have their first unit before unit `in` of it
  __device__ __forceinline__ int32_t tiles_before(int64_t in) const {
    const int64_t u = unit_cost == 2 ? (in + 1) >> 1 : in;  // units of one row tile, rounded up
    if (u <= kChunkFixed) return 0;
    if (u >= kChunkFixed + span) return tiles;
    return static_cast<int32_t>(min(static_cast<int64_t>(tiles), (u - kChunkFixed + 127) >> 7));
  }
  __device__ __forceinline__ int64_t first_unit(int32_t tile) const {
    return (kChunkFixed + min(static_cast<int64_t>(tile) << 7, span - 1)) * unit_cost;
  }
};
// The item of a team's member in a super: one without tiles where the sequence
// has no such group.
__device__ __forceinline__ ChunkItem chunk_item(const ChunkParams& p, const ChunkSeq& s, int32_t super, int32_t member) {
  ChunkItem item{};
  const int32_t g = super * s.team + member;
  item.unit_cost = super + 1 == s.supers ? s.last_cost : p.q_tiles;
  item.span = chunk_span(p, s, super);
  if (g >= s.groups) return item;
  const int32_t t0 = g * p.item_tokens, tokens = min(s.n - t0, p.item_tokens);
  item.row0 = t0 * p.group, item.rows = tokens * p.group;
  item.cost = item.rows > p.tile_rows ? 2 : 1;
  item.hi = min(s.ctx + t0 + tokens, s.keys);
  item.lo = p.window ? max(0, s.ctx + t0 - p.window + 1) : 0;
  item.sinks = min(p.sinks, item.hi);
  const int32_t end = (item.hi + 127) >> 7;
  item.low_tile = item.lo >> 7;
  item.sink_tiles = min((item.sinks + 127) >> 7, item.low_tile);
  // rows that attend to nothing still have a tile, so that they are written
  if (item.low_tile >= end && item.sink_tiles == 0) item.low_tile = end - 1;
  item.tiles = item.sink_tiles + max(end - item.low_tile, 0);
  return item;
}

// The first unit of team c, and the team that has unit u, when `total` units
// are cut into `ctas` equal ranges.
__device__ __forceinline__ int64_t chunk_from(int64_t total, int32_t ctas, int32_t c) { return total * c / ctas; }
__device__ __forceinline__ int32_t chunk_owner(int64_t total, int32_t ctas, int64_t u) {
  return static_cast<int32_t>(((u + 1) * ctas + total - 1) / total) - 1;
}

constexpr int kChunkNear = 16;  // sequences whose lengths a CTA keeps in shared memory

// Consecutive key tiles of one item.
struct ChunkSegment {
  ChunkSeq seq;
  ChunkItem item;
  int32_t b, head;
  int32_t first, count;
  int32_t more;        // 0: there is none
  int64_t begin;       // the first unit of its item
  __device__ __forceinline__ bool whole() const { return first == 0 && count == item.tiles; }
  // the first place of the segment's tile i
  __device__ __forceinline__ int32_t place(int32_t i) const {
    const int32_t k = first + i;
    return (k < item.sink_tiles ? k : item.low_tile + k - item.sink_tiles) << 7;
  }
};

// A walk over a CTA's range, one segment at a time.
struct ChunkWalk : ChunkSegment {
  int64_t at, to;
  int32_t super, member;      // the super that `at` is in, and which of its groups this CTA has
  const int32_t (*near_)[4];  // start, n, ctx of the sequences from near_b on
  int32_t near_b;

  __device__ __forceinline__ void load(const ChunkParams& p) {
    const int i = b - near_b;
    seq = i < kChunkNear ? chunk_seq(p, seq.team, near_[i][0], near_[i][1], near_[i][2]) : chunk_seq(p, seq.team, b);
  }
  // to unit `from`, in sequence b, whose units start at `before`
  __device__ __forceinline__ void start(const ChunkParams& p, int32_t team, int32_t member_, int32_t b_, int64_t before, int64_t from, int64_t to_) {
    b = b_, at = from, to = to_, member = member_;
    seq.team = team;
    load(p);
    const int64_t each = chunk_of_head(p, seq), in = from - before;
    head = static_cast<int32_t>(in / each);
    const int64_t rest = in - head * each;
    int32_t low = 0, high = seq.supers - 1;  // the last super whose units start at `rest` or before
    while (low < high) {
      const int32_t mid = (low + high + 1) >> 1;
      if (chunk_before(p, seq, mid) <= rest) low = mid;
      else high = mid - 1;
    }
    super = low;
    begin = before + head * each + chunk_before(p, seq, super);
    item = chunk_item(p, seq, super, member);
  }
  __device__ __forceinline__ bool next(const ChunkParams& p) {
    for (;;) {
      if (at >= to) return false;
      if (at >= begin + item.units()) {
        begin += item.units();
        if (++super == seq.supers) {
          super = 0;
          if (++head == p.kv_heads) {
            head = 0;
            do {
              ++b;
              load(p);
            } while (seq.supers == 0);
          }
        }
        item = chunk_item(p, seq, super, member);
      }
      const int64_t in = at - begin, take = min(item.units() - in, to - at);
      at += take;
      first = item.tiles_before(in);
      count = item.tiles_before(in + take) - first;
      if (count > 0) return true;
    }
  }
};

// Shared state after the tiles.
struct ChunkShared {
  uint64_t full[12], empty[12];   // ring stages
  uint64_t s_full[2], p_ready[2], o_done[2];
  uint64_t q_full, q_empty, exchange, drained;
  uint64_t turn[2];               // a pair's issuers issue in turn
  uint64_t told[2], done[2];      // segments for the softmax warpgroups
  uint32_t tmem;
  int32_t abort;
  int32_t poisoned[2][2];         // a warpgroup's last odd and even segment (counted from 1) that found a value that is not finite
  int32_t b;
  int32_t joins;                  // this CTA has the last part of an item
  int64_t before;
  int32_t near_[kChunkNear][4];
  ChunkSegment segments[2];
  union {
    float2 stats[2][128];         // a warpgroup's row references and weights
    int64_t warps[2][12];         // before any: units of each warp's sequences,
    int64_t sums[5][12];          // and what the size of teams is chosen by
  };
};
static_assert(sizeof(ChunkShared) <= ChunkSmem<64>::kExtra, "fits the room after the tiles");

// GROUPED: a box holds both halves of the columns, which lie in shared memory by
// turns, 8 keys of each (ChunkParams::grouped); else each half has a box, and
// all keys of the first half come first.
template <typename T, int HD, bool GROUPED>
__global__ void __launch_bounds__(kChunkThreads, 1)
    chunk_kernel(const ChunkParams p, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v) {
  constexpr uint32_t kTile = ChunkSmem<HD>::kTileBytes;
  constexpr int kChunks = HD / 64;           // 64-column parts of a tile, 16 KB each
  constexpr uint32_t kPart = 128u * 128u;    // bytes of one part
  // keys and values: bytes from 8 keys to the next 8, and from the first half of the columns to the other
  constexpr uint32_t kKeys8 = GROUPED ? 2048u : 1024u, kHalf = GROUPED ? 1024u : kPart;
  constexpr uint32_t kFmt = sizeof(T) == 2 && El<T>::kBf16 ? 1u : 0u;
  // the scores' reference lies this far below their maximum, so that small
  // weights keep their bits as fp16 (its normal numbers end at 2^-14)
  constexpr float kShift = El<T>::kBf16 ? 0.0f : 7.0f;
  constexpr float kGrow = 8.0f;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* q_smem = smem;
  uint8_t* ring = smem + p.q_tiles * kTile;
  ChunkShared& sh = *reinterpret_cast<ChunkShared*>(ring + p.stages * kTile);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t stages = p.stages;

  griddep_launch_dependents();

  if (tid == 0) {
    for (uint32_t i = 0; i < stages; ++i) mbar_init(&sh.full[i], 1), mbar_init(&sh.empty[i], 2);
    for (int i = 0; i < 2; ++i) mbar_init(&sh.s_full[i], 1), mbar_init(&sh.p_ready[i], 4), mbar_init(&sh.o_done[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sh.told[i], 1), mbar_init(&sh.done[i], 8);
    mbar_init(&sh.turn[0], 1), mbar_init(&sh.turn[1], 1);
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 2);
    mbar_init(&sh.exchange, 256);
    mbar_init(&sh.drained, 2);
    fence_mbar_init();
    sh.abort = 0;
    for (int i = 0; i < 4; ++i) sh.poisoned[i >> 1][i & 1] = 0;
  }

  // ---- CTAs of a team.  Where a sequence's row groups on different CTAs go
  // through more keys and values than the L2 keeps, each read them from memory
  // by itself (two chunks of 512 tokens after 65536 and 98304 places: 5.4 GB for
  // 0.69 GB, 1029 us for 966); as a team they read them once.  A team of eight, four
  // or two is taken where its CTAs without a group and its rounding up cost at
  // most a sixteenth more.
  int32_t team = 1;
  if (p.teams) {
    int64_t sums[5] = {0, 0, 0, 0, 0};  // units of one, two, four, eight; places
    for (int b = tid; b < p.batch; b += kChunkThreads) {
      ChunkSeq s = chunk_seq(p, 1, b);
      sums[0] += chunk_units(p, s);
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        s = chunk_seq(p, 1 << i, s.start, s.n, s.ctx);
        sums[i] += chunk_units(p, s) << i;
      }
      if (s.groups > 1) sums[4] += p.window ? min(static_cast<int64_t>(s.keys), static_cast<int64_t>(p.window) + s.n) : s.keys;
    }
#pragma unroll
    for (int i = 0; i < 5; ++i) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sums[i] += __shfl_xor_sync(0xffffffffu, sums[i], o);
      if (lane == 0) sh.sums[i][warp] = sums[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      sums[i] = 0;
#pragma unroll
      for (int w = 0; w < kChunkThreads / 32; ++w) sums[i] += sh.sums[i][w];
    }
    if (sums[4] * p.kv_heads * HD * 4 > kChunkKept)
#pragma unroll
      for (int i = 1; i < 4; ++i)
        if (sums[i] * 16 <= sums[0] * 17) team = 1 << i;
    __syncthreads();
  }

  // ---- this CTA's range of units.  One pass over the sequences where every
  // thread has one; else a pass for the total and one to find the place.
  const bool once = p.batch <= kChunkThreads;
  int64_t mine = 0;
  ChunkSeq seq{};
  for (int b = tid; b < p.batch; b += kChunkThreads) {
    seq = chunk_seq(p, team, b);
    mine += chunk_units(p, seq);
  }
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) sh.warps[0][warp] = upto;
  __syncthreads();
  int64_t total = 0, base = 0;
#pragma unroll
  for (int w = 0; w < kChunkThreads / 32; ++w) {
    if (w < warp) base += sh.warps[0][w];
    total += sh.warps[0][w];
  }
  // a range is no shorter than a tile's units, so that a CTA between the first
  // and the last of an item has a tile of it
  const int32_t ctas = static_cast<int32_t>(min(static_cast<int64_t>(gridDim.x / team), total >> (p.q_tiles == 2 ? 8 : 7)));
  const int32_t number = blockIdx.x / team, member = blockIdx.x % team;
  if (number >= ctas) {
    if (tid == 0 && !p.arrivals) p.meta[blockIdx.x].rows = 0;
    return;
  }
  const int64_t from = chunk_from(total, ctas, number), to = chunk_from(total, ctas, number + 1);
  if (once) {
    if (base + upto - mine <= from && from < base + upto) sh.b = tid, sh.before = base + upto - mine;
  } else {
    int64_t before = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kChunkThreads) {
      const int64_t units = b0 + tid < p.batch ? chunk_units(p, chunk_seq(p, team, b0 + tid)) : 0;
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
      for (int w = 0; w < kChunkThreads / 32; ++w) {
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
  if (once ? tid >= near_b && tid < min(near_b + kChunkNear, p.batch) : tid < kChunkNear && near_b + tid < p.batch) {
    if (!once) seq = chunk_seq(p, team, near_b + tid);
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
  ChunkWalk walk;
  walk.near_ = sh.near_, walk.near_b = near_b;
  walk.start(p, team, member, near_b, sh.before, from, to);
  if (warp == 8) {
    // ------------------------------------------------------- producer ----
    uint32_t pos = 0;  // loads so far
    bool ok = true;
    const int boxes = 128 / p.box_rows;
    if (lane == 0) tma_prefetch_desc(&map_k), tma_prefetch_desc(&map_v);
    while (ok && walk.next(p)) {
      const int32_t* table = p.block_table + walk.b * p.table_stride;
      auto place = [&](int tile, int* page, int* off) {
        const int key = walk.place(tile) + lane * p.box_rows;
        // a box none of whose places any row attends to is left out
        const bool has = lane < boxes && key < walk.item.hi && (key < walk.item.sinks || key + p.box_rows > walk.item.lo);
        *page = -1, *off = 0;
        if (has) {
          *page = __ldg(table + key / p.page_size);
          *off = key % p.page_size;
        }
        return has;
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
          const uint32_t dst = smem_u32(ring + slot * kTile) + lane * p.box_rows * (kKeys8 / 8);
          if constexpr (GROUPED) {
            const bool there = page >= 0 && page < p.num_pages;  // reads as zeros else
            if (p.grouped == 1) tma_load_5d(dst, map, &sh.full[slot], 0, 0, 2 * walk.head, off >> 3, page);
            else tma_load_5d(dst, map, &sh.full[slot], 0, 0, 0, off >> 3, there ? page * p.kv_heads + walk.head : -1);
          } else {
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
              tma_load_4d(dst + c * kPart, map, &sh.full[slot], c * 64, p.heads_inner ? walk.head : off, p.heads_inner ? off : walk.head, page);
          }
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
  } else if (warp != 11) {
    // -------------------------------------------------------- issuers ----
    // The first gives both softmax warpgroups their products where they take
    // turns on the key tiles.  For a pair each has a warpgroup of its own, so
    // that what one of them waits for and computes between its products passes
    // behind the other's; they issue in turn: else the two fall into step, with
    // both warpgroups at their weights while the tensor cores wait and the
    // other way round.  The whole warp walks, so that addresses stay in uniform
    // registers; one elected lane issues; places in the ring are stepped, not
    // divided out.
    //
    // Loads need not end in their order, and a wait for a turn of the ring
    // passes at once while the turn before is not over.  So whoever waits for
    // a place has waited for the one a ring's length before, or knows of
    // products that came after it.
    constexpr uint32_t kIdescS = idesc_f32acc(kFmt, kFmt, 128, 128);
    constexpr uint32_t kIdescO = idesc_f32acc(kFmt, kFmt, 128, HD) | (1u << 16);  // values: keys are the strided index
    const uint32_t mine = warp - 9;
    const uint64_t q_desc = sdesc_k_sw128(smem_u32(q_smem));
    constexpr uint64_t kMore = static_cast<uint64_t>((kKeys8 - 1024) >> 4) << 32;  // of the stride from 8 keys to the next
    const uint64_t k_desc = sdesc_k_sw128(smem_u32(ring)) + kMore, v_desc = sdesc_mn_sw128(smem_u32(ring), kHalf) + kMore;
    uint32_t segment = 0, used0 = 0, used1 = 0;  // segments, and tiles given to each warpgroup
    uint32_t slot0 = 0, turn0 = 0;               // the segment's first place in the ring, and how often the ring was full
    uint32_t turns = 0;                          // of a pair
    auto step = [&](uint32_t& slot, uint32_t& turn, uint32_t by) {
      slot += by;
      if (slot >= stages) slot -= stages, ++turn;
    };
    auto my_turn = [&]() { return wait_all(&sh.turn[mine], mine ? turns : turns + 1); };
    auto pass = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.turn[mine ^ 1]);
      ++turns;
    };
    // The second warpgroup's products change hands between a pair and other
    // items.  Who takes them over waits until the last of the other issuer's
    // are over: else scores come where that warpgroup's weights still lie, and
    // a wait for its weights passes at once.  The other's turns are over first,
    // so the wait for its last sums is for no earlier ones.
    bool theirs = false;
    bool ok = true;
    while (ok && walk.next(p)) {
      const uint32_t count = walk.count;
      const bool pair = walk.item.cost == 2;
      if (pair != (mine == 1)) theirs = true;
      uint32_t slot_k = slot0, turn_k = turn0, slot_v = slot0, turn_v = turn0;
      step(slot_v, turn_v, count == 1 ? 1 : 2);
      if (!(ok = wait_all(&sh.q_full, segment))) break;
      // O += P V of a warpgroup's tile
      auto sums = [&](uint32_t s, bool add) {
        const uint64_t v = v_desc + (slot_v * kTile >> 4);
        const uint32_t w = tmem + s * 128, o = w + 256;
        umma_f16_ts(o, w, v, kIdescO, add ? 1 : 0);
#pragma unroll
        for (int k = 1; k < 8; ++k) umma_f16_ts_add(o, w + k * 8, v + k * (2 * kKeys8 >> 4), kIdescO);
        umma_commit(&sh.o_done[s]);
        umma_commit(&sh.empty[slot_v]);
        if (!pair) umma_commit(&sh.empty[slot_v]);  // for the other issuer
      };
      // S = Q K^T of its next one
      auto scores = [&](uint32_t s) {
        const uint64_t q = q_desc + (pair && s ? kTile >> 4 : 0), key = k_desc + (slot_k * kTile >> 4);
        const uint32_t d = tmem + s * 128;
        umma_f16(d, q, key, kIdescS, 0);
#pragma unroll
        for (int k = 1; k < HD / 16; ++k) {
          umma_f16_add(d, q + (((k / 4) * kPart + (k % 4) * 32) >> 4), key + (((k / 4) * kHalf + (k % 4) * 32) >> 4), kIdescS);
        }
        umma_commit(&sh.s_full[s]);
        umma_commit(&sh.empty[slot_k]);
        if (!pair) umma_commit(&sh.empty[slot_k]);
      };
      // the keys of tile i are 2 i - 1 places on (those of tile 0 at none),
      // its values 2 i + 2, the last tile's one less
      auto next_k = [&](uint32_t i) { step(slot_k, turn_k, i == 0 ? 1 : 2); };
      auto next_v = [&](uint32_t i) { step(slot_v, turn_v, i + 2 == count ? 1 : 2); };
      if (pair) {
        // tile i's keys, then the values of the one before, in the ring's order
        if (!(ok = wait_all(&sh.full[slot_k], turn_k) && my_turn())) break;
        if (mine && theirs) {
          if (used1 > 0 && !(ok = wait_all(&sh.o_done[1], used1 - 1))) break;
          theirs = false;
        }
        tc_fence_after();
        if (elect_one()) scores(mine);
        pass();
        next_k(0);
        uint32_t weights = mine ? used1 : used0;
        for (uint32_t i = 1; i < count; ++i, ++weights) {
          if (!(ok = wait_all(&sh.full[slot_k], turn_k) && wait_all(&sh.full[slot_v], turn_v) && my_turn() && wait_all(&sh.p_ready[mine], weights))) break;
          tc_fence_after();
          if (elect_one()) sums(mine, i > 1), scores(mine);
          pass();
          next_k(i);
          next_v(i - 1);
        }
        if (!ok) break;
        if (elect_one()) umma_commit(&sh.q_empty);
        if (!(ok = wait_all(&sh.full[slot_v], turn_v) && my_turn() && wait_all(&sh.p_ready[mine], weights))) break;
        tc_fence_after();
        if (elect_one()) sums(mine, count > 1);
        pass();
        used0 += count, used1 += count;
      } else if (mine == 0) {
        // scores run two tiles ahead of the sums
        for (uint32_t j = 0; j < count + 2; ++j) {
          const uint32_t s = j & 1;
          if (j >= 2) {
            if (!(ok = wait_all(&sh.full[slot_v], turn_v) && wait_all(&sh.p_ready[s], (s ? used1 : used0) + (j >> 1) - 1))) break;
            tc_fence_after();
            if (elect_one()) sums(s, j >= 4);
            __syncwarp();
            next_v(j - 2);
          }
          if (j < count) {
            if (!(ok = wait_all(&sh.full[slot_k], turn_k))) break;
            if (s && theirs) {
              if (!(ok = my_turn() && wait_all(&sh.o_done[1], used1 - 1))) break;
              theirs = false;
            }
            tc_fence_after();
            if (elect_one()) {
              scores(s);
              if (j + 1 == count) umma_commit(&sh.q_empty), umma_commit(&sh.q_empty);
            }
            __syncwarp();
            next_k(j);
          }
        }
      }
      if (!ok) break;
      if (!pair) used0 += (count + 1) / 2, used1 += count / 2;
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
    // ---------------------------------- the walk's segments and queries ----
    if (tid == kChunkThreads - 1 && !p.arrivals) {
      // The joining kernel's work at this cut: the item that it divides, where
      // it is the item's first.  The CTAs with the item's first tile and with
      // its last: those between them have some too.
      ChunkMeta m{};
      if (number > 0 && from > walk.begin && chunk_from(total, ctas, number - 1) <= walk.begin) {
        m.lead = chunk_owner(total, ctas, walk.begin + walk.item.first_unit(0)) * team + member;
        m.last = chunk_owner(total, ctas, walk.begin + walk.item.first_unit(max(walk.item.tiles - 1, 0))) * team + member;
        m.team = team, m.rows = m.lead == m.last ? 0 : walk.item.rows;
        m.start = walk.seq.start, m.row0 = walk.item.row0, m.head = walk.head;
      }
      p.meta[blockIdx.x] = m;
    }
    // The walk for the softmax warpgroups, whose registers have no room for it,
    // and the queries: a box is `box_tokens` tokens by the heads that share a
    // cached one; lane i has box i of each tile.
    const int box = p.box_tokens * p.group, boxes = p.tile_rows / box;
    uint32_t segment = 0;
    for (bool more = true; more; ) {
      if (!wait_all(&sh.done[segment & 1], (segment >> 1) + 1)) break;
      more = walk.next(p);
      walk.more = more;
      if (lane == 0) {
        sh.segments[segment & 1] = walk;
        mbar_arrive(&sh.told[segment & 1]);
      }
      if (!more || !wait_all(&sh.q_empty, segment + 1)) break;
      const int all = (walk.item.rows + box - 1) / box;  // boxes that hold a row
      if (lane == 0) mbar_arrive_expect_tx(&sh.q_full, all * box * 128u * kChunks);
      __syncwarp();
      for (int i = lane; i < all; i += 32) {
        const int tile = i >= boxes ? 1 : 0, in = i - tile * boxes;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          tma_load_3d(smem_u32(q_smem) + tile * kTile + c * kPart + in * box * 128u, &map_q, &sh.q_full, c * 64, walk.head * p.group,
                      walk.seq.start + walk.item.row0 / p.group + i * p.box_tokens);
      }
      ++segment;
    }
    if (segment > 0) mbar_wait(&sh.q_full, (segment - 1) & 1, p.wait_limit_ns);  // leaves no copy in flight behind
  }
  } else {
    // -------------------------------------------------------- softmax ----
    setmaxnreg_inc<208>();
    const int s = warp >> 2;            // the warpgroup
    const int row_in = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t t_s = tmem + lanes + s * 128, t_o = tmem + lanes + 256;
    const float c = p.scale_log2;
    const uint64_t c2 = pack64(__float_as_uint(c), __float_as_uint(c));
    uint32_t base = 0, uses = 0, exchanges = 0;
    int32_t segment = 0;
    bool ok = true;
    for (;;) {
      const ChunkSegment& walk = sh.segments[segment & 1];
      if (!(ok = wait_all(&sh.told[segment & 1], segment >> 1)) || !walk.more) break;
      ++segment;
      const bool pair = walk.item.cost == 2;
      const int count = walk.count, hi = walk.item.hi, lo = walk.item.lo, sinks = walk.item.sinks;
      const int tile_row0 = pair ? s * p.tile_rows : 0;
      const int r = tile_row0 + row_in;
      const bool valid = row_in < p.tile_rows && r < walk.item.rows;
      const bool busy = __any_sync(0xffffffffu, valid);  // the warp has a row
      const int t = (walk.item.row0 + r) / p.group;
      const int64_t packed = walk.seq.start + t;
      const int head = walk.head * p.group + (walk.item.row0 + r) - t * p.group;
      // what this row attends to: [from_place, to_place) and the places before `sinks`
      const int to_place = valid ? min(walk.seq.ctx + t + 1, hi) : 0;
      const int from_place = p.window ? max(walk.seq.ctx + t - p.window + 1, 0) : 0;
      // what every row of the warpgroup's tile attends to
      const int all_to = min(walk.seq.ctx + (walk.item.row0 + tile_row0) / p.group + 1, hi);
      const int all_from = p.window ? walk.seq.ctx + (walk.item.row0 + min(tile_row0 + p.tile_rows, walk.item.rows) - 1) / p.group - p.window + 1 : 0;
      // and what every row of the item does
      const int item_to = min(walk.seq.ctx + walk.item.row0 / p.group + 1, hi);
      const int item_from = p.window ? walk.seq.ctx + (walk.item.row0 + walk.item.rows - 1) / p.group - p.window + 1 : 0;
      // 32 bits of which places from `place` on this row attends to
      auto seen_bits = [&](int place) -> uint32_t {
        auto first_bits = [](int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; };
        const int sink = valid ? sinks - place : 0;
        return first_bits(to_place - place) & (~first_bits(from_place - place) | first_bits(sink));
      };
      float m = -CUDART_INF_F, l = 0.0f;  // m: the reference (log2), before the shift
      bool fresh = true;                  // no tile of this segment yet
      for (int i = pair ? 0 : s; ok && i < count; i += pair ? 1 : 2) {
        const int key0 = walk.place(i);
        const int key1 = key0 + static_cast<int>(kChunkKeys);
        const bool edge = key1 > all_to || (key0 < all_from && key1 > sinks);
        if (key1 > item_to || (key0 < item_from && key1 > sinks)) {
          // Before a pair's scores come: values of places that no row attends to
          // become zero, and so do other values that are not finite: a weight
          // of zero times one would reach rows that do not attend to it
          // (`repair` adds it to those that do).  The flag is there before the
          // zeros, for the other warpgroup that may find those.
          // A wait for a turn of the ring needs the turn before to be over: a
          // pair's warpgroup has used the keys of tile i - 1, which lie behind
          // that in a ring of five or more; one that takes every other tile
          // has to have the scores of this one, whose keys do in any.
          if (!pair && !(ok = wait_all(&sh.s_full[s], uses))) break;
          const uint32_t at = base + attn_pos_v(i, count), slot = at % stages;
          if (!(ok = wait_all(&sh.full[slot], at / stages))) break;
          const int key = key0 + row_in;
          uint8_t* v_row = ring + slot * kTile + (row_in >> 3) * kKeys8 + (row_in & 7) * 128;
          // a lane's pieces of its row, in an order that keeps lanes off each other's banks
          auto piece = [&](int j) { return reinterpret_cast<uint4*>(v_row + (j >> 3) * kHalf + ((j ^ lane) & 7) * 16); };
          if (key >= hi || (key < lo && key >= sinks)) {
#pragma unroll
            for (int j = 0; j < kChunks * 8; ++j) *piece(j) = make_uint4(0, 0, 0, 0);
          } else {
            // an exponent of ones carries into the sign's place
            constexpr uint32_t kInf = El<T>::kBf16 ? 0x7F80u : 0x7C00u, kInf2 = kInf << 16 | kInf, kOne2 = 0x80008000u - kInf2;
            uint32_t bad = 0;
#pragma unroll
            for (int j = 0; j < kChunks * 8; ++j) {
              const uint4 v = *piece(j);
              bad |= ((v.x & kInf2) + kOne2) | ((v.y & kInf2) + kOne2) | ((v.z & kInf2) + kOne2) | ((v.w & kInf2) + kOne2);
            }
            if (bad & 0x80008000u) {
              *reinterpret_cast<volatile int32_t*>(&sh.poisoned[s][segment & 1]) = segment;
              __threadfence_block();
#pragma unroll 1
              for (int j = 0; j < kChunks * 8; ++j) {
                uint32_t* word = reinterpret_cast<uint32_t*>(piece(j));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if ((word[k] & kInf) == kInf) word[k] &= 0xFFFF0000u;
                  if ((word[k] & (kInf << 16)) == (kInf << 16)) word[k] &= 0x0000FFFFu;
                }
              }
            }
          }
          fence_proxy_async_smem();
        }
        if (!(ok = wait_all(&sh.s_full[s], uses))) break;
        tc_fence_after();
        if (busy) {
          uint32_t w[64];  // the weights, two 16-bit values a word
          float high = -CUDART_INF_F, sum = 0.0f;
          bool careful = edge || fresh;
          if (!careful) {
            // Weights against the reference at hand, their maximum beside
            // them: where that turns out too high the tile is done again.
            const float ref = m == -CUDART_INF_F ? 0.0f : kShift - m;
            const uint64_t ref2 = pack64(__float_as_uint(ref), __float_as_uint(ref));
            uint32_t x[2][32];
            float top[2] = {-CUDART_INF_F, -CUDART_INF_F};
            uint64_t sum2[2] = {0, 0};
            tmem_ld32p(t_s, x[0]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t* y = x[q & 1];
              tmem_ld_wait();
              reg_fence<32>(y);
              if (q < 3) tmem_ld32p(t_s + (q + 1) * 32, x[(q + 1) & 1]);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                top[j & 1] = max3(top[j & 1], __uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1]));
                float a, b;
                unpack64(fma2(pack64(y[2 * j], y[2 * j + 1]), c2, ref2), &a, &b);
                a = attn_ex2(a), b = attn_ex2(b);
                sum2[j & 1] = add2(sum2[j & 1], pack64(__float_as_uint(a), __float_as_uint(b)));
                w[q * 16 + j] = El<T>::pack2(a, b);
              }
            }
            high = fmaxf(top[0], top[1]) * c;
            float sum_a, sum_b;
            unpack64(add2(sum2[0], sum2[1]), &sum_a, &sum_b);
            sum = sum_a + sum_b;
            careful = __any_sync(0xffffffffu, valid && high > m + kGrow);
          }
          if (careful) {
            uint32_t x[128];
#pragma unroll
            for (int j = 0; j < 4; ++j) tmem_ld32p(t_s + j * 32, x + j * 32);
            tmem_ld_wait();
            reg_fence<128>(x);
            if (edge) {
              // -infinity where the row does not attend to
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t bits = seen_bits(key0 + 32 * k);
                if (__all_sync(0xffffffffu, bits == 0xFFFFFFFFu)) continue;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (!(bits >> j & 1u)) x[k * 32 + j] = 0xFF800000u;
              }
            }
            float top[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
            for (int j = 0; j < 64; ++j) top[j & 1] = max3(top[j & 1], __uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
            high = fmaxf(top[0], top[1]);
            high = high == -CUDART_INF_F || !valid ? -CUDART_INF_F : high * c;
            if (fresh) {
              m = high;
            } else if (__any_sync(0xffffffffu, high > m + kGrow)) {
              // bring this row's sums to its new maximum
              const float next = fmaxf(m, high);
              const float f = next == m ? 1.0f : attn_ex2(m - next);
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
            const uint64_t ref2 = pack64(__float_as_uint(ref), __float_as_uint(ref));
            uint64_t sum2[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 64; ++j) {
              float a, b;
              unpack64(fma2(pack64(x[2 * j], x[2 * j + 1]), c2, ref2), &a, &b);
              a = attn_ex2(a), b = attn_ex2(b);
              sum2[j & 1] = add2(sum2[j & 1], pack64(__float_as_uint(a), __float_as_uint(b)));
              w[j] = El<T>::pack2(a, b);
            }
            float sum_a, sum_b;
            unpack64(add2(sum2[0], sum2[1]), &sum_a, &sum_b);
            sum = sum_a + sum_b;
          }
          l += sum;
          tmem_st32(t_s, w);
          tmem_st32(t_s + 32, w + 32);
          tmem_st_wait();
        }
        fresh = false;
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
      // A pair's warpgroups have rows of their own and go on by themselves; else
      // each has half the keys of all rows, and half the columns of the result.
      float2 own = make_float2(m, l), other = make_float2(-CUDART_INF_F, 0.0f);
      if (!pair) {
        sh.stats[s][row_in] = own;
        tc_fence_before();
        mbar_arrive(&sh.exchange);
        if (!(ok = wait_all(&sh.exchange, exchanges))) break;
        ++exchanges;
        tc_fence_after();
        other = sh.stats[s ^ 1][row_in];
      }
      // either warpgroup may have met the value first
      __threadfence_block();
      const bool repair = *reinterpret_cast<volatile int32_t*>(&sh.poisoned[0][segment & 1]) == segment ||
                          *reinterpret_cast<volatile int32_t*>(&sh.poisoned[1][segment & 1]) == segment;
      const float both = fmaxf(own.x, other.x);
      const float ref = both == -CUDART_INF_F ? 0.0f : both;
      const float f_own = attn_ex2(own.x - ref), f_other = attn_ex2(other.x - ref);
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
        // a lane's row goes out in whole sectors where they lie on them
        const bool wide = ((reinterpret_cast<uintptr_t>(p.o) | static_cast<uint64_t>(p.o_token) * 2 | static_cast<uint64_t>(p.o_head) * 2) & 31) == 0 &&
                          p.head_dim % 16 == 0;
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
          if (whole && wide) {
#pragma unroll
            for (int k = 0; k < kCols; k += 16) {
              if (j + k >= p.head_dim) continue;
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                y[e] = weight == 0.0f ? 0u : El<T>::pack2(__uint_as_float(a[k + 2 * e]) * scale, __uint_as_float(a[k + 2 * e + 1]) * scale);
              st_global_32(o + j + k, y);
            }
            continue;
          }
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
          // values that are not finite, to the rows that attend to them
          for (int k = 0; k < count * static_cast<int>(kChunkKeys); ++k) {
            const int key = walk.place(k >> 7) + (k & 127);
            if (!(seen_bits(key) & 1u)) continue;
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
      const bool joining = !whole && p.arrivals;
      if (joining) __threadfence();
      tc_fence_before();
      if (!pair || joining) {
        // the other warpgroup's accumulator is read: it may be written again
        mbar_arrive(&sh.exchange);
        if (!(ok = wait_all(&sh.exchange, exchanges))) break;
        ++exchanges;
      }
      tc_fence_after();
      if (joining) {
        // the CTA that leaves the last part of the item joins all of them
        const int32_t lead = chunk_owner(total, ctas, walk.begin + walk.item.first_unit(0)) * team + member;
        const int32_t last = chunk_owner(total, ctas, walk.begin + walk.item.first_unit(walk.item.tiles - 1)) * team + member;
        if (tid == 0) {
          const int before = atomicAdd(p.arrivals + lead, 1);
          sh.joins = before == (last - lead) / team;
          if (sh.joins) p.arrivals[lead] = 0;
          __threadfence();
        }
        mbar_arrive(&sh.exchange);
        if (!(ok = wait_all(&sh.exchange, exchanges))) break;
        ++exchanges;
        if (sh.joins) {
          const int rows = walk.item.rows, pieces = rows * (HD / 4);
          for (int i = tid; i < pieces; i += 256) {
            const int at_row = walk.item.row0 + i % rows, t_ = at_row / p.group;
            attn_join_piece<T, HD>(p, lead, last, team, i % rows, i / rows * 4, walk.seq.start + t_, walk.head * p.group + at_row - t_ * p.group);
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
// the main kernel leaves that to it: the blocks of cut x (where CTA x starts)
// serve the item whose first cut it is, eight rows each; which CTAs have parts
// of it the main kernel found (its two divisions of 64 bits in every thread
// here: 18 us for the prompt of 8192, so 13).  A thread has
// four columns of a row; a warp has eight rows of 16 columns, which is how they
// lie side by side.
template <typename T, int HD>
__global__ void __launch_bounds__(HD * 2) chunk_join_kernel(const ChunkParams p) {
  griddep_wait();
  const ChunkMeta m = p.meta[blockIdx.x + 1];
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.y * 8 + (lane & 7);
  if (r >= m.rows) return;
  const int t = (m.row0 + r) / p.group;
  attn_join_piece<T, HD>(p, m.lead, m.last, m.team, r, ((threadIdx.x >> 5) * 4 + (lane >> 3)) * 4, m.start + t, m.head * p.group + (m.row0 + r) - t * p.group);
}

}  // namespace eg
