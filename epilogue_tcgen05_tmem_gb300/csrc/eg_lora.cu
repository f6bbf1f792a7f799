// eg_lora.cu -- low-rank adapters of many requests beside a shared projection
// (include/eg_prompt.h has the formula).
//
// Two kernels over tiles of up to 128 rows of one sequence, so of one adapter.
// The first forms h = x A^T: a cluster shares a tile's columns of x, each CTA
// streams its part of x and A through a ring of TMA boxes into tcgen05.mma, and
// the parts are added through distributed shared memory in the cluster's order.
// The second, launched as the first's dependent, streams B in tiles of 128
// outputs, forms h B^T and adds base in its epilogue.  h goes between them as
// two 16-bit parts: h / 2^e = hi + lo with 2^e the row's size, so that the
// second product's operands lose nothing that shows next to the output's own
// rounding (fp16 needs the common size for its range); hi and lo are side by
// side along its inner dimension, against the same tile of B.
//
// Tiles of at most 16 rows (single tokens) take the second product the other
// way round: 128 outputs are the rows of tensor memory and the tokens its
// columns, so that one product covers 128 outputs with no idle rows and a warp
// writes neighbouring outputs of a token.  In other tiles a lane has a row, and
// rows go out through shared memory: stored from the lanes themselves, 32 rows
// an instruction, the second kernel took 96 us for the five prompts below, so
// 37 us.
//
// Measured in succession, bf16 (a copy reaches 6.8 TB/s).  Five prompts of 8191
// tokens, 5120 to 5120, rank 64, added to a base: 70 us, 3.7 TB/s; each kernel
// streams at 5.5 to 7 TB/s (11.6 us in the first, 29 in the second), and the
// rest is what they cannot overlap: finding the work, the first boxes, the sum
// over the cluster, the wait of the second for the first.  64 single tokens,
// nearly each with its own adapter, 4096 to 12288, rank 64: 41 us, 3.0 TB/s (45
// us with h's two parts one after the other and 64 inputs a stage).  Two prompts
// among 31 single tokens, 12288 to 4096, rank 128, fp16: 84 us; the first kernel
// reads x and A of 6 MB a tile from L2 at what an SM takes in.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <algorithm>
#include <atomic>

#include "../../include/eg_prompt.h"
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

constexpr int kTileRows = 128;  // rows of a tile, and outputs of one of the second product
constexpr int kBox = 16;        // rows of one TMA box of x; tiles of at most as many are small
constexpr int kFew = 8;         // rows of one box of h; tiles of at most as many have h's two parts side by side
constexpr int kInnerThreads = 224, kOuterThreads = 320;
constexpr uint32_t kRowTile = 128u * 128u;  // bytes of 128 rows of 64 elements

struct LoraParams {
  int32_t rows, sequences, adapters, outputs, rank;
  int32_t rank16;       // rank rounded up to the products' step of 16
  int32_t chunks;       // columns of x, in 64s
  int32_t splits;       // CTAs of a cluster that share them
  int32_t subs;         // tiles of 128 outputs
  int32_t ring;         // bytes of the first kernel's ring
  int32_t stages_out;   // of the second's
  const int32_t *seq_start, *adapter;
  const float* scales;
  const void* base;
  int64_t base_row;
  void* out;
  int64_t out_row;
  void* h;              // [rows][2 rank16]
  float* row_scale;     // [rows]: 2^e times the adapter's scale
  uint64_t wait_limit_ns;
  int32_t stall;        // test hook: the loading warps load nothing
};

// Set when a wait of either kernel ran past its limit (one for each device).
__device__ int32_t g_lora_status;

struct LoraTile {
  int32_t row0, rows, adapter;  // rows 0: there is no such tile
};

constexpr int kStages = 12;  // of a ring, at most
constexpr int kAhead = 8;    // boxes of base that a group has for a small tile

struct LoraShared {
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full[2], acc_empty[2], h_full, h_empty, done, drained;
  uint64_t base_half[2][2], base_ahead[2][kAhead];
  uint32_t tmem;
  int32_t abort;
  LoraTile tile;
  int32_t b;
  int64_t before;
  union {
    int32_t warps[2][12];
    int64_t units[12];
  };
};

// Bounded wait: false once any wait of the CTA has run past its limit.
__device__ __forceinline__ bool lora_wait(LoraShared& sh, uint64_t* bar, uint32_t phase, uint64_t limit_ns) {
  if (mbar_try_wait(bar, phase & 1)) return true;
  volatile int32_t* abort = &sh.abort;
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, phase & 1)) return true;
    if ((it & 63u) == 0) {
      if (*abort) return false;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit_ns) {
        *abort = 1;
        *reinterpret_cast<volatile int32_t*>(&g_lora_status) = 1;
        return false;
      }
    }
  }
}

// The tile of number `index`, found by the whole CTA.
template <int THREADS>
__device__ __forceinline__ LoraTile find_tile(const LoraParams& p, LoraShared& sh, int index) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) sh.tile.rows = 0;
  int before = 0;
  for (int b0 = 0, turn = 0; b0 < p.sequences && before <= index; b0 += THREADS, turn ^= 1) {
    const int b = b0 + tid;
    int start = 0, n = 0;
    if (b < p.sequences) {
      start = min(max(__ldg(p.seq_start + b), 0), p.rows);
      n = min(max(__ldg(p.seq_start + b + 1), start), p.rows) - start;
    }
    const int tiles = (n + kTileRows - 1) / kTileRows;
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) sh.warps[turn][warp] = upto;
    __syncthreads();
    int base = before;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) base += sh.warps[turn][w];
      before += sh.warps[turn][w];
    }
    const int first = base + upto - tiles;
    if (first <= index && index < first + tiles) {
      const int row0 = (index - first) * kTileRows;
      int a = __ldg(p.adapter + b);
      if (a < 0 || a >= p.adapters) a = -1;
      sh.tile = LoraTile{start + row0, min(n - row0, kTileRows), a};
    }
  }
  __syncthreads();
  return sh.tile;
}

__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
  return p != 0;
}

// Products in flight have to end before tensor memory is freed.
__device__ __forceinline__ void drain(LoraShared& sh, uint64_t limit_ns) {
  if (elected()) umma_commit(&sh.drained);
  __syncwarp();
  if (!mbar_wait(&sh.drained, 0, limit_ns)) mbar_wait(&sh.drained, 0, 8 * limit_ns);
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// ------------------------------------------------------ h = x A^T ---------

template <typename T>
__global__ void __launch_bounds__(kInnerThreads) lora_inner_kernel(const LoraParams p, const __grid_constant__ CUtensorMap map_x,
                                                                   const __grid_constant__ CUtensorMap map_box, const __grid_constant__ CUtensorMap map_a) {
  constexpr uint32_t kFmt = El<T>::kBf16 ? 1u : 0u;
  extern __shared__ __align__(1024) uint8_t smem[];
  LoraShared& sh = *reinterpret_cast<LoraShared*>(smem + p.ring);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int index = blockIdx.x / p.splits, part = blockIdx.x % p.splits;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&sh.full[i], 1), mbar_init(&sh.empty[i], 2);
    mbar_init(&sh.done, 2);
    mbar_init(&sh.drained, 2);
    fence_mbar_init();
    sh.abort = 0;
  }
  const LoraTile tile = find_tile<kInnerThreads>(p, sh, index);
  // the whole cluster has the same tile
  if (tile.rows == 0 || tile.adapter < 0) return;
  if (warp == 1) tmem_alloc(&sh.tmem, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // not before every CTA has its tensor memory: the second kernel's CTAs hold
  // theirs while they wait for this kernel
  griddep_launch_dependents();
  const uint32_t tmem = sh.tmem;
  // Rows come in one box of 128, or 16 a box where that is less to read; then a
  // stage has two times 64 columns, since a stage's turn costs more than its
  // few rows.  A product reads 128 rows of x, the idle ones from whatever
  // follows, so that much follows the last stage too.
  const int boxes = (tile.rows + kBox - 1) / kBox;
  const bool big = boxes > 4;
  const int wide = big ? 1 : 2, units = (p.chunks + wide - 1) / wide;  // the last one's second half may be past x: zeros
  const int from = units * part / p.splits, to = units * (part + 1) / p.splits;
  const int count = to - from;
  const uint32_t x_one = big ? kRowTile : boxes * kBox * 128u, a_one = (p.rank16 * 128u + 1023u) / 1024u * 1024u;
  const uint32_t a_at = wide * x_one, stage_bytes = wide * (x_one + a_one);
  const int stages = min(kStages, static_cast<int>((p.ring - max(stage_bytes, (wide - 1) * x_one + kRowTile)) / stage_bytes) + 1);

  if (warp == 0) {
    // ------------------------------------------------------- loads ----
    const uint32_t bytes = wide * (x_one + p.rank * 128u);
    int i = 0, slot = 0, turn = 0;
    for (; i < count; ++i) {
      if (!__all_sync(0xffffffffu, lora_wait(sh, &sh.empty[slot], turn + 1, p.wait_limit_ns))) break;
      uint8_t* stage = smem + slot * stage_bytes;
      if (!p.stall) {
        if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], bytes);
        __syncwarp();
        const int k0 = (from + i) * wide * 64;
        if (big) {
          if (lane == 0) tma_load_2d(stage, &map_x, &sh.full[slot], k0, tile.row0);
        } else if (lane < 2 * boxes) {
          tma_load_2d(stage + (lane & 1) * x_one + (lane >> 1) * kBox * 128, &map_box, &sh.full[slot], k0 + (lane & 1) * 64, tile.row0 + (lane >> 1) * kBox);
        }
        if (lane >= 32 - wide) tma_load_2d(stage + a_at + (31 - lane) * a_one, &map_a, &sh.full[slot], k0 + (31 - lane) * 64, tile.adapter * p.rank);
      }
      if (++slot == stages) slot = 0, ++turn;
    }
    // no copy in flight is left behind
    if (!p.stall)
      for (int j = max(i - stages, 0); j < i; ++j)
        if (!mbar_wait(&sh.full[j % stages], (j / stages) & 1, p.wait_limit_ns)) break;
  } else if (warp <= 2) {
    // ---------------------------------------------------- products ----
    // Two issuers take every other stage, each to an accumulator of its own:
    // what one waits for passes behind the other's products.  Each waits for
    // every stage and gives every one back: loads need not end in their order,
    // and a wait for a turn of a stage whose last turn is not over would pass
    // at once.
    const int which = warp - 1;
    const uint32_t idesc = idesc_f32acc(kFmt, kFmt, 128, p.rank16), d = tmem + which * 128;
    const uint64_t x0 = sdesc_k_sw128(smem_u32(smem)), a0 = sdesc_k_sw128(smem_u32(smem + a_at));
    int slot = 0, turn = 0;
    for (int i = 0; i < count; ++i) {
      if (!__all_sync(0xffffffffu, lora_wait(sh, &sh.full[slot], turn, p.wait_limit_ns))) break;
      if ((i & 1) == which) {
        tc_fence_after();
        const uint64_t x = x0 + (slot * stage_bytes >> 4), a = a0 + (slot * stage_bytes >> 4);
        if (elected()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) umma_f16(d, x + k * 2, a + k * 2, idesc, i >= 2 || k > 0);
          if (wide == 2)
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_f16(d, x + (x_one >> 4) + k * 2, a + (a_one >> 4) + k * 2, idesc, 1);
          umma_commit(&sh.empty[slot]);
        }
      } else if (lane == 0) {
        mbar_arrive(&sh.empty[slot]);
      }
      __syncwarp();
      if (++slot == stages) slot = 0, ++turn;
    }
    if (elected()) umma_commit(&sh.done);
    __syncwarp();
    drain(sh, p.wait_limit_ns);
  }
  __syncwarp();
  // ------------------------------------------------------- the sum ----
  const int pitch = p.rank16 + 4;  // floats: rows start on different banks
  float* mine = reinterpret_cast<float*>(smem);
  if (warp >= 3) {
    // the ring has been read when the products are done: it takes this CTA's part of h
    const bool ok = __all_sync(0xffffffffu, lora_wait(sh, &sh.done, 0, p.wait_limit_ns));
    tc_fence_after();
    const int quarter = warp & 3, row = quarter * 32 + lane;
    if (ok && quarter * 32 < tile.rows) {
      for (int c = 0; c < p.rank16; c += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + (static_cast<uint32_t>(quarter) << 21) + c, v);
        if (count > 1) {
          uint32_t w[16];
          tmem_ld16(tmem + (static_cast<uint32_t>(quarter) << 21) + 128 + c, w);
          tmem_ld_wait();
          reg_fence<16>(v), reg_fence<16>(w);
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(w[j]));
        } else {
          tmem_ld_wait();
          reg_fence<16>(v);
        }
        if (row < tile.rows)
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            *reinterpret_cast<float4*>(mine + row * pitch + c + j) =
                make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]), __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
      }
    }
  }
  __syncwarp();
  if (p.splits > 1) cluster_sync_all();
  else __syncthreads();
  {
    // Rows in turn over the cluster's CTAs and all their warps; a lane has four
    // columns, so half a warp has a row of rank 64 or less.
    const float scale = p.scales ? __ldg(p.scales + tile.adapter) : 1.0f;
    const int width = p.rank16 <= 64 ? 16 : 32, sub = lane / width, col = lane % width * 4, at_once = 32 / width;
    for (int row0 = (part * (kInnerThreads / 32) + warp) * at_once; row0 < tile.rows; row0 += p.splits * (kInnerThreads / 32) * at_once) {
      const int row = row0 + sub;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (col < p.rank && row < tile.rows) {
        if (p.splits == 1) {
          v = *reinterpret_cast<const float4*>(mine + row * pitch + col);
        } else {
          // all on their way before the first is added
          const uint32_t at = smem_u32(mine + row * pitch + col);
          float4 w[8];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < p.splits) w[c] = ld_cluster4(cluster_map(at, c));
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < p.splits) v.x += w[c].x, v.y += w[c].y, v.z += w[c].z, v.w += w[c].w;
        }
      }
      // bits of the largest magnitude: a NaN's are above infinity's
      uint32_t most = max(max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu),
                          max(__float_as_uint(v.z) & 0x7FFFFFFFu, __float_as_uint(v.w) & 0x7FFFFFFFu));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (o < width) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
      // 2^e of the largest, at most 2^126 either way so that its inverse is normal too
      const int e = most >= 0x7F800000u || most == 0 ? 127 : min(max(static_cast<int>(most >> 23), 1), 253);
      const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23), up = __uint_as_float(static_cast<uint32_t>(e) << 23);
      if (row < tile.rows && col < p.rank16) {
        if (col == 0) p.row_scale[tile.row0 + row] = up * scale;
        const float y[4] = {v.x * down, v.y * down, v.z * down, v.w * down};
        float hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          hi[j] = El<T>::to_float(El<T>::from_float(y[j]));
          lo[j] = fabsf(hi[j]) < CUDART_INF_F ? y[j] - hi[j] : 0.0f;
        }
        T* out = static_cast<T*>(p.h) + static_cast<int64_t>(tile.row0 + row) * (2 * p.rank16) + col;
        *reinterpret_cast<uint2*>(out) = make_uint2(El<T>::pack2(hi[0], hi[1]), El<T>::pack2(hi[2], hi[3]));
        *reinterpret_cast<uint2*>(out + p.rank16) = make_uint2(El<T>::pack2(lo[0], lo[1]), El<T>::pack2(lo[2], lo[3]));
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  if (p.splits > 1) cluster_sync_all();  // no CTA's shared memory goes while it is read
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    tmem_relinquish();
    tmem_dealloc(tmem, 256);
  }
}

// ---------------------------------------------- out = base + h B^T --------

// Barrier of the four warps of an epilogue group.
__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, 128;" ::"r"(group + 1) : "memory"); }

// Work of the second kernel: every tile has units for its tiles of outputs, one
// each where it is small, else kBigCost; all units in a row are cut into equal
// ranges, one a CTA.  A tile of outputs belongs to the CTA that has its first.
constexpr int kBigCost = 3;

// Consecutive tiles of outputs of one tile of rows, and the walk over a CTA's range.
struct LoraWalk {
  LoraTile tile;
  int32_t sub0, count;
  int32_t b, start, n, k;  // the sequence, its rows, the tile in it
  int64_t begin, at, to;   // the tile's first unit, the range that is left

  __device__ __forceinline__ void load(const LoraParams& p) {
    start = min(max(__ldg(p.seq_start + b), 0), p.rows);
    n = min(max(__ldg(p.seq_start + b + 1), start), p.rows) - start;
  }
  __device__ __forceinline__ static int64_t units_of(const LoraParams& p, int n) {
    const int tiles = (n + kTileRows - 1) / kTileRows, rest = n - (tiles - 1) * kTileRows;
    return n == 0 ? 0 : static_cast<int64_t>(p.subs) * ((tiles - 1) * kBigCost + (rest <= kBox ? 1 : kBigCost));
  }
  __device__ __forceinline__ void start_at(const LoraParams& p, int b_, int64_t before, int64_t from, int64_t to_) {
    b = b_, at = from, to = to_;
    load(p);
    k = static_cast<int32_t>((from - before) / (static_cast<int64_t>(p.subs) * kBigCost));
    begin = before + static_cast<int64_t>(k) * p.subs * kBigCost;
  }
  __device__ __forceinline__ bool next(const LoraParams& p) {
    while (at < to) {
      const int rows = min(n - k * kTileRows, kTileRows), cost = rows <= kBox ? 1 : kBigCost;
      const int64_t end = begin + static_cast<int64_t>(p.subs) * cost, upto = min(end, to);
      sub0 = static_cast<int32_t>((at - begin + cost - 1) / cost);
      count = static_cast<int32_t>((upto - begin + cost - 1) / cost) - sub0;
      if (count > 0) {
        const int a = __ldg(p.adapter + b);
        tile = LoraTile{start + k * kTileRows, rows, a < 0 || a >= p.adapters ? -1 : a};
      }
      at = upto;
      if (upto == end) {
        begin = end;
        if (++k * kTileRows >= n && at < to) {
          k = 0;
          do ++b, load(p);
          while (n == 0);
        }
      }
      if (count > 0) return true;
    }
    return false;
  }
};

// The range of this CTA, found by all its threads: false where it has none.
template <int THREADS>
__device__ __forceinline__ bool find_range(const LoraParams& p, LoraShared& sh, LoraWalk* walk) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto units_at = [&](int b) -> int64_t {
    if (b >= p.sequences) return 0;
    const int start = min(max(__ldg(p.seq_start + b), 0), p.rows);
    return LoraWalk::units_of(p, min(max(__ldg(p.seq_start + b + 1), start), p.rows) - start);
  };
  // the total, then the place: each thread has consecutive sequences
  const int each = (p.sequences + THREADS - 1) / THREADS;
  int64_t mine = 0;
  for (int i = 0; i < each; ++i) mine += units_at(tid * each + i);
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) sh.units[warp] = upto;
  __syncthreads();
  int64_t total = 0, before = upto - mine;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += sh.units[w];
    total += sh.units[w];
  }
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);
  if (blockIdx.x >= ctas) return false;
  const int64_t from = total * blockIdx.x / ctas, to = total * (blockIdx.x + 1) / ctas;
  if (before <= from && from < before + mine) {
    for (int i = 0; i < each; ++i) {
      const int64_t units = units_at(tid * each + i);
      if (from < before + units) {
        sh.b = tid * each + i, sh.before = before;
        break;
      }
      before += units;
    }
  }
  __syncthreads();
  walk->start_at(p, sh.b, sh.before, from, to);
  return true;
}

// D = h B^T of STEPS steps of 16 for the high parts, and as many for the low
// ones against the same B.  HOW 1: D^T; 2: D^T of both parts at once, which are
// rows of the same tile.
template <int HOW, int STEPS>
__device__ __forceinline__ void outer_products(uint32_t d, uint64_t h, uint64_t b, uint32_t idesc) {
#pragma unroll
  for (int k = 0; k < (HOW == 2 ? STEPS : 2 * STEPS); ++k) {
    const int kb = k % STEPS;
    const uint64_t hk = h + (k / 4) * (kRowTile >> 4) + (k % 4) * 2, bk = b + (kb / 4) * (kRowTile >> 4) + (kb % 4) * 2;
    umma_f16(d, HOW ? bk : hk, HOW ? hk : bk, idesc, k > 0);
  }
}
template <int HOW>
__device__ __forceinline__ void outer_products(int steps, uint32_t d, uint64_t h, uint64_t b, uint32_t idesc) {
  switch (steps) {
    case 1: return outer_products<HOW, 1>(d, h, b, idesc);
    case 2: return outer_products<HOW, 2>(d, h, b, idesc);
    case 3: return outer_products<HOW, 3>(d, h, b, idesc);
    case 4: return outer_products<HOW, 4>(d, h, b, idesc);
    case 5: return outer_products<HOW, 5>(d, h, b, idesc);
    case 6: return outer_products<HOW, 6>(d, h, b, idesc);
    case 7: return outer_products<HOW, 7>(d, h, b, idesc);
    default: return outer_products<HOW, 8>(d, h, b, idesc);
  }
}

template <typename T>
__global__ void __launch_bounds__(kOuterThreads, 1) lora_outer_kernel(const LoraParams p, const __grid_constant__ CUtensorMap map_h,
                                                                      const __grid_constant__ CUtensorMap map_b,
                                                                      const __grid_constant__ CUtensorMap map_base) {
  constexpr uint32_t kFmt = El<T>::kBf16 ? 1u : 0u;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int parts = (p.rank16 + 63) / 64;            // 64-column parts of a tile of B
  const int h_parts = (2 * p.rank16 + 63) / 64;      // and of h
  const uint32_t b_bytes = parts * kRowTile;
  uint8_t* h_smem = smem;
  uint8_t* staged = smem + h_parts * kRowTile;       // base and results: two boxes of 128 rows of 64 outputs for each epilogue group
  uint8_t* ring = staged + 2 * 2 * kRowTile;
  LoraShared& sh = *reinterpret_cast<LoraShared*>(ring + p.stages_out * b_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < p.stages_out; ++i) mbar_init(&sh.full[i], 1), mbar_init(&sh.empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.acc_full[i], 1), mbar_init(&sh.acc_empty[i], 4);
      mbar_init(&sh.base_half[i][0], 1), mbar_init(&sh.base_half[i][1], 1);
      for (int j = 0; j < kAhead; ++j) mbar_init(&sh.base_ahead[i][j], 1);
    }
    mbar_init(&sh.h_full, 1);
    mbar_init(&sh.h_empty, 1);
    mbar_init(&sh.drained, 1);
    fence_mbar_init();
    sh.abort = 0;
  }
  LoraWalk walk;
  if (!find_range<kOuterThreads>(p, sh, &walk)) {
    griddep_wait();  // this kernel does not end before the first
    return;
  }
  const T* base = static_cast<const T*>(p.base);
  T* out = static_cast<T*>(p.out);

  if (warp == 0) {
    // ------------------------------------------------------- loads ----
    int slot = 0, turn = 0, sent = 0;
    uint32_t segment = 0;
    bool ok = true;
    while (ok && walk.next(p)) {
      const LoraTile& tile = walk.tile;
      if (tile.adapter < 0) continue;
      // B does not wait for the first kernel, whose h follows the ring's filling
      const int ahead = min(walk.count, p.stages_out);
      for (int i = 0; i <= walk.count; ++i) {
        if (i == ahead) {
          if (segment == 0) griddep_wait();
          if (!(ok = __all_sync(0xffffffffu, lora_wait(sh, &sh.h_empty, segment + 1, p.wait_limit_ns)))) break;
          if (!p.stall) {
            // a few rows: the low parts follow the high ones, 8 rows on
            const bool few = tile.rows <= kFew;
            const int boxes = few ? 2 : (tile.rows + kFew - 1) / kFew, of_parts = few ? parts : h_parts;
            if (lane == 0) mbar_arrive_expect_tx(&sh.h_full, boxes * of_parts * kFew * 128u);
            __syncwarp();
            for (int j = lane; j < boxes * of_parts; j += 32) {
              const int part = j / boxes, box = j % boxes;
              tma_load_2d(h_smem + part * kRowTile + box * kFew * 128, &map_h, &sh.h_full, part * 64 + (few ? box * p.rank16 : 0),
                          tile.row0 + (few ? 0 : box * kFew));
            }
          }
          ++segment;
        }
        if (i == walk.count) break;
        if (!(ok = __all_sync(0xffffffffu, lora_wait(sh, &sh.empty[slot], turn + 1, p.wait_limit_ns)))) break;
        if (!p.stall) {
          const int n0 = (walk.sub0 + i) * kTileRows;
          if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], b_bytes);
          __syncwarp();
          // rows past the adapter's last output are the next one's, or zeros: their products are not stored
          if (lane < parts) tma_load_2d(ring + slot * b_bytes + lane * kRowTile, &map_b, &sh.full[slot], lane * 64, tile.adapter * p.outputs + n0);
        }
        ++sent;
        if (++slot == p.stages_out) slot = 0, ++turn;
      }
    }
    if (!p.stall) {
      // no copy in flight is left behind
      for (int j = max(sent - p.stages_out, 0); j < sent; ++j)
        if (!mbar_wait(&sh.full[j % p.stages_out], (j / p.stages_out) & 1, p.wait_limit_ns)) break;
      if (segment > 0) mbar_wait(&sh.h_full, (segment - 1) & 1, p.wait_limit_ns);
    }
  } else {
    if (warp == 1) tmem_alloc(&sh.tmem, 256);
    tc_fence_before();
    asm volatile("bar.sync 3, %0;" ::"n"(kOuterThreads - 32) : "memory");  // all but the loading warp
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    if (warp == 1) {
      // -------------------------------------------------- products ----
      const int steps = p.rank16 / 16;
      const uint64_t h0 = sdesc_k_sw128(smem_u32(h_smem)), b0 = sdesc_k_sw128(smem_u32(ring));
      int slot = 0, turn = 0;
      uint32_t segment = 0, used = 0;  // tiles of outputs so far: the two accumulators in turn
      bool ok = true;
      while (ok && walk.next(p)) {
        if (walk.tile.adapter < 0) continue;
        const bool small = walk.tile.rows <= kBox;
        const uint32_t idesc = small ? idesc_f32acc(kFmt, kFmt, 128, kBox) : idesc_f32acc(kFmt, kFmt, 128, kTileRows);
        if (!(ok = __all_sync(0xffffffffu, lora_wait(sh, &sh.h_full, segment, p.wait_limit_ns)))) break;
        ++segment;
        for (int i = 0; i < walk.count; ++i, ++used) {
          const uint32_t buf = used & 1;
          ok = __all_sync(0xffffffffu, lora_wait(sh, &sh.acc_empty[buf], (used >> 1) + 1, p.wait_limit_ns) &&
                                           lora_wait(sh, &sh.full[slot], turn, p.wait_limit_ns));
          if (!ok) break;
          tc_fence_after();
          const uint64_t bs = b0 + (slot * b_bytes >> 4);
          if (elected()) {
            if (walk.tile.rows <= kFew) outer_products<2>(steps, tmem + buf * kTileRows, h0, bs, idesc);
            else if (small) outer_products<1>(steps, tmem + buf * kTileRows, h0, bs, idesc);
            else outer_products<0>(steps, tmem + buf * kTileRows, h0, bs, idesc);
            umma_commit(&sh.empty[slot]);
            umma_commit(&sh.acc_full[buf]);
            if (i + 1 == walk.count) umma_commit(&sh.h_empty);
          }
          __syncwarp();
          if (++slot == p.stages_out) slot = 0, ++turn;
        }
      }
      drain(sh, p.wait_limit_ns);
    } else {
      // -------------------------------------------------- epilogue ----
      // two groups of four warps take every other tile of outputs
      const int group = (warp - 2) >> 2, quarter = warp & 3, in = tid - 64 - group * 128;
      const uint32_t acc = tmem + (static_cast<uint32_t>(quarter) << 21) + group * kTileRows;
      const int row = quarter * 32 + lane;
      uint8_t* mine = staged + group * 2 * kRowTile;
      uint32_t used = 0;                   // tiles of outputs before this segment
      uint32_t turn = 0, halves = 0, aheads = 0;  // this group's tiles; those with base in halves, and in small boxes
      bool ok = true, waited = false;
      while (ok && walk.next(p)) {
        const LoraTile tile = walk.tile;
        const int count = walk.count, sub0 = walk.sub0;
        if (tile.adapter < 0) {
          // nothing is added
          if (base == out) continue;
          const int width = (min(p.outputs, (sub0 + count) * kTileRows) - sub0 * kTileRows) / 8;
          for (int i = tid - 64; i < tile.rows * width; i += 256) {
            const int64_t r = tile.row0 + i / width;
            const int col = sub0 * kTileRows + i % width * 8;
            const uint4 v = base ? *reinterpret_cast<const uint4*>(base + r * p.base_row + col) : make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(out + r * p.out_row + col) = v;
          }
          continue;
        }
        const int first = (used ^ group) & 1, boxes = (tile.rows + kBox - 1) / kBox;
        used += count;
        if (tile.rows <= kBox) {
          // Lanes are outputs, columns rows.  Base comes kAhead tiles ahead, in
          // two boxes of 64 outputs each.
          auto fetch = [&](int i, uint32_t number) {
            if (!base || i >= count || p.stall) return;
            uint8_t* box = mine + number % kAhead * (2 * kBox * 128);
            uint64_t* bar = &sh.base_ahead[group][number % kAhead];
            if (lane == 0) mbar_arrive_expect_tx(bar, 2 * kBox * 128u);
            __syncwarp();
            if (lane < 2) tma_load_2d(box + lane * kBox * 128, &map_base, bar, (sub0 + i) * kTileRows + lane * 64, tile.row0);
          };
          if (in < 32)
            for (int j = 0; j < kAhead; ++j) fetch(first + 2 * j, aheads + j);
          if (!waited) griddep_wait(), waited = true;  // before row_scale is read
          int i = first;
          for (; i < count; i += 2, ++turn, ++aheads) {
            if (!(ok = __all_sync(0xffffffffu, lora_wait(sh, &sh.acc_full[group], turn, p.wait_limit_ns) &&
                                                   (!base || lora_wait(sh, &sh.base_ahead[group][aheads % kAhead], aheads / kAhead, p.wait_limit_ns)))))
              break;
            tc_fence_after();
            uint32_t v[kBox];
            tmem_ld16(acc, v);
            tmem_ld_wait();
            reg_fence<kBox>(v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.acc_empty[group]);
            if (tile.rows <= kFew)
#pragma unroll
              for (int t = 0; t < kFew; ++t) v[t] = __float_as_uint(__uint_as_float(v[t]) + __uint_as_float(v[t + kFew]));
            const int n = (sub0 + i) * kTileRows + row;
            const uint8_t* box = mine + aheads % kAhead * (2 * kBox * 128) + (row >> 6) * kBox * 128;
#pragma unroll
            for (int t = 0; t < kBox; ++t) {
              if (t >= tile.rows) break;
              const int64_t r = tile.row0 + t;
              const float b = base ? El<T>::to_float(*reinterpret_cast<const T*>(box + t * 128 + (((row >> 3) ^ t) & 7) * 16 + (row & 7) * 2)) : 0.0f;
              if (n < p.outputs) out[r * p.out_row + n] = El<T>::from_float(fmaf(__uint_as_float(v[t]), p.row_scale[r], b));
            }
            group_sync(group);  // the box has been read
            if (in < 32) fetch(i + 2 * kAhead, aheads + kAhead);
          }
          // no copy in flight is left behind
          if (!ok && base && !p.stall)
            for (uint32_t j = aheads; i < count && j < aheads + kAhead; ++j, i += 2)
              mbar_wait(&sh.base_ahead[group][j % kAhead], (j / kAhead) & 1, p.wait_limit_ns);
        } else {
          // A lane has a row.  Base comes to shared memory in boxes of 64
          // outputs, the sum replaces it there, and goes out a row of 128 bytes
          // to eight lanes; the next tile's box is on its way while the other
          // half is worked on.
          const bool busy = quarter * 32 < tile.rows;
          auto fetch = [&](int i, int half) {
            if (!base || i >= count || p.stall) return;
            if (lane == 0) mbar_arrive_expect_tx(&sh.base_half[group][half], boxes * kBox * 128u);
            __syncwarp();
            if (lane < boxes)
              tma_load_2d(mine + half * kRowTile + lane * kBox * 128, &map_base, &sh.base_half[group][half], (sub0 + i) * kTileRows + half * 64,
                          tile.row0 + lane * kBox);
          };
          if (in < 32) fetch(first, 0), fetch(first, 1);
          if (!waited) griddep_wait(), waited = true;
          const float scale = row < tile.rows ? p.row_scale[tile.row0 + row] : 0.0f;
          for (int i = first; i < count; i += 2, ++turn, ++halves) {
            if (!(ok = __all_sync(0xffffffffu, lora_wait(sh, &sh.acc_full[group], turn, p.wait_limit_ns)))) break;
            tc_fence_after();
            const int n0 = (sub0 + i) * kTileRows;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
              uint8_t* box = mine + half * kRowTile;
              if (base && !(ok = __all_sync(0xffffffffu, lora_wait(sh, &sh.base_half[group][half], halves, p.wait_limit_ns)))) break;
              if (busy) {
                uint32_t v[64];
                tmem_ld32p(acc + half * 64, v);
                tmem_ld32p(acc + half * 64 + 32, v + 32);
                tmem_ld_wait();
                reg_fence<64>(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  uint8_t* at = box + row * 128 + ((j ^ row) & 7) * 16;  // pieces of 8 outputs, in the order that boxes are swizzled in
                  Chunk<T, 8> sum;
                  if (base) sum.load(reinterpret_cast<const T*>(at));
                  else sum.zero();
                  float f[8];
                  sum.get(f);
#pragma unroll
                  for (int e = 0; e < 8; ++e) f[e] = fmaf(__uint_as_float(v[j * 8 + e]), scale, f[e]);
                  sum.set(f);
                  sum.store(reinterpret_cast<T*>(at));
                }
              }
              if (half == 1) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.acc_empty[group]);
              }
              group_sync(group);
              const int piece = in & 7, col = n0 + half * 64 + piece * 8;
              if (col < p.outputs) {
#pragma unroll 4
                for (int r = in >> 3; r < tile.rows; r += 16) {
                  const uint4 v = *reinterpret_cast<const uint4*>(box + r * 128 + ((piece ^ r) & 7) * 16);
                  *reinterpret_cast<uint4*>(out + (tile.row0 + r) * p.out_row + col) = v;
                }
              }
              fence_proxy_async_smem();  // the next box of base goes where these reads and writes were
              group_sync(group);
              if (in < 32) fetch(i + 2, half);
            }
            if (!ok) break;
          }
          // no copy in flight is left behind
          if (!ok && base && !p.stall)
            for (int half = 0; half < 2; ++half) mbar_wait(&sh.base_half[group][half], halves & 1, p.wait_limit_ns);
        }
      }
      if (!waited) griddep_wait();  // this kernel does not end before the first
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    const uint32_t tmem = sh.tmem;
    tmem_relinquish();
    tmem_dealloc(tmem, 256);
  }
}

// ------------------------------------------------------------------- host --

std::atomic<uint64_t> g_limit_ns{0};
std::atomic<int32_t> g_stall{0};

bool multiple16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int rank16_of(const eg_lora_args& a) { return (a.rank + 15) / 16 * 16; }
size_t h_bytes(const eg_lora_args& a) { return static_cast<size_t>(a.rows) * 2 * rank16_of(a) * 2; }
size_t workspace_of(const eg_lora_args& a) { return h_bytes(a) + (static_cast<size_t>(a.rows) * 4 + 15) / 16 * 16; }

eg_status check_shape(const eg_lora_args* a) {
  if (!a) return host_fail(EG_ERR_INVALID_ARG, "args is NULL");
  if (a->rows < 0 || a->sequences < 0 || a->adapters < 0)
    return host_fail(EG_ERR_INVALID_ARG, "negative size (rows=%d sequences=%d adapters=%d)", a->rows, a->sequences, a->adapters);
  if (a->dtype != EG_EL_BF16 && a->dtype != EG_EL_F16)
    return host_fail(a->dtype == EG_EL_F32 ? EG_ERR_UNSUPPORTED : EG_ERR_INVALID_ARG, "dtype must be bf16 or fp16 (got %d)", a->dtype);
  if (a->rows > (1 << 24) || a->sequences > 65536) return host_fail(EG_ERR_UNSUPPORTED, "at most 2^24 rows and 65536 sequences a call");
  for (int n : {a->inputs, a->outputs})
    if (n < 8 || n % 8 || n > (1 << 20)) return host_fail(EG_ERR_UNSUPPORTED, "inputs and outputs must be multiples of 8 in 8..2^20 (got %d and %d)", a->inputs, a->outputs);
  if (a->rank < 8 || a->rank % 8 || a->rank > 128) return host_fail(EG_ERR_UNSUPPORTED, "rank must be a multiple of 8 in 8..128 (got %d)", a->rank);
  if (static_cast<int64_t>(a->adapters) * std::max(a->outputs, a->rank) > INT32_MAX)
    return host_fail(EG_ERR_UNSUPPORTED, "%d adapters of %d outputs exceed 2^31 rows", a->adapters, a->outputs);
  return EG_OK;
}

eg_status check_matrix(const char* name, const void* p, int64_t stride, int width, int rows, bool output) {
  if (!p || !multiple16(p)) return host_fail(EG_ERR_INVALID_ARG, "%s is NULL or not 16-byte aligned", name);
  if (rows > 1 && (stride % 8 || stride < (output ? width : 8) || stride > (1ll << 38)))
    return host_fail(EG_ERR_INVALID_ARG, "the rows of %s must be a positive multiple of 8 elements apart%s (got %lld)", name,
                     output ? ", their width at least" : "", (long long)stride);
  return EG_OK;
}

eg_status encode(const eg_lora_args& a, const void* base, uint64_t cols, uint64_t rows, uint64_t row_elements, uint32_t box_rows, CUtensorMap* map) {
  EncodeTiledFn fn = host_encode_tiled();
  if (!fn) return host_fail(EG_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {row_elements * 2};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t steps[2] = {1, 1};
  const CUresult r = fn(map, a.dtype == EG_EL_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims,
                        strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? EG_OK : host_fail(EG_ERR_INVALID_ARG, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
}

template <typename T>
eg_status launch(const eg_lora_args& a, LoraParams p, int tiles, int sms, int dev, cudaStream_t st) {
  static std::atomic<uint64_t> allowed_inner{0}, allowed_outer{0};
  CUtensorMap map_x, map_box, map_a, map_h, map_b, map_base;
  const uint64_t x_row = a.rows > 1 ? a.x_row : a.inputs;
  EG_TRY(encode(a, a.x, a.inputs, a.rows, x_row, kBox, &map_box));
  if (a.rows > 4 * kBox) EG_TRY(encode(a, a.x, a.inputs, a.rows, x_row, kTileRows, &map_x));
  else map_x = map_box;  // not used
  // nothing is read of an empty bank, but a map has to have some place
  const uint64_t bank = std::max(a.adapters, 1);
  EG_TRY(encode(a, a.adapters ? a.a : a.x, a.inputs, bank * a.rank, a.inputs, a.rank, &map_a));
  EG_TRY(encode(a, p.h, 2 * p.rank16, a.rows, 2 * p.rank16, kFew, &map_h));
  EG_TRY(encode(a, a.adapters ? a.b : a.x, a.rank, bank * a.outputs, a.rank, kTileRows, &map_b));

  if (a.base) EG_TRY(encode(a, a.base, a.outputs, a.rows, a.rows > 1 ? a.base_row : a.outputs, kBox, &map_base));
  else map_base = map_h;  // not used

  // First kernel: two CTAs an SM, a cluster as large as lets them all run at
  // once (80 tiles of up to 12288 inputs as 320 CTAs: 58 us, as 160 50 us), at
  // least four columns of 64 each.
  p.ring = (113 * 1024 - static_cast<int>(sizeof(LoraShared))) / 1024 * 1024;
  const int inner_bytes = p.ring + static_cast<int>(sizeof(LoraShared));
  p.splits = 1;
  while (p.splits < 8 && tiles * p.splits * 2 <= sms * 2 && p.chunks >= p.splits * 8) p.splits *= 2;
  // Second kernel: one CTA an SM, whose tiles of outputs and of base come far ahead.
  const int h_tile = (2 * p.rank16 + 63) / 64 * static_cast<int>(kRowTile), b_tile = (p.rank16 + 63) / 64 * static_cast<int>(kRowTile);
  const int staged = 4 * static_cast<int>(kRowTile);
  p.stages_out = std::min(kStages, (226 * 1024 - static_cast<int>(sizeof(LoraShared)) - h_tile - staged) / b_tile);
  const int outer_bytes = h_tile + staged + p.stages_out * b_tile + static_cast<int>(sizeof(LoraShared));
  p.subs = (a.outputs + kTileRows - 1) / kTileRows;

  auto inner = lora_inner_kernel<T>;
  auto outer = lora_outer_kernel<T>;
  EG_TRY(host_allow_smem(reinterpret_cast<const void*>(inner), 114 * 1024, dev, &allowed_inner));
  EG_TRY(host_allow_smem(reinterpret_cast<const void*>(outer), 227 * 1024, dev, &allowed_outer));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles) * p.splits);
  cfg.blockDim = dim3(kInnerThreads);
  cfg.dynamicSmemBytes = inner_bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.splits, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, inner, p, map_x, map_box, map_a);
  if (e != cudaSuccess) return host_cuda_fail(e, "launching lora's first product");
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(sms, static_cast<int64_t>(tiles) * p.subs)));
  cfg.blockDim = dim3(kOuterThreads);
  cfg.dynamicSmemBytes = outer_bytes;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  e = cudaLaunchKernelEx(&cfg, outer, p, map_h, map_b, map_base);
  return e == cudaSuccess ? EG_OK : host_cuda_fail(e, "launching lora's second product");
}

}  // namespace
}  // namespace eg

using namespace eg;

extern "C" {

eg_status eg_lora_workspace_bytes(const eg_lora_args* args, size_t* out) {
  EG_TRY(check_shape(args));
  if (!out) return host_fail(EG_ERR_INVALID_ARG, "out is NULL");
  *out = workspace_of(*args);
  return EG_OK;
}

eg_status eg_lora(const eg_lora_args* args, void* stream) {
  EG_TRY(check_shape(args));
  const eg_lora_args& a = *args;
  if (a.rows == 0 || a.sequences == 0) return EG_OK;
  EG_TRY(check_matrix("out", a.out, a.out_row, a.outputs, a.rows, true));
  if (a.base) EG_TRY(check_matrix("base", a.base, a.base_row, a.outputs, a.rows, false));
  if (a.base == a.out && a.rows > 1 && a.base_row != a.out_row)
    return host_fail(EG_ERR_INVALID_ARG, "out is base with another stride");
  EG_TRY(check_matrix("x", a.x, a.x_row, a.inputs, a.rows, false));
  if (a.adapters > 0 && (!a.a || !a.b || !multiple16(a.a) || !multiple16(a.b)))
    return host_fail(EG_ERR_INVALID_ARG, "a or b is NULL or not 16-byte aligned");
  if (!a.seq_start || !a.adapter) return host_fail(EG_ERR_INVALID_ARG, "seq_start or adapter is NULL");
  for (const void* x : {static_cast<const void*>(a.seq_start), static_cast<const void*>(a.adapter), static_cast<const void*>(a.scales)})
    if (reinterpret_cast<uintptr_t>(x) % 4) return host_fail(EG_ERR_INVALID_ARG, "a side tensor is not aligned to its elements");
  if (!a.workspace || !multiple16(a.workspace)) return host_fail(EG_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned");
  if (a.workspace_bytes < workspace_of(a)) return host_fail(EG_ERR_INVALID_ARG, "workspace holds %zu bytes of %zu", a.workspace_bytes, workspace_of(a));
  int dev = 0, sms = 0;
  EG_TRY(host_check_device(&dev, &sms));
  LoraParams p{};
  p.rows = a.rows, p.sequences = a.sequences, p.adapters = a.adapters, p.outputs = a.outputs, p.rank = a.rank, p.rank16 = rank16_of(a);
  p.chunks = (a.inputs + 63) / 64;
  p.seq_start = a.seq_start, p.adapter = a.adapter, p.scales = a.scales;
  p.base = a.base, p.base_row = a.base_row, p.out = a.out, p.out_row = a.out_row;
  p.h = a.workspace, p.row_scale = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + h_bytes(a));
  const uint64_t limit = g_limit_ns.load(std::memory_order_relaxed);
  p.wait_limit_ns = limit ? limit : host_wait_limit_ns();
  p.stall = g_stall.load(std::memory_order_relaxed);
  // tiles that the sequences can have at most: one more each than whole ones
  const int tiles = a.rows / kTileRows + std::min(a.sequences, a.rows);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a.dtype == EG_EL_BF16 ? launch<__nv_bfloat16>(a, p, tiles, sms, dev, st) : launch<__half>(a, p, tiles, sms, dev, st);
}

eg_status eg_lora_device_status(void) {
  int dev = 0;
  EG_TRY(host_check_device(&dev));
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return host_cuda_fail(e, "synchronising the current device");
  int32_t status = 0;
  if ((e = cudaMemcpyFromSymbol(&status, g_lora_status, 4)) != cudaSuccess) return host_cuda_fail(e, "reading the status of lora");
  if (status == 0) return EG_OK;
  status = 0;
  e = cudaMemcpyToSymbol(g_lora_status, &status, 4);
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);  // later calls may be on streams that do not wait for this one
  if (e != cudaSuccess) return host_cuda_fail(e, "clearing the status of lora");
  return host_fail(EG_ERR_DEVICE_TIMEOUT, "a wait of the lora kernels ran past its limit");
}

eg_status eg_lora_set_test_stall(uint64_t wait_limit_ns, int32_t stall_loader) {
  if (stall_loader != 0 && stall_loader != 1) return host_fail(EG_ERR_INVALID_ARG, "stall_loader must be 0 or 1");
  g_limit_ns.store(wait_limit_ns, std::memory_order_relaxed);
  g_stall.store(stall_loader, std::memory_order_relaxed);
  return EG_OK;
}

}  // extern "C"
