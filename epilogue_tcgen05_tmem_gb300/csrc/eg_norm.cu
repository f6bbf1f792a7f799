// eg_norm.cu -- addition to the residual stream with the root-mean-square norm
// and the codes and scales that a linear plan takes, in one pass, and the
// gradient (include/eg_prompt.h has the formulas).
//
// Each value is read once and written once.  In succession: 8191 rows of 5120
// in bf16 with a residual, to E4M3 with a scale for each 128 columns, 53 us (5.6
// TB/s of the 6.8 that a copy reaches); the gradient of 16384 rows of 4096 92 to
// 94 us (5.8 TB/s).
//
// Forward: a CTA (for short rows a warp) has a row, a thread some 16-byte
// vectors of it in registers from the first read to the codes.  What bounded it
// before memory did was the number of instructions: two values in one
// instruction where there is one, a conversion of two codes, and a product with
// the scale's reciprocal in place of a division for each code took it from 64 to
// 53 us.  Gradient: a CTA walks rows and a thread has the same columns of each,
// so the weight's gradient adds up in registers; rows come to shared memory by
// asynchronous copies four ahead, for with one ahead in registers an SM had too
// little on its way (111 us).
//
// Rows of an odd width start at any place of a vector.  Where all tensors' do at
// the same, vectors that begin before the row and end behind it are used (8191
// rows of 5121 to E4M3 73 us, element by element 180 us, 5120 columns 49 us;
// gradient 80, 383 and 55 us).
//
// The sums of squares are float32, at most 32 a thread before the trees of a
// warp and of the CTA (a 256th of the row where registers do not hold it).
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <initializer_list>

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

struct NormParams {
  int32_t rows, width, quant;
  float eps, inv_width;
  const void *x, *residual, *weight;
  int64_t x_row, residual_row;
  void *sum, *out;
  int64_t sum_row, out_row;
  uint8_t* codes;
  int64_t codes_row;
  float* scales;
};

struct NormGradParams {
  int32_t rows, width;
  float eps, inv_width;
  const void *d_out, *sum, *weight, *d_sum;
  int64_t d_out_row, sum_row, d_sum_row;
  void* dx;
  int64_t dx_row;
  float* partial;  // [CTAs][width] sums of d_weight, or NULL
  int32_t stages;  // rows in shared memory
};

// The scale of values whose largest magnitude has the bits `most` (a NaN's are
// above all numbers').
__device__ __forceinline__ float scale_of(uint32_t most, float top) {
  const float s = __fdiv_rn(__uint_as_float(most), top);
  return s == 0.0f ? 1.0f : s;
}

// What h is multiplied by for its code; 0 where that would overflow and h is
// divided by the scale instead.
__device__ __forceinline__ float inverse_of(float scale) { return scale < 0x1p-126f ? 0.0f : __frcp_rn(scale); }

// The codes of two values, the first in the low byte.
__device__ __forceinline__ uint32_t codes_of(uint64_t h, float scale, float inverse, bool int8) {
  float a, b;
  if (inverse != 0.0f) {
    unpack64(mul2(h, pack64(inverse, inverse)), &a, &b);
  } else {
    unpack64(h, &a, &b);
    a = __fdiv_rn(a, scale), b = __fdiv_rn(b, scale);
  }
  if (!int8) return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const int x = min(max(__float2int_rn(a), -127), 127), y = min(max(__float2int_rn(b), -127), 127);
  return static_cast<uint32_t>(x & 0xFF) | static_cast<uint32_t>(y & 0xFF) << 8;
}

// The larger of a and |b|, NaN where either is.
__device__ __forceinline__ float max_abs(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(fabsf(b)));
  return y;
}

// Sum, or largest bits, over the threads of a row: a warp, or the whole CTA.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (WARP) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < (blockDim.x >> 5) ? red[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <bool WARP>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  if constexpr (WARP) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < (blockDim.x >> 5) ? red[lane] : 0u;
  return __reduce_max_sync(0xffffffffu, v);
}

// A vector of a row's elements from k0 on, of which only those in [0, width)
// are the row's: the others are zeros, and are not stored.
template <typename T, int CH>
__device__ __forceinline__ void load_part(Chunk<T, CH>& c, const T* row, int k0, int width) {
  if (k0 >= 0 && k0 + CH <= width) return c.load(row + k0);
  float f[CH];
#pragma unroll
  for (int e = 0; e < CH; ++e) f[e] = k0 + e >= 0 && k0 + e < width ? El<T>::to_float(row[k0 + e]) : 0.0f;
  c.set(f);
}
template <typename T, int CH>
__device__ __forceinline__ void store_part(const Chunk<T, CH>& c, T* row, int k0, int width) {
  if (k0 >= 0 && k0 + CH <= width) return c.store(row + k0);
  float f[CH];
  c.get(f);
#pragma unroll
  for (int e = 0; e < CH; ++e)
    if (k0 + e >= 0 && k0 + e < width) row[k0 + e] = El<T>::from_float(f[e]);
}
// The same from any address.
template <typename T, int CH>
__device__ __forceinline__ void load_singles(Chunk<T, CH>& c, const T* row, int k0, int width) {
  float f[CH];
#pragma unroll
  for (int e = 0; e < CH; ++e) f[e] = k0 + e >= 0 && k0 + e < width ? El<T>::to_float(row[k0 + e]) : 0.0f;
  c.set(f);
}

// Rows whose vectors of CH elements are aligned.  A thread keeps V vectors of
// its row; WARP: a row is a warp's, else a CTA's.  SHIFT: rows start at any
// element, all tensors' at the same place of a vector; the first vector starts
// before the row and the last one ends behind it, and only the weight is read
// by elements.
template <typename T, int CH, int V, bool WARP, bool SHIFT>
__global__ void __launch_bounds__(WARP ? 128 : SHIFT && V == 2 ? 512 : 1024) norm_kernel(const NormParams p) {
  // a linear plan launched as this kernel's dependent may stream its weights
  griddep_launch_dependents();
  __shared__ float red_sum[32];
  __shared__ uint32_t red_max[32];
  const int row = WARP ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= p.rows) return;
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, step = WARP ? 32 : blockDim.x;
  const int shift = SHIFT ? static_cast<int>(row * (p.x_row & (CH - 1)) & (CH - 1)) : 0;  // elements before the row in its first vector
  const int vectors = SHIFT ? (p.width + shift + CH - 1) / CH : p.width / CH;
  const T* x = static_cast<const T*>(p.x) + row * p.x_row;
  const T* w = static_cast<const T*>(p.weight);
  Chunk<T, CH> c[V], wc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * step + tid;
    if (v < vectors) SHIFT ? load_part(c[i], x, v * CH - shift, p.width) : c[i].load(x + v * CH);
    else c[i].zero();
  }
  uint64_t s[V][CH / 2];  // the sum's pairs, then the normed ones
  if (p.residual) {
    const T* r = static_cast<const T*>(p.residual) + row * p.residual_row;
    T* sum = static_cast<T*>(p.sum) + row * p.sum_row;
    Chunk<T, CH> d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * step + tid;
      if (v < vectors) SHIFT ? load_part(d[i], r, v * CH - shift, p.width) : d[i].load(r + v * CH);
      else d[i].zero();
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * step + tid;
#pragma unroll
      for (int j = 0; j < CH / 2; ++j) c[i].set_pair(j, add2(c[i].pair(j), d[i].pair(j)));
      if (v < vectors) SHIFT ? store_part(c[i], sum, v * CH - shift, p.width) : c[i].store(sum + v * CH);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * step + tid;
    if (v < vectors) SHIFT ? load_singles(wc[i], w, v * CH - shift, p.width) : wc[i].load(w + v * CH);
    else wc[i].zero();
  }
  uint64_t square2 = 0;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < CH / 2; ++j) {
      s[i][j] = c[i].pair(j);
      square2 = fma2(s[i][j], s[i][j], square2);
    }
  float square, other;
  unpack64(square2, &square, &other);
  square = row_sum<WARP>(square + other, red_sum);
  const float r = rsqrtf(fmaf(square, p.inv_width, p.eps));
  const uint64_t r2 = pack64(r, r);
  float most[V], top = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * step + tid;
    most[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < CH / 2; ++j) {
      s[i][j] = mul2(mul2(s[i][j], r2), wc[i].pair(j));
      float a, b;
      unpack64(s[i][j], &a, &b);
      most[i] = max_abs(max_abs(most[i], a), b);
    }
    // a row without a vector here has zeros, which may be no numbers after the product
    if (v >= vectors) most[i] = 0.0f;
    if (SHIFT && v < vectors && (v * CH < shift || v * CH - shift + CH > p.width)) {
      most[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < CH / 2; ++j) {
        const int k0 = v * CH - shift + 2 * j;
        float a, b;
        unpack64(s[i][j], &a, &b);
        if (k0 >= 0 && k0 < p.width) most[i] = max_abs(most[i], a);
        if (k0 + 1 >= 0 && k0 + 1 < p.width) most[i] = max_abs(most[i], b);
      }
    }
    top = max_abs(top, most[i]);
    if (p.out && v < vectors) {
      Chunk<T, CH> o;
#pragma unroll
      for (int j = 0; j < CH / 2; ++j) o.set_pair(j, s[i][j]);
      T* out = static_cast<T*>(p.out) + row * p.out_row;
      SHIFT ? store_part(o, out, v * CH - shift, p.width) : o.store(out + v * CH);
    }
  }
  if (p.quant == EG_NORM_PLAIN) return;
  const bool int8 = p.quant == EG_NORM_INT8;
  float scale = 1.0f, inverse = 1.0f;
  if (p.quant != EG_NORM_E4M3_BLOCK) {
    scale = scale_of(row_max<WARP>(__float_as_uint(top), red_max), int8 ? 127.0f : 448.0f);
    inverse = inverse_of(scale);
    if (tid == 0) p.scales[row] = scale;
  }
  uint8_t* codes = p.codes + row * p.codes_row;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * step + tid;
    if (p.quant == EG_NORM_E4M3_BLOCK) {
      // a block is 128 / CH neighbouring lanes; the lanes past the row's end hold zeros of no block
#pragma unroll
      for (int o = 64 / CH; o > 0; o >>= 1) most[i] = max_abs(most[i], __shfl_xor_sync(0xffffffffu, most[i], o));
      scale = scale_of(__float_as_uint(most[i]), 448.0f);
      inverse = inverse_of(scale);
      if (v < vectors && v % (128 / CH) == 0) p.scales[static_cast<int64_t>(row) * (p.width >> 7) + v / (128 / CH)] = scale;
    }
    if (v >= vectors) continue;
    uint32_t word[CH / 4];
#pragma unroll
    for (int j = 0; j < CH / 4; ++j) word[j] = codes_of(s[i][2 * j], scale, inverse, int8) | codes_of(s[i][2 * j + 1], scale, inverse, int8) << 16;
    if (SHIFT && (v * CH < shift || v * CH - shift + CH > p.width)) {
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        const int k0 = v * CH - shift + e;
        if (k0 >= 0 && k0 < p.width) codes[k0] = static_cast<uint8_t>(word[e >> 2] >> (8 * (e & 3)));
      }
      continue;
    }
    if constexpr (CH == 8) *reinterpret_cast<uint2*>(codes + v * CH - shift) = make_uint2(word[0], word[1]);
    else *reinterpret_cast<uint32_t*>(codes + v * CH - shift) = word[0];
  }
}

// Rows that start at different places of a vector: element by element, V of
// them in a thread's registers.  A warp has 128 neighbouring columns at a time,
// a lane every 32nd of them, so a block of the block scales is a warp's.
template <typename T, int V>
__global__ void __launch_bounds__(1024) norm_single_kernel(const NormParams p) {
  griddep_launch_dependents();
  __shared__ float red_sum[32];
  __shared__ uint32_t red_max[32];
  const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  auto place = [&](int i) { return ((i >> 2) * warps + warp) * 128 + (i & 3) * 32 + lane; };
  const T* x = static_cast<const T*>(p.x) + row * p.x_row;
  const T* w = static_cast<const T*>(p.weight);
  float s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = place(i) < p.width ? El<T>::to_float(x[place(i)]) : 0.0f;
  if (p.residual) {
    const T* r = static_cast<const T*>(p.residual) + row * p.residual_row;
    T* sum = static_cast<T*>(p.sum) + row * p.sum_row;
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = place(i) < p.width ? El<T>::to_float(r[place(i)]) : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const T v = El<T>::from_float(s[i] + d[i]);
      s[i] = El<T>::to_float(v);
      if (place(i) < p.width) sum[place(i)] = v;
    }
  }
  float square = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) square = fmaf(s[i], s[i], square);
  square = row_sum<false>(square, red_sum);
  const float r = rsqrtf(fmaf(square, p.inv_width, p.eps));
  float top = 0.0f, most[V / 4];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if ((i & 3) == 0) most[i >> 2] = 0.0f;
    if (place(i) >= p.width) continue;
    s[i] = s[i] * r * El<T>::to_float(w[place(i)]);
    most[i >> 2] = max_abs(most[i >> 2], s[i]);
    if (p.out) static_cast<T*>(p.out)[row * p.out_row + place(i)] = El<T>::from_float(s[i]);
  }
  if (p.quant == EG_NORM_PLAIN) return;
  const bool int8 = p.quant == EG_NORM_INT8, block = p.quant == EG_NORM_E4M3_BLOCK;
  float scale = 1.0f, inverse = 1.0f;
  if (!block) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) top = max_abs(top, most[i]);
    scale = scale_of(row_max<false>(__float_as_uint(top), red_max), int8 ? 127.0f : 448.0f);
    inverse = inverse_of(scale);
    if (threadIdx.x == 0) p.scales[row] = scale;
  }
  uint8_t* codes = p.codes + row * p.codes_row;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (block && (i & 3) == 0) {
      scale = scale_of(__reduce_max_sync(0xffffffffu, __float_as_uint(most[i >> 2])), 448.0f);
      inverse = inverse_of(scale);
      if (lane == 0 && place(i) < p.width) p.scales[static_cast<int64_t>(row) * (p.width >> 7) + (place(i) >> 7)] = scale;
    }
    if (place(i) < p.width) codes[place(i)] = static_cast<uint8_t>(codes_of(pack64(s[i], 0.0f), scale, inverse, int8));
  }
}

// Any width and alignment: the row read again from the cache after each
// reduction.  Taken where the registers above do not hold a row.
constexpr int kAnyThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kAnyThreads) norm_any_kernel(const NormParams p) {
  griddep_launch_dependents();
  __shared__ float red_sum[32];
  __shared__ uint32_t red_max[32];
  const int row = blockIdx.x, tid = threadIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.x_row;
  const T* w = static_cast<const T*>(p.weight);
  float square = 0.0f;
  if (p.residual) {
    const T* r = static_cast<const T*>(p.residual) + row * p.residual_row;
    T* s = static_cast<T*>(p.sum) + row * p.sum_row;
    for (int k = tid; k < p.width; k += kAnyThreads) {
      const T v = El<T>::from_float(El<T>::to_float(x[k]) + El<T>::to_float(r[k]));
      s[k] = v;
      const float f = El<T>::to_float(v);
      square = fmaf(f, f, square);
    }
    x = s;
  } else {
    for (int k = tid; k < p.width; k += kAnyThreads) {
      const float f = El<T>::to_float(x[k]);
      square = fmaf(f, f, square);
    }
  }
  square = row_sum<false>(square, red_sum);
  const float r = rsqrtf(fmaf(square, p.inv_width, p.eps));
  auto normed = [&](int k) { return El<T>::to_float(x[k]) * r * El<T>::to_float(w[k]); };
  uint8_t* codes = p.codes + row * p.codes_row;
  if (p.quant == EG_NORM_E4M3_BLOCK) {
    // a warp has a block of 128 columns, four a lane
    for (int b = tid >> 5; b < p.width >> 7; b += kAnyThreads / 32) {
      float h[4];
      uint32_t most = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[e] = normed(b * 128 + e * 32 + (tid & 31));
        most = max(most, __float_as_uint(h[e]) & 0x7FFFFFFFu);
      }
      const float scale = scale_of(__reduce_max_sync(0xffffffffu, most), 448.0f), inverse = inverse_of(scale);
      if ((tid & 31) == 0) p.scales[static_cast<int64_t>(row) * (p.width >> 7) + b] = scale;
#pragma unroll
      for (int e = 0; e < 4; ++e) codes[b * 128 + e * 32 + (tid & 31)] = static_cast<uint8_t>(codes_of(pack64(h[e], 0.0f), scale, inverse, false));
    }
  } else if (p.quant != EG_NORM_PLAIN) {
    uint32_t most = 0;
    for (int k = tid; k < p.width; k += kAnyThreads) most = max(most, __float_as_uint(normed(k)) & 0x7FFFFFFFu);
    const float scale = scale_of(row_max<false>(most, red_max), p.quant == EG_NORM_INT8 ? 127.0f : 448.0f);
    if (tid == 0) p.scales[row] = scale;
    const float inverse = inverse_of(scale);
    for (int k = tid; k < p.width; k += kAnyThreads)
      codes[k] = static_cast<uint8_t>(codes_of(pack64(normed(k), 0.0f), scale, inverse, p.quant == EG_NORM_INT8));
  }
  if (p.out) {
    if (p.quant == EG_NORM_E4M3_BLOCK) __syncthreads();  // out may be x: every block has been read
    T* o = static_cast<T*>(p.out) + row * p.out_row;
    for (int k = tid; k < p.width; k += kAnyThreads) o[k] = El<T>::from_float(normed(k));
  }
}

// The gradient.  A CTA walks rows; a thread has the same columns of each, so
// the weight's gradient adds up in its registers.
__device__ __forceinline__ float2 cta_sum2(float2 v, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v.x += __shfl_xor_sync(0xffffffffu, v.x, o), v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < (blockDim.x >> 5) ? red[lane] : make_float2(0.0f, 0.0f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v.x += __shfl_xor_sync(0xffffffffu, v.x, o), v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  return v;
}

// SHIFT: as in norm_kernel; the CTAs are a multiple of CH in number, so that all
// rows of one start at the same place of a vector.
template <typename T, int CH, int V, bool SHIFT, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_backward_kernel(const NormGradParams p) {
  griddep_launch_dependents();
  __shared__ float2 red[2][32];
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, step = blockDim.x;
  const int shift = SHIFT ? static_cast<int>(blockIdx.x * (p.sum_row & (CH - 1)) & (CH - 1)) : 0;
  const int vectors = SHIFT ? (p.width + shift + CH - 1) / CH : p.width / CH;
  uint64_t dw[V][CH / 2];
  Chunk<T, CH> d[V], z[V], add[V], w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < CH / 2; ++j) dw[i][j] = 0;
    const int v = i * step + tid;
    w[i].zero();
    if (v < vectors) SHIFT ? load_singles(w[i], static_cast<const T*>(p.weight), v * CH - shift, p.width) : w[i].load(static_cast<const T*>(p.weight) + v * CH);
  }
  // Rows come to shared memory some turns ahead; a thread copies what it will
  // read itself, so they need no barrier.
  auto place = [&](int stage, int tensor, int i) { return smem + ((stage * 3 + tensor) * V + i) * (step * 16) + tid * 16; };
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = i * step + tid;
        if (v >= vectors) continue;
        // what lies behind the row is not read; what lies before it in the first vector is the row before's
        const int k0 = v * CH - shift;
        const uint32_t bytes = SHIFT ? min(CH, p.width - k0) * static_cast<int>(sizeof(T)) : 16;
        cp_async_16(place(stage, 0, i), static_cast<const T*>(p.d_out) + row * p.d_out_row + k0, bytes);
        cp_async_16(place(stage, 1, i), static_cast<const T*>(p.sum) + row * p.sum_row + k0, bytes);
        if (p.d_sum) cp_async_16(place(stage, 2, i), static_cast<const T*>(p.d_sum) + row * p.d_sum_row + k0, bytes);
      }
    }
    cp_async_commit();
  };
  const int stages = p.stages;
  for (int s = 0; s < stages; ++s) fetch(blockIdx.x + static_cast<int64_t>(s) * gridDim.x, s);
  int turn = 0, stage = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    if (stages == 4) cp_async_wait<3>();
    else if (stages == 2) cp_async_wait<1>();
    else cp_async_wait<0>();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      d[i].zero(), z[i].zero(), add[i].zero();
      if (i * step + tid >= vectors) continue;
      d[i].load(reinterpret_cast<const T*>(place(stage, 0, i)));
      z[i].load(reinterpret_cast<const T*>(place(stage, 1, i)));
      if (p.d_sum) add[i].load(reinterpret_cast<const T*>(place(stage, 2, i)));
      if (SHIFT && i == 0 && tid == 0) {
        float f[CH], g[CH];
        d[0].get(f), z[0].get(g);
#pragma unroll
        for (int e = 0; e < CH; ++e)
          if (e < shift) f[e] = g[e] = 0.0f;
        d[0].set(f), z[0].set(g);
      }
    }
    uint64_t square2 = 0, gz2 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < CH / 2; ++j) {
        const uint64_t b = z[i].pair(j);
        square2 = fma2(b, b, square2);
        gz2 = fma2(mul2(d[i].pair(j), w[i].pair(j)), b, gz2);
      }
    float2 both, other;  // sums of z^2 and of g z
    unpack64(square2, &both.x, &other.x), unpack64(gz2, &both.y, &other.y);
    both.x += other.x, both.y += other.y;
    both = cta_sum2(both, red[turn]);
    // this row has been read: its place is free
    fetch(row + static_cast<int64_t>(stages) * gridDim.x, stage);
    if (++stage == stages) stage = 0;
    const float r = rsqrtf(fmaf(both.x, p.inv_width, p.eps));
    const float back = -(r * r * (both.y * p.inv_width) * r);
    const uint64_t r2 = pack64(r, r), back2 = pack64(back, back);
    T* dx = static_cast<T*>(p.dx) + row * p.dx_row;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * step + tid;
      Chunk<T, CH> o;
#pragma unroll
      for (int j = 0; j < CH / 2; ++j) {
        const uint64_t a = d[i].pair(j), b = z[i].pair(j);
        o.set_pair(j, fma2(mul2(a, w[i].pair(j)), r2, fma2(b, back2, add[i].pair(j))));
        dw[i][j] = fma2(a, mul2(b, r2), dw[i][j]);
      }
      if (v < vectors) SHIFT ? store_part(o, dx, v * CH - shift, p.width) : o.store(dx + v * CH);
    }
  }
  if (!p.partial) return;
  float* out = p.partial + static_cast<int64_t>(blockIdx.x) * p.width;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * step + tid;
    if (v >= vectors) continue;
    if constexpr (SHIFT) {
#pragma unroll
      for (int j = 0; j < CH / 2; ++j) {
        const int k0 = v * CH - shift + 2 * j;
        float a, b;
        unpack64(dw[i][j], &a, &b);
        if (k0 >= 0 && k0 < p.width) out[k0] = a;
        if (k0 + 1 >= 0 && k0 + 1 < p.width) out[k0 + 1] = b;
      }
    } else {
#pragma unroll
      for (int j = 0; j < CH / 2; j += 2) *reinterpret_cast<ulonglong2*>(out + v * CH + 2 * j) = make_ulonglong2(dw[i][j], dw[i][j + 1]);
    }
  }
}

// The same for rows that start at different places of a vector.
template <typename T, int V, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) norm_backward_single_kernel(const NormGradParams p) {
  griddep_launch_dependents();
  __shared__ float2 red[2][32];
  const int tid = threadIdx.x, step = blockDim.x;
  float dw[V], w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) dw[i] = 0.0f, w[i] = i * step + tid < p.width ? El<T>::to_float(static_cast<const T*>(p.weight)[i * step + tid]) : 0.0f;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const T* d_row = static_cast<const T*>(p.d_out) + row * p.d_out_row;
    const T* z_row = static_cast<const T*>(p.sum) + row * p.sum_row;
    const T* add_row = p.d_sum ? static_cast<const T*>(p.d_sum) + row * p.d_sum_row : nullptr;
    T* dx = static_cast<T*>(p.dx) + row * p.dx_row;
    float d[V], z[V];
    T add[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = i * step + tid;
      d[i] = k < p.width ? El<T>::to_float(d_row[k]) : 0.0f;
      z[i] = k < p.width ? El<T>::to_float(z_row[k]) : 0.0f;
      add[i] = k < p.width && add_row ? add_row[k] : El<T>::from_float(0.0f);
    }
    float2 both = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) both.x = fmaf(z[i], z[i], both.x), both.y = fmaf(d[i] * w[i], z[i], both.y);
    both = cta_sum2(both, red[turn]);
    const float r = rsqrtf(fmaf(both.x, p.inv_width, p.eps));
    const float back = r * r * (both.y * p.inv_width) * r;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = i * step + tid;
      dw[i] = fmaf(d[i], z[i] * r, dw[i]);
      if (k < p.width) dx[k] = El<T>::from_float(fmaf(d[i] * w[i], r, fmaf(-back, z[i], El<T>::to_float(add[i]))));
    }
  }
  if (!p.partial) return;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i * step + tid < p.width) p.partial[static_cast<int64_t>(blockIdx.x) * p.width + i * step + tid] = dw[i];
}

// The same for rows that the registers do not hold; the sums of the weight's
// gradient stay in the workspace, each column its thread's.
template <typename T>
__global__ void __launch_bounds__(kAnyThreads) norm_backward_any_kernel(const NormGradParams p) {
  griddep_launch_dependents();
  __shared__ float2 red[2][32];
  const int tid = threadIdx.x;
  const T* w = static_cast<const T*>(p.weight);
  float* mine = p.partial ? p.partial + static_cast<int64_t>(blockIdx.x) * p.width : nullptr;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const T* d = static_cast<const T*>(p.d_out) + row * p.d_out_row;
    const T* z = static_cast<const T*>(p.sum) + row * p.sum_row;
    const T* add = p.d_sum ? static_cast<const T*>(p.d_sum) + row * p.d_sum_row : nullptr;
    T* dx = static_cast<T*>(p.dx) + row * p.dx_row;
    float2 both = make_float2(0.0f, 0.0f);
    for (int k = tid; k < p.width; k += kAnyThreads) {
      const float a = El<T>::to_float(d[k]), b = El<T>::to_float(z[k]);
      both.x = fmaf(b, b, both.x), both.y = fmaf(a * El<T>::to_float(w[k]), b, both.y);
    }
    both = cta_sum2(both, red[turn]);
    const float r = rsqrtf(fmaf(both.x, p.inv_width, p.eps));
    const float back = r * r * (both.y * p.inv_width) * r;
    for (int k = tid; k < p.width; k += kAnyThreads) {
      const float a = El<T>::to_float(d[k]), b = El<T>::to_float(z[k]);
      const float s = add ? El<T>::to_float(add[k]) : 0.0f;
      if (mine) mine[k] = fmaf(a, b * r, row == blockIdx.x ? 0.0f : mine[k]);
      dx[k] = El<T>::from_float(fmaf(a * El<T>::to_float(w[k]), r, fmaf(-back, b, s)));
    }
  }
}

// Sums of the CTAs' parts, in their order: a warp has 32 columns of every 32nd.
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float* partial, int ctas, int width, float* out) {
  griddep_wait();
  __shared__ float shared[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int column = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (column < width)
#pragma unroll 8
    for (int c = warp; c < ctas; c += 32) v += partial[static_cast<int64_t>(c) * width + column];
  shared[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && column < width) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += shared[i][lane];
    out[column] = v;
  }
}

// ------------------------------------------------------------------- host --

int el_bytes(int dtype) { return dtype == EG_EL_F32 ? 4 : 2; }

eg_status check_shape(int64_t rows, int64_t width, int32_t dtype, float eps) {
  if (rows < 0 || width < 0) return host_fail(EG_ERR_INVALID_ARG, "negative size (rows=%lld width=%lld)", (long long)rows, (long long)width);
  if (dtype != EG_EL_BF16 && dtype != EG_EL_F16 && dtype != EG_EL_F32) return host_fail(EG_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (rows > (1 << 24)) return host_fail(EG_ERR_UNSUPPORTED, "at most 2^24 rows a call (got %lld)", (long long)rows);
  if (width < 1 || width > 65536) return host_fail(EG_ERR_UNSUPPORTED, "width must be in 1..65536 (got %lld)", (long long)width);
  if (!(eps >= 0.0f)) return host_fail(EG_ERR_INVALID_ARG, "eps must not be negative");
  return EG_OK;
}

eg_status check_rows(const char* name, const void* ptr, int64_t stride, int64_t rows, int64_t width, int bytes) {
  if (rows == 0) return EG_OK;
  if (!ptr) return host_fail(EG_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(ptr) % bytes) return host_fail(EG_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
  if (rows > 1 && stride < width) return host_fail(EG_ERR_INVALID_ARG, "the rows of %s are %lld apart, less than their width", name, (long long)stride);
  return EG_OK;
}

// Inputs may be broadcast over the rows (stride 0), outputs may not.
eg_status check_input(const char* name, const void* ptr, int64_t stride, int64_t rows, int64_t width, int bytes) {
  return check_rows(name, ptr, stride == 0 ? width : stride, rows, width, bytes);
}

struct Operand {
  const void* ptr;
  int64_t stride;
};

// Whether every row starts on a vector of `ch` elements of `bytes` bytes.
bool vectors_fit(int64_t width, int64_t rows, int ch, int bytes, std::initializer_list<Operand> operands) {
  if (width % ch) return false;
  for (const Operand& o : operands)
    if (o.ptr && (reinterpret_cast<uintptr_t>(o.ptr) % (ch * bytes) || (rows > 1 && o.stride % ch))) return false;
  return true;
}

// Whether all rows start at the same place of a vector, those of the first row
// on one.
bool vectors_shift(int64_t width, int64_t rows, int ch, int bytes, int64_t stride, std::initializer_list<Operand> operands) {
  if (width < ch) return false;
  for (const Operand& o : operands)
    if (o.ptr && (reinterpret_cast<uintptr_t>(o.ptr) % (ch * bytes) || (rows > 1 && (o.stride - stride) % ch))) return false;
  return true;
}

// Vectors a thread holds of a row of `vectors` (`want`, or as many as it takes
// for at most `most` threads, at most `limit`), and the threads of a row.
void split_row(int vectors, int want, int most, int limit, int* v, int* threads) {
  *v = want;
  while (*v < limit && (vectors + *v - 1) / *v > most) *v *= 2;
  *threads = std::max(32, ((vectors + *v - 1) / *v + 31) / 32 * 32);
}

template <typename T, int CH>
void launch_shifted(const NormParams& p, cudaStream_t st) {
  int v = 0, threads = 0;
  split_row(p.width / CH + 2, 2, 512, 4, &v, &threads);
  if (v == 2) norm_kernel<T, CH, 2, false, true><<<p.rows, threads, 0, st>>>(p);
  else norm_kernel<T, CH, 4, false, true><<<p.rows, threads, 0, st>>>(p);
}

template <typename T, int CH>
void launch_norm(const NormParams& p, int v, int threads, cudaStream_t st) {
  if (threads == 32) {
    // four rows a CTA
    norm_kernel<T, CH, 4, true, false><<<static_cast<unsigned>((p.rows + 3) / 4), 128, 0, st>>>(p);
    return;
  }
  if (v == 4) norm_kernel<T, CH, 4, false, false><<<p.rows, threads, 0, st>>>(p);
  else norm_kernel<T, CH, 8, false, false><<<p.rows, threads, 0, st>>>(p);
}

// Threads of a row that holds `v` elements each.
int threads_of(int width, int v) { return ((width + v - 1) / v + 31) / 32 * 32; }

// Rows that are no vectors: four elements a thread up to 4096 columns, sixteen
// up to 16384, else from the cache.
template <typename T>
void launch_singles(const NormParams& p, cudaStream_t st) {
  if (p.width <= 4096) norm_single_kernel<T, 4><<<p.rows, threads_of(p.width, 4), 0, st>>>(p);
  else if (p.width <= 16384) norm_single_kernel<T, 16><<<p.rows, threads_of(p.width, 16), 0, st>>>(p);
  else norm_any_kernel<T><<<p.rows, kAnyThreads, 0, st>>>(p);
}
template <typename T>
void launch_singles(const NormGradParams& p, int grid, cudaStream_t st) {
  if (p.width <= 2048) norm_backward_single_kernel<T, 4, 512><<<grid, threads_of(p.width, 4), 0, st>>>(p);
  else if (p.width <= 8192) norm_backward_single_kernel<T, 16, 512><<<grid, threads_of(p.width, 16), 0, st>>>(p);
  else if (p.width <= 16384) norm_backward_single_kernel<T, 16, 1024><<<grid, threads_of(p.width, 16), 0, st>>>(p);
  else norm_backward_any_kernel<T><<<grid, kAnyThreads, 0, st>>>(p);
}

template <typename T, int CH, int V, bool SHIFT = false, int THREADS = 512>
eg_status launch_backward(NormGradParams p, int threads, int grid, int dev, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  // four rows ahead where two CTAs an SM have room for that, else two, else none
  const int stage = 3 * V * threads * 16;
  p.stages = 4 * stage <= 110 * 1024 ? 4 : 2 * stage <= 220 * 1024 ? 2 : 1;
  EG_TRY(host_allow_smem(reinterpret_cast<const void*>(norm_backward_kernel<T, CH, V, SHIFT, THREADS>), 224 * 1024, dev, &allowed));
  norm_backward_kernel<T, CH, V, SHIFT, THREADS><<<grid, threads, p.stages * stage, st>>>(p);
  return EG_OK;
}
// Rows of `vectors` vectors; more than 512 threads only in float32, whose rows
// of up to 16384 columns are twice as many vectors.
template <typename T, int CH, bool SHIFT>
eg_status launch_rows(const NormGradParams& p, int vectors, int grid, int dev, cudaStream_t st) {
  int v = 0, threads = 0;
  split_row(vectors, 1, 512, 4, &v, &threads);
  if (v == 1) return launch_backward<T, CH, 1, SHIFT>(p, threads, grid, dev, st);
  if (v == 2) return launch_backward<T, CH, 2, SHIFT>(p, threads, grid, dev, st);
  if constexpr (CH == 4)
    if (threads > 512) return launch_backward<T, CH, 4, SHIFT, 1024>(p, threads, grid, dev, st);
  return launch_backward<T, CH, 4, SHIFT>(p, threads, grid, dev, st);
}

// Most CTAs of the gradient: each leaves a row of sums.
int backward_ctas(int sms, int64_t rows) { return static_cast<int>(std::min<int64_t>(std::max<int64_t>(rows, 1), sms * 2)); }

eg_status check_grads(const eg_norm_grads* a) {
  if (!a) return host_fail(EG_ERR_INVALID_ARG, "args is NULL");
  return check_shape(a->rows, a->width, a->dtype, a->eps);
}

}  // namespace
}  // namespace eg

using namespace eg;

extern "C" {

eg_status eg_add_rms_norm(const eg_norm_args* args, void* stream) {
  if (!args) return host_fail(EG_ERR_INVALID_ARG, "args is NULL");
  const eg_norm_args& a = *args;
  EG_TRY(check_shape(a.rows, a.width, a.dtype, a.eps));
  if (a.quant < EG_NORM_PLAIN || a.quant > EG_NORM_E4M3_BLOCK) return host_fail(EG_ERR_INVALID_ARG, "unknown quant mode %d", a.quant);
  if (a.quant == EG_NORM_E4M3_BLOCK && a.width % 128)
    return host_fail(EG_ERR_UNSUPPORTED, "block scales need a width that is a multiple of 128 (got %lld)", (long long)a.width);
  const int bytes = el_bytes(a.dtype);
  EG_TRY(check_input("x", a.x, a.x_row, a.rows, a.width, bytes));
  EG_TRY(check_input("weight", a.weight, 0, a.rows, a.width, bytes));
  if (a.residual) {
    EG_TRY(check_input("residual", a.residual, a.residual_row, a.rows, a.width, bytes));
    EG_TRY(check_rows("sum", a.sum, a.sum_row, a.rows, a.width, bytes));
  }
  if (a.out || a.quant == EG_NORM_PLAIN) EG_TRY(check_rows("out", a.out, a.out_row, a.rows, a.width, bytes));
  if (a.quant != EG_NORM_PLAIN) {
    EG_TRY(check_rows("codes", a.codes, a.codes_row, a.rows, a.width, 1));
    EG_TRY(check_rows("scales", a.scales, 1, std::min<int64_t>(a.rows, 1), 1, 4));
  }
  if (a.rows == 0) return EG_OK;
  int dev = 0;
  EG_TRY(host_check_device(&dev));
  NormParams p{};
  p.rows = static_cast<int32_t>(a.rows), p.width = static_cast<int32_t>(a.width), p.quant = a.quant;
  p.eps = a.eps, p.inv_width = 1.0f / static_cast<float>(a.width);
  p.x = a.x, p.residual = a.residual, p.weight = a.weight, p.x_row = a.x_row, p.residual_row = a.residual_row;
  p.sum = a.sum, p.out = a.out, p.sum_row = a.sum_row, p.out_row = a.out_row;
  p.codes = static_cast<uint8_t*>(a.codes), p.codes_row = a.codes_row, p.scales = a.scales;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int ch = 16 / bytes;
  const bool quant = a.quant != EG_NORM_PLAIN;
  const bool fits = a.width / ch <= 8 * 1024 && vectors_fit(a.width, a.rows, ch, bytes, {{a.x, a.x_row}, {a.residual, a.residual_row}, {a.residual ? a.sum : nullptr, a.sum_row}, {a.out, a.out_row}, {a.weight, 0}}) &&
                    (!quant || vectors_fit(a.width, a.rows, ch, 1, {{a.codes, a.codes_row}}));
  if (fits) {
    int v = 0, threads = 0;
    split_row(p.width / ch, 4, 1024, 8, &v, &threads);
    if (a.dtype == EG_EL_F32) launch_norm<float, 4>(p, v, threads, st);
    else if (a.dtype == EG_EL_BF16) launch_norm<__nv_bfloat16, 8>(p, v, threads, st);
    else launch_norm<__half, 8>(p, v, threads, st);
  } else if (a.quant != EG_NORM_E4M3_BLOCK && a.width / ch + 2 <= 4 * 1024 &&
             vectors_shift(a.width, a.rows, ch, bytes, a.x_row, {{a.x, a.x_row}, {a.residual, a.residual_row}, {a.residual ? a.sum : nullptr, a.sum_row}, {a.out, a.out_row}}) &&
             (!quant || vectors_shift(a.width, a.rows, ch, 1, a.x_row, {{a.codes, a.codes_row}}))) {
    if (a.dtype == EG_EL_F32) launch_shifted<float, 4>(p, st);
    else if (a.dtype == EG_EL_BF16) launch_shifted<__nv_bfloat16, 8>(p, st);
    else launch_shifted<__half, 8>(p, st);
  } else if (a.dtype == EG_EL_F32) launch_singles<float>(p, st);
  else if (a.dtype == EG_EL_BF16) launch_singles<__nv_bfloat16>(p, st);
  else launch_singles<__half>(p, st);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? EG_OK : host_cuda_fail(e, "launching add_rms_norm");
}

eg_status eg_add_rms_norm_workspace_bytes(const eg_norm_grads* args, size_t* out) {
  EG_TRY(check_grads(args));
  if (!out) return host_fail(EG_ERR_INVALID_ARG, "out is NULL");
  int dev = 0, sms = 0;
  EG_TRY(host_check_device(&dev, &sms));
  *out = static_cast<size_t>(backward_ctas(sms, args->rows)) * args->width * 4;
  return EG_OK;
}

eg_status eg_add_rms_norm_backward(const eg_norm_grads* args, void* stream) {
  EG_TRY(check_grads(args));
  const eg_norm_grads& a = *args;
  const int bytes = el_bytes(a.dtype);
  EG_TRY(check_input("d_out", a.d_out, a.d_out_row, a.rows, a.width, bytes));
  EG_TRY(check_input("sum", a.sum, a.sum_row, a.rows, a.width, bytes));
  EG_TRY(check_input("weight", a.weight, 0, a.rows, a.width, bytes));
  if (a.d_sum) EG_TRY(check_input("d_sum", a.d_sum, a.d_sum_row, a.rows, a.width, bytes));
  EG_TRY(check_rows("dx", a.dx, a.dx_row, a.rows, a.width, bytes));
  if (reinterpret_cast<uintptr_t>(a.d_weight) % 4) return host_fail(EG_ERR_INVALID_ARG, "d_weight is not aligned to its elements");
  int dev = 0, sms = 0;
  EG_TRY(host_check_device(&dev, &sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.rows == 0) {
    if (!a.d_weight) return EG_OK;
    const cudaError_t e = cudaMemsetAsync(a.d_weight, 0, static_cast<size_t>(a.width) * 4, st);
    return e == cudaSuccess ? EG_OK : host_cuda_fail(e, "clearing the weight's gradient");
  }
  const int grid = backward_ctas(sms, a.rows);
  if (a.d_weight) {
    const size_t need = static_cast<size_t>(grid) * a.width * 4;
    if (!a.workspace || reinterpret_cast<uintptr_t>(a.workspace) % 16)
      return host_fail(EG_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned");
    if (a.workspace_bytes < need) return host_fail(EG_ERR_INVALID_ARG, "workspace holds %zu bytes of %zu", a.workspace_bytes, need);
  }
  NormGradParams p{};
  p.rows = static_cast<int32_t>(a.rows), p.width = static_cast<int32_t>(a.width);
  p.eps = a.eps, p.inv_width = 1.0f / static_cast<float>(a.width);
  p.d_out = a.d_out, p.sum = a.sum, p.weight = a.weight, p.d_sum = a.d_sum;
  p.d_out_row = a.d_out_row, p.sum_row = a.sum_row, p.d_sum_row = a.d_sum_row;
  p.dx = a.dx, p.dx_row = a.dx_row;
  p.partial = a.d_weight ? static_cast<float*>(a.workspace) : nullptr;
  const int ch = 16 / bytes;
  const bool fits = a.width / ch <= (ch == 4 ? 4 * 1024 : 4 * 512) && vectors_fit(a.width, a.rows, ch, bytes, {{a.d_out, a.d_out_row}, {a.sum, a.sum_row}, {a.weight, 0}, {a.d_sum, a.d_sum_row}, {a.dx, a.dx_row}});
  if (fits) {
    const int vectors = p.width / ch;
    EG_TRY(a.dtype == EG_EL_F32    ? (launch_rows<float, 4, false>(p, vectors, grid, dev, st))
           : a.dtype == EG_EL_BF16 ? (launch_rows<__nv_bfloat16, 8, false>(p, vectors, grid, dev, st))
                                   : (launch_rows<__half, 8, false>(p, vectors, grid, dev, st)));
  } else if (a.width / ch + 2 <= (ch == 4 ? 4 * 1024 : 4 * 512) && (grid == a.rows || grid % ch == 0) &&
             vectors_shift(a.width, a.rows, ch, bytes, a.sum_row, {{a.d_out, a.d_out_row}, {a.sum, a.sum_row}, {a.d_sum, a.d_sum_row}, {a.dx, a.dx_row}})) {
    const int vectors = p.width / ch + 2;
    EG_TRY(a.dtype == EG_EL_F32    ? (launch_rows<float, 4, true>(p, vectors, grid, dev, st))
           : a.dtype == EG_EL_BF16 ? (launch_rows<__nv_bfloat16, 8, true>(p, vectors, grid, dev, st))
                                   : (launch_rows<__half, 8, true>(p, vectors, grid, dev, st)));
  } else if (a.dtype == EG_EL_F32) launch_singles<float>(p, grid, st);
  else if (a.dtype == EG_EL_BF16) launch_singles<__nv_bfloat16>(p, grid, st);
  else launch_singles<__half>(p, grid, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return host_cuda_fail(e, "launching the gradient of add_rms_norm");
  if (!a.d_weight) return EG_OK;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((a.width + 31) / 32));
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, norm_weight_kernel, static_cast<const float*>(p.partial), grid, static_cast<int>(a.width), a.d_weight);
  return e == cudaSuccess ? EG_OK : host_cuda_fail(e, "launching the sum of the weight's gradient");
}

}  // extern "C"
