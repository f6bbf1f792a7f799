// eg_attn.cuh -- what the attention kernels over a paged cache share: tensor
// loads, operand descriptors, products, packed float32 arithmetic, and the join
// of partial results.
#pragma once
#include <math_constants.h>

#include "eg_el.cuh"
#include "eg_ptx.cuh"

namespace eg {

// 4-D tiled bulk-tensor load global -> shared.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y, int32_t z,
                                            int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// 5-D tiled bulk-tensor load global -> shared.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y, int32_t z,
                                            int32_t w, int32_t u) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(u)
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

// 32 bytes, to a multiple of 32.
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(__cvta_generic_to_global(p)), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// The largest of three.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ float attn_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Position of a tile's values in the ring's order: K0, K1, V0, K2, V1, ...
__device__ __forceinline__ uint32_t attn_pos_v(uint32_t i, uint32_t count) { return i + 1 < count ? 2 * i + 2 : 2 * count - 1; }

// Four columns of one row of an item that CTAs lead, lead + step, ... last have
// parts of, joined in the order of the CTAs.
template <typename T, int HD, typename Params>
__device__ __forceinline__ void attn_join_piece(const Params& p, int lead, int last, int step, int r, int col, int64_t packed, int head) {
  constexpr float kShift = El<T>::kBf16 ? 0.0f : 7.0f;
  const int64_t rows = static_cast<int64_t>(128) * p.q_tiles;
  const float2* ml = reinterpret_cast<const float2*>(p.partial_ml) + r;
  const float* part = p.partial + static_cast<int64_t>(col) * rows + r * 4;
  // both to the reference of the largest maximum so far
  float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float top = -CUDART_INF_F, weight = 0.0f;
#pragma unroll 4
  for (int c = lead; c <= last; c += step) {
    const int64_t slot = (static_cast<int64_t>(c) * 2 + (c == lead ? 1 : 0)) * rows;
    const float2 w = __ldcg(ml + slot);
    const float4 x = __ldcg(reinterpret_cast<const float4*>(part + slot * HD));
    const float next = fmaxf(top, w.x);
    const float ref = next == -CUDART_INF_F ? 0.0f : next;
    const float f_old = attn_ex2(top - ref), f = attn_ex2(w.x - ref);
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

}  // namespace eg
