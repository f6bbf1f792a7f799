// eg_el.cuh -- element types of the decoder operators: conversion of packed
// 16-byte / 8-byte words of bf16, fp16 or float32 to float32 and back
// (nearest even).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace eg {

// Two float32 values.
using pk_t = float2;
__device__ __forceinline__ pk_t pk(float lo, float hi) { return make_float2(lo, hi); }
__device__ __forceinline__ float2 unpk(pk_t v) { return v; }
__device__ __forceinline__ pk_t pk_fma(pk_t a, pk_t b, pk_t c) { return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)); }
__device__ __forceinline__ pk_t pk_mul(pk_t a, pk_t b) { return make_float2(a.x * b.x, a.y * b.y); }
__device__ __forceinline__ pk_t pk_swap(pk_t v) { return make_float2(v.y, v.x); }
__device__ __forceinline__ float pk_sum(pk_t v) { return v.x + v.y; }

template <typename T>
struct El;

template <>
struct El<__nv_bfloat16> {
  static constexpr bool kBf16 = true;
  static __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
  // the two elements of one 32-bit word (low half first)
  static __device__ __forceinline__ float2 unpack2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

template <>
struct El<__half> {
  static constexpr bool kBf16 = false;
  static __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
  static __device__ __forceinline__ float2 unpack2(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

template <>
struct El<float> {
  static __device__ __forceinline__ float to_float(float x) { return x; }
  static __device__ __forceinline__ float from_float(float x) { return x; }
};

// CH consecutive elements of type T held as raw 32-bit words.
template <typename T, int CH>
struct Chunk {
  static constexpr int kWords = CH * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      static_assert(kWords == 2, "a chunk is 8 or 16 bytes");
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kWords == 4)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void get(float (&f)[CH]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < CH; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const float2 v = El<T>::unpack2(w[i]);
        f[2 * i] = v.x, f[2 * i + 1] = v.y;
      }
    }
  }
  // the elements in pairs
  __device__ __forceinline__ void get(pk_t (&f)[CH / 2]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) f[i] = pk(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const float2 v = El<T>::unpack2(w[i]);
        f[i] = pk(v.x, v.y);
      }
    }
  }
  __device__ __forceinline__ void set(const pk_t (&f)[CH / 2]) {
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) {
      const float2 v = unpk(f[i]);
      if constexpr (sizeof(T) == 4) w[2 * i] = __float_as_uint(v.x), w[2 * i + 1] = __float_as_uint(v.y);
      else w[i] = El<T>::pack2(v.x, v.y);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[CH]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < CH; ++i) w[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = El<T>::pack2(f[2 * i], f[2 * i + 1]);
    }
  }
};

}  // namespace eg
