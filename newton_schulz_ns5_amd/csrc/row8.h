// 8 consecutive values of a row in registers, loaded and stored whole or, at the
// end of a row, in part; any alignment to the element.
#pragma once

#include "linear_epilogue.h"

namespace muon {

// 8 consecutive values as they are stored, the first `valid` of which exist.
// A part of a chunk (only at the end of a row whose width is no multiple of 8)
// moves through the words value by value; without EDGE there are none, and a
// thread without a chunk makes no call.
template <typename T, bool EDGE = true>
struct Raw8 {
  static constexpr int W = 2 * (int)sizeof(T);
  uint32_t w[W];
  __device__ __forceinline__ void load(const void* base, uint32_t at, int valid) {
    const T* const p = (const T*)base + at;
    if (!EDGE || valid >= 8) {
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        const u32x4 t = load16((const uint32_t*)(const void*)p + 4 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * q + e] = t[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e) w[e] = 0;
#pragma unroll 1
      for (int i = valid - 1; i >= 0; --i) {
#pragma unroll
        for (int e = W - 1; e > 0; --e) w[e] = sizeof(T) == 4 ? w[e - 1] : (w[e] << 16) | (w[e - 1] >> 16);
        if constexpr (sizeof(T) == 4) w[0] = __builtin_bit_cast(uint32_t, p[i]);
        else w[0] = (w[0] << 16) | (uint32_t)p[i];
      }
    }
  }
  __device__ __forceinline__ float value(int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  }
  __device__ __forceinline__ void round(const float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < W; ++e) {
      if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(v[e]);
      else w[e] = pack_bf2(v[2 * e], v[2 * e + 1]);
    }
  }
  __device__ __forceinline__ void store(void* base, uint32_t at, int valid) {
    T* const p = (T*)base + at;
    if (!EDGE || valid >= 8) {
#pragma unroll
      for (int q = 0; q < W / 4; ++q) store16((uint32_t*)(void*)p + 4 * q, u32x4{w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]});
    } else {
#pragma unroll 1
      for (int i = 0; i < valid; ++i) {
        if constexpr (sizeof(T) == 4) p[i] = __builtin_bit_cast(T, w[0]);
        else p[i] = (T)w[0];
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const uint32_t up = e + 1 < W ? w[e + 1 < W ? e + 1 : 0] : 0u;
          w[e] = sizeof(T) == 4 ? up : (w[e] >> 16) | (up << 16);
        }
      }
    }
  }
};

template <typename T, bool EDGE>
__device__ __forceinline__ void round_store(void* base, uint32_t at, int valid, const float (&v)[8]) {
  Raw8<T, EDGE> r;
  r.round(v);
  r.store(base, at, valid);
}
// The same with the type known at run time.
template <bool EDGE>
__device__ __forceinline__ void load_values(const void* base, uint32_t at, bool bf16, int valid, float (&v)[8]) {
  if (bf16) {
    Raw8<uint16_t, EDGE> r;
    r.load(base, at, valid);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = r.value(e);
  } else {
    Raw8<float, EDGE> r;
    r.load(base, at, valid);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = r.value(e);
  }
}
template <bool EDGE>
__device__ __forceinline__ void store_values(void* base, uint32_t at, bool bf16, int valid, const float (&v)[8]) {
  if (bf16) round_store<uint16_t, EDGE>(base, at, valid, v);
  else round_store<float, EDGE>(base, at, valid, v);
}

}  // namespace muon
