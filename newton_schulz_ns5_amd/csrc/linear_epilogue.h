// Epilogue of the linear product on 8 consecutive columns of a row:
// z = v + bias, Z = z, Y = act(z) + add, in fp32 with one rounding on store.
#pragma once

#include "layer_internal.h"
#include "layer_math.h"

namespace muon {

// 16 bytes at any address (global memory takes unaligned 16-byte accesses).
__device__ __forceinline__ u32x4 load16(const void* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ void store16(void* p, u32x4 v) { __builtin_memcpy(p, &v, 16); }

// Elements idx .. idx + 7 as fp32; only the first `valid` of them exist.
__device__ __forceinline__ void get8(const void* base, int64_t idx, bool bf, int valid, float (&v)[8]) {
  if (valid >= 8) {
    if (bf) {
      const u32x4 a = load16((const uint16_t*)base + idx);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        v[2 * w] = __uint_as_float(a[w] << 16);
        v[2 * w + 1] = __uint_as_float(a[w] & 0xffff0000u);
      }
    } else {
      const u32x4 a = load16((const float*)base + idx), b = load16((const float*)base + idx + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) { v[e] = __uint_as_float(a[e]); v[4 + e] = __uint_as_float(b[e]); }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < valid ? load_elem(base, idx + e, bf) : 0.f;
  }
}

__device__ __forceinline__ void put8(void* base, int64_t idx, bool bf, int valid, const float (&v)[8]) {
  if (valid >= 8) {
    if (bf) {
      u32x4 a;
#pragma unroll
      for (int w = 0; w < 4; ++w) a[w] = pack_bf2(v[2 * w], v[2 * w + 1]);
      store16((uint16_t*)base + idx, a);
    } else {
      u32x4 a, b;
#pragma unroll
      for (int e = 0; e < 4; ++e) { a[e] = __float_as_uint(v[e]); b[e] = __float_as_uint(v[4 + e]); }
      store16((float*)base + idx, a);
      store16((float*)base + idx + 4, b);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < valid) store_elem(base, idx + e, v[e], bf);
  }
}

// The bias of columns j .. j + 7 (zeros without one).
__device__ __forceinline__ void bias8(const LinGemm& p, int64_t j, int valid, float (&b)[8]) {
  if (p.bias) {
    get8(p.bias, j, p.bias_dtype == MUON_BF16, valid, b);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = 0.f;
  }
}

template <int ACT, bool BF>
__device__ __forceinline__ void finish8(const LinGemm& p, int64_t i, int64_t j, int valid, const float (&b)[8],
                                        float (&v)[8]) {
  float r[8];
  if (p.add) get8(p.add, i * p.ldadd + j, p.add_dtype == MUON_BF16, valid, r);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] += b[e];
  if (p.Z) put8(p.Z, i * p.ldz + j, BF, valid, v);
  if constexpr (ACT != MUON_ACT_NONE) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = act_fwd<ACT, BF>(v[e]);
  }
  if (p.add) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += r[e];
  }
  put8(p.Y, i * p.ldy + j, p.y_dtype == MUON_BF16, valid, v);
}

}  // namespace muon
