// Epilogue of the linear product on 8 consecutive columns of a row:
// z = v + bias, Z = z, Y = act(z) + add, in fp32 with one rounding on store.
#pragma once

#include "layer_internal.h"
#include "layer_math.h"

namespace muon {

// Element `idx` .. + 7 as fp32; the first `valid` of them where they are not
// whole, aligned chunks.
__device__ __forceinline__ void get8(const void* base, int64_t idx, bool bf, bool vec, int valid, float (&v)[8]) {
  if (vec && valid >= 8) {
    if (bf) {
      const u32x4 a = *(const u32x4*)((const uint16_t*)base + idx);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        v[2 * w] = __uint_as_float(a[w] << 16);
        v[2 * w + 1] = __uint_as_float(a[w] & 0xffff0000u);
      }
    } else {
      const f32x4 a = *(const f32x4*)((const float*)base + idx), b = *(const f32x4*)((const float*)base + idx + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[4 + e] = b[e]; }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < valid ? load_elem(base, idx + e, bf) : 0.f;
  }
}

__device__ __forceinline__ void put8(void* base, int64_t idx, bool bf, bool vec, int valid, const float (&v)[8]) {
  if (vec && valid >= 8) {
    if (bf) {
      u32x4 a;
#pragma unroll
      for (int w = 0; w < 4; ++w) a[w] = pack_bf2(v[2 * w], v[2 * w + 1]);
      *(u32x4*)((uint16_t*)base + idx) = a;
    } else {
      *(f32x4*)((float*)base + idx) = f32x4{v[0], v[1], v[2], v[3]};
      *(f32x4*)((float*)base + idx + 4) = f32x4{v[4], v[5], v[6], v[7]};
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
    get8(p.bias, j, p.bias_dtype == MUON_BF16, (p.vec & kVecBias) != 0, valid, b);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = 0.f;
  }
}

template <int ACT, bool BF>
__device__ __forceinline__ void finish8(const LinGemm& p, int64_t i, int64_t j, int valid, const float (&b)[8],
                                        float (&v)[8]) {
  float r[8];
  if (p.add) get8(p.add, i * p.ldadd + j, p.add_dtype == MUON_BF16, (p.vec & kVecAdd) != 0, valid, r);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] += b[e];
  if (p.Z) put8(p.Z, i * p.ldz + j, BF, (p.vec & kVecZ) != 0, valid, v);
  if constexpr (ACT != MUON_ACT_NONE) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = act_fwd<ACT>(v[e]);
  }
  if (p.add) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += r[e];
  }
  put8(p.Y, i * p.ldy + j, p.y_dtype == MUON_BF16, (p.vec & kVecY) != 0, valid, v);
}

}  // namespace muon
