// Chunks of consecutive values of a row in registers: loaded and stored whole
// or, at the end of a row, in part, at any alignment to the element; and sums
// over lanes without LDS.
#pragma once

#include "device_util.h"

namespace muon {

typedef u32x4 u32x4_any __attribute__((aligned(2)));  // at any element's address
typedef u32x2 u32x2_any __attribute__((aligned(2)));

// How a chunk goes to memory: `kStream` for results that are larger than the
// caches and written once (nontemporal: they do not push out what is read
// again).  It pays where a wave's store instruction covers whole lines, and
// costs where two instructions share them.
enum StorePolicy { kPlain, kStream };

// V values of type T (uint16_t for bf16), the first `valid` of which exist.
// Without EDGE all do, and a thread without a chunk makes no call.
template <typename T, int V, bool EDGE>
struct Chunk {
  static constexpr int W = V * (int)sizeof(T) / 4;
  static constexpr bool kEdge = EDGE;
  static_assert(W == 2 || W == 4 || W == 8, "8, 16 or 32 bytes");
  uint32_t w[W];

  __device__ __forceinline__ void load_whole(const T* p) {
    if constexpr (W == 2) {
      const u32x2 t = *(const u32x2_any*)(const void*)p;
      w[0] = t[0];
      w[1] = t[1];
    } else {
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        const u32x4 t = ((const u32x4_any*)(const void*)p)[q];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * q + e] = t[e];
      }
    }
  }
  // Values at .. at + valid - 1 of a row from `base` on.  A part of a chunk is
  // the end of the row's last V values, moved down; only a row shorter than
  // that is read value by value.
  __device__ __forceinline__ void load(const void* base, uint32_t at, int valid) {
    const T* const p = (const T*)base;
    if constexpr (!EDGE) {
      load_whole(p + at);
    } else {
      const int miss = V - valid;
      if ((int)at >= miss) {
        load_whole(p + (at - miss));
        if (miss) {
          constexpr int PER = 4 / (int)sizeof(T);  // values of a word
#pragma unroll
          for (int s = V / 2; s >= 1; s /= 2) {
            const bool on = miss & s;
#pragma unroll
            for (int e = 0; e < W; ++e) {
              if (s >= PER) {
                const int from = e + s / PER;
                const uint32_t up = from < W ? w[from < W ? from : 0] : 0u;
                w[e] = on ? up : w[e];
              } else {
                const uint32_t up = e + 1 < W ? w[e + 1 < W ? e + 1 : 0] : 0u;
                w[e] = on ? (w[e] >> 16) | (up << 16) : w[e];
              }
            }
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e) w[e] = 0;
#pragma unroll 1
        for (int i = valid - 1; i >= 0; --i) {
#pragma unroll
          for (int e = W - 1; e > 0; --e) w[e] = sizeof(T) == 4 ? w[e - 1] : (w[e] << 16) | (w[e - 1] >> 16);
          if constexpr (sizeof(T) == 4) w[0] = __builtin_bit_cast(uint32_t, p[at + i]);
          else w[0] = (w[0] << 16) | (uint32_t)p[at + i];
        }
      }
    }
  }
  __device__ __forceinline__ float value(int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  }
  __device__ __forceinline__ void round(const float (&v)[V]) {
#pragma unroll
    for (int e = 0; e < W; ++e) {
      if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(v[e]);
      else w[e] = pack_bf2(v[2 * e], v[2 * e + 1]);
    }
  }
  template <StorePolicy POLICY>
  __device__ __forceinline__ void store(void* base, uint32_t at, int valid) {
    T* const p = (T*)base + at;
    if (!EDGE || valid >= V) {
      if constexpr (W == 2) {
        const u32x2 t = {w[0], w[1]};
        if constexpr (POLICY == kStream) __builtin_nontemporal_store(t, (u32x2_any*)(void*)p);
        else *(u32x2_any*)(void*)p = t;
      } else {
#pragma unroll
        for (int q = 0; q < W / 4; ++q) {
          const u32x4 t = {w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]};
          if constexpr (POLICY == kStream) __builtin_nontemporal_store(t, (u32x4_any*)(void*)p + q);
          else ((u32x4_any*)(void*)p)[q] = t;
        }
      }
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

template <typename T, int V, bool EDGE, StorePolicy POLICY>
__device__ __forceinline__ void round_store(void* base, uint32_t at, int valid, const float (&v)[V]) {
  Chunk<T, V, EDGE> r;
  r.round(v);
  r.template store<POLICY>(base, at, valid);
}
// The same with the type known at run time.
template <int V, bool EDGE>
__device__ __forceinline__ void load_values(const void* base, uint32_t at, bool bf16, int valid, float (&v)[V]) {
  if (bf16) {
    Chunk<uint16_t, V, EDGE> r;
    r.load(base, at, valid);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = r.value(e);
  } else {
    Chunk<float, V, EDGE> r;
    r.load(base, at, valid);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = r.value(e);
  }
}
template <int V, bool EDGE>
__device__ __forceinline__ void store_values(void* base, uint32_t at, bool bf16, int valid, const float (&v)[V]) {
  if (bf16) round_store<uint16_t, V, EDGE, kPlain>(base, at, valid, v);
  else round_store<float, V, EDGE, kPlain>(base, at, valid, v);
}

// Values that a lane's chunk holds where tensors of these types are read and
// written together: 16 bytes of the wider type, so that the lanes of a wave
// cover memory without gaps in every instruction.
template <typename A, typename B>
constexpr int chunk_values() { return sizeof(A) == 2 && sizeof(B) == 2 ? 8 : 4; }

// v of another lane: within 16 lanes by the data-parallel primitives, which
// take no LDS access.
template <int CTRL>
__device__ __forceinline__ float lane_move(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// Sum over groups of N lanes (8, 16 or 32), the same bits in each of them.
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
  v += lane_move<0xB1>(v);   // lanes 1 0 3 2
  v += lane_move<0x4E>(v);   // lanes 2 3 0 1
  v += lane_move<0x141>(v);  // the other four of eight, mirrored
  if constexpr (N >= 16) v += lane_move<0x140>(v);  // the other eight of sixteen, mirrored
  if constexpr (N >= 32) v += __shfl_xor(v, 16, 64);
  return v;
}
// Sum over a wave in its last lane.
__device__ __forceinline__ float lanes_sum_last(float v) {
  v = lanes_sum<16>(v);
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x142, 0xa, 0xf, true));  // lane 15 of the row before, to rows 1 and 3
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x143, 0xc, 0xf, true));  // lane 31, to rows 2 and 3
  return v;
}

}  // namespace muon
