// What the forward and backward kernels of the norms around a block share: a
// row in the registers of a group of threads.
#pragma once

#include "pass_internal.h"
#include "row8.h"

namespace muon {

// Row r of a tensor of `bf16` (or fp32) values.  Where a wave holds one row its
// address is made scalar: the lanes add 32-bit offsets to it.
template <int GS>
__device__ __forceinline__ void* row_of(const void* base, int64_t r, int64_t ld, int bytes) {
  uint64_t a = (uint64_t)base + (uint64_t)(r * ld * bytes);
  if constexpr (GS >= 64) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a), hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
    a = ((uint64_t)hi << 32) | lo;
  }
  return (void*)a;
}

// Threads of a workgroup that holds rows with groups of GS, and the rows it
// holds at once.
template <int GS>
struct Rows8 {
  static constexpr int NT = GS < 256 && GS <= 64 ? 256 : GS;
  static constexpr int RPW = NT / GS;
};

// Sums of N values over the group that holds a row, the same bits in all its
// threads.  Above a wave's 64 threads through LDS, two buffers in turn: one
// barrier per sum, since a buffer is written again only after the other one's
// barrier.
template <int GS, int N>
struct GroupSum {
  float (*red)[2][N][GS > 64 ? GS / 64 : 1];
  int turn = 0;
  template <int M>
  __device__ __forceinline__ void operator()(float (&v)[M]) {
    static_assert(M <= N, "more sums than the buffer holds");
    constexpr int L = GS < 64 ? GS : 64;
#pragma unroll
    for (int off = L / 2; off >= 1; off >>= 1) {
#pragma unroll
      for (int i = 0; i < M; ++i) v[i] += __shfl_xor(v[i], off, 64);
    }
    if constexpr (GS > 64) {
      const int wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int i = 0; i < M; ++i) (*red)[turn][i][wave] = v[i];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < M; ++i) {
        float t = (*red)[turn][i][0];
#pragma unroll
        for (int w = 1; w < GS / 64; ++w) t += (*red)[turn][i][w];
        v[i] = t;
      }
      turn ^= 1;
    }
  }
};

// The vectors of every row (weights, a gate for all rows) in fp32: in LDS where
// a thread has one chunk, read again for every row where it has two.
template <int GS, int K, int N, bool EDGE>
struct Vectors {
  static constexpr bool kLds = K == 1;
  static constexpr int kFloats = kLds ? N * 8 * GS : 4;
  const void* p[N];
  bool bf16[N];
  float offset[N];  // added
  float* lds;
  __device__ __forceinline__ void set(int i, const void* ptr, int bf, float off) {
    p[i] = ptr;
    bf16[i] = bf != 0;
    offset[i] = off;
  }
  // Fills the LDS copies (threads of the first group); a barrier follows.
  __device__ __forceinline__ void fill(int cols) {
    if constexpr (kLds) {
      if ((int)threadIdx.x < GS) {
        const int col = 8 * threadIdx.x, valid = cols - col < 0 ? 0 : (cols - col < 8 ? cols - col : 8);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float v[8] = {};
          if (valid > 0) read(i, col, valid, v);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            ((f32x4*)lds)[(2 * i + h) * GS + threadIdx.x] = f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
        }
      }
      __syncthreads();
    }
  }
  __device__ __forceinline__ void read(int i, int col, int valid, float (&v)[8]) const {
    if (p[i]) {
      load_values<EDGE>(p[i], col, bf16[i], valid, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += offset[i];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 1.f;
    }
  }
  // Columns col .. col + 7, chunk j of the group.
  __device__ __forceinline__ void get(int i, int j, int col, int valid, float (&v)[8]) const {
    if constexpr (kLds) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 t = ((const f32x4*)lds)[(2 * i + h) * GS + j];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * h + e] = t[e];
      }
    } else {
      read(i, col, valid, v);
    }
  }
};

// f called with the group size and chunk count of a row of `cols` columns.
template <class F>
hipError_t with_norm_shape(const NormShape& s, bool edge, F&& f) {
#define MUON_SHAPE(G, K)                                                                                                \
  if (s.group == G && s.chunks == K)                                                                                    \
    return edge ? f(std::integral_constant<int, G>{}, std::integral_constant<int, K>{}, std::integral_constant<bool, true>{}) \
                : f(std::integral_constant<int, G>{}, std::integral_constant<int, K>{}, std::integral_constant<bool, false>{})
  MUON_SHAPE(8, 1);
  MUON_SHAPE(16, 1);
  MUON_SHAPE(32, 1);
  MUON_SHAPE(64, 1);
  MUON_SHAPE(128, 1);
  MUON_SHAPE(256, 1);
  MUON_SHAPE(512, 1);
  MUON_SHAPE(1024, 1);
  MUON_SHAPE(1024, 2);
#undef MUON_SHAPE
  return hipErrorInvalidValue;
}

}  // namespace muon
