// What the forward and backward kernels of the norms around a block share: a
// row in the registers of a group of threads.
#pragma once

#include "chunks.h"
#include "pass_internal.h"

namespace muon {

// A row is held by GS threads of a wave (8 or 32), or by a whole workgroup
// (GS 0), which has as many waves as the row needs.
template <int GS>
struct Group {
  static constexpr int kRows = GS ? 256 / GS : 1;  // rows of a workgroup
  static constexpr int kMaxThreads = GS ? 256 : 1024;
  static __device__ __forceinline__ int size() { return GS ? GS : (int)blockDim.x; }
  static __device__ __forceinline__ int lane() { return GS ? (int)threadIdx.x % (GS ? GS : 1) : (int)threadIdx.x; }
  static __device__ __forceinline__ int row() { return GS ? (int)threadIdx.x / (GS ? GS : 1) : 0; }
};

// Row r of a tensor.  Where a wave holds one row its address is made scalar:
// the lanes add 32-bit offsets to it.
template <int GS>
__device__ __forceinline__ void* row_of(const void* base, int64_t r, int64_t ld, int bytes) {
  uint64_t a = (uint64_t)base + (uint64_t)(r * ld * bytes);
  if constexpr (GS == 0) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a), hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
    a = ((uint64_t)hi << 32) | lo;
  }
  return (void*)a;
}

// Sums of N values over the group that holds a row, the same bits in all its
// threads.  Over a workgroup through LDS, two buffers in turn: one barrier per
// sum, since a buffer is written again only after the other one's barrier.
template <int GS, int N>
struct GroupSum {
  struct Buffer { __attribute__((aligned(16))) float v[2][N][GS ? 4 : 16]; };
  Buffer* red;
  int turn = 0;
  __device__ __forceinline__ explicit GroupSum(Buffer* b) : red(b) {
    if constexpr (GS == 0) {
      for (int i = threadIdx.x; i < 2 * N * 16; i += blockDim.x) (&red->v[0][0][0])[i] = 0.f;  // of waves that are not there
      __syncthreads();
    }
  }
  template <int M>
  __device__ __forceinline__ void operator()(float (&v)[M]) {
    static_assert(M <= N, "more sums than the buffer holds");
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] = GS ? lanes_sum<GS ? GS : 64>(v[i]) : lanes_sum_last(v[i]);
    if constexpr (GS == 0) {
      if ((threadIdx.x & 63) == 63) {
#pragma unroll
        for (int i = 0; i < M; ++i) red->v[turn][i][threadIdx.x >> 6] = v[i];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < M; ++i) v[i] = 0.f;
      for (int w = 0; w < (int)blockDim.x; w += 256) {
#pragma unroll
        for (int i = 0; i < M; ++i) {
          const f32x4 t = *(const f32x4*)&red->v[turn][i][w >> 6];
          v[i] += (t[0] + t[1]) + (t[2] + t[3]);
        }
      }
      turn ^= 1;
    }
  }
};

// The vectors of every row (weights, a gate for all rows or the gate of those
// at hand): held in LDS in fp32, 16 bytes of a thread beside those of the others,
// or read from memory again for every row.
template <int GS, int K, int V, int N, bool EDGE>
struct Vectors {
  static constexpr int Q = K * V / 4;  // quarters of a thread
  const void* p[N];
  int bf16[N];
  float offset[N];  // added
  f32x4* lds[N];    // null: not held
  __device__ __forceinline__ void set(int i, const void* ptr, int bf, float off, f32x4*& at, int held) {
    p[i] = ptr;
    bf16[i] = bf;
    offset[i] = off;
    lds[i] = held && ptr ? at : nullptr;
    if (lds[i]) at += Q * Group<GS>::size();
  }
  __device__ __forceinline__ void read(int i, int col, int valid, float (&v)[V]) const {
    load_values<V, EDGE>(p[i], col, bf16[i] != 0, valid, v);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] += offset[i];
  }
  // This thread's chunks of vector i.  Where a workgroup holds one row no other
  // thread reads them.
  __device__ __forceinline__ void hold(int i, const int (&col)[K], const int (&valid)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (valid[k] <= 0) continue;
      float v[V];
      read(i, col[k], valid[k], v);
#pragma unroll
      for (int h = 0; h < V / 4; ++h)
        lds[i][(k * (V / 4) + h) * Group<GS>::size() + Group<GS>::lane()] = f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
    }
  }
  // Threads of the workgroup's first row; a barrier follows.
  __device__ __forceinline__ void fill(const int (&col)[K], const int (&valid)[K]) {
    if (Group<GS>::row() == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (lds[i]) hold(i, col, valid);
      }
    }
    __syncthreads();
  }
  // Another vector in the place of vector i, by all threads of the workgroup.
  __device__ __forceinline__ void refill(int i, const void* ptr, const int (&col)[K], const int (&valid)[K]) {
    p[i] = ptr;
    if (!lds[i]) return;
    if constexpr (Group<GS>::kRows > 1) __syncthreads();  // the other rows have read the one before
    if (Group<GS>::row() == 0) hold(i, col, valid);
    if constexpr (Group<GS>::kRows > 1) __syncthreads();
  }
  // Chunk k of this thread: ones without a vector.
  __device__ __forceinline__ void get(int i, int k, int col, int valid, float (&v)[V]) const {
    if (lds[i]) {
#pragma unroll
      for (int h = 0; h < V / 4; ++h) {
        const f32x4 t = lds[i][(k * (V / 4) + h) * Group<GS>::size() + Group<GS>::lane()];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * h + e] = t[e];
      }
    } else if (p[i]) {
      read(i, col, valid, v);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = 1.f;
    }
  }
};

// f called with what a kernel is compiled for: the threads that hold a row and
// the columns of each, a norm after the block, a gate, rows that end in part of
// a chunk.
template <int GS, int C, typename F>
hipError_t with_norm_flags(const ResidualNorm& p, F&& f) {
  using std::bool_constant;
  const std::integral_constant<int, GS> g;
  const std::integral_constant<int, C> c;
  auto edge = [&](auto post, auto gate) { return p.cols % 8 ? f(g, c, post, gate, bool_constant<true>{}) : f(g, c, post, gate, bool_constant<false>{}); };
  if (p.post) return p.gate ? edge(bool_constant<true>{}, bool_constant<true>{}) : edge(bool_constant<true>{}, bool_constant<false>{});
  return p.gate ? edge(bool_constant<false>{}, bool_constant<true>{}) : edge(bool_constant<false>{}, bool_constant<false>{});
}
template <typename F>
hipError_t with_norm_form(const NormShape& s, const ResidualNorm& p, F&& f) {
  if (s.group == 8 && s.columns == 8) return with_norm_flags<8, 8>(p, f);
  if (s.group == 32 && s.columns == 8) return with_norm_flags<32, 8>(p, f);
  if (s.group >= 64 && s.columns == 8) return with_norm_flags<0, 8>(p, f);
  if (s.group >= 64 && s.columns == 16) return with_norm_flags<0, 16>(p, f);
  return hipErrorInvalidValue;
}

}  // namespace muon
