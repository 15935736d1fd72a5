// The norms before and after a block with its gate and its residual:
//   u = b / sqrt(mean(b^2) + eps) pw    (or u = b)
//   s = residual_scale x + scale gate u
//   y = s / sqrt(mean(s^2) + eps) w
//
// Bound by HBM: b and x are read once, s and y written once.  A row stays in
// the registers of a group of threads, 8 columns each (16 bytes of bf16), from
// its loads to its stores; the two sums of squares are the only traffic between
// the threads.  The next row's loads are in flight during this row's sums.
// 8192 rows of 4096 in bf16, both norms, a gate and a residual: 53 us for
// 268 MB, 5.0 TB/s, a large copy's rate.  One row: 2.7 us, of which the loads,
// two sums over a workgroup and the launch are all.
#include "residual_norm.h"

namespace muon {
namespace {

template <typename T, typename R, int GS, int C, bool POST, bool GATE, bool EDGE>
__global__ __launch_bounds__(Group<GS>::kMaxThreads) void residual_norm_kernel(const ResidualNorm p) {
  constexpr int V = chunk_values<T, R>(), K = C / V;
  constexpr bool AHEAD = C == 8;     // the next row's loads in flight
  // What is stored is read next: nontemporal stores gain 2 us of 100 alone and
  // cost the product that reads y 5 (a norm and its product: 153 and 158 us).
  constexpr StorePolicy TO_STREAM = kPlain, TO_Y = kPlain;
  enum { W, PW, G };
  extern __shared__ __attribute__((aligned(16))) f32x4 held[];
  __shared__ typename GroupSum<GS, 1>::Buffer red;
  GroupSum<GS, 1> sum(&red);
  int col[K], valid[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    col[k] = V * (Group<GS>::lane() + k * Group<GS>::size());
    valid[k] = p.cols - col[k] < 0 ? 0 : (p.cols - col[k] < V ? p.cols - col[k] : V);
  }
  const bool gate_all = GATE && p.gate_each >= p.rows;  // one row of the gate
  Vectors<GS, K, V, 3, EDGE> vec;
  f32x4* at = held;
  vec.set(W, p.norm ? p.weight : nullptr, p.weight_bf16, p.offset, at, p.held);
  vec.set(PW, POST ? p.post_weight : nullptr, p.weight_bf16, p.offset, at, p.held);
  vec.set(G, gate_all ? p.gate : nullptr, p.gate_bf16, 0.f, at, p.held);
  vec.fill(col, valid);
  const float inv = 1.f / (float)p.cols;
  Chunk<T, V, EDGE> bn[K];
  Chunk<R, V, EDGE> xn[K];
  auto load_row = [&](int64_t r) {
    const void* const b = row_of<GS>(p.block, r, p.ldb, sizeof(T));
    const void* const x = row_of<GS>(p.residual, r, p.ldr, sizeof(R));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (valid[k] <= 0) continue;
      bn[k].load(b, col[k], valid[k]);
      if (p.residual) xn[k].load(x, col[k], valid[k]);
    }
  };
  const int64_t step = (int64_t)gridDim.x * Group<GS>::kRows;
  int64_t r = (int64_t)blockIdx.x * Group<GS>::kRows + Group<GS>::row();
  if (AHEAD && r < p.rows) load_row(r);
  for (; r < p.rows; r += step) {
    if constexpr (!AHEAD) load_row(r);
    float v[K][V];
    Chunk<R, V, EDGE> x[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int e = 0; e < V; ++e) v[k][e] = valid[k] > 0 ? bn[k].value(e) : 0.f;
      x[k] = xn[k];
    }
    if (AHEAD && r + step < p.rows) load_row(r + step);
    if (POST) {
      float ss[1] = {0.f};
#pragma unroll
      for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < V; ++e) ss[0] += v[k][e] * v[k][e];
      }
      sum(ss);
      const float rs = __frsqrt_rn(ss[0] * inv + p.eps);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (valid[k] <= 0) continue;
        float t[V];
        vec.get(PW, k, col[k], valid[k], t);
#pragma unroll
        for (int e = 0; e < V; ++e) v[k][e] *= rs * t[e];
      }
    }
    const int64_t gr = !GATE || gate_all ? 0 : (int64_t)((uint32_t)r / (uint32_t)p.gate_each);
    const void* const gate = row_of<GS>(p.gate, gr, p.ldg, p.gate_bf16 ? 2 : 4);
    void* const stream = row_of<GS>(p.stream, r, p.lds, sizeof(R));
    float ss[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (valid[k] <= 0) continue;
      if (GATE) {
        float t[V];
        if (gate_all) vec.get(G, k, col[k], valid[k], t);
        else load_values<V, EDGE>(gate, col[k], p.gate_bf16 != 0, valid[k], t);
#pragma unroll
        for (int e = 0; e < V; ++e) v[k][e] *= t[e];
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        v[k][e] *= p.scale;
        if (p.residual) v[k][e] = fmaf(p.residual_scale, x[k].value(e), v[k][e]);
        ss[0] += v[k][e] * v[k][e];
      }
      if (p.stream) round_store<R, V, EDGE, TO_STREAM>(stream, col[k], valid[k], v[k]);
    }
    if (p.norm) {
      sum(ss);
      const float rs = __frsqrt_rn(ss[0] * inv + p.eps);
      void* const y = row_of<GS>(p.y, r, p.ldy, sizeof(T));
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (valid[k] <= 0) continue;
        float t[V];
        vec.get(W, k, col[k], valid[k], t);
#pragma unroll
        for (int e = 0; e < V; ++e) v[k][e] *= rs * t[e];
        round_store<T, V, EDGE, TO_Y>(y, col[k], valid[k], v[k]);
      }
    }
  }
}

template <typename T, typename R>
hipError_t launch_types(const ResidualNorm& p, int blocks, hipStream_t s) {
  const NormShape shape = norm_shape(p.cols);
  return with_norm_form(shape, p, [&](auto g, auto c, auto post, auto gate, auto e) {
    return launch_kernel(residual_norm_kernel<T, R, decltype(g)::value, decltype(c)::value, decltype(post)::value, decltype(gate)::value,
                                              decltype(e)::value>,
                         dim3((unsigned)blocks), p, s, norm_threads(shape), p.held);
  });
}

}  // namespace

// Eight threads up to 64 columns (262144 x 64 in bf16: forward 21 us, backward
// 32; by 32 threads 29 and 51), 32 up to 256 (65536 x 256 backward: 32 us, by a
// wave 42; 131072 x 128: 33 and 63), then a workgroup of as many waves as the
// row needs, 16 columns to a thread where 8 would take more than 1024 threads.
NormShape norm_shape(int64_t cols) {
  const int64_t chunks = (cols + 7) / 8;
  if (chunks <= 32) return {chunks <= 8 ? 8 : 32, 8};
  if (chunks <= 1024) return {(int)((chunks + 63) / 64 * 64), 8};
  return {(int)((chunks + 127) / 128 * 64), 16};
}

hipError_t launch_residual_norm(const ResidualNorm& p, bool bf16, bool stream_bf16, int blocks, hipStream_t s) {
  if (bf16) return stream_bf16 ? launch_types<uint16_t, uint16_t>(p, blocks, s) : launch_types<uint16_t, float>(p, blocks, s);
  return stream_bf16 ? launch_types<float, uint16_t>(p, blocks, s) : launch_types<float, float>(p, blocks, s);
}

}  // namespace muon
