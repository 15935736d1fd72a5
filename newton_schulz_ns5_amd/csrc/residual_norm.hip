// The norms before and after a block with its gate and its residual:
//   u = b / sqrt(mean(b^2) + eps) pw    (or u = b)
//   s = residual_scale x + scale gate u
//   y = s / sqrt(mean(s^2) + eps) w
//
// Bound by HBM: b and x are read once, s and y written once.  A row stays in
// the registers of a group of threads, 8 columns each (16 bytes of bf16), from
// its loads to its stores; the two sums of squares are the only traffic between
// the threads.  The next row's loads are in flight during this row's sums.
#include "residual_norm.h"

namespace muon {
namespace {

template <typename T, typename R, int GS, int K, bool EDGE>
__global__ __launch_bounds__(Rows8<GS>::NT) void residual_norm_kernel(const ResidualNorm p) {
  constexpr int RPW = Rows8<GS>::RPW;
  constexpr bool AHEAD = K == 1;     // the next row's loads in flight
  enum { W, PW, G };
  __shared__ float red[2][1][GS > 64 ? GS / 64 : 1];
  __shared__ __attribute__((aligned(16))) float held[Vectors<GS, K, 3, EDGE>::kFloats];
  GroupSum<GS, 1> sum{&red};
  const int j = threadIdx.x % GS, grp = threadIdx.x / GS;
  int col[K], valid[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    col[k] = 8 * (j + k * GS);
    valid[k] = p.cols - col[k] < 0 ? 0 : (p.cols - col[k] < 8 ? p.cols - col[k] : 8);
  }
  const bool gate_all = p.gate && p.gate_each >= p.rows;  // one row of the gate
  Vectors<GS, K, 3, EDGE> vec;
  vec.lds = held;
  vec.set(W, p.weight, p.weight_bf16, p.offset);
  vec.set(PW, p.post_weight, p.weight_bf16, p.offset);
  vec.set(G, gate_all ? p.gate : nullptr, p.gate_bf16, 0.f);
  vec.fill(p.cols);
  const float inv = 1.f / (float)p.cols;
  Raw8<T, EDGE> bn[K];
  Raw8<R, EDGE> xn[K];
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
  const int64_t step = (int64_t)gridDim.x * RPW;
  int64_t r = (int64_t)blockIdx.x * RPW + grp;
  if (AHEAD && r < p.rows) load_row(r);
  for (; r < p.rows; r += step) {
    if constexpr (!AHEAD) load_row(r);
    float v[K][8];
    Raw8<R, EDGE> x[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = valid[k] > 0 ? bn[k].value(e) : 0.f;
      x[k] = xn[k];
    }
    if (AHEAD && r + step < p.rows) load_row(r + step);
    if (p.post) {
      float ss[1] = {0.f};
#pragma unroll
      for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) ss[0] += v[k][e] * v[k][e];
      }
      sum(ss);
      const float rs = __frsqrt_rn(ss[0] * inv + p.eps);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (valid[k] <= 0) continue;
        float t[8];
        vec.get(PW, j, col[k], valid[k], t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] *= rs * t[e];
      }
    }
    const int64_t gr = !p.gate || gate_all ? 0 : (int64_t)((uint32_t)r / (uint32_t)p.gate_each);
    const void* const gate = row_of<GS>(p.gate, gr, p.ldg, p.gate_bf16 ? 2 : 4);
    void* const stream = row_of<GS>(p.stream, r, p.lds, sizeof(R));
    float ss[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (valid[k] <= 0) continue;
      if (p.gate) {
        float t[8];
        if (gate_all) vec.get(G, j, col[k], valid[k], t);
        else load_values<EDGE>(gate, col[k], p.gate_bf16 != 0, valid[k], t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] *= t[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[k][e] *= p.scale;
        if (p.residual) v[k][e] = fmaf(p.residual_scale, x[k].value(e), v[k][e]);
        ss[0] += v[k][e] * v[k][e];
      }
      if (p.stream) round_store<R, EDGE>(stream, col[k], valid[k], v[k]);
    }
    if (p.norm) {
      sum(ss);
      const float rs = __frsqrt_rn(ss[0] * inv + p.eps);
      void* const y = row_of<GS>(p.y, r, p.ldy, sizeof(T));
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (valid[k] <= 0) continue;
        float t[8];
        vec.get(W, j, col[k], valid[k], t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] *= rs * t[e];
        round_store<T, EDGE>(y, col[k], valid[k], v[k]);
      }
    }
  }
}

template <typename T, typename R>
hipError_t launch_types(const ResidualNorm& p, int blocks, hipStream_t s) {
  return with_norm_shape(norm_shape(p.cols), p.cols % 8 != 0, [&](auto g, auto k, auto e) {
    constexpr int GS = decltype(g)::value, K = decltype(k)::value;
    return launch_kernel(residual_norm_kernel<T, R, GS, K, decltype(e)::value>, dim3((unsigned)blocks), p, s, Rows8<GS>::NT);
  });
}

}  // namespace

NormShape norm_shape(int64_t cols) {
  const int64_t chunks = (cols + 7) / 8;
  int g = 8;
  while (g < 1024 && g < chunks) g *= 2;
  int k = 1;
  while ((int64_t)k * g < chunks) k *= 2;
  return {g, k};
}
int norm_threads(const NormShape& s) { return s.group <= 64 ? 256 : s.group; }

hipError_t launch_residual_norm(const ResidualNorm& p, bool bf16, bool stream_bf16, int blocks, hipStream_t s) {
  if (bf16) return stream_bf16 ? launch_types<uint16_t, uint16_t>(p, blocks, s) : launch_types<uint16_t, float>(p, blocks, s);
  return stream_bf16 ? launch_types<float, uint16_t>(p, blocks, s) : launch_types<float, float>(p, blocks, s);
}

}  // namespace muon
