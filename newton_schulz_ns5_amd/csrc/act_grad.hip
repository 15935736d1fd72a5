// Gradient at the pre-activation, G = dy act'(z), with the bias gradient's
// column sums in the same pass, and the sum of their partials.
//
// Bound by HBM: dy and z are read once and G written once.  A workgroup owns
// 256 columns of a chunk of rows; a thread owns 8 consecutive columns of every
// eighth row of it, keeps their sums in registers, and the eight row groups
// are added in order through LDS, so a column's sum is added in an order that
// depends on the sizes only.  4096 x 14336 in bf16 (352 MB, 69 us at the rate
// of a copy): 80 us.  For gradients in fp32 it stores a second term, what the
// rounding of G left, 117 MB more there.
#include "layer_internal.h"
#include "linear_epilogue.h"

namespace muon {
namespace {

constexpr int CW = 256;  // columns per workgroup

template <bool BF>
__global__ __launch_bounds__(256) void act_grad_kernel(const ActGrad p) {
  __shared__ float red[8][CW + 8];
  const int tid = threadIdx.x, rg = tid >> 5, cg = (tid & 31) * 8;
  const int64_t j = (int64_t)blockIdx.x * CW + cg;
  const int valid = j >= p.N ? 0 : (p.N - j < 8 ? (int)(p.N - j) : 8);
  const int64_t r0 = (int64_t)blockIdx.y * p.rows_per;
  const int64_t r1 = r0 + p.rows_per < p.M ? r0 + p.rows_per : p.M;
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
  if (valid > 0) {
    with_act(p.act, [&](auto act_c) {
      constexpr int ACT = decltype(act_c)::value;
#pragma unroll 2
      for (int64_t i = r0 + rg; i < r1; i += 8) {
        float g[8];
        get8(p.dy, i * p.lddy + j, p.dy_dtype == MUON_BF16, valid, g);
        if constexpr (ACT != MUON_ACT_NONE) {
          float z[8];
          get8(p.z, i * p.ldz + j, BF, valid, z);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] *= act_slope<ACT, BF>(z[e]);
        }
        if (p.G) put8(p.G, i * p.ldg + j, BF, 8, g);  // values past N are zero
        if constexpr (BF) {
          if (p.low) {  // what the rounding left (nothing where it overflowed)
            float l[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float h = bf2f(f2bf(g[e]));
              l[e] = fabsf(h) < __builtin_huge_valf() ? g[e] - h : 0.f;
            }
            put8(p.low, i * p.ldg + j, true, 8, l);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += g[e];
      }
    });
  }
  if (!p.partial) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) red[rg][cg + e] = sum[e];
  __syncthreads();
  const int64_t c = (int64_t)blockIdx.x * CW + tid;
  if (c >= p.N) return;
  float t = red[0][tid];
#pragma unroll
  for (int g = 1; g < 8; ++g) t += red[g][tid];
  p.partial[(int64_t)blockIdx.y * p.N + c] = t;
}

struct ColSum {
  const float* partial; int32_t chunks; int64_t n;
  void* out; int32_t out_dtype; int32_t accumulate;
};

// 16 threads per column add every 16th chunk, then the 16 sums in order.
__global__ __launch_bounds__(256) void col_sum_kernel(const ColSum p) {
  __shared__ float red[16][17];
  const int col = threadIdx.x & 15, q = threadIdx.x >> 4;
  const int64_t j = (int64_t)blockIdx.x * 16 + col;
  float t = 0.f;
  if (j < p.n) {
#pragma unroll 8
    for (int c = q; c < p.chunks; c += 16) t += p.partial[(int64_t)c * p.n + j];
  }
  red[q][col] = t;
  __syncthreads();
  if (q || j >= p.n) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) t += red[i][col];
  const bool bf = p.out_dtype == MUON_BF16;
  if (p.accumulate) t += load_elem(p.out, j, bf);
  store_elem(p.out, j, t, bf);
}

}  // namespace

hipError_t launch_act_grad(const ActGrad& g, bool bf16, hipStream_t s) {
  const int64_t cols = (g.N + CW - 1) / CW;
  if (cols <= 0 || g.M <= 0) return hipSuccess;
  if (cols > INT32_MAX || g.chunks > 65535 || g.chunks * g.rows_per < g.M) return hipErrorInvalidValue;
  const dim3 grid((unsigned)cols, (unsigned)g.chunks);
  return bf16 ? launch_kernel(act_grad_kernel<true>, grid, g, s) : launch_kernel(act_grad_kernel<false>, grid, g, s);
}

hipError_t launch_col_sum(const float* partial, int chunks, int64_t n, void* out, int32_t out_dtype, bool accumulate,
                          hipStream_t s) {
  const int64_t blocks = (n + 15) / 16;
  if (blocks <= 0) return hipSuccess;
  if (blocks > INT32_MAX) return hipErrorInvalidValue;
  const ColSum p{partial, chunks, n, out, out_dtype, accumulate ? 1 : 0};
  return launch_kernel(col_sum_kernel, dim3((unsigned)blocks), p, s);
}

}  // namespace muon
