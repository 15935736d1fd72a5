// Gradients of the norms around a block, from the stream s as the forward pass
// stored it.  With n = s / sqrt(mean(s^2) + eps), h = dy w:
//   D = dstream + (h - n mean(h n)) / sqrt(..),  dweight = sum over rows of dy n
//   dresidual = residual_scale D,  t = scale D
//   dgate = sum over the rows of a gate of t u,  d = t gate
//   with m = b / sqrt(mean(b^2) + eps), k = d pw:  dpost_weight = sum of d m,
//   dblock = (k - m mean(k m)) / sqrt(..);  without that norm dblock = d.
//
// Bound by HBM: dy, dstream, s and b are read once, dblock and dresidual
// written once.  A row stays in a group's registers as in the forward pass;
// sum s^2, sum h s and sum b^2 are taken together, sum k m behind them.  The
// sums over rows stay in registers over all rows of a workgroup, whose partials
// a second launch adds in order.
#include "residual_norm.h"

namespace muon {
namespace {

template <typename T, typename R, int GS, int K, bool EDGE>
__global__ __launch_bounds__(Rows8<GS>::NT, 4) void residual_norm_grad_kernel(const ResidualNorm p) {
  constexpr int RPW = Rows8<GS>::RPW, NT = Rows8<GS>::NT;
  constexpr bool AHEAD = K == 1;     // the next row's loads in flight
  enum { W, PW, G };
  __shared__ float red[2][3][GS > 64 ? GS / 64 : 1];
  __shared__ float rows[RPW > 1 ? NT / 64 : 1][RPW > 1 ? 8 * GS : 1];
  __shared__ __attribute__((aligned(16))) float held[Vectors<GS, K, 3, EDGE>::kFloats];
  GroupSum<GS, 3> sum{&red};
  const int j = threadIdx.x % GS, grp = threadIdx.x / GS;
  int col[K], valid[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    col[k] = 8 * (j + k * GS);
    valid[k] = p.cols - col[k] < 0 ? 0 : (p.cols - col[k] < 8 ? p.cols - col[k] : 8);
  }
  const bool gate_all = p.gate && p.gate_each >= p.rows;
  const bool gate_row = p.gate && p.gate_each == 1 && !gate_all;  // a gate for every row: its gradient is not a sum
  Vectors<GS, K, 3, EDGE> vec;
  vec.lds = held;
  vec.set(W, p.weight, p.weight_bf16, p.offset);
  vec.set(PW, p.post_weight, p.weight_bf16, p.offset);
  vec.set(G, gate_all ? p.gate : nullptr, p.gate_bf16, 0.f);
  vec.fill(p.cols);
  float aw[K][8], ap[K][8], ag[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int e = 0; e < 8; ++e) aw[k][e] = ap[k][e] = ag[k][e] = 0.f;
  }
  // A sum over a workgroup's rows: its groups' sums in order, by the threads
  // of the first group.
  auto total = [&](float (&a)[8]) {
    if constexpr (RPW > 1) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int off = 32; off >= GS; off >>= 1) a[e] += __shfl_xor(a[e], off, 64);
      }
      __syncthreads();  // what was there has been read
      if ((threadIdx.x & 63) < GS) {
#pragma unroll
        for (int e = 0; e < 8; ++e) rows[threadIdx.x >> 6][8 * j + e] = a[e];
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = rows[0][8 * j + e];
#pragma unroll
        for (int q = 1; q < NT / 64; ++q) a[e] += rows[q][8 * j + e];
      }
    }
  };
  const float inv = 1.f / (float)p.cols;
  const bool need_b = p.post || p.gate;
  struct Row {
    Raw8<T, EDGE> dy[K], b[K];
    Raw8<R, EDGE> s[K], ds[K];
  };
  auto load_row = [&](int64_t r, Row& w) {
    const void* const dy = row_of<GS>(p.dy, r, p.lddy, sizeof(T));
    const void* const st = row_of<GS>(p.stream, r, p.lds, sizeof(R));
    const void* const ds = row_of<GS>(p.dstream, r, p.ldds, sizeof(R));
    const void* const b = row_of<GS>(p.block, r, p.ldb, sizeof(T));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (valid[k] <= 0) continue;
      if (p.norm) {
        w.dy[k].load(dy, col[k], valid[k]);
        w.s[k].load(st, col[k], valid[k]);
      }
      if (p.dstream) w.ds[k].load(ds, col[k], valid[k]);
      if (need_b) w.b[k].load(b, col[k], valid[k]);
    }
  };
  for (int64_t u = blockIdx.x; u < p.units; u += gridDim.x) {
    const int64_t g = u / p.gate_chunks;
    const int64_t r0 = g * p.span + (u - g * p.gate_chunks) * p.unit_rows;
    const int64_t end = (g + 1) * p.span < p.rows ? (g + 1) * p.span : p.rows;
    const int64_t r1 = r0 + p.unit_rows < end ? r0 + p.unit_rows : end;
    int64_t r = r0 + grp;
    Row row, next;
    if (AHEAD && r < r1) load_row(r, next);
    for (; r < r1; r += RPW) {
      if constexpr (AHEAD) {
        row = next;
        if (r + RPW < r1) load_row(r + RPW, next);
      } else {
        load_row(r, row);
      }
      float q[3] = {0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (valid[k] <= 0) continue;
        if (p.norm) {
          float w[8];
          vec.get(W, j, col[k], valid[k], w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            q[0] += row.s[k].value(e) * row.s[k].value(e);
            q[1] += row.dy[k].value(e) * w[e] * row.s[k].value(e);
          }
        }
        if (p.post) {
#pragma unroll
          for (int e = 0; e < 8; ++e) q[2] += row.b[k].value(e) * row.b[k].value(e);
        }
      }
      if (p.norm || p.post) sum(q);
      const float rs = p.norm ? __frsqrt_rn(q[0] * inv + p.eps) : 0.f, mean = q[1] * rs * inv;
      const float rb = p.post ? __frsqrt_rn(q[2] * inv + p.eps) : 1.f;
      const int64_t gr = !p.gate || gate_all ? 0 : (int64_t)((uint32_t)r / (uint32_t)p.gate_each);
      void* const dres = row_of<GS>(p.dresidual, r, p.lddr, sizeof(R));
      const void* const gate = row_of<GS>(p.gate, gr, p.ldg, p.gate_bf16 ? 2 : 4);
      float d[K][8];
      float dot[1] = {0.f};
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (valid[k] <= 0) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) d[k][e] = p.dstream ? row.ds[k].value(e) : 0.f;
        if (p.norm) {
          float w[8];
          vec.get(W, j, col[k], valid[k], w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float n = row.s[k].value(e) * rs, dy = row.dy[k].value(e);
            aw[k][e] += dy * n;
            d[k][e] += rs * (dy * w[e] - n * mean);
          }
        }
        if (p.dresidual) {
          float t[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) t[e] = p.residual_scale * d[k][e];
          round_store<R, EDGE>(dres, col[k], valid[k], t);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) d[k][e] *= p.scale;       // t
        float pw[8];
        if (p.post) {
          vec.get(PW, j, col[k], valid[k], pw);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) pw[e] = 1.f;
        }
        if (p.gate) {
          float gt[8], dg[8];
          if (gate_all) vec.get(G, j, col[k], valid[k], gt);
          else load_values<EDGE>(gate, col[k], p.gate_bf16 != 0, valid[k], gt);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            dg[e] = d[k][e] * (row.b[k].value(e) * rb) * pw[e];
            d[k][e] *= gt[e];
          }
          if (gate_row) {
            if (p.dgate) store_values<EDGE>(row_of<GS>(p.dgate, r, p.lddg, p.gate_bf16 ? 2 : 4), col[k], p.gate_bf16 != 0, valid[k], dg);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) ag[k][e] += dg[e];
          }
        }
        if (p.post) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float m = row.b[k].value(e) * rb;
            ap[k][e] += d[k][e] * m;
            d[k][e] *= pw[e];                                  // k
            dot[0] += d[k][e] * m;
          }
        }
      }
      if (p.post) {
        sum(dot);
        const float mk = dot[0] * inv;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (valid[k] <= 0) continue;
#pragma unroll
          for (int e = 0; e < 8; ++e) d[k][e] = rb * (d[k][e] - row.b[k].value(e) * rb * mk);
        }
      }
      if (p.dblock) {
        void* const db = row_of<GS>(p.dblock, r, p.lddb, sizeof(T));
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (valid[k] > 0) round_store<T, EDGE>(db, col[k], valid[k], d[k]);
        }
      }
    }
    if (p.gate && !gate_row && (p.dgate || p.part[2])) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        total(ag[k]);
        if (grp == 0 && valid[k] > 0) {
          if (p.part[2]) round_store<float, EDGE>(p.part[2] + u * p.cols, col[k], valid[k], ag[k]);
          else store_values<EDGE>((char*)p.dgate + g * p.lddg * (p.gate_bf16 ? 2 : 4), col[k], p.gate_bf16 != 0, valid[k], ag[k]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ag[k][e] = 0.f;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (p.part[0]) {
      total(aw[k]);
      if (grp == 0 && valid[k] > 0) round_store<float, EDGE>(p.part[0] + (int64_t)blockIdx.x * p.cols, col[k], valid[k], aw[k]);
    }
    if (p.part[1]) {
      total(ap[k]);
      if (grp == 0 && valid[k] > 0) round_store<float, EDGE>(p.part[1] + (int64_t)blockIdx.x * p.cols, col[k], valid[k], ap[k]);
    }
  }
}

// 32 columns by 32 parts: a part adds every 32nd row, then the parts are added
// pairwise.
constexpr int SC = 32, SP = 32;
__global__ __launch_bounds__(SC * SP) void norm_sums_kernel(const NormSums p) {
  __shared__ float red[SP][SC + 1];
  int o = 0, g = blockIdx.y;
  while (o < 2 && g >= p.groups[o]) g -= p.groups[o++];
  const int c = threadIdx.x % SC, part = threadIdx.x / SC;
  const int j = blockIdx.x * SC + c;
  const float* const src = p.part[o] + (int64_t)g * p.count[o] * p.cols;
  float t = 0.f;
  if (j < p.cols) {
#pragma unroll 8
    for (int i = part; i < p.count[o]; i += SP) t += src[(int64_t)i * p.cols + j];
  }
  red[part][c] = t;
#pragma unroll
  for (int half = SP / 2; half >= 1; half >>= 1) {
    __syncthreads();
    if (part < half) red[part][c] += red[part + half][c];
  }
  if (part == 0 && j < p.cols) store_elem(p.out[o], g * p.ld[o] + j, red[0][c], p.bf16[o] != 0);
}

template <typename T, typename R>
hipError_t launch_types(const ResidualNorm& p, int blocks, hipStream_t s) {
  return with_norm_shape(norm_shape(p.cols), p.cols % 8 != 0, [&](auto g, auto k, auto e) {
    constexpr int GS = decltype(g)::value, K = decltype(k)::value;
    return launch_kernel(residual_norm_grad_kernel<T, R, GS, K, decltype(e)::value>, dim3((unsigned)blocks), p, s, Rows8<GS>::NT);
  });
}

}  // namespace

hipError_t launch_residual_norm_grad(const ResidualNorm& p, bool bf16, bool stream_bf16, int blocks, hipStream_t s) {
  if (bf16) return stream_bf16 ? launch_types<uint16_t, uint16_t>(p, blocks, s) : launch_types<uint16_t, float>(p, blocks, s);
  return stream_bf16 ? launch_types<float, uint16_t>(p, blocks, s) : launch_types<float, float>(p, blocks, s);
}

hipError_t launch_norm_sums(const NormSums& p, hipStream_t s) {
  const int y = p.groups[0] + p.groups[1] + p.groups[2];
  if (!y || !p.cols) return hipSuccess;
  if (y > 65535) return hipErrorInvalidValue;
  return launch_kernel(norm_sums_kernel, dim3((unsigned)((p.cols + SC - 1) / SC), (unsigned)y), p, s, SC * SP);
}

}  // namespace muon
