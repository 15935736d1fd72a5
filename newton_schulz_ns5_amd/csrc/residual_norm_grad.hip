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
// a second launch adds in order.  Four waves per SIMD fill the registers, so the
// latency of one row's loads and sums shows: 8192 x 4096 in bf16 takes 71 us
// (335 MB, 4.7 TB/s) with one norm, 91 (403 MB, 4.4 TB/s) with both and a gate,
// where vector instructions are issued in 60 % of the cycles too.
#include "residual_norm.h"

namespace muon {
namespace {

template <typename T, typename R, int GS, int C, bool POST, bool GATE, bool EDGE>
__global__ __launch_bounds__(Group<GS>::kMaxThreads, 4) void residual_norm_grad_kernel(const ResidualNorm p) {
  constexpr int V = chunk_values<T, R>(), K = C / V;
  constexpr int ROWS = Group<GS>::kRows;
  // The next row's loads are in flight but where V is 4 with both the norm after
  // the block and a gate, or C is 16: this row is unpacked to fp32 first and they
  // take its place (8192 x 4096 in bf16 with both: 96 us; with registers of their
  // own 99; 5105 x 2050 with both and an fp32 stream, left out: 61 us so, 56
  // without).  The choice was timed at these shapes only, and spilled registers
  // stand on both sides of it.  With loads ahead: none to 9 of a workgroup per row,
  // 19 to 30 of 8 or 32 threads with both at V = 8, up to 28 with a gate alone at
  // V = 4.  Without: 4 to 20 of a workgroup, 20 to 35 of 8 or 32 threads, and at
  // C = 16 up to 15 with neither, 135 with one, 49 to 143 with both.
  constexpr bool AHEAD = C == 8 && (V == 8 || !(POST && GATE));
  constexpr bool NEED_B = POST || GATE;
  // The sums of PW and G over rows stay in LDS where both are there.  2048 rows of
  // 16384 columns in bf16: both take 158 us there, 252 from spilled registers; one
  // of them alone 112 and 110 there, 109 and 107 in registers.  Beside fp32 a kernel
  // with one of them spills 30 to 135 registers and was not timed in LDS: with a
  // norm after the block and an fp32 stream it takes 152 us, both 242.
  constexpr bool LDS_SUMS = C == 16 && POST && GATE;
  constexpr int KR = LDS_SUMS ? 1 : K;
  enum { W, PW, G };
  extern __shared__ __attribute__((aligned(16))) f32x4 held[];
  __shared__ typename GroupSum<GS, 3>::Buffer red;
  __shared__ float rows[ROWS > 1 ? 4 : 1][ROWS > 1 ? V * GS : 1];
  GroupSum<GS, 3> sum(&red);
  const int lane = Group<GS>::lane(), grp = Group<GS>::row();
  int col[K], valid[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    col[k] = V * (lane + k * Group<GS>::size());
    valid[k] = p.cols - col[k] < 0 ? 0 : (p.cols - col[k] < V ? p.cols - col[k] : V);
  }
  const bool gate_row = GATE && p.gate_each == 1 && p.rows > 1;  // a gate for every row: its gradient is not a sum
  const int gate_bytes = p.gate_bf16 ? 2 : 4;
  Vectors<GS, K, V, 3, EDGE> vec;
  f32x4* at = held;
  vec.set(W, p.norm ? p.weight : nullptr, p.weight_bf16, p.offset, at, p.held);
  vec.set(PW, POST ? p.post_weight : nullptr, p.weight_bf16, p.offset, at, p.held);
  vec.set(G, GATE && !gate_row ? p.gate : nullptr, p.gate_bf16, 0.f, at, p.held);
  vec.fill(col, valid);
  float aw[K][V], ap[KR][V], ag[KR][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int e = 0; e < V; ++e) aw[k][e] = ap[LDS_SUMS ? 0 : k][e] = ag[LDS_SUMS ? 0 : k][e] = 0.f;
  }
  // A thread's own places in LDS, behind the vectors: no other thread's.
  auto slot = [&](bool post, int k, int h) -> f32x4& {
    return at[((post ? C / 4 : 0) + k * (V / 4) + h) * Group<GS>::size() + Group<GS>::lane()];
  };
  auto clear = [&](bool post) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int h = 0; h < V / 4; ++h) slot(post, k, h) = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  };
  auto add = [&](bool post, int k, const float (&v)[V]) {
#pragma unroll
    for (int h = 0; h < V / 4; ++h) slot(post, k, h) += f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
  };
  auto sums_of = [&](bool post, int k, float (&v)[V]) {
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
      const f32x4 t = slot(post, k, h);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * h + e] = t[e];
    }
  };
  if constexpr (LDS_SUMS) {
    clear(false);
    clear(true);
  }
  // A sum over a workgroup's rows: its groups' sums in order, by the threads
  // of the first group.
  auto total = [&](float (&a)[V]) {
    if constexpr (ROWS > 1) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int off = 32; off >= (GS ? GS : 64); off >>= 1) a[e] += __shfl_xor(a[e], off, 64);
      }
      __syncthreads();  // what was there has been read
      if ((threadIdx.x & 63) < GS) {
#pragma unroll
        for (int e = 0; e < V; ++e) rows[threadIdx.x >> 6][V * lane + e] = a[e];
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < V; ++e) {
        a[e] = rows[0][V * lane + e];
#pragma unroll
        for (int q = 1; q < 4; ++q) a[e] += rows[q][V * lane + e];
      }
    }
  };
  const float inv = 1.f / (float)p.cols;
  struct Row {
    Chunk<T, V, EDGE> dy[K], b[K];
    Chunk<R, V, EDGE> s[K], ds[K];
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
      if (NEED_B) w.b[k].load(b, col[k], valid[k]);
    }
  };
  int64_t gate_at = 0;  // the gate that vec has: the first one, then that of the unit
  for (int64_t u = blockIdx.x; u < p.units; u += gridDim.x) {
    const int64_t g = u / p.gate_chunks;
    const int64_t r0 = g * p.span + (u - g * p.gate_chunks) * p.unit_rows;
    const int64_t end = (g + 1) * p.span < p.rows ? (g + 1) * p.span : p.rows;
    const int64_t r1 = r0 + p.unit_rows < end ? r0 + p.unit_rows : end;
    if (GATE && !gate_row && g != gate_at) {
      vec.refill(G, row_of<GS>(p.gate, g, p.ldg, gate_bytes), col, valid);
      gate_at = g;
    }
    const void* gate = nullptr;
    int64_t r = r0 + grp;
    Row raw;
    if (AHEAD && r < r1) load_row(r, raw);
    for (; r < r1; r += ROWS) {
      if constexpr (!AHEAD) load_row(r, raw);
      // The row's values: unpacked where the next row's loads take their place.
      float dyv[AHEAD ? K : 1][V], sv[AHEAD ? K : 1][V], bv[AHEAD ? K : 1][V], d[K][V];
#pragma unroll
      for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if constexpr (AHEAD) {
            dyv[k][e] = raw.dy[k].value(e);
            sv[k][e] = raw.s[k].value(e);
            bv[k][e] = NEED_B ? raw.b[k].value(e) : 0.f;
          }
          d[k][e] = p.dstream ? raw.ds[k].value(e) : 0.f;
        }
      }
      auto dy = [&](int k, int e) { return AHEAD ? dyv[AHEAD ? k : 0][e] : raw.dy[k].value(e); };
      auto s = [&](int k, int e) { return AHEAD ? sv[AHEAD ? k : 0][e] : raw.s[k].value(e); };
      auto b = [&](int k, int e) { return AHEAD ? bv[AHEAD ? k : 0][e] : NEED_B ? raw.b[k].value(e) : 0.f; };
      if (AHEAD && r + ROWS < r1) load_row(r + ROWS, raw);
      if (gate_row) gate = row_of<GS>(p.gate, r, p.ldg, gate_bytes);
      // sum s^2, sum dy w s, sum b^2
      float q[3] = {0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (valid[k] <= 0) continue;
        if (p.norm) {
          float w[V];
          vec.get(W, k, col[k], valid[k], w);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            q[0] += s(k, e) * s(k, e);
            q[1] += dy(k, e) * w[e] * s(k, e);
          }
        }
        if (POST) {
#pragma unroll
          for (int e = 0; e < V; ++e) q[2] += b(k, e) * b(k, e);
        }
      }
      if constexpr (POST) {
        sum(q);
      } else if (p.norm) {
        float two[2] = {q[0], q[1]};
        sum(two);
        q[0] = two[0];
        q[1] = two[1];
      }
      // D = ds + rs dy w - c s, c = rs^3 mean(dy w s)
      const float rs = p.norm ? __frsqrt_rn(q[0] * inv + p.eps) : 0.f, c = q[1] * inv * rs * rs * rs;
      const float rb = POST ? __frsqrt_rn(q[2] * inv + p.eps) : 1.f;
      auto m = [&](int k, int e) { return POST && !AHEAD ? b(k, e) * rb : b(k, e); };  // b holds m from here on where it can
      void* const dres = row_of<GS>(p.dresidual, r, p.lddr, sizeof(R));
      float dot[1] = {0.f};
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (valid[k] <= 0) continue;
        if (p.norm) {
          float w[V];
          vec.get(W, k, col[k], valid[k], w);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            aw[k][e] += dy(k, e) * (s(k, e) * rs);
            d[k][e] = fmaf(-c, s(k, e), fmaf(rs, dy(k, e) * w[e], d[k][e]));
          }
        }
        if (p.dresidual) {
          float t[V];
#pragma unroll
          for (int e = 0; e < V; ++e) t[e] = p.residual_scale * d[k][e];
          round_store<R, V, EDGE, kPlain>(dres, col[k], valid[k], t);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) d[k][e] *= p.scale;        // t
        float gt[V], pw[V], dg[V], dp[V];
        if (GATE) {
          if (!gate_row) vec.get(G, k, col[k], valid[k], gt);
          else load_values<V, EDGE>(gate, col[k], p.gate_bf16 != 0, valid[k], gt);
        }
        if (POST) vec.get(PW, k, col[k], valid[k], pw);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if constexpr (POST && AHEAD) bv[k][e] *= rb;
          const float tm = d[k][e] * m(k, e);
          if (GATE) {
            dg[e] = POST ? tm * pw[e] : tm;
            d[k][e] *= gt[e];
          }
          if (POST) {
            if constexpr (LDS_SUMS) dp[e] = GATE ? tm * gt[e] : tm;
            else ap[k][e] += GATE ? tm * gt[e] : tm;
            d[k][e] *= pw[e];                                  // k
            dot[0] += d[k][e] * m(k, e);
          }
        }
        if constexpr (POST && LDS_SUMS) add(true, k, dp);
        if (GATE) {
          if (gate_row) {
            if (p.dgate) store_values<V, EDGE>(row_of<GS>(p.dgate, r, p.lddg, gate_bytes), col[k], p.gate_bf16 != 0, valid[k], dg);
          } else if constexpr (LDS_SUMS) {
            add(false, k, dg);
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) ag[k][e] += dg[e];
          }
        }
      }
      if (POST) {
        sum(dot);
        const float cb = dot[0] * inv * rb;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
          for (int e = 0; e < V; ++e) d[k][e] = fmaf(-cb, m(k, e), rb * d[k][e]);
        }
      }
      if (p.dblock) {
        void* const db = row_of<GS>(p.dblock, r, p.lddb, sizeof(T));
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (valid[k] > 0) round_store<T, V, EDGE, kPlain>(db, col[k], valid[k], d[k]);
        }
      }
    }
    if (GATE && !gate_row && (p.dgate || p.part[2])) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if constexpr (LDS_SUMS) sums_of(false, k, ag[0]);
        float (&a)[V] = ag[LDS_SUMS ? 0 : k];
        total(a);
        if (grp == 0 && valid[k] > 0) {
          if (p.part[2]) round_store<float, V, EDGE, kPlain>(p.part[2] + u * p.cols, col[k], valid[k], a);
          else store_values<V, EDGE>((char*)p.dgate + g * p.lddg * gate_bytes, col[k], p.gate_bf16 != 0, valid[k], a);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) a[e] = 0.f;
      }
      if constexpr (LDS_SUMS) clear(false);
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (p.part[0]) {
      total(aw[k]);
      if (grp == 0 && valid[k] > 0) round_store<float, V, EDGE, kPlain>(p.part[0] + (int64_t)blockIdx.x * p.cols, col[k], valid[k], aw[k]);
    }
    if (POST && p.part[1]) {
      auto& a = ap[LDS_SUMS ? 0 : k];
      if constexpr (LDS_SUMS) sums_of(true, k, a);
      total(a);
      if (grp == 0 && valid[k] > 0) round_store<float, V, EDGE, kPlain>(p.part[1] + (int64_t)blockIdx.x * p.cols, col[k], valid[k], a);
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
  const NormShape shape = norm_shape(p.cols);
  return with_norm_form(shape, p, [&](auto g, auto c, auto post, auto gate, auto e) {
    return launch_kernel(residual_norm_grad_kernel<T, R, decltype(g)::value, decltype(c)::value, decltype(post)::value,
                                                   decltype(gate)::value, decltype(e)::value>,
                         dim3((unsigned)blocks), p, s, norm_threads(shape), p.held + p.sums);
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
