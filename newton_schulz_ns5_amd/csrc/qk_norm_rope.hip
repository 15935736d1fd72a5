// Per-head norm of queries and keys with the position rotation in the same
// pass, its backward pass, and the rotation alone.
//
// Per head row x of D values, with n = x / sqrt(mean(x^2) + eps), u = n w:
//   y = R u, R turning pair p = (a, b) by theta = pos[axis(p)] inv_freq[p]:
//   (u_a c - u_b s, u_b c + u_a s), c = scale cos(theta), s = scale sin(theta);
//   values past the rotated ones pass through.
// Backward, g = R^T dy:  dw += g n,  dx = (g w - n mean(g w n)) / sqrt(..).
//
// Bound by HBM: every value is read and written once.  A wave takes one token
// (or a few, when a token has fewer head rows than a wave holds): its lanes
// first compute the token's cos and sin, one pair each, into LDS, then groups
// of LPR lanes take one head row each.  A lane owns both members of its pairs
// (chunks of VEC consecutive values from the two halves of the rotated part,
// or of adjacent pairs), so a row never leaves its lanes' registers.
//
// 8192 tokens of 32 + 8 heads of 128 in bf16 (168 MB; a copy of as much takes
// 33 us): forward 38 us; backward (252 MB, 49 us) 50 us and 5 for the weight
// gradients.  A workgroup works on q or on k alone and keeps the norm weights
// in LDS, which holds the registers at five waves per SIMD (four backward):
// with both tensors' weights in registers 46 and 67 us; with six waves the
// compiler spills (63 us).  Loading the next row while this one is turned gave
// the last 10 %; loading four rows at once cost more in waves than it gained.
//
// The angle is formed in turns: pos * (inv_freq / 2 pi) less its nearest
// integer, in a fused multiply-add, the factor in two fp64 terms, so that sine
// and cosine are fp32's at any position that fp64 holds (2^53).  A rounded fp64
// product would be off by pos 2^-52 radians, one in fp32 by whole radians at
// 10^7.  What rounding the turns to fp32 leaves turns the sine and cosine once
// more, to first order.
#include "layer_internal.h"
#include "device_util.h"
#include "muon_mi355x.h"

#include <algorithm>

namespace muon {
namespace {

constexpr int NT = 256;
constexpr int kCsPairs = 512;  // (cos, sin) pairs of LDS per wave

// Batch entry of a token (a division only where there are several).
__device__ __forceinline__ int64_t batch_of(const QkParams& p, int64_t tok) { return p.seq == p.tokens ? 0 : tok / p.seq; }

__device__ __forceinline__ int64_t pos_of(const QkParams& p, int64_t tok, int axis) {
  const int64_t b = batch_of(p, tok), t = tok - b * p.seq;
  const int64_t at = axis * p.pos_sa + b * p.pos_sb + t * p.pos_st;
  return p.pos_i64 ? ((const int64_t*)p.pos)[at] : (int64_t)((const int32_t*)p.pos)[at];
}

__device__ __forceinline__ f32x2_t cos_sin(const QkParams& p, int64_t tok, int pair) {
  const double f = p.inv_freq_f64 ? ((const double*)p.inv_freq)[pair] : (double)((const float*)p.inv_freq)[pair];
  const double pos = (double)pos_of(p, tok, p.axis[pair]);
  const double h = f * 0.15915494309189535, l = fma(f, 0.15915494309189535, -h) + f * -9.839338337591243e-18;  // f / 2 pi
  const double half = 2.0 * (fma(pos, h, -rint(pos * h)) + pos * l);  // in half turns
  const float x = (float)half, d = (float)((half - (double)x) * 3.14159265358979323846);
  float s0, c0;
  sincospif(x, &s0, &c0);
  const float c = c0 - s0 * d, s = s0 + c0 * d;
  return f32x2_t{c * p.scale, s * p.scale * p.sign};
}

// VEC consecutive values as they are stored, in registers of 4 bytes.
template <typename T, int VEC>
struct Chunk {
  static constexpr int W = VEC * (int)sizeof(T) / 4;
  uint32_t w[W];
  __device__ __forceinline__ void load(const T* src) {
    if constexpr (W >= 4) {
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        const u32x4 t = ((const u32x4*)src)[q];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * q + e] = t[e];
      }
    } else if constexpr (W == 2) {
      const u32x2 t = *(const u32x2*)src;
      w[0] = t[0]; w[1] = t[1];
    } else {
      w[0] = *(const uint32_t*)src;
    }
  }
  __device__ __forceinline__ void values(float* v) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < W; ++e) v[e] = __uint_as_float(w[e]);
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    }
  }
};

template <typename T, int VEC>
__device__ __forceinline__ void store_chunk(T* dst, const float* v) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (VEC >= 4) {
#pragma unroll
      for (int q = 0; q < VEC / 4; ++q) ((f32x4*)dst)[q] = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    } else {
      *(f32x2_t*)dst = f32x2_t{v[0], v[1]};
    }
  } else {
    if constexpr (VEC == 8) {
      *(u32x4*)dst = u32x4{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7])};
    } else if constexpr (VEC == 4) {
      *(u32x2*)dst = u32x2{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3])};
    } else {
      *(uint32_t*)dst = pack_bf2(v[0], v[1]);
    }
  }
}

template <typename T>
__device__ __forceinline__ T* row_ptr(const QkTensor& x, const QkParams& p, int64_t tok, int head) {
  const int64_t b = batch_of(p, tok), t = tok - b * p.seq;
  return (T*)x.p + b * x.sb + t * x.st + head * x.sh;
}

// MODE 0: rotation; 1: norm and rotation; 2: backward of 1.  A workgroup works
// on q (the first blocks[0] workgroups) or on k.
template <typename T, int MODE, bool INTER, int VEC, int LPR>
__global__ __launch_bounds__(NT, MODE == 2 ? 4 : 5) void qk_kernel(const QkParams p) {
  constexpr int RPW = 64 / LPR;           // head rows a wave takes at once
  __shared__ f32x2_t cs_all[NT / 64][kCsPairs];
  __shared__ __attribute__((aligned(16))) float wts[MODE == 0 ? 4 : 2 * VEC * LPR];
  __shared__ float red[MODE == 2 ? NT / 64 : 1][MODE == 2 ? 2 * VEC * LPR : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q = (int)blockIdx.x >= p.blocks[0];
  const int block = (int)blockIdx.x - (q ? p.blocks[0] : 0);
  const int H = p.heads[q], tw = p.tw[q], parts = p.parts[q];
  const QkTensor px = p.x[q], pg = p.g[q], py = p.y[q];
  f32x2_t* const cs = cs_all[wave];
  const int pairs = p.rot / 2;
  const int j = lane % LPR, grp = lane / LPR;
  const int nch = p.dim / (2 * VEC);      // chunk pairs of a head row
  const bool live = j < nch;
  // The lane's two chunks and the pairs they hold.  Halves: chunk j of the
  // first half of the rotated part with chunk j of the second; the chunks past
  // the rotated part in twos.  Adjacent pairs: chunks j and j + nch.
  const int rch = p.rot / (2 * VEC);      // chunk pairs of the rotated part (halves)
  int c0, c1;
  bool rot0, rot1;
  if constexpr (INTER) {
    c0 = j * VEC; c1 = (j + nch) * VEC;
    rot0 = c0 < p.rot; rot1 = c1 < p.rot;
  } else {
    rot0 = rot1 = j < rch;
    c0 = rot0 ? j * VEC : p.rot + (j - rch) * 2 * VEC;
    c1 = rot0 ? c0 + p.rot / 2 : c0 + VEC;
  }
  float acc[MODE == 2 ? 2 * VEC : 1];
  if constexpr (MODE == 2) {
#pragma unroll
    for (int e = 0; e < 2 * VEC; ++e) acc[e] = 0.f;
  }
  if constexpr (MODE != 0) {
    for (int d = threadIdx.x; d < p.dim; d += NT) wts[d] = p.w[q] ? load_elem(p.w[q], d, p.w_dtype == MUON_BF16) : 1.f;
    __syncthreads();
  }
  const float inv_d = 1.f / (float)p.dim;
  const int64_t groups = (p.tokens + tw - 1) / tw;
  const int64_t items = groups * parts;
  for (int64_t item = (int64_t)block * (NT / 64) + wave; item < items; item += (int64_t)p.blocks[q] * (NT / 64)) {
    const int64_t grp_tok = item / parts;
    const int part = (int)(item - grp_tok * parts);
    const int64_t tok0 = grp_tok * tw;
    const int ntok = (int)(p.tokens - tok0 < tw ? p.tokens - tok0 : tw);
    const int rows = ntok * H, step = parts * RPW;
    Chunk<T, VEC> xc[2], gc[2];
    // Row r of the item: its token and head, and its values in xc (and gc).
    auto load_row = [&](int r) {
      if (!live || r >= rows) return;
      const int t = ntok == 1 ? 0 : r / H;
      const T* const xr = row_ptr<const T>(px, p, tok0 + t, r - t * H);
      xc[0].load(xr + c0);
      xc[1].load(xr + c1);
      if constexpr (MODE == 2) {
        const T* const gr = row_ptr<const T>(pg, p, tok0 + t, r - t * H);
        gc[0].load(gr + c0);
        gc[1].load(gr + c1);
      }
    };
    const int r0 = part * RPW + grp;
    load_row(r0);                         // in flight while the angles are formed
    for (int i = lane; i < ntok * pairs; i += 64) {
      const int t = i / pairs;
      cs[i] = cos_sin(p, tok0 + t, i - t * pairs);
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);   // the wave's own LDS writes before its reads
    __builtin_amdgcn_wave_barrier();
    for (int r = r0; r < rows; r += step) {
      const int t = ntok == 1 ? 0 : r / H;
      float x[2 * VEC], g[2 * VEC];
      float ss = 0.f;
      if (live) {
        xc[0].values(x);
        xc[1].values(x + VEC);
        if constexpr (MODE == 2) {
          gc[0].values(g);
          gc[1].values(g + VEC);
        }
        if constexpr (MODE != 0) {
#pragma unroll
          for (int e = 0; e < 2 * VEC; ++e) ss += x[e] * x[e];
        }
      }
      load_row(r + step);                 // in flight during this row's arithmetic
      const f32x2_t* const at = cs + t * pairs;
      // v <- R v
      auto turn = [&](float (&v)[2 * VEC]) {
        if constexpr (INTER) {
#pragma unroll
          for (int e = 0; e < 2 * VEC; e += 2) {
            const bool on = e < VEC ? rot0 : rot1;
            const f32x2_t cv = on ? at[((e < VEC ? c0 + e : c1 + e - VEC)) / 2] : f32x2_t{1.f, 0.f};
            const float va = v[e], vb = v[e + 1];
            v[e] = va * cv[0] - vb * cv[1];
            v[e + 1] = vb * cv[0] + va * cv[1];
          }
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const f32x2_t cv = rot0 ? at[c0 + e] : f32x2_t{1.f, 0.f};
            const float va = v[e], vb = v[VEC + e];
            v[e] = va * cv[0] - vb * cv[1];
            v[VEC + e] = vb * cv[0] + va * cv[1];
          }
        }
      };
      auto weight = [&](int e) { return wts[e < VEC ? c0 + e : c1 + e - VEC]; };
      auto row_sum = [&](float v) {
#pragma unroll
        for (int off = LPR / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
        return v;
      };
      if constexpr (MODE == 0) {
        if (live) turn(x);
      } else {
        const float rs = __frsqrt_rn(row_sum(ss) * inv_d + p.eps);
        if constexpr (MODE == 1) {
          if (live) {
#pragma unroll
            for (int e = 0; e < 2 * VEC; ++e) x[e] = x[e] * rs * weight(e);
            turn(x);
          }
        } else {
          float dot = 0.f;
          if (live) {
            turn(g);
#pragma unroll
            for (int e = 0; e < 2 * VEC; ++e) {
              x[e] *= rs;
              acc[e] += g[e] * x[e];
              g[e] *= weight(e);
              dot += g[e] * x[e];
            }
          }
          dot = row_sum(dot) * inv_d;
          if (live) {
#pragma unroll
            for (int e = 0; e < 2 * VEC; ++e) x[e] = rs * (g[e] - x[e] * dot);
          }
        }
      }
      if (live) {
        T* const yr = row_ptr<T>(py, p, tok0 + t, r - t * H);
        store_chunk<T, VEC>(yr + c0, x);
        store_chunk<T, VEC>(yr + c1, x + VEC);
      }
    }
    // the next token's cos and sin go where this one's were read from
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_wave_barrier();
  }
  if constexpr (MODE == 2) {
    // Weight gradients: the row groups of a wave, then the waves, in order.
#pragma unroll
    for (int e = 0; e < 2 * VEC; ++e) {
      float v = acc[e];
#pragma unroll
      for (int off = 32; off >= LPR; off >>= 1) v += __shfl_xor(v, off, 64);
      if (grp == 0 && live) red[wave][(e < VEC ? c0 + e : c1 + e - VEC)] = v;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < p.dim; d += NT)
      p.partial[(int64_t)blockIdx.x * p.dim + d] = ((red[0][d] + red[1][d]) + red[2][d]) + red[3][d];
  }
}

// Any head size, stride and alignment: a workgroup of one wave takes a token,
// its lanes the values of one head row at a time, both members of a value's
// pair read from global memory.  In place is safe: a row is read whole into
// LDS before any of it is written.
constexpr int kMaxDim = 1024;
template <typename T, int MODE, bool INTER>
__global__ __launch_bounds__(64) void qk_plain_kernel(const QkParams p) {
  constexpr bool BF = sizeof(T) == 2;
  __shared__ f32x2_t cs[kMaxPairs];
  __shared__ float xs[kMaxDim], gs[kMaxDim], dws[MODE == 2 ? kMaxDim : 1];
  const int lane = threadIdx.x, pairs = p.rot / 2;
  const int q = (int)blockIdx.x >= p.blocks[0];
  const int block = (int)blockIdx.x - (q ? p.blocks[0] : 0);
  if constexpr (MODE == 2) {
    for (int d = lane; d < p.dim; d += 64) dws[d] = 0.f;
  }
  // partner of value d, its pair and the sign of the sine term
  auto turned = [&](const float* v, int d) {
    if (d >= p.rot) return v[d];
    int pair, other;
    bool first;
    if (INTER) { pair = d >> 1; first = !(d & 1); other = d ^ 1; }
    else { first = d < pairs; pair = first ? d : d - pairs; other = first ? d + pairs : d - pairs; }
    const f32x2_t a = cs[pair];
    return v[d] * a[0] + (first ? -v[other] : v[other]) * a[1];
  };
  for (int64_t tok = block; tok < p.tokens; tok += p.blocks[q]) {
    __syncthreads();
    for (int i = lane; i < pairs; i += 64) cs[i] = cos_sin(p, tok, i);
      for (int head = 0; head < p.heads[q]; ++head) {
        const T* const xr = row_ptr<const T>(p.x[q], p, tok, head);
        T* const yr = row_ptr<T>(p.y[q], p, tok, head);
        auto wt = [&](int d) { return p.w[q] ? load_elem(p.w[q], d, p.w_dtype == MUON_BF16) : 1.f; };
        __syncthreads();
        float ss = 0.f;
        for (int d = lane; d < p.dim; d += 64) {
          const float v = load_elem(xr, d, BF);
          xs[d] = v;
          ss += v * v;
          if (MODE == 2) gs[d] = load_elem(row_ptr<const T>(p.g[q], p, tok, head), d, BF);
        }
        const float rs = MODE == 0 ? 1.f : __frsqrt_rn(wave_sum(ss) / (float)p.dim + p.eps);
        if (MODE == 1)
          for (int d = lane; d < p.dim; d += 64) xs[d] = xs[d] * rs * wt(d);
        __syncthreads();
        if (MODE != 2) {
          for (int d = lane; d < p.dim; d += 64) store_elem(yr, d, turned(xs, d), BF);
        } else {
          float dot = 0.f;
          for (int d = lane; d < p.dim; d += 64) {
            const float g = turned(gs, d), n = xs[d] * rs;
            dws[d] += g * n;
            dot += g * wt(d) * n;
          }
          dot = wave_sum(dot) / (float)p.dim;
          for (int d = lane; d < p.dim; d += 64)
            store_elem(yr, d, rs * (turned(gs, d) * wt(d) - xs[d] * rs * dot), BF);
        }
      }
  }
  if constexpr (MODE == 2) {
    __syncthreads();
    for (int d = lane; d < p.dim; d += 64) p.partial[(int64_t)blockIdx.x * p.dim + d] = dws[d];
  }
}

template <typename T, int MODE, bool INTER, int VEC>
hipError_t launch_vec(const QkParams& p, hipStream_t s) {
  const int nch = p.dim / (2 * VEC);
  const dim3 g((unsigned)(p.blocks[0] + p.blocks[1]));
  if (nch <= 4) return launch_kernel(qk_kernel<T, MODE, INTER, VEC, 4>, g, p, s, NT);
  if (nch <= 8) return launch_kernel(qk_kernel<T, MODE, INTER, VEC, 8>, g, p, s, NT);
  if (nch <= 16) return launch_kernel(qk_kernel<T, MODE, INTER, VEC, 16>, g, p, s, NT);
  if (nch <= 32) return launch_kernel(qk_kernel<T, MODE, INTER, VEC, 32>, g, p, s, NT);
  if (nch <= 64) return launch_kernel(qk_kernel<T, MODE, INTER, VEC, 64>, g, p, s, NT);
  return hipErrorInvalidValue;
}

template <typename T, int MODE, bool INTER>
hipError_t launch_mode(const QkParams& p, int vec, hipStream_t s) {
  if (vec > 1 && (p.dim % (2 * vec) || p.rot % (2 * vec) || std::max(p.tw[0], p.tw[1]) * (p.rot / 2) > kCsPairs)) return hipErrorInvalidValue;
  switch (vec) {
    case 8:  // 16 bytes of bf16; fp32 takes 4 values, twice the bytes per lane would spill
      if constexpr (sizeof(T) == 2) return launch_vec<T, MODE, INTER, 8>(p, s);
      else return hipErrorInvalidValue;
    case 4: return launch_vec<T, MODE, INTER, 4>(p, s);
    case 2: return launch_vec<T, MODE, INTER, 2>(p, s);
    default: return p.dim <= kMaxDim ? launch_kernel(qk_plain_kernel<T, MODE, INTER>, dim3((unsigned)(p.blocks[0] + p.blocks[1])), p, s, 64)
                                     : hipErrorInvalidValue;
  }
}

template <typename T>
hipError_t launch_type(const QkParams& p, int mode, bool inter, int vec, hipStream_t s) {
  if (mode == 0) return inter ? launch_mode<T, 0, true>(p, vec, s) : launch_mode<T, 0, false>(p, vec, s);
  if (mode == 1) return inter ? launch_mode<T, 1, true>(p, vec, s) : launch_mode<T, 1, false>(p, vec, s);
  return inter ? launch_mode<T, 2, true>(p, vec, s) : launch_mode<T, 2, false>(p, vec, s);
}

struct WeightSum {
  const float* partial; int32_t blocks[2], dim;
  void* out[2]; int32_t out_dtype;
};

// dw[q][d] = the sum of tensor q's workgroups' partials: 64 threads per value
// each add every 64th, then the 64 sums are added pairwise.  1024 workgroups of
// 128 values: 4.8 us (16 threads per value, one load at a time: 20.6 us).
__global__ __launch_bounds__(1024) void qk_weight_sum_kernel(const WeightSum p) {
  __shared__ float red[64][17];
  const int v = threadIdx.x & 15, part = threadIdx.x >> 4, q = blockIdx.y;
  const int d = blockIdx.x * 16 + v;
  const float* const src = p.partial + (q ? (int64_t)p.blocks[0] * p.dim : 0);
  float t = 0.f;
  if (d < p.dim) {
#pragma unroll 8
    for (int b = part; b < p.blocks[q]; b += 64) t += src[(int64_t)b * p.dim + d];
  }
  red[part][v] = t;
#pragma unroll
  for (int half = 32; half >= 1; half >>= 1) {
    __syncthreads();
    if (part < half) red[part][v] += red[part + half][v];
  }
  if (part == 0 && d < p.dim && p.out[q]) store_elem(p.out[q], d, red[0][v], p.out_dtype == MUON_BF16);
}

}  // namespace

hipError_t launch_qk(const QkParams& p, int mode, bool bf16, bool interleaved, int vec, hipStream_t s) {
  if (p.blocks[0] + p.blocks[1] <= 0) return hipErrorInvalidValue;
  return bf16 ? launch_type<uint16_t>(p, mode, interleaved, vec, s) : launch_type<float>(p, mode, interleaved, vec, s);
}

hipError_t launch_qk_weight_sum(const QkParams& p, void* const out[2], int32_t out_dtype, hipStream_t s) {
  const WeightSum w{p.partial, {p.blocks[0], p.blocks[1]}, p.dim, {out[0], out[1]}, out_dtype};
  return launch_kernel(qk_weight_sum_kernel, dim3((unsigned)((p.dim + 15) / 16), 2), w, s, 1024);
}

}  // namespace muon
