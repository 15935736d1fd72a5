// The linear product for few rows (decoding: 1 to 64 tokens).
//
// Bound by HBM: the weight is read once, 2 bytes per 2 M operations.  A
// workgroup owns 16 NB weight rows and all tokens; its eight waves take the
// 128-byte steps of K in turn (so together they read a kilobyte of each row at
// a time) and stream them straight into registers, 32 bytes per lane of every
// row, as one operand of 16x16 MFMAs whose other operand is the tokens (16 MB,
// from the caches).  The order of K within a step differs between the lanes'
// layout and memory, but in the same way for both operands, so every product
// is formed once.  The waves' sums are added in order through LDS and finished
// there.
//
// Every workgroup reads all tokens, M / (16 NB) of what it reads of the
// weight, so NB is 4 where that leaves the chip full; a weight with fewer rows
// has its K split over workgroups (launch_split_finish adds them).  us by NB and
// split, against the weight's bytes at 5.1 TB/s (a call of one launch takes 8
// at least, of two 11):
//   bf16, rows x K  tokens   bytes   1/1   1/2   1/4   1/8   4/1   4/2   4/4   4/8
//   14336 x 4096        48    23.2     -     -     -     -  31.9  38.5     -     -
//   6144 x 4096          1     9.8  12.5  15.3  15.2  17.7  18.4  15.0  15.0  16.4
//   6144 x 4096         10     9.8  15.6  16.1  16.8  19.2  19.9  15.8  15.9  17.4
//   6144 x 4096         16     9.8  18.3  17.7  18.3  20.5  20.9  16.1  16.5  18.1
//   6144 x 4096         38     9.8  28.4  26.4  26.8  30.3  28.5  20.6  23.0  23.6
//   4096 x 8192         16    13.1  20.1  24.2  22.8  25.7  38.8  25.2  20.9  19.5
//   4096 x 8192         24    13.1  22.4  27.3  26.3  29.1  43.9  27.6  21.8  20.0
//   1024 x 8192          1     3.3  11.3  11.1  11.1  11.1  32.1  20.2  12.8  11.0
//   1024 x 8192         16     3.3  16.6  12.9  11.1  11.3  37.4  23.4  14.7  11.2
//   1024 x 16384         1     6.5  20.0  14.1  12.2  12.4  61.2  34.8  20.2  13.3
//   512 x 14336         64     2.9  63.7  36.7  21.5  14.6  99.5  55.0  31.1  19.7
//   5921 x 10391*       38    23.9   169   133   133   134   160    87    89    76
//   fp32, rows x K
//   576 x 3456           4     1.5  11.2  12.3  12.4  12.1  32.9  21.7  13.9  12.3
//   576 x 3456          16     1.5  14.6  12.4  12.3  12.3  35.3  23.0  14.5  12.3
//   384 x 13973*        62     4.2   123  66.9  37.6  23.1   329   173  92.8  52.5
//   9472 x 2504         40    18.5  61.1  56.1  56.5  56.4  58.9  63.5  54.6  56.0
// (* rows that are not 16-byte aligned: every load takes two lines.)
// More steps in flight per wave (two or four loaded together) gained nothing.
#include "layer_internal.h"
#include "linear_epilogue.h"

namespace muon {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
// Weight and token rows may start anywhere: unaligned 16-byte loads.
template <typename T>
struct Loads;
template <>
struct Loads<uint16_t> { typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(2))); };
template <>
struct Loads<float> { typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(4))); };

constexpr int NWV = 8;

template <typename T, int MB, int NB>
__global__ __launch_bounds__(NWV * 64, 2) void linear_small_kernel(const LinGemm p) {
  constexpr bool BF = sizeof(T) == 2;
  constexpr int E = 32 / sizeof(T);        // values of K per lane and step
  constexpr int KS = 4 * E;                // values of K per step
  constexpr int NR = 16 * NB, PITCH = NR + 4;
  typedef typename Loads<T>::v4 v4u;
  __shared__ __attribute__((aligned(16))) float red[NWV][16 * MB * PITCH];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * NR;
  const T* wrow[NB];
  const T* xrow[MB];
  bool tok[MB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int64_t n = n0 + 16 * b + r;
    wrow[b] = (const T*)p.B + (n < p.N ? n : p.N - 1) * p.ldb + g * E;
  }
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    tok[b] = 16 * b + r < p.M;
    xrow[b] = (const T*)p.A + (tok[b] ? 16 * b + r : 0) * p.lda + g * E;
  }
  f32x4 acc[MB][NB];
#pragma unroll
  for (int a = 0; a < MB; ++a)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto products = [&](const u32x4 (&w)[NB][2], const u32x4 (&x)[MB][2]) {
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if constexpr (BF) {
            acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[b][q]),
                                                                __builtin_bit_cast(bf16x8, x[a][q]), acc[a][b], 0, 0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[b][q][e]), __uint_as_float(x[a][q][e]),
                                                               acc[a][b], 0, 0, 0);
          }
        }
  };
  const int64_t all = (p.K + KS - 1) / KS;
  const int64_t first = p.split > 1 ? (int64_t)blockIdx.y * all / p.split : 0;
  const int64_t steps = p.split > 1 ? (int64_t)(blockIdx.y + 1) * all / p.split : all;  // this workgroup's, up to here
  const int64_t full = p.K / KS < steps ? p.K / KS : steps;
  int64_t s = first + wave;
  for (; s < full; s += NWV) {
    u32x4 w[NB][2], x[MB][2];
    const int64_t k = s * KS;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      w[b][0] = *(const v4u*)(wrow[b] + k);
      w[b][1] = *(const v4u*)(wrow[b] + k + E / 2);
    }
#pragma unroll
    for (int a = 0; a < MB; ++a) {
      x[a][0] = x[a][1] = u32x4{0, 0, 0, 0};
      if (tok[a]) {
        x[a][0] = *(const v4u*)(xrow[a] + k);
        x[a][1] = *(const v4u*)(xrow[a] + k + E / 2);
      }
    }
    products(w, x);
  }
  for (; s < steps; s += NWV) {  // the rest, values of K past the end as zeros
    u32x4 w[NB][2], x[MB][2];
    const int64_t k = s * KS;
    auto part = [&](const T* row, int q, bool on) -> u32x4 {
      const T* at = row + k + q * (E / 2);
      const int64_t left = p.K - (k + g * E + q * (E / 2));
      if (on && left >= E / 2) return *(const v4u*)at;
      T v[E / 2];
#pragma unroll
      for (int e = 0; e < E / 2; ++e) v[e] = on && e < left ? at[e] : T(0);
      u32x4 o;
      __builtin_memcpy(&o, v, 16);
      return o;
    };
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int b = 0; b < NB; ++b) w[b][q] = part(wrow[b], q, true);
#pragma unroll
      for (int a = 0; a < MB; ++a) x[a][q] = part(xrow[a], q, tok[a]);
    }
    products(w, x);
  }
  // D of a 16 x 16 block: lane l holds token l % 16, weight rows 4 (l / 16) .. + 3.
#pragma unroll
  for (int a = 0; a < MB; ++a)
#pragma unroll
    for (int b = 0; b < NB; ++b) *(f32x4*)(&red[wave][(16 * a + r) * PITCH + 16 * b + 4 * g]) = acc[a][b];
  __syncthreads();
  with_act(p.act, [&](auto act_c) {
    constexpr int ACT = decltype(act_c)::value;
    for (int at = threadIdx.x; at < (int)p.M * (NR / 8); at += NWV * 64) {
      const int i = at / (NR / 8), c8 = (at % (NR / 8)) * 8;
      const int64_t j = n0 + c8;
      const int valid = j >= p.N ? 0 : (p.N - j < 8 ? (int)(p.N - j) : 8);
      if (valid <= 0) continue;
      float v[8], b[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = red[0][i * PITCH + c8 + e];
#pragma unroll
      for (int w = 1; w < NWV; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += red[w][i * PITCH + c8 + e];
      if (p.part) {
        float* const d = p.part + ((int64_t)blockIdx.y * p.M + i) * p.ldpart + j;
        *(f32x4*)d = f32x4{v[0], v[1], v[2], v[3]};
        *(f32x4*)(d + 4) = f32x4{v[4], v[5], v[6], v[7]};
        continue;
      }
      bias8(p, j, valid, b);
      finish8<ACT, BF>(p, i, j, valid, b, v);
    }
  });
}

template <typename T, int MB, int NB>
hipError_t launch_one(const LinGemm& g, hipStream_t s) {
  const int64_t grid = (g.N + 16 * NB - 1) / (16 * NB);
  if (grid > INT32_MAX || g.split < 1 || g.split > 65535 || (g.split > 1 && !g.part)) return hipErrorInvalidValue;
  return launch_kernel(linear_small_kernel<T, MB, NB>, dim3((unsigned)grid, (unsigned)g.split), g, s, NWV * 64);
}

template <typename T>
hipError_t launch_type(const LinGemm& g, int nb, hipStream_t s) {
  if (g.M <= 0 || g.N <= 0) return hipSuccess;
  if (nb != 1 && nb != 4) return hipErrorInvalidValue;
  switch ((g.M + 15) / 16) {
    case 1: return nb == 4 ? launch_one<T, 1, 4>(g, s) : launch_one<T, 1, 1>(g, s);
    case 2: return nb == 4 ? launch_one<T, 2, 4>(g, s) : launch_one<T, 2, 1>(g, s);
    case 3: return nb == 4 ? launch_one<T, 3, 4>(g, s) : launch_one<T, 3, 1>(g, s);
    case 4: return nb == 4 ? launch_one<T, 4, 4>(g, s) : launch_one<T, 4, 1>(g, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_linear_small(const LinGemm& g, bool bf16, int nb, hipStream_t s) {
  return bf16 ? launch_type<uint16_t>(g, nb, s) : launch_type<float>(g, nb, s);
}

}  // namespace muon
