// The linear product's simple kernel: one 64 x 64 output tile per workgroup,
// operands staged element by element through registers into LDS, products on
// MFMA with fp32 sums, the epilogue on the accumulators.  Right for every
// size, stride and alignment.
#include "layer_internal.h"
#include "layer_math.h"

namespace muon {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int BT = 64, KS = 32;

template <typename T, int KIND>
__global__ __launch_bounds__(256) void linear_simple_kernel(const LinGemm p) {
  constexpr bool BF = sizeof(T) == 2;
  constexpr int PITCH = KS + 16 / sizeof(T);
  __shared__ __attribute__((aligned(16))) T As[BT * PITCH], Bs[BT * PITCH];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t tiles_n = (p.N + BT - 1) / BT;
  const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * BT, n0 = (int64_t)(blockIdx.x % tiles_n) * BT;
  auto stage = [&](T* dst, const void* src, int64_t ld, int64_t r0, int64_t R, int64_t k0, bool col) {
    const T* s = (const T*)src;
#pragma unroll
    for (int e = 0; e < BT * KS / 256; ++e) {
      const int i = tid + e * 256;
      const int r = col ? i % BT : i / KS, k = col ? i / BT : i % KS;
      const int64_t gr = r0 + r, gk = k0 + k;
      T v = 0;
      if (gr < R && gk < p.K) v = col ? s[gk * ld + gr] : s[gr * ld + gk];
      dst[r * PITCH + k] = v;
    }
  };
  f32x16 acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  const int r = lane & 31, h = lane >> 5;
  for (int64_t k0 = 0; k0 < p.K; k0 += KS) {
    stage(As, p.A, p.lda, m0, p.M, k0, KIND == kColCol);
    stage(Bs, p.B, p.ldb, n0, p.N, k0, KIND != kRowRow);
    __syncthreads();
    if constexpr (BF) {
#pragma unroll
      for (int ks = 0; ks < KS / 16; ++ks) {
        const bf16x8 a = *(const bf16x8*)(As + (wm + r) * PITCH + ks * 16 + h * 8);
        const bf16x8 b = *(const bf16x8*)(Bs + (wn + r) * PITCH + ks * 16 + h * 8);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int k = 0; k < KS; k += 2)
        acc = __builtin_amdgcn_mfma_f32_32x32x2f32(As[(wm + r) * PITCH + k + h], Bs[(wn + r) * PITCH + k + h], acc, 0, 0, 0);
    }
    __syncthreads();
  }
  const int64_t j = n0 + wn + r;
  if (j >= p.N) return;
  const float b = p.bias ? load_elem(p.bias, j, p.bias_dtype == MUON_BF16) : 0.f;
  with_act(p.act, [&](auto act_c) {
    constexpr int ACT = decltype(act_c)::value;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int64_t i = m0 + wm + 8 * (e >> 2) + 4 * h + (e & 3);
      if (i >= p.M) continue;
      const float z = acc[e] + b;
      if (p.Z) store_elem(p.Z, i * p.ldz + j, z, BF);
      float y = act_fwd<ACT>(z);
      if (p.add) y += load_elem(p.add, i * p.ldadd + j, p.add_dtype == MUON_BF16);
      store_elem(p.Y, i * p.ldy + j, y, p.y_dtype == MUON_BF16);
    }
  });
}

template <typename T>
hipError_t launch_kind(const LinGemm& g, LinKind kind, hipStream_t s) {
  const int64_t grid = ((g.M + BT - 1) / BT) * ((g.N + BT - 1) / BT);
  if (grid <= 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  const dim3 G((unsigned)grid);
  if (kind == kRowRow) return launch_kernel(linear_simple_kernel<T, kRowRow>, G, g, s);
  if (kind == kRowCol) return launch_kernel(linear_simple_kernel<T, kRowCol>, G, g, s);
  return launch_kernel(linear_simple_kernel<T, kColCol>, G, g, s);
}

}  // namespace

hipError_t launch_linear_simple(const LinGemm& g, bool bf16, LinKind kind, hipStream_t s) {
  return bf16 ? launch_kind<uint16_t>(g, kind, s) : launch_kind<float>(g, kind, s);
}

}  // namespace muon
