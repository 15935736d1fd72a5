// The norm over all gradients and their clipping:
//   N = sqrt(sum over tensors of sum g^2), or the largest |g|;
//   y = f g, f = 1 where max_norm >= N + eps, else max_norm / (N + eps).
//
// Bound by HBM: the norm reads every gradient once, clipping reads them again
// and writes them.  Squares are added in fp64, so that neither values whose
// squares leave fp32's range nor the length of the sum cost digits; the matrix
// units and fp32 would not be faster, since the loads bound it.  The order of
// the additions depends on the sizes alone: lanes, waves and workgroups take
// fixed items, and the partials are added in order.
//
// Items of kListItem elements, so that tensors of all sizes share one launch: a
// wave finds an item's tensor by bisection in the kernel's arguments and has
// eight 16-byte loads per lane in flight.  3.5 GB of bf16 in eight layers' tensors
// are normed in 508 us (6.9 TB/s, which reads alone reach); 436 MB are clipped
// in 216 us, 68 of the norm and 148 of the scaling (5.9 TB/s read and written).
#include "chunks.h"
#include "pass_internal.h"

namespace muon {
namespace {

constexpr int NT = 256;

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const uint32_t o = __shfl_xor(v, off, 64);
    v = o > v ? o : v;
  }
  return v;
}

// The tensor that holds an item, and the item's first element in it.
__device__ __forceinline__ int find_item(const TensorList& l, int item, int64_t& first) {
  int lo = 0, hi = l.n - 1;  // the first i with end[i] > item
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (l.end[mid] > item) hi = mid;
    else lo = mid + 1;
  }
  first = (int64_t)(item - (lo ? l.end[lo - 1] : 0)) * kListItem;
  return lo;
}
__device__ __forceinline__ bool bit(const uint64_t* words, int i) { return (words[i >> 6] >> (i & 63)) & 1; }

// What a lane adds up: squares, or the largest pattern of a magnitude (a NaN's
// is larger than infinity's, so a NaN stays).
template <bool MAX>
struct Acc {
  double sum[2] = {0.0, 0.0};
  uint32_t top = 0;
  __device__ __forceinline__ void add(float v, int e) {
    if constexpr (MAX) {
      const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
      top = b > top ? b : top;
    } else {
      const double d = (double)v;
      sum[e & 1] = fma(d, d, sum[e & 1]);
    }
  }
};

// Nontemporal: 1 GiB of bf16 in 168 us, 186 by plain loads; lists that the
// caches hold take the same time either way, the second read of clipping too
// (200 MiB: 100 us).
__device__ __forceinline__ u32x4 load_words(const void* p) { return __builtin_nontemporal_load((const u32x4_any*)p); }

template <bool MAX, bool BF>
__device__ __forceinline__ void add_item(const void* base, int64_t first, int64_t n, int lane, Acc<MAX>& acc) {
  constexpr int W = BF ? 8 : 4;                      // elements of a 16-byte load
  constexpr int U = kListItem / (64 * W) < 8 ? kListItem / (64 * W) : 8;  // loads in flight
  const char* const p = (const char*)base + first * (BF ? 2 : 4);
  auto use = [&](u32x4 a) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if constexpr (BF) {
        acc.add(__uint_as_float(a[w] << 16), 0);
        acc.add(__uint_as_float(a[w] & 0xffff0000u), 1);
      } else {
        acc.add(__uint_as_float(a[w]), w);
      }
    }
  };
  if (n >= kListItem) {
#pragma unroll
    for (int r = 0; r < kListItem / (64 * W * U); ++r) {
      u32x4 a[U];
#pragma unroll
      for (int u = 0; u < U; ++u) a[u] = load_words(p + ((r * U + u) * 64 + lane) * 16);
#pragma unroll
      for (int u = 0; u < U; ++u) use(a[u]);
    }
    return;
  }
  const int whole = (int)n / W;
  for (int v = lane; v < whole; v += 64) use(load_words(p + v * 16));
  for (int e = whole * W + lane; e < n; e += 64) acc.add(load_elem(p, e, BF), 0);
}

template <bool MAX>
__global__ __launch_bounds__(NT) void norm_partial_kernel(const NormPartial p) {
  __shared__ uint64_t red[NT / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Acc<MAX> acc;
  for (int item = __builtin_amdgcn_readfirstlane((int)blockIdx.x * (NT / 64) + wave); item < p.list.items; item += gridDim.x * (NT / 64)) {
    int64_t first;
    const int t = find_item(p.list, item, first);
    const int64_t left = p.list.numel[t] - first;
    if (bit(p.list.x_bf16, t)) add_item<MAX, true>(p.list.x[t], first, left, lane, acc);
    else add_item<MAX, false>(p.list.x[t], first, left, lane, acc);
  }
  uint64_t v;
  if constexpr (MAX) v = wave_max(acc.top);
  else v = __builtin_bit_cast(uint64_t, wave_sum64(acc.sum[0] + acc.sum[1]));
  if (lane == 0) red[wave] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    if constexpr (MAX) {
#pragma unroll
      for (int w = 1; w < NT / 64; ++w) v = red[w] > v ? red[w] : v;
    } else {
      double t = __builtin_bit_cast(double, v);
#pragma unroll
      for (int w = 1; w < NT / 64; ++w) t += __builtin_bit_cast(double, red[w]);
      v = __builtin_bit_cast(uint64_t, t);
    }
    p.partial[blockIdx.x] = v;
  }
}

// The norm, the same in every thread of the workgroup; the sum of squares
// through `square` (kind 2 only).
__device__ __forceinline__ double total_norm(const NormTotal& p, double& square) {
  __shared__ uint64_t red[NT / 64];
  square = 0.0;
  if (p.total) {
    if (!p.total_f64) return (double)*(const float*)p.total;
    square = *(const double*)p.total;
    return sqrt(square);
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (p.max_norm_kind) {
    uint32_t top = 0;
    for (int64_t i = threadIdx.x; i < p.count; i += NT) {
      const uint32_t b = (uint32_t)p.partial[i];
      top = b > top ? b : top;
    }
    top = wave_max(top);
    if (lane == 0) red[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) top = (uint32_t)red[w] > top ? (uint32_t)red[w] : top;
    return (double)__uint_as_float(top);
  }
  double t = 0.0;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < p.count; i += NT) t += __builtin_bit_cast(double, p.partial[i]);
  t = wave_sum64(t);
  if (lane == 0) red[wave] = __builtin_bit_cast(uint64_t, t);
  __syncthreads();
  t = 0.0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) t += __builtin_bit_cast(double, red[w]);
  square = t;
  return sqrt(t);
}

__global__ __launch_bounds__(NT) void norm_total_kernel(const NormTotal p) {
  double square;
  const double norm = total_norm(p, square);
  if (threadIdx.x == 0) {
    if (p.norm) *p.norm = (float)norm;
    if (p.square) *p.square = square;
    if (p.store) *p.store = p.max_norm_kind ? __float_as_uint((float)norm) : __builtin_bit_cast(uint64_t, square);
  }
}

// X, Y: uint16_t for bf16.  Nontemporal stores: nothing reads the gradients
// again before the caches have seen all of them.
template <typename X, typename Y>
__device__ __forceinline__ void scale_item(const void* x, void* y, int64_t first, int64_t n, int lane, float f) {
  constexpr int V = chunk_values<X, Y>(), U = 4;
  const X* const from = (const X*)x + first;
  Y* const to = (Y*)y + first;
  auto store = [&](auto chunk, int at, int valid) {
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = chunk.value(e) * f;
    round_store<Y, V, decltype(chunk)::kEdge, kStream>(to, at, valid, v);
  };
  if (n >= kListItem) {
#pragma unroll
    for (int r = 0; r < kListItem / (64 * V * U); ++r) {
      Chunk<X, V, false> c[U];
#pragma unroll
      for (int u = 0; u < U; ++u) c[u].load(from, ((r * U + u) * 64 + lane) * V, V);
#pragma unroll
      for (int u = 0; u < U; ++u) store(c[u], ((r * U + u) * 64 + lane) * V, V);
    }
    return;
  }
  for (int at = lane * V; at < n; at += 64 * V) {
    const int valid = n - at < V ? (int)(n - at) : V;
    Chunk<X, V, true> c;
    c.load(from, at, valid);
    store(c, at, valid);
  }
}

__global__ __launch_bounds__(NT) void clip_kernel(const ClipParams p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double square;
  const double norm = total_norm(p.total, square);
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.total.norm) *p.total.norm = (float)norm;
  // a NaN norm gives a NaN factor, an infinite one zero (and NaN from infinite gradients)
  const float f = p.max_norm >= norm + p.eps ? 1.f : (float)(p.max_norm / (norm + p.eps));
  if (f == 1.f && p.in_place) return;
  for (int item = __builtin_amdgcn_readfirstlane((int)blockIdx.x * (NT / 64) + wave); item < p.list.items; item += gridDim.x * (NT / 64)) {
    int64_t first;
    const int t = find_item(p.list, item, first);
    const int64_t left = p.list.numel[t] - first;
    const bool xb = bit(p.list.x_bf16, t), yb = bit(p.list.y_bf16, t);
    const void* const x = p.list.x[t];
    void* const y = p.list.y[t];
    if (xb && yb) scale_item<uint16_t, uint16_t>(x, y, first, left, lane, f);
    else if (xb) scale_item<uint16_t, float>(x, y, first, left, lane, f);
    else if (yb) scale_item<float, uint16_t>(x, y, first, left, lane, f);
    else scale_item<float, float>(x, y, first, left, lane, f);
  }
}

}  // namespace

hipError_t launch_norm_partial(const NormPartial& p, int blocks, hipStream_t s) {
  return launch_kernel(p.max_norm_kind ? norm_partial_kernel<true> : norm_partial_kernel<false>, dim3(blocks), p, s, NT);
}
hipError_t launch_norm_total(const NormTotal& p, hipStream_t s) { return launch_kernel(norm_total_kernel, dim3(1), p, s, NT); }
hipError_t launch_clip(const ClipParams& p, int blocks, hipStream_t s) { return launch_kernel(clip_kernel, dim3(blocks), p, s, NT); }

}  // namespace muon
