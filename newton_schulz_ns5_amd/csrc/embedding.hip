// Embedding lookup with scaling, and its gradient by sorted tokens.
//   y[t] = scale W[row(t)],  row(t) = id[t] - first, zeros where there is no such row
//   dW[v] (+)= scale sum over the tokens t of row v of dy[t]
//
// Lookup: bound by HBM, every row read once per token (L2 and the infinity
// cache serve frequent ones) and written once.
//
// Gradient: bound by HBM too, dy read once and dW written once, rows without a
// token as zeros.  The token numbers are sorted by row, stable, so that a row's
// tokens are neighbours in token order; then pieces of the sorted list are
// summed by workgroups that are alike however often a token occurs.  A run of
// one row inside a piece is written at once; what reaches over a piece's end
// goes into slots that a second launch joins in order.  No value is added by
// an atomic, so the bits depend on the call alone.
#include "pass_internal.h"
#include "row8.h"

namespace muon {
namespace {

constexpr int NT = 256;

__device__ __forceinline__ int64_t row_of_token(const EmbedIds& p, int64_t t, bool gradient) {
  const int64_t id = p.i64 ? ((const int64_t*)p.ids)[t] : (int64_t)((const int32_t*)p.ids)[t];
  // as unsigned, so that no difference of two ids overflows
  const uint64_t row = (uint64_t)id - (uint64_t)p.first;
  const bool inside = id >= p.first && row < (uint64_t)p.rows && !(gradient && p.has_padding && id == p.padding);
  return inside ? (int64_t)row : -1;
}

// G threads hold a row; U tokens in flight.
template <typename T, typename O, int G, bool EDGE>
__global__ __launch_bounds__(NT) void embed_kernel(const Embed p) {
  constexpr int U = 4;
  const int j = threadIdx.x % G, grp = threadIdx.x / G;
  const int col = 8 * (int)(blockIdx.y * G + j);
  const int valid = p.dim - col < 0 ? 0 : (p.dim - col < 8 ? p.dim - col : 8);
  if (valid <= 0) return;
  const int64_t step = (int64_t)gridDim.x * (NT / G);
  for (int64_t t0 = (int64_t)blockIdx.x * (NT / G) + grp; t0 < p.tokens; t0 += U * step) {
    int64_t row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) row[u] = t0 + u * step < p.tokens ? row_of_token(p.ids, t0 + u * step, false) : -1;
    Raw8<T, EDGE> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (row[u] >= 0) x[u].load((const T*)p.w + row[u] * p.ldw, col, valid);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t0 + u * step >= p.tokens) continue;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = row[u] >= 0 ? x[u].value(e) * p.scale : 0.f;
      round_store<O, EDGE>((O*)p.y + (t0 + u * step) * p.ldy, col, valid, v);
    }
  }
}

// ---- the sort ------------------------------------------------------------------------
__device__ __forceinline__ uint32_t sort_key(const EmbedSort& p, int64_t i) {
  if (!p.first_pass) return p.key_in[i];
  const int64_t row = row_of_token(p.ids, i, true);
  return row < 0 ? (uint32_t)p.ids.rows : (uint32_t)row;
}
__device__ __forceinline__ int digit_of(const EmbedSort& p, uint32_t key) { return (int)((key >> p.shift) & ((1u << p.bits) - 1)); }

__global__ __launch_bounds__(NT) void sort_hist_kernel(const EmbedSort p) {
  __shared__ uint32_t bins[kSortBins];
  for (int d = threadIdx.x; d < kSortBins; d += NT) bins[d] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * NT * p.rounds;
  for (int r = 0; r < p.rounds; ++r) {
    const int64_t i = base + (int64_t)r * NT + threadIdx.x;
    if (i < p.n) atomicAdd(&bins[digit_of(p, sort_key(p, i))], 1u);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < kSortBins; d += NT) p.hist[(int64_t)blockIdx.x * kSortBins + d] = bins[d];
}

// Exclusive sum of v over the workgroup, and its total.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* red, uint32_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t s = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = __shfl_up(s, off, 64);
    if (lane >= off) s += o;
  }
  __syncthreads();
  if (lane == 63) red[wave] = s;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    if (w < wave) before += red[w];
    total += red[w];
  }
  return before + s - v;
}

// One digit's counts, replaced by their sums over the tiles before.
__global__ __launch_bounds__(NT) void sort_scan_kernel(const EmbedSort p, int tiles) {
  __shared__ uint32_t red[NT / 64];
  const int d = blockIdx.x;
  uint32_t carry = 0;
  for (int t0 = 0; t0 < tiles; t0 += NT) {
    const int t = t0 + threadIdx.x;
    const uint32_t v = t < tiles ? p.hist[(int64_t)t * kSortBins + d] : 0;
    uint32_t total;
    const uint32_t s = block_scan(v, red, total);
    if (t < tiles) p.hist[(int64_t)t * kSortBins + d] = carry + s;
    carry += total;
  }
  if (threadIdx.x == 0) p.totals[d] = carry;
}

__global__ __launch_bounds__(NT) void sort_scatter_kernel(const EmbedSort p, int tiles) {
  constexpr int W = NT / 64;
  __shared__ uint32_t red[W];
  __shared__ uint32_t place[W][kSortBins];  // a wave's next place for every digit
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // Where this tile's tokens of the thread's two digits begin.
  static_assert(kSortBins == 2 * NT, "two digits per thread");
  uint32_t before[2] = {0, 0}, total[2] = {0, 0};
  const int d0 = 2 * threadIdx.x;
  if (p.scanned) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      before[e] = p.hist[(int64_t)blockIdx.x * kSortBins + d0 + e];
      total[e] = p.totals[d0 + e];
    }
  } else {
#pragma unroll 8
    for (int t = 0; t < tiles; ++t) {
      const u32x2 h = *(const u32x2*)(p.hist + (int64_t)t * kSortBins + d0);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        total[e] += h[e];
        if (t < (int)blockIdx.x) before[e] += h[e];
      }
    }
  }
  uint32_t all;
  const uint32_t lower = block_scan(total[0] + total[1], red, all);
  for (int d = threadIdx.x; d < W * kSortBins; d += NT) (&place[0][0])[d] = 0;
  __syncthreads();
  // The waves take consecutive quarters of the tile.
  const int64_t base = (int64_t)blockIdx.x * NT * p.rounds + (int64_t)wave * 64 * p.rounds;
  for (int r = 0; r < p.rounds; ++r) {
    const int64_t i = base + (int64_t)r * 64 + lane;
    if (i < p.n) atomicAdd(&place[wave][digit_of(p, sort_key(p, i))], 1u);
  }
  __syncthreads();
  {
    uint32_t at[2] = {lower + before[0], lower + total[0] + before[1]};
#pragma unroll
    for (int w = 0; w < W; ++w) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t c = place[w][d0 + e];
        place[w][d0 + e] = at[e];
        at[e] += c;
      }
    }
  }
  __syncthreads();
  for (int r = 0; r < p.rounds; ++r) {
    const int64_t i = base + (int64_t)r * 64 + lane;
    const bool here = i < p.n;
    const uint32_t key = here ? sort_key(p, i) : 0;
    const int d = digit_of(p, key);
    // the lanes with the same digit
    uint64_t peers = __ballot(here);
    for (int b = 0; b < p.bits; ++b) {
      const uint64_t m = __ballot((d >> b) & 1);
      peers &= (d >> b) & 1 ? m : ~m;
    }
    const int rank = __popcll(peers & (((uint64_t)1 << lane) - 1));
    uint32_t at = 0;
    if (here) at = place[wave][d];
    __builtin_amdgcn_s_waitcnt(0xC07F);  // every lane has read its place before it moves
    __builtin_amdgcn_wave_barrier();
    if (here && rank == 0) place[wave][d] = at + (uint32_t)__popcll(peers);
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_wave_barrier();
    if (here) {
      p.key_out[at + rank] = key;
      p.tok_out[at + rank] = p.first_pass ? (uint32_t)i : p.tok_in[i];
    }
  }
}

// ---- the sums ------------------------------------------------------------------------
// The first position in the sorted list whose key is not below `key`.
__device__ __forceinline__ int64_t lower_bound(const uint32_t* key, int64_t n, uint32_t k) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (key[mid] < k) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

template <typename O, bool EDGE>
__device__ __forceinline__ void write_row(const EmbedGrad& p, uint32_t row, int col, int valid, const float (&a)[8]) {
  O* const at = (O*)p.dw + (int64_t)row * p.lddw;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = a[e] * p.scale;
  if (p.accumulate) {
    Raw8<O, EDGE> old;
    old.load(at, col, valid);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += old.value(e);
  }
  round_store<O, EDGE>(at, col, valid, v);
}

constexpr int kClearRows = 64;

template <typename T, typename O, int G, bool EDGE>
__global__ __launch_bounds__(NT) void embed_grad_kernel(const EmbedGrad p) {
  __shared__ uint8_t touched[kClearRows];
  const int j = threadIdx.x % G, grp = threadIdx.x / G;
  if ((int)blockIdx.x >= p.sum_blocks) {
    // Clears the rows that no token has, kClearRows of them.
    const int64_t r0 = (int64_t)(blockIdx.x - p.sum_blocks) * kClearRows;
    if (threadIdx.x < kClearRows) {
      const int64_t r = r0 + threadIdx.x;
      bool has = true;
      if (r < p.rows) {
        const int64_t at = lower_bound(p.key, p.n, (uint32_t)r);
        has = at < p.n && p.key[at] == (uint32_t)r;
      }
      touched[threadIdx.x] = has;
    }
    __syncthreads();
    const float zero[8] = {};
    for (int i = grp; i < kClearRows; i += NT / G) {
      if (touched[i]) continue;
      O* const at = (O*)p.dw + (r0 + i) * p.lddw;
      for (int col = 8 * j; col < p.dim; col += 8 * G) round_store<O, EDGE>(at, col, p.dim - col < 8 ? p.dim - col : 8, zero);
    }
    return;
  }
  constexpr int U = 8;
  const int64_t piece = (int64_t)(blockIdx.x / p.col_blocks) * (NT / G) + grp;
  const int col = 8 * (int)(blockIdx.x % p.col_blocks * G + j);
  const int valid = p.dim - col < 0 ? 0 : (p.dim - col < 8 ? p.dim - col : 8);
  const int64_t i0 = piece * p.piece, i1 = i0 + p.piece < p.n ? i0 + p.piece : p.n;
  const uint32_t none = (uint32_t)p.rows;
  if (valid <= 0 || i0 >= p.n || p.key[i0] == none) return;
  float acc[8] = {};
  uint32_t run = p.key[i0];
  bool open = i0 > 0 && p.key[i0 - 1] == run;  // the run began in a piece before
  for (int64_t i = i0; i < i1; i += U) {
    uint32_t key[U];
    Raw8<T, EDGE> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      key[u] = i + u < i1 ? p.key[i + u] : none;
      if (key[u] != none) x[u].load((const T*)p.dy + (int64_t)p.tok[i + u] * p.lddy, col, valid);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (key[u] != run) {
        if (run != none && i + u > i0 && i + u <= i1) {
          if (open) round_store<float, EDGE>(p.slots + (2 * piece) * p.dim, col, valid, acc);
          else if (i + u < i1 || i1 == p.n || p.key[i1] != run) write_row<O, EDGE>(p, run, col, valid, acc);
          else round_store<float, EDGE>(p.slots + (2 * piece + 1) * p.dim, col, valid, acc);
        }
        open = false;
        run = key[u];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      }
      if (key[u] != none) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += x[u].value(e);
      }
    }
  }
  if (run == none) return;
  // the piece's last run, where the piece ends with the loop's last step
  if (open) round_store<float, EDGE>(p.slots + (2 * piece) * p.dim, col, valid, acc);
  else if (i1 == p.n || p.key[i1] != run) write_row<O, EDGE>(p, run, col, valid, acc);
  else round_store<float, EDGE>(p.slots + (2 * piece + 1) * p.dim, col, valid, acc);
}

// Joins the runs that reach over pieces.  A workgroup looks at one piece and
// 512 columns: where a run begins in the piece and goes on, it adds the slots
// of the pieces it reaches, four parts of them at once, then the parts.
constexpr int kJoinParts = 4;
template <typename O, bool EDGE>
__global__ __launch_bounds__(NT) void embed_join_kernel(const EmbedGrad p) {
  __shared__ float red[kJoinParts][64][9];
  const int64_t piece = blockIdx.x;
  const int64_t i0 = piece * p.piece, i1 = i0 + p.piece;
  if (i1 >= p.n) return;
  const uint32_t run = p.key[i1 - 1];
  if (run == (uint32_t)p.rows || p.key[i1] != run || (p.key[i0] == run && i0 > 0 && p.key[i0 - 1] == run)) return;
  const int64_t last = (lower_bound(p.key, p.n, run + 1) - 1) / p.piece;
  const int j = threadIdx.x & 63, part = threadIdx.x >> 6;
  const int col = 8 * (int)(blockIdx.y * 64 + j);
  const int valid = p.dim - col < 0 ? 0 : (p.dim - col < 8 ? p.dim - col : 8);
  float acc[8] = {};
  if (valid > 0) {
    auto add = [&](int64_t slot) {
      Raw8<float, EDGE> x;
      x.load(p.slots + slot * p.dim, col, valid);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += x.value(e);
    };
    if (part == 0) add(2 * piece + 1);
#pragma unroll 4
    for (int64_t q = piece + 1 + part; q <= last; q += kJoinParts) add(2 * q);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) red[part][j][e] = acc[e];
  __syncthreads();
  if (part || valid <= 0) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int q = 1; q < kJoinParts; ++q) acc[e] += red[q][j][e];
  }
  write_row<O, EDGE>(p, run, col, valid, acc);
}

// f called with the group size and whether rows end in part of a chunk.
template <class F>
hipError_t with_group(int64_t dim, F&& f) {
  const bool edge = dim % 8 != 0;
  switch (embed_group(dim)) {
#define MUON_GROUP(G)                                                                                        \
  case G:                                                                                                    \
    return edge ? f(std::integral_constant<int, G>{}, std::integral_constant<bool, true>{})                  \
                : f(std::integral_constant<int, G>{}, std::integral_constant<bool, false>{})
    MUON_GROUP(8);
    MUON_GROUP(16);
    MUON_GROUP(32);
    MUON_GROUP(64);
    MUON_GROUP(128);
    MUON_GROUP(256);
#undef MUON_GROUP
  }
  return hipErrorInvalidValue;
}

template <typename T, typename O>
hipError_t launch_embed_types(const Embed& p, hipStream_t s) {
  return with_group(p.dim, [&](auto g, auto e) {
    constexpr int G = decltype(g)::value;
    const int64_t want = (p.tokens + NT / G - 1) / (NT / G);
    const unsigned y = (unsigned)((p.dim + 8 * G - 1) / (8 * G));
    const int64_t most = 8192 / y > 256 ? 8192 / y : 256;
    return launch_kernel(embed_kernel<T, O, G, decltype(e)::value>, dim3((unsigned)(want < most ? want : most), y), p, s, NT);
  });
}
template <typename T, typename O>
hipError_t launch_grad_types(const EmbedGrad& p, int blocks, hipStream_t s) {
  return with_group(p.dim, [&](auto g, auto e) {
    return launch_kernel(embed_grad_kernel<T, O, decltype(g)::value, decltype(e)::value>, dim3((unsigned)blocks), p, s, NT);
  });
}

hipError_t launch_sort(void (*kernel)(const EmbedSort, int), dim3 grid, const EmbedSort& p, int tiles, hipStream_t s) {
  void* args[] = {const_cast<EmbedSort*>(&p), &tiles};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(NT), args, 0, s);
}

}  // namespace

int embed_group(int64_t dim) {
  const int64_t chunks = (dim + 7) / 8;
  int g = 8;
  while (g < kEmbedCols / 8 && g < chunks) g *= 2;
  return g;
}

hipError_t launch_embed(const Embed& p, bool w_bf16, bool y_bf16, hipStream_t s) {
  if (w_bf16) return y_bf16 ? launch_embed_types<uint16_t, uint16_t>(p, s) : launch_embed_types<uint16_t, float>(p, s);
  return y_bf16 ? launch_embed_types<float, uint16_t>(p, s) : launch_embed_types<float, float>(p, s);
}

hipError_t launch_sort_hist(const EmbedSort& p, int tiles, hipStream_t s) { return launch_kernel(sort_hist_kernel, dim3((unsigned)tiles), p, s, NT); }
hipError_t launch_sort_scan(const EmbedSort& p, int tiles, hipStream_t s) { return launch_sort(sort_scan_kernel, dim3(kSortBins), p, tiles, s); }
hipError_t launch_sort_scatter(const EmbedSort& p, int tiles, hipStream_t s) {
  return launch_sort(sort_scatter_kernel, dim3((unsigned)tiles), p, tiles, s);
}

hipError_t launch_embed_grad(const EmbedGrad& p, bool dy_bf16, bool dw_bf16, int blocks, hipStream_t s) {
  if (dy_bf16) return dw_bf16 ? launch_grad_types<uint16_t, uint16_t>(p, blocks, s) : launch_grad_types<uint16_t, float>(p, blocks, s);
  return dw_bf16 ? launch_grad_types<float, uint16_t>(p, blocks, s) : launch_grad_types<float, float>(p, blocks, s);
}

hipError_t launch_embed_join(const EmbedGrad& p, bool dw_bf16, hipStream_t s) {
  const int64_t pieces = (p.n + p.piece - 1) / p.piece;
  const dim3 grid((unsigned)pieces, (unsigned)((p.dim + 511) / 512));
  if (p.dim % 8)
    return dw_bf16 ? launch_kernel(embed_join_kernel<uint16_t, true>, grid, p, s, NT) : launch_kernel(embed_join_kernel<float, true>, grid, p, s, NT);
  return dw_bf16 ? launch_kernel(embed_join_kernel<uint16_t, false>, grid, p, s, NT) : launch_kernel(embed_join_kernel<float, false>, grid, p, s, NT);
}

}  // namespace muon
