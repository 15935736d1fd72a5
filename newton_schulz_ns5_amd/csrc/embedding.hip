// Embedding lookup with scaling, and its gradient by sorted tokens.
//   y[t] = scale W[row(t)],  row(t) = id[t] - first, zeros where there is no such row
//   dW[v] (+)= scale sum over the tokens t of row v of dy[t]
//
// Lookup: bound by HBM, every row read once per token (L2 and the infinity
// cache serve frequent ones) and written once.  8192 tokens of 4096 from bf16 to
// fp32: 27.8 us for 201 MB, 7.2 TB/s, since caches hold some of the rows; one
// token 2.6 us.
//
// Gradient: bound by HBM too, dy read once and dW written once, rows without a
// token as zeros.  The token numbers are sorted by row, stable, so that a row's
// tokens are neighbours in token order; then pieces of the sorted list are
// summed by workgroups that are alike however often a token occurs.  A run of
// one row inside a piece is written at once; what reaches over a piece's end
// goes into slots that a second launch joins in order.  No value is added by
// an atomic, so the bits depend on the call alone.  8192 tokens of 4096 over
// 131072 rows in bf16: 218 us for 1141 MB (5.2 TB/s), 12 of the sort, 200 of the
// sums with the zeros between them, 6 of the join.  A row's slots are joined by
// one workgroup per 32 to 256 columns, so a row with most of the tokens costs more
// than many rare ones: 65536 tokens of 512 over 32000 rows take 55 us spread evenly,
// 68 with half of them one row's, 81 with all; 32768 of 4096 140, 152 and 169.
#include "chunks.h"
#include "pass_internal.h"

namespace muon {
namespace {

constexpr int NT = 256;
// Nontemporal: the lookup of 8192 tokens takes 28 us, by plain stores 42, and
// with a norm behind it as long as with those.
constexpr StorePolicy EMBED_STORE = kStream, CLEAR_STORE = kStream, SUM_STORE = kStream;

__device__ __forceinline__ int64_t row_of_token(const EmbedIds& p, int64_t t, bool gradient) {
  const int64_t id = p.i64 ? ((const int64_t*)p.ids)[t] : (int64_t)((const int32_t*)p.ids)[t];
  // as unsigned, so that no difference of two ids overflows
  const uint64_t row = (uint64_t)id - (uint64_t)p.first;
  const bool inside = id >= p.first && row < (uint64_t)p.rows && !(gradient && p.has_padding && id == p.padding);
  return inside ? (int64_t)row : -1;
}

// G threads hold V G columns of a row; U tokens in flight.
template <typename T, typename O, int G, bool EDGE>
__global__ __launch_bounds__(NT) void embed_kernel(const Embed p) {
  constexpr int U = 4, V = chunk_values<T, O>();
  const int j = threadIdx.x % G, grp = threadIdx.x / G;
  const int col = V * (int)(blockIdx.y * G + j);
  const int valid = p.dim - col < 0 ? 0 : (p.dim - col < V ? p.dim - col : V);
  if (valid <= 0) return;
  const int64_t step = (int64_t)gridDim.x * (NT / G);
  for (int64_t t0 = (int64_t)blockIdx.x * (NT / G) + grp; t0 < p.tokens; t0 += U * step) {
    int64_t row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) row[u] = t0 + u * step < p.tokens ? row_of_token(p.ids, t0 + u * step, false) : -1;
    Chunk<T, V, EDGE> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (row[u] >= 0) x[u].load((const T*)p.w + row[u] * p.ldw, col, valid);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t0 + u * step >= p.tokens) continue;
      float v[V];
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = row[u] >= 0 ? x[u].value(e) * p.scale : 0.f;
      round_store<O, V, EDGE, EMBED_STORE>((O*)p.y + (t0 + u * step) * p.ldy, col, valid, v);
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

static_assert(kSortThreads >= kSortBins, "a thread for every digit");

// The lanes of the wave that hold the same digit, among those that are here.
__device__ __forceinline__ uint64_t same_digit(const EmbedSort& p, int d, bool here) {
  uint64_t peers = __ballot(here);
  for (int b = 0; b < p.bits; ++b) {
    const uint64_t m = __ballot((d >> b) & 1);
    peers &= (d >> b) & 1 ? m : ~m;
  }
  return peers;
}
__device__ __forceinline__ int lanes_before(uint64_t peers) { return __popcll(peers & (((uint64_t)1 << (threadIdx.x & 63)) - 1)); }

// Counts of every digit: one addition per digit and wave, since many tokens
// share one.
__global__ __launch_bounds__(kSortThreads) void sort_hist_kernel(const EmbedSort p) {
  __shared__ uint32_t bins[kSortBins];
  const int64_t base = (int64_t)blockIdx.x * kSortThreads * kSortBatch + threadIdx.x;
  if (threadIdx.x < kSortBins) bins[threadIdx.x] = 0;
  __syncthreads();
  uint32_t key[kSortBatch];
#pragma unroll
  for (int u = 0; u < kSortBatch; ++u) {
    const int64_t i = base + (int64_t)u * kSortThreads;
    key[u] = i < p.n ? sort_key(p, i) : 0;
  }
#pragma unroll
  for (int u = 0; u < kSortBatch; ++u) {
    const bool here = base + (int64_t)u * kSortThreads < p.n;
    const int d = digit_of(p, key[u]);
    const uint64_t peers = same_digit(p, d, here);
    if (here && lanes_before(peers) == 0) atomicAdd(&bins[d], (uint32_t)__popcll(peers));
  }
  __syncthreads();
  if (threadIdx.x < kSortBins) p.hist[(int64_t)blockIdx.x * kSortBins + threadIdx.x] = bins[threadIdx.x];
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
  for (int w = 0; w < kSortThreads / 64; ++w) {
    if (w < wave) before += red[w];
    total += red[w];
  }
  return before + s - v;
}

// One digit's counts, replaced by their sums over the tiles before.
__global__ __launch_bounds__(kSortThreads) void sort_scan_kernel(const EmbedSort p, int tiles) {
  __shared__ uint32_t red[kSortThreads / 64];
  const int d = blockIdx.x;
  uint32_t carry = 0;
  for (int t0 = 0; t0 < tiles; t0 += kSortThreads) {
    const int t = t0 + threadIdx.x;
    const uint32_t v = t < tiles ? p.hist[(int64_t)t * kSortBins + d] : 0;
    uint32_t total;
    const uint32_t s = block_scan(v, red, total);
    if (t < tiles) p.hist[(int64_t)t * kSortBins + d] = carry + s;
    carry += total;
  }
  if (threadIdx.x == 0) p.totals[d] = carry;
}

// A thread's keys are kSortBatch, its wave's consecutive.  A key's place is
// where its digit begins in this tile, the keys of the digit in the waves
// before, and those before it in its own wave.
__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(const EmbedSort p, int tiles) {
  constexpr int W = kSortThreads / 64;
  __shared__ uint32_t red[W];
  __shared__ uint32_t place[W][kSortBins];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t base = ((int64_t)blockIdx.x * kSortThreads + (int64_t)wave * 64) * kSortBatch + lane;
  uint32_t key[kSortBatch], tok[kSortBatch], rank[kSortBatch];
#pragma unroll
  for (int u = 0; u < kSortBatch; ++u) {
    const int64_t i = base + (int64_t)u * 64;
    key[u] = i < p.n ? sort_key(p, i) : 0;
    tok[u] = p.first_pass || i >= p.n ? (uint32_t)i : p.tok_in[i];
  }
  // Where this tile's tokens of the thread's digit begin.
  uint32_t before = 0, total = 0;
  const int own = threadIdx.x;
  if (own < kSortBins) {
    if (p.scanned) {
      before = p.hist[(int64_t)blockIdx.x * kSortBins + own];
      total = p.totals[own];
    } else {
#pragma unroll 16
      for (int t = 0; t < tiles; ++t) {
        const uint32_t h = p.hist[(int64_t)t * kSortBins + own];
        total += h;
        if (t < (int)blockIdx.x) before += h;
      }
    }
  }
  for (int d = lane; d < kSortBins; d += 64) place[wave][d] = 0;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int u = 0; u < kSortBatch; ++u) {
    const bool here = base + (int64_t)u * 64 < p.n;
    const int d = digit_of(p, key[u]);
    const uint64_t peers = same_digit(p, d, here);
    const uint32_t at = place[wave][d];   // every lane reads before one of them writes: a wave's LDS accesses are in order
    rank[u] = at + (uint32_t)lanes_before(peers);
    __builtin_amdgcn_wave_barrier();
    if (here && lanes_before(peers) == 0) place[wave][d] = at + (uint32_t)__popcll(peers);
    __builtin_amdgcn_wave_barrier();
  }
  uint32_t all;
  const uint32_t lower = block_scan(total, red, all);  // its barriers stand between the waves' counts and their sums
  if (own < kSortBins) {
    uint32_t at = lower + before;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const uint32_t c = place[w][own];
      place[w][own] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kSortBatch; ++u) {
    if (base + (int64_t)u * 64 >= p.n) continue;
    const uint32_t at = place[wave][digit_of(p, key[u])] + rank[u];
    p.key_out[at] = key[u];
    p.tok_out[at] = tok[u];
  }
}

// Few tokens: every token's place in the sorted list is the number of tokens
// before it there, counted against all of them, kRankTokens tokens per
// workgroup, whose half waves take one 32nd of the list each.
constexpr int kRankThreads = 1024, kRankParts = kRankThreads / kRankTokens;
static_assert(kRankTokens == 32, "half a wave");
__global__ __launch_bounds__(kRankThreads) void sort_rank_kernel(const EmbedSort p) {
  __shared__ __attribute__((aligned(16))) uint32_t keys[kRankMost];
  __shared__ uint32_t count[kRankParts][kRankTokens + 1];
  const int n = (int)p.n, up = (n + kRankTokens - 1) / kRankTokens * kRankTokens;
  {
    constexpr int B = kRankMost / kRankThreads;  // all loads in flight
    uint32_t k[B];
#pragma unroll
    for (int u = 0; u < B; ++u) {
      const int i = u * kRankThreads + threadIdx.x;
      k[u] = i < n ? sort_key(p, i) : 0xffffffffu;  // behind every token
    }
#pragma unroll
    for (int u = 0; u < B; ++u) {
      const int i = u * kRankThreads + threadIdx.x;
      if (i < up) keys[i] = k[u];
    }
  }
  __syncthreads();
  const int t = threadIdx.x & (kRankTokens - 1), part = threadIdx.x / kRankTokens;
  const int own = blockIdx.x, i = own * kRankTokens + t;
  const uint32_t key = keys[i];
  uint32_t c = 0;
  for (int b = part; b < up / kRankTokens; b += kRankParts) {
    const u32x4* const k = (const u32x4*)(keys + b * kRankTokens);
    if (b == own) {
#pragma unroll
      for (int q = 0; q < kRankTokens / 4; ++q) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c += k[q][e] < key + (4 * q + e < t ? 1u : 0u);
      }
    } else {
      const uint32_t limit = key + (b < own ? 1u : 0u);  // of equal keys those before come first
#pragma unroll
      for (int q = 0; q < kRankTokens / 4; ++q) {
        const u32x4 v = k[q];
#pragma unroll
        for (int e = 0; e < 4; ++e) c += v[e] < limit;
      }
    }
  }
  count[part][t] = c;
  __syncthreads();
  if (threadIdx.x >= kRankTokens || i >= n) return;
  uint32_t at = 0;
#pragma unroll
  for (int q = 0; q < kRankParts; ++q) at += count[q][t];
  p.key_out[at] = key;
  p.tok_out[at] = (uint32_t)i;
}

// ---- the sums ------------------------------------------------------------------------
// The first position from lo to hi of the sorted list whose key is not below k
// (hi where there is none), found by a wave: each step asks 64 places at once.
__device__ __forceinline__ int64_t wave_lower_bound(const uint32_t* key, int64_t lo, int64_t hi, uint32_t k) {
  const int lane = threadIdx.x & 63;
  while (hi > lo) {
    const int64_t step = (hi - lo + 63) / 64, at = lo + lane * step;
    const int below = __popcll(__ballot(at < hi && key[at] < k));
    if (!below) return lo;
    const int64_t next = lo + below * step;
    lo += (below - 1) * step + 1;
    hi = next < hi ? next : hi;
  }
  return lo;
}

template <typename O, int V, bool EDGE>
__device__ __forceinline__ void write_row(const EmbedGrad& p, uint32_t row, int col, int valid, const float (&a)[V]) {
  O* const at = (O*)p.dw + (int64_t)row * p.lddw;
  float v[V];
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = a[e] * p.scale;
  if (p.accumulate) {
    Chunk<O, V, EDGE> old;
    old.load(at, col, valid);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] += old.value(e);
  }
  round_store<O, V, EDGE, SUM_STORE>(at, col, valid, v);
}

// Clears `bytes` bytes from an address aligned to 2: the 16-byte words inside
// it, lane beside lane, and what is left at its ends.
template <int G>
__device__ __forceinline__ void clear_bytes(char* p, int64_t bytes, int j) {
  const int64_t head = (int64_t)(-(uintptr_t)p & 15) < bytes ? (int64_t)(-(uintptr_t)p & 15) : bytes;
  const int64_t words = (bytes - head) / 16, tail = head + 16 * words;
  u32x4* const at = (u32x4*)(p + head);
  const u32x4 zero = {0, 0, 0, 0};
  for (int64_t i = j; i < words; i += G) {
    if constexpr (CLEAR_STORE == kStream) __builtin_nontemporal_store(zero, at + i);
    else at[i] = zero;
  }
  for (int64_t i = 2 * j; i < head; i += 2 * G) *(uint16_t*)(p + i) = 0;
  for (int64_t i = tail + 2 * j; i < bytes; i += 2 * G) *(uint16_t*)(p + i) = 0;
}

template <typename T, typename O, int G, bool EDGE>
__global__ __launch_bounds__(NT) void embed_grad_kernel(const EmbedGrad p) {
  constexpr int V = chunk_values<T, O>();
  __shared__ uint8_t touched[kClearRows];
  __shared__ int64_t bounds[2];
  const int j = threadIdx.x % G, grp = threadIdx.x / G;
  if ((int)blockIdx.x >= p.sum_blocks) {
    // Clears the rows that no token has, kClearRows of them.
    const int64_t r0 = (int64_t)(blockIdx.x - p.sum_blocks) * kClearRows;
    const int64_t r1 = r0 + kClearRows < p.rows ? r0 + kClearRows : p.rows;
    const int wave = threadIdx.x >> 6;
    if (wave < 2) {
      const int64_t at = wave_lower_bound(p.key, 0, p.n, (uint32_t)(wave ? r1 : r0));
      if ((threadIdx.x & 63) == 0) bounds[wave] = at;
    } else if (threadIdx.x < 128 + kClearRows) {
      touched[threadIdx.x - 128] = 0;
    }
    __syncthreads();
    const int64_t lo = bounds[0], hi = bounds[1];
    if (hi - lo <= 2 * NT) {
      for (int64_t i = lo + threadIdx.x; i < hi; i += NT) touched[p.key[i] - (uint32_t)r0] = 1;
    } else {  // many tokens: each row is searched for
      for (int64_t r = r0 + wave; r < r1; r += NT / 64) {
        const int64_t at = wave_lower_bound(p.key, lo, hi, (uint32_t)r);
        if ((threadIdx.x & 63) == 0) touched[r - r0] = at < hi && p.key[at] == (uint32_t)r;
      }
    }
    __syncthreads();
    for (int i = grp; r0 + i < r1; i += NT / G)
      if (!touched[i]) clear_bytes<G>((char*)((O*)p.dw + (r0 + i) * p.lddw), (int64_t)p.dim * sizeof(O), j);
    return;
  }
  // The piece's keys and tokens, and the keys beside it.
  constexpr int U = 8;
  __shared__ uint32_t keys[NT / G][kPieceMost + 2], toks[NT / G][kPieceMost];
  const int64_t piece = (int64_t)(blockIdx.x / p.col_blocks) * (NT / G) + grp;
  const int64_t i0 = piece * p.piece;
  const uint32_t none = (uint32_t)p.rows;
  for (int i = j; i < p.piece + 2; i += G) {
    const int64_t at = i0 + i - 1;
    keys[grp][i] = at >= 0 && at < p.n ? p.key[at] : none;
    if (i < p.piece) toks[grp][i] = i0 + i < p.n ? p.tok[i0 + i] : 0;
  }
  __syncthreads();
  const uint32_t* const key = keys[grp] + 1;
  const int col = V * (int)(blockIdx.x % p.col_blocks * G + j);
  const int valid = p.dim - col < 0 ? 0 : (p.dim - col < V ? p.dim - col : V);
  uint32_t run = key[0];
  if (valid <= 0 || run == none) return;
  bool open = key[-1] == run;                  // the run began in a piece before
  float acc[V] = {};
  // The end of a run; at_end: it is the end of the piece.
  auto flush = [&](bool at_end) {
    if (open) round_store<float, V, EDGE, kPlain>(p.slots + (2 * piece) * p.dim, col, valid, acc);
    else if (!at_end || key[p.piece] != run) write_row<O, V, EDGE>(p, run, col, valid, acc);
    else round_store<float, V, EDGE, kPlain>(p.slots + (2 * piece + 1) * p.dim, col, valid, acc);
  };
  // The next tokens' loads are issued before this batch's stores: loads and
  // stores complete in order, so the loads would else wait for the stores.
  Chunk<T, V, EDGE> next[U];
  auto load = [&](int i) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (key[i + u] != none) next[u].load((const T*)p.dy + (int64_t)toks[grp][i + u] * p.lddy, col, valid);
  };
  load(0);
  for (int i = 0; i < p.piece; i += U) {
    Chunk<T, V, EDGE> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = next[u];
    if (i + U < p.piece) load(i + U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t k = key[i + u];
      if (k != run) {
        if (run != none) flush(false);
        open = false;
        run = k;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.f;
      }
      if (k != none) {
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += x[u].value(e);
      }
    }
  }
  if (run != none) flush(true);
}

// Joins the runs that reach over pieces.  A workgroup looks at one piece and
// 4 G columns: where a run begins in the piece and goes on, it adds the slots
// of the pieces it reaches, NT / G parts of them at once, then the parts.  Narrow
// rows take few lanes, so that a frequent token's many slots go by in parts.
template <typename O, int G, bool EDGE>
__global__ __launch_bounds__(NT) void embed_join_kernel(const EmbedGrad p) {
  constexpr int V = 4, PARTS = NT / G;
  __shared__ float red[PARTS][G][V + 1];
  const int64_t piece = blockIdx.x;
  const int64_t i0 = piece * p.piece, i1 = i0 + p.piece;
  if (i1 >= p.n) return;
  const uint32_t run = p.key[i1 - 1], next = p.key[i1], first = p.key[i0], before = p.key[i0 ? i0 - 1 : 0];
  if (run == (uint32_t)p.rows || next != run || (first == run && i0 && before == run)) return;
  // The last piece that begins with the run, 64 pieces looked at together.
  const int64_t pieces = (p.n + p.piece - 1) / p.piece;
  const int look = threadIdx.x & 63;
  int64_t last = piece + 1;
  for (int64_t q = piece + 1;; q += 64) {
    const uint64_t same = __ballot(q + look < pieces && p.key[q + look < pieces ? (q + look) * p.piece : 0] == run);
    const int count = same == ~(uint64_t)0 ? 64 : __ffsll((unsigned long long)~same) - 1;
    if (count) last = q + count - 1;
    if (count < 64) break;
  }
  const int j = threadIdx.x % G, part = threadIdx.x / G;
  const int col = V * (int)(blockIdx.y * G + j);
  const int valid = p.dim - col < 0 ? 0 : (p.dim - col < V ? p.dim - col : V);
  float acc[V] = {};
  if (valid > 0) {
    auto add = [&](int64_t slot) {
      Chunk<float, V, EDGE> x;
      x.load(p.slots + slot * p.dim, col, valid);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += x.value(e);
    };
    if (part == 0) add(2 * piece + 1);
#pragma unroll 8
    for (int64_t q = piece + 1 + part; q <= last; q += PARTS) add(2 * q);
  }
#pragma unroll
  for (int e = 0; e < V; ++e) red[part][j][e] = acc[e];
#pragma unroll
  for (int half = PARTS / 2; half >= 1; half >>= 1) {
    __syncthreads();
    if (part < half) {
#pragma unroll
      for (int e = 0; e < V; ++e) red[part][j][e] += red[part + half][j][e];
    }
  }
  if (part || valid <= 0) return;
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = red[0][j][e];
  write_row<O, V, EDGE>(p, run, col, valid, acc);
}

// f called with the group size and whether rows end in part of a chunk.
template <class F>
hipError_t with_group(int64_t dim, int group, F&& f) {
  const bool edge = dim % 8 != 0;
  switch (group) {
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
  constexpr int V = chunk_values<T, O>();
  return with_group(p.dim, embed_group(p.dim, V), [&](auto g, auto e) {
    constexpr int G = decltype(g)::value;
    const int64_t want = (p.tokens + NT / G - 1) / (NT / G);
    const unsigned y = (unsigned)((p.dim + V * G - 1) / (V * G));
    const int64_t most = 8192 / y > 256 ? 8192 / y : 256;
    return launch_kernel(embed_kernel<T, O, G, decltype(e)::value>, dim3((unsigned)(want < most ? want : most), y), p, s, NT);
  });
}
template <typename T, typename O>
hipError_t launch_grad_types(const EmbedGrad& p, int blocks, hipStream_t s) {
  return with_group(p.dim, embed_group(p.dim, chunk_values<T, O>()), [&](auto g, auto e) {
    return launch_kernel(embed_grad_kernel<T, O, decltype(g)::value, decltype(e)::value>, dim3((unsigned)blocks), p, s, NT);
  });
}

hipError_t launch_sort(void (*kernel)(const EmbedSort, int), dim3 grid, const EmbedSort& p, int tiles, hipStream_t s) {
  void* args[] = {const_cast<EmbedSort*>(&p), &tiles};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(kSortThreads), args, 0, s);
}

}  // namespace

int embed_chunk(bool a_bf16, bool b_bf16) { return a_bf16 && b_bf16 ? chunk_values<uint16_t, uint16_t>() : chunk_values<float, float>(); }
int embed_group(int64_t dim, int values) {
  const int64_t chunks = (dim + values - 1) / values;
  int g = 8;
  while (g < NT && g < chunks) g *= 2;
  return g;
}

hipError_t launch_embed(const Embed& p, bool w_bf16, bool y_bf16, hipStream_t s) {
  if (w_bf16) return y_bf16 ? launch_embed_types<uint16_t, uint16_t>(p, s) : launch_embed_types<uint16_t, float>(p, s);
  return y_bf16 ? launch_embed_types<float, uint16_t>(p, s) : launch_embed_types<float, float>(p, s);
}

hipError_t launch_sort_rank(const EmbedSort& p, hipStream_t s) {
  if (p.n > kRankMost) return hipErrorInvalidValue;
  return launch_kernel(sort_rank_kernel, dim3((unsigned)((p.n + kRankTokens - 1) / kRankTokens)), p, s, kRankThreads);
}
hipError_t launch_sort_hist(const EmbedSort& p, int tiles, hipStream_t s) { return launch_kernel(sort_hist_kernel, dim3((unsigned)tiles), p, s, kSortThreads); }
hipError_t launch_sort_scan(const EmbedSort& p, int tiles, hipStream_t s) { return launch_sort(sort_scan_kernel, dim3(kSortBins), p, tiles, s); }
hipError_t launch_sort_scatter(const EmbedSort& p, int tiles, hipStream_t s) {
  return launch_sort(sort_scatter_kernel, dim3((unsigned)tiles), p, tiles, s);
}

hipError_t launch_embed_grad(const EmbedGrad& p, bool dy_bf16, bool dw_bf16, int blocks, hipStream_t s) {
  if (dy_bf16) return dw_bf16 ? launch_grad_types<uint16_t, uint16_t>(p, blocks, s) : launch_grad_types<uint16_t, float>(p, blocks, s);
  return dw_bf16 ? launch_grad_types<float, uint16_t>(p, blocks, s) : launch_grad_types<float, float>(p, blocks, s);
}

template <typename O>
hipError_t launch_join_type(const EmbedGrad& p, hipStream_t s) {
  const int64_t pieces = (p.n + p.piece - 1) / p.piece;
  auto launch = [&](auto g, auto edge) {
    constexpr int G = decltype(g)::value;
    return launch_kernel(embed_join_kernel<O, G, decltype(edge)::value>, dim3((unsigned)pieces, (unsigned)((p.dim + 4 * G - 1) / (4 * G))), p, s, NT);
  };
  using std::integral_constant;
  const bool edge = p.dim % 8 != 0;
  if (p.dim <= 32) return edge ? launch(integral_constant<int, 8>{}, std::true_type{}) : launch(integral_constant<int, 8>{}, std::false_type{});
  if (p.dim <= 256) return edge ? launch(integral_constant<int, 16>{}, std::true_type{}) : launch(integral_constant<int, 16>{}, std::false_type{});
  return edge ? launch(integral_constant<int, 64>{}, std::true_type{}) : launch(integral_constant<int, 64>{}, std::false_type{});
}
hipError_t launch_embed_join(const EmbedGrad& p, bool dw_bf16, hipStream_t s) {
  return dw_bf16 ? launch_join_type<uint16_t>(p, s) : launch_join_type<float>(p, s);
}

}  // namespace muon
