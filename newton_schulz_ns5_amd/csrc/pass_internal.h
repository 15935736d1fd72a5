// Internal declarations of the operators around a layer's products in a pass:
// the gradient norm and clipping, the embedding with its gradient, the norms
// around a block.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace muon {

// ---- gradient norm and clipping ----------------------------------------------------
// Tensors of one launch.  A wave takes an item, kListItem consecutive elements
// of one tensor (or what is left of it); end[i] is the items up to and with
// tensor i.
constexpr int kListMax = 128;
constexpr int kListItem = 2048;
struct TensorList {
  const void* x[kListMax];
  void* y[kListMax];                       // clipping only
  int64_t numel[kListMax];
  int32_t end[kListMax];
  uint64_t x_bf16[kListMax / 64], y_bf16[kListMax / 64];
  int32_t n, items;
};
// Partials are 64-bit words, one per workgroup: a sum of squares (a double's
// bits), or the largest magnitude (an fp32 pattern without its sign).
struct NormPartial {
  TensorList list;
  uint64_t* partial;                       // of this launch's workgroups
  int32_t max_norm_kind;                   // 1: largest magnitude
};
// The norm from `count` partials (or `total`), and what becomes of it.
struct NormTotal {
  const uint64_t* partial; int64_t count;
  const void* total; int32_t total_f64;    // given instead: fp64 sum of squares, or fp32 norm
  int32_t max_norm_kind;
  float* norm; double* square;             // outputs, may be null
  uint64_t* store;                         // launch_norm_total: the one partial that stands for all, may be null
};
struct ClipParams {
  TensorList list;
  NormTotal total;
  double max_norm, eps;
  int32_t in_place;                        // no output differs from its input
};
hipError_t launch_norm_partial(const NormPartial& p, int blocks, hipStream_t s);
hipError_t launch_norm_total(const NormTotal& p, hipStream_t s);
hipError_t launch_clip(const ClipParams& p, int blocks, hipStream_t s);

// ---- norms around a block -----------------------------------------------------------
// A row is held by a group of threads, 8 or 16 columns each.
constexpr int kNormMaxCols = 16384;
struct ResidualNorm {
  int64_t rows;
  int32_t cols;
  int32_t post, norm;                      // norm of the block's output, norm of the stream
  const void* block; int64_t ldb;
  const void* residual; int64_t ldr;       // may be null
  void* stream; int64_t lds;               // forward: may be null; backward: read
  void* y; int64_t ldy;
  const void *weight, *post_weight; int32_t weight_bf16;  // may be null: ones
  const void* gate; int64_t ldg; int32_t gate_bf16;       // may be null
  int64_t gate_each;                       // rows that share a row of the gate
  float scale, residual_scale, eps, offset;
  // backward
  const void* dy; int64_t lddy;
  const void* dstream; int64_t ldds;       // may be null
  void* dblock; int64_t lddb;              // may be null
  void* dresidual; int64_t lddr;           // may be null
  void* dgate; int64_t lddg;               // written here where a workgroup has all rows of a gate's row
  float* part[3];                          // of dweight, dpost_weight [workgroup][cols], of dgate [unit][cols]; may be null
  // Units of rows: gate_chunks for every row of the gate (or for all rows), of
  // unit_rows each but the last.
  int64_t units, unit_rows, span;          // span: rows that gate_chunks units cover
  int32_t gate_chunks;
  int32_t held;                            // bytes of LDS that hold the vectors of every row; 0: not held
  int32_t sums;                            // bytes of LDS behind them, of the gradients' sums where they are not in registers
};
// Threads that hold a row (8 or 32, or the whole waves of a workgroup), and
// columns of each.
struct NormShape { int group, columns; };
NormShape norm_shape(int64_t cols);
inline int norm_threads(const NormShape& s) { return s.group < 64 ? 256 : s.group; }  // of a workgroup
inline int norm_rows(const NormShape& s) { return s.group < 64 ? 256 / s.group : 1; }
hipError_t launch_residual_norm(const ResidualNorm& p, bool bf16, bool stream_bf16, int blocks, hipStream_t s);
hipError_t launch_residual_norm_grad(const ResidualNorm& p, bool bf16, bool stream_bf16, int blocks, hipStream_t s);
// out[o][j] = the sum over count[o] rows of part[o], for each of groups[o]
// consecutive sets of rows.
struct NormSums {
  const float* part[3]; void* out[3]; int64_t ld[3];
  int32_t count[3], groups[3], bf16[3], cols;
};
hipError_t launch_norm_sums(const NormSums& p, hipStream_t s);

// ---- embedding -------------------------------------------------------------------------
// A group of threads holds a row, or as much of it as a workgroup's, one chunk
// of embed_chunk() columns each.
int embed_chunk(bool a_bf16, bool b_bf16);
int embed_group(int64_t dim, int chunk);   // threads of a group
struct EmbedIds {
  const void* ids; int32_t i64;
  int64_t first, rows, padding;            // padding: an id without a gradient (has_padding)
  int32_t has_padding;
};
struct Embed {
  EmbedIds ids;
  int64_t tokens;
  int32_t dim;
  const void* w; int64_t ldw;
  void* y; int64_t ldy;
  float scale;
};
hipError_t launch_embed(const Embed& p, bool w_bf16, bool y_bf16, hipStream_t s);

// Sorting token numbers by their row, stable: digits of `bits` bits from the
// lowest on, by tiles of kSortTile tokens.  A token without a row has the
// key `rows`.
constexpr int kSortBits = 9, kSortBins = 1 << kSortBits, kSortThreads = 512;
constexpr int kSortBatch = 4, kSortTile = kSortThreads * kSortBatch;  // tokens of a thread, of a workgroup
struct EmbedSort {
  EmbedIds ids;                            // first pass: where keys come from
  const uint32_t *key_in, *tok_in;         // later passes
  uint32_t *key_out, *tok_out;
  uint32_t* hist;                          // [tiles][kSortBins]
  uint32_t* totals;                        // [kSortBins], where hist holds sums over the tiles before
  int32_t first_pass, shift, bits, scanned;
  int64_t n;
};
// One launch for up to kRankMost tokens; n^2 comparisons.  A gradient of 2048
// tokens takes 18 us so, 33 by digits; of 8192 30 and 43.  The keys of all tokens
// are in LDS, 32 KiB; longer lists were not ranked, and the two cross above the
// bound: 8192 tokens of 512 over 1000 rows take 25 us, 8193 take 34, 16384 36.
constexpr int kRankMost = 8192, kRankTokens = 32;
hipError_t launch_sort_rank(const EmbedSort& p, hipStream_t s);
hipError_t launch_sort_hist(const EmbedSort& p, int tiles, hipStream_t s);
hipError_t launch_sort_scan(const EmbedSort& p, int tiles, hipStream_t s);
hipError_t launch_sort_scatter(const EmbedSort& p, int tiles, hipStream_t s);

// Sums over the sorted tokens, by pieces of `piece` of them.
struct EmbedGrad {
  const uint32_t *key, *tok;               // sorted
  int64_t n, rows;
  int32_t dim, piece;
  const void* dy; int64_t lddy;
  void* dw; int64_t lddw;
  float scale;
  int32_t accumulate;
  float* slots;                            // [pieces][2][dim]: sums that go on in the next or come from the last piece
  int32_t sum_blocks, col_blocks;          // workgroups of the sums; those behind them clear rows without tokens
};
constexpr int kPieceLeast = 16, kPieceMost = 64;  // multiples of 8
constexpr int kClearRows = 16;             // rows that a workgroup clears
constexpr int kJoinCols = 256;             // columns that a workgroup joins (fewer of narrow rows)
hipError_t launch_embed_grad(const EmbedGrad& p, bool dy_bf16, bool dw_bf16, int blocks, hipStream_t s);
hipError_t launch_embed_join(const EmbedGrad& p, bool dw_bf16, hipStream_t s);

}  // namespace muon
