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
constexpr int kListItem = 4096;
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

}  // namespace muon
