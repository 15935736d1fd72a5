// Internal declarations of the layer operators (linear product and its
// gradients, per-head norms with rotation) shared by host code and kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stddef.h>

namespace muon {

// Records `msg` as this thread's last error and returns `code`.
int report(int code, const char* msg) noexcept;

// ---- products with an epilogue -------------------------------------------------
// C(i, j) = sum_l A(i, l) B(j, l), i < M, j < N, l < K, with fp32 sums.  An
// operand is stored either with l contiguous ("row": A[i * lda + l]) or with
// its own index contiguous ("col": A[l * lda + i]):
//   forward          x [M][K] row, w [N][K] row
//   input gradient   g [M][N] row, w [N][K] col  (M x K out, sum over N)
//   weight gradient  g [M][N] col, x [M][K] col  (N x K out, sum over M)
// Epilogue: z = C + bias_j; zout = z; y = act(z) + add(i, j).
struct LinGemm {
  const void* A; int64_t lda;
  const void* B; int64_t ldb;
  int64_t M, N, K;
  int64_t Kcol;                                        // K values a col operand holds (K, or fewer: zeros from there on)
  const void* bias; int32_t bias_dtype;
  const void* add; int32_t add_dtype; int64_t ldadd;  // residual, or the output itself (accumulation)
  void* Y; int32_t y_dtype; int64_t ldy;
  void* Z; int64_t ldz;                                // pre-activation (operand type), or null
  int32_t act;
  float* part; int64_t ldpart;                         // split sum: [split][M][ldpart] fp32, else null
  int32_t split;                                       // chunks of the sum, >= 1
};
enum LinKind { kRowRow = 0, kRowCol = 1, kColCol = 2 };

// Tiled kernels (fp32: kTile256x128 and kTile64).  Operand rows
// must start 16-byte aligned, and a row operand's K be a multiple of 16 bytes
// (launch_pack makes such a copy); with split > 1 the kernel stores the
// chunks' products and launch_split_finish adds them and runs the epilogue.
enum LinTile { kTile256 = 0, kTile256x128 = 1, kTile128 = 2, kTile64 = 3 };
hipError_t launch_linear_tiles(const LinGemm& g, bool bf16, LinKind kind, LinTile tile, hipStream_t s);
hipError_t launch_split_finish(const LinGemm& g, bool bf16, hipStream_t s);
// Few rows (M <= kSmallRows), kRowRow: any stride and alignment; 16 nb weight
// rows per workgroup (nb 1 or 4), split as above.
constexpr int kSmallRows = 64;
hipError_t launch_linear_small(const LinGemm& g, bool bf16, int nb, hipStream_t s);
// dst [rows][ldd] = src [rows][cols] with zeros in columns cols .. ldd - 1, up
// to two matrices per launch.
struct PackJob { const void* src; int64_t lds; void* dst; int64_t ldd; int64_t rows, cols; };
struct PackJobs { PackJob job[2]; int32_t n; };
hipError_t launch_pack(const PackJobs& p, bool bf16, hipStream_t s);

// ---- gradient at the pre-activation ----------------------------------------------
// G = round(dy * act'(z)) in the operand type (G null: not stored), with zeros
// in columns N .. ldg - 1 (ldg the next multiple of 8); low (bf16 operands, may
// be null) = round(dy * act'(z) - G), laid out the same; and, when
// partial is not null, partial[c][j] = the sum over row chunk c of dy * act'(z)
// (unrounded), rows c * rows_per .. of M.
struct ActGrad {
  const void* dy; int32_t dy_dtype; int64_t lddy;
  const void* z; int64_t ldz;          // operand type; null: act' = 1
  void* G; int64_t ldg;
  void* low;
  float* partial; int32_t chunks; int64_t rows_per;
  int64_t M, N;
  int32_t act;
};
hipError_t launch_act_grad(const ActGrad& g, bool bf16, hipStream_t s);
// out[j] (+)= sum over chunks of partial[c][j], c ascending.
hipError_t launch_col_sum(const float* partial, int chunks, int64_t n, void* out, int32_t out_dtype, bool accumulate,
                          hipStream_t s);

// ---- per-head norms and rotation ---------------------------------------------------
constexpr int kMaxPairs = 256;
constexpr int kMaxAxes = 4;
struct QkTensor { const void* p; int64_t sb, st, sh; };   // strides in elements: batch, token, head
struct QkParams {
  QkTensor x[2];        // q, k (forward input, or the backward's saved input)
  QkTensor g[2];        // backward: gradients of the outputs
  QkTensor y[2];        // outputs (rotated q, k, or dq, dk)
  int32_t heads[2];
  const void* w[2]; int32_t w_dtype;       // norm weights [dim], may be null
  int64_t seq, tokens;                     // tokens per batch entry, tokens in all
  int32_t dim, rot;
  const void* pos; int32_t pos_i64; int64_t pos_sa, pos_sb, pos_st;
  const void* inv_freq; int32_t inv_freq_f64;
  float scale, sign;                       // cos and sin times scale, sin times sign
  float eps;
  float* partial;                          // backward: [blocks[0] + blocks[1]][dim]
  int32_t tw[2], parts[2], blocks[2];      // of q and k: tokens per wave item, row parts per item, workgroups
  uint8_t axis[kMaxPairs];
};
// mode 0: rotation only; 1: norm and rotation; 2: backward of 1.  vec is the
// elements per chunk (8, 4, 2: vector kernels; 1: the element-wise kernel).
hipError_t launch_qk(const QkParams& p, int mode, bool bf16, bool interleaved, int vec, hipStream_t s);
hipError_t launch_qk_weight_sum(const QkParams& p, void* const out[2], int32_t out_dtype, hipStream_t s);

}  // namespace muon
