// Host side of the layer operators: validation, workspace carve-up and launch
// sequences of the linear product, its gradients and the per-head norms with
// rotation.  Every argument is checked before anything is enqueued.
#include <cmath>
#include <algorithm>

#include "host_check.h"
#include "layer_internal.h"
#include "muon_mi355x.h"

using namespace muon;

namespace {

// ---- the linear product -------------------------------------------------------------
// Dimensions stay below 2^30 and a row stride (rounded up to 32 bytes, as
// copies are) below 2^23 bytes, so that a tile's panel of rows is addressed
// with 32-bit offsets.
constexpr int64_t kMaxSize = (int64_t)1 << 30, kMaxRowBytes = ((int64_t)1 << 23) - 32;

int check_sizes(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || n < 0 || k < 0) return fail(MUON_ERR_INVALID_ARG, "negative size (m=%lld n=%lld k=%lld)", (long long)m, (long long)n, (long long)k);
  if (m > kMaxSize || n > kMaxSize || k > kMaxSize) return fail(MUON_ERR_INVALID_ARG, "m, n and k must be at most 2^30");
  // one workgroup per 64 x 64 tile of an output, and a grid holds fewer than 2^31
  if (std::max({cdiv(m, 64) * cdiv(n, 64), cdiv(m, 64) * cdiv(k, 64), cdiv(n, 64) * cdiv(k, 64)}) > INT32_MAX)
    return fail(MUON_ERR_INVALID_ARG, "an output has too many tiles");
  return MUON_OK;
}

int check_matrix(const char* name, const void* p, int32_t dt, int64_t rows, int64_t cols, int64_t ld) {
  if (!dtype_ok(dt)) return fail(MUON_ERR_UNSUPPORTED, "%s dtype %d is not MUON_F32 or MUON_BF16", name, dt);
  if (rows == 0 || cols == 0) return MUON_OK;
  if (!p) return fail(MUON_ERR_INVALID_ARG, "%s is NULL", name);
  if (ld < cols && rows > 1) return fail(MUON_ERR_INVALID_ARG, "%s row stride %lld is smaller than its %lld columns", name, (long long)ld, (long long)cols);
  if (cols * esize(dt) > kMaxRowBytes || (rows > 1 && ld * esize(dt) > kMaxRowBytes))
    return fail(MUON_ERR_INVALID_ARG, "%s rows must be at most 2^23 - 32 bytes apart", name);
  if ((uintptr_t)p % esize(dt)) return fail(MUON_ERR_INVALID_ARG, "%s is not aligned to its element size", name);
  return MUON_OK;
}

int check_act(int32_t act) {
  if (act < MUON_ACT_NONE || act > MUON_ACT_GELU_TANH) return fail(MUON_ERR_UNSUPPORTED, "activation %d is not one of MUON_ACT_*", act);
  return MUON_OK;
}

int check_linear(const muon_linear_problem* q) {
  if (!q) return fail(MUON_ERR_INVALID_ARG, "problem is NULL");
  if (q->reserved) return fail(MUON_ERR_INVALID_ARG, "reserved must be 0");
  int rc;
  if ((rc = check_sizes(q->m, q->n, q->k)) || (rc = check_act(q->activation))) return rc;
  if ((rc = check_matrix("x", q->x, q->dtype, q->m, q->k, q->x_row_stride))) return rc;
  if ((rc = check_matrix("w", q->w, q->dtype, q->n, q->k, q->w_row_stride))) return rc;
  if ((rc = check_matrix("y", q->y, q->y_dtype, q->m, q->n, q->y_row_stride))) return rc;
  if (q->bias && (rc = check_matrix("bias", q->bias, q->bias_dtype, 1, q->n, q->n))) return rc;
  if (q->residual && (rc = check_matrix("residual", q->residual, q->residual_dtype, q->m, q->n, q->residual_row_stride))) return rc;
  if (q->preact && (rc = check_matrix("preact", q->preact, q->dtype, q->m, q->n, q->preact_row_stride))) return rc;
  const Rows y = rows_of("y", q->y, q->y_dtype, q->m, q->n, q->y_row_stride);
  const Rows z = rows_of("preact", q->preact, q->dtype, q->m, q->n, q->preact_row_stride);
  const Rows in[] = {rows_of("x", q->x, q->dtype, q->m, q->k, q->x_row_stride),
                     rows_of("w", q->w, q->dtype, q->n, q->k, q->w_row_stride),
                     rows_of("bias", q->bias, q->bias_dtype, 1, q->n, q->n),
                     rows_of("residual", q->residual, q->residual_dtype, q->m, q->n, q->residual_row_stride)};
  for (const Rows& r : in) {
    const bool same = r.at == y.at && r.name == in[3].name && q->residual_dtype == q->y_dtype &&
                      (q->m <= 1 || q->residual_row_stride == q->y_row_stride);
    if (!same && meet(y, r)) return fail(MUON_ERR_INVALID_ARG, "y overlaps %s (only y == residual is allowed)", r.name);
    if (meet(z, r)) return fail(MUON_ERR_INVALID_ARG, "preact overlaps %s", r.name);
  }
  if (meet(y, z)) return fail(MUON_ERR_INVALID_ARG, "preact overlaps y");
  return MUON_OK;
}

int check_linear_grad(const muon_linear_grad* q) {
  if (!q) return fail(MUON_ERR_INVALID_ARG, "problem is NULL");
  if (q->reserved) return fail(MUON_ERR_INVALID_ARG, "reserved must be 0");
  int rc;
  if ((rc = check_sizes(q->m, q->n, q->k)) || (rc = check_act(q->activation))) return rc;
  if (!dtype_ok(q->dtype)) return fail(MUON_ERR_UNSUPPORTED, "dtype %d is not MUON_F32 or MUON_BF16", q->dtype);
  if ((rc = check_matrix("dy", q->dy, q->dy_dtype, q->m, q->n, q->dy_row_stride))) return rc;
  // the gradient at the pre-activation is a matrix of the operands' type
  if (q->n * esize(q->dtype) > kMaxRowBytes) return fail(MUON_ERR_INVALID_ARG, "rows of n elements of dtype must be at most 2^23 - 32 bytes");
  const bool act = q->activation != MUON_ACT_NONE;
  if (act && (rc = check_matrix("preact", q->preact, q->dtype, q->m, q->n, q->preact_row_stride))) return rc;
  if (q->dw && (rc = check_matrix("x", q->x, q->dtype, q->m, q->k, q->x_row_stride))) return rc;
  if (q->dx && (rc = check_matrix("w", q->w, q->dtype, q->n, q->k, q->w_row_stride))) return rc;
  if (q->dx && (rc = check_matrix("dx", q->dx, q->dx_dtype, q->m, q->k, q->dx_row_stride))) return rc;
  if (q->dw && (rc = check_matrix("dw", q->dw, q->dw_dtype, q->n, q->k, q->dw_row_stride))) return rc;
  if (q->dbias && (rc = check_matrix("dbias", q->dbias, q->dbias_dtype, 1, q->n, q->n))) return rc;
  if (q->accumulate != 0 && q->accumulate != 1) return fail(MUON_ERR_INVALID_ARG, "accumulate must be 0 or 1");
  const Rows in[] = {rows_of("dy", q->dy, q->dy_dtype, q->m, q->n, q->dy_row_stride),
                     rows_of("preact", act ? q->preact : nullptr, q->dtype, q->m, q->n, q->preact_row_stride),
                     rows_of("x", q->dw ? q->x : nullptr, q->dtype, q->m, q->k, q->x_row_stride),
                     rows_of("w", q->dx ? q->w : nullptr, q->dtype, q->n, q->k, q->w_row_stride)};
  const Rows out[] = {rows_of("dx", q->dx, q->dx_dtype, q->m, q->k, q->dx_row_stride),
                      rows_of("dw", q->dw, q->dw_dtype, q->n, q->k, q->dw_row_stride),
                      rows_of("dbias", q->dbias, q->dbias_dtype, 1, q->n, q->n)};
  for (int i = 0; i < 3; ++i) {
    for (const Rows& r : in)
      if (meet(out[i], r)) return fail(MUON_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, r.name);
    for (int j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return fail(MUON_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, out[j].name);
  }
  return MUON_OK;
}

// Elements per 16 bytes.
int64_t per16(int32_t dt) { return 16 / esize(dt); }

// An operand of a product: a [rows][cols] matrix, used in place where the
// tiled kernels can load it (16-byte aligned rows, whole 16-byte chunks of K
// in a row operand), else copied into the workspace with zeros behind its
// rows (one read and one write of it, against the product's many).
struct Operand {
  const void* p;
  int64_t rows, cols, ld;
  bool pack;
  size_t off;  // of the copy in the workspace
};

Operand operand(const void* p, int64_t rows, int64_t cols, int64_t ld, int32_t dt, bool row_kind) {
  Operand o{p, rows, cols, ld, false, 0};
  if (rows <= 1) o.ld = cdiv(cols, per16(dt)) * per16(dt);  // a single row's stride means nothing
  o.pack = ((uintptr_t)p & 15) || (o.ld % per16(dt)) || (row_kind && cols % per16(dt));
  return o;
}

// How a product M x N over K runs: rows 0 .. m1 - 1 and columns 0 .. n1 - 1 in
// tiles `first`, the others (rows or columns, not both) in tiles `rest`, and
// the sum in `split` chunks.
//
// Workgroups of a tile run in rounds of as many as the chip holds at once; a
// round takes a fixed time (pipeline start, epilogue) and a time per slice of
// K, which is bounded by latency (u0) while few workgroups run and by the
// chip's rate (u1) in a full round.  Measured for every tile with 16 to 1024
// workgroups.  bf16, us in tiles of 256 x 256, 256 x 128, 128 and 64, and with
// the last, part-empty round of the largest tile in the next (one box):
//   4096 x 14336 over 4096   417  409  500  704  399
//   14336 x 4096 over 4096   398  432  546  791  388
//   6144 x 4096 over 2048    104  101  121  158   96
//   2048 x 4096 over 6144    129   91  112  161
//   1037 x 1001 over 2056      -   22*  23*   18      * split, with its addition
struct Tiling { LinTile first, rest; int64_t m1, n1; int split; double us; };  // us: by the model above

//
// fp32 64-edge tiles, four to a CU: the last round takes as long as its fullest
// CU, so their rate goes by whole workgroups per CU, and their start and
// epilogue run under each other's products.  us, the tiles chosen without and
// with that in the model, and the library's product:
//   260 x 4096 over 14336   474  297  255
//   227 x 9174 over 4920    238  197  193
//   87 x 8583 over 4288     110   91   66
//   16 x 6812 over 7680      91   68   40
//   2339 x 704 over 4736    160  137  121
//   7680 x 6812 over 16      81   62   77
//   260 x 14336 over 4096   326  326  239
struct TileCost { LinTile tile; int bm, bn, slots; double fixed, u0, u1; bool by_cu; };
constexpr TileCost kCostBf16[] = {{kTile256, 256, 256, 256, 8.0, 1.15, 1.65, false},
                                  {kTile256x128, 256, 128, 256, 6.0, 0.58, 0.87, false},
                                  {kTile128, 128, 128, 512, 6.0, 0.75, 1.13, false},
                                  {kTile64, 64, 64, 768, 6.0, 0.30, 0.62, false}};
constexpr TileCost kCostF32[] = {{kTile256x128, 256, 128, 256, 9.0, 3.6, 3.77, false},
                                 {kTile64, 64, 64, 1024, 3.0, 0.5, 2.0, true}};

// Microseconds of `wgs` workgroups of `slices` slices each.
double tile_time(const TileCost& c, int64_t wgs, int64_t slices) {
  const int64_t full = wgs / c.slots, last = wgs % c.slots;
  double t = (double)full * (c.fixed + (double)slices * c.u1);
  const int cus = 256, per_cu = c.slots / cus;
  const double share = c.by_cu ? (double)cdiv(last, cus) / per_cu : (double)last / c.slots;
  if (last) t += c.fixed + (double)slices * std::max(c.u0, c.u1 * share);
  return t;
}

Tiling choose_tiling(int64_t M, int64_t N, int64_t K, bool bf) {
  const TileCost* costs = bf ? kCostBf16 : kCostF32;
  const int n = bf ? 4 : 2;
  const int64_t slices = std::max<int64_t>(1, cdiv(K, bf ? 64 : 32));
  Tiling best{kTile64, kTile64, M, N, 1, 0};
  double least = 1e30;
  for (int i = 0; i < n; ++i) {
    const TileCost& c = costs[i];
    const int64_t tiles = cdiv(M, c.bm) * cdiv(N, c.bn);
    if (tiles >= (int64_t)1 << 23) continue;  // a launch has fewer than 2^32 threads, of up to 512 per tile
    for (int split : {1, 2, 3, 4, 6, 8, 12, 16}) {
      // chunks of at least two slices, and at most two rounds of them
      if (split > 1 && (split > slices / 2 || tiles * split > 2 * c.slots)) break;
      double t = tile_time(c, tiles * split, cdiv(slices, split));
      if (split > 1) t += 4.0 + (double)(M * N) * 4.0 * (split + 1) / 4e6;  // a launch, and the products at 4 TB/s
      if (t < least) {
        least = t;
        best = {c.tile, c.tile, M, N, split, t};
      }
    }
  }
  if (bf) {  // whole rounds of the largest tile, the rest in the next smaller
    const int64_t tm = cdiv(M, 256), tn = cdiv(N, 256), rounds = tm * tn / 256;
    const int64_t cols = rounds * 256 / tm, rows = rounds * 256 / tn;  // whole columns or rows of tiles in them
    if (cols > 0 && cols < tn) {
      const double t = tile_time(kCostBf16[0], cols * tm, slices) + tile_time(kCostBf16[1], tm * cdiv(N - cols * 256, 128), slices);
      if (t < least) {
        least = t;
        best = {kTile256, kTile256x128, M, cols * 256, 1, t};
      }
    }
    if (rows > 0 && rows < tm) {
      const double t = tile_time(kCostBf16[0], rows * tn, slices) + tile_time(kCostBf16[1], (tm - rows) * cdiv(N, 128), slices);
      if (t < least) best = {kTile256, kTile256x128, rows * 256, N, 1, t};
    }
  }
  return best;
}

int64_t part_ld(int64_t N) { return cdiv(N, 8) * 8; }
size_t part_bytes(int64_t M, int64_t N, int split) {
  return split > 1 ? align256((size_t)split * (size_t)M * (size_t)part_ld(N) * 4) : 0;
}

// Pack launches of the operands that need one, two per launch.
hipError_t pack_all(Operand* const* ops, int n, int32_t dt, char* ws, hipStream_t s) {
  PackJobs jobs{};
  for (int i = 0; i < n; ++i) {
    Operand& o = *ops[i];
    if (o.pack) {
      const int64_t ld = cdiv(o.cols, per16(dt)) * per16(dt);
      jobs.job[jobs.n++] = PackJob{o.p, o.ld, ws + o.off, ld, o.rows, o.cols};
      o.p = ws + o.off;
      o.ld = ld;
    }
    if (jobs.n == 2 || (i == n - 1 && jobs.n)) {
      const hipError_t e = launch_pack(jobs, dt == MUON_BF16, s);
      if (e != hipSuccess) return e;
      jobs.n = 0;
    }
  }
  return hipSuccess;
}

size_t pack_bytes(const Operand& o, int32_t dt) {
  return o.pack ? align256((size_t)(o.rows * cdiv(o.cols, per16(dt)) * 16)) : 0;
}

hipError_t run_product(LinGemm g, int32_t dt, LinKind kind, const Tiling& t, char* part, hipStream_t s) {
  const bool bf = dt == MUON_BF16;
  g.Kcol = g.K;
  // a row operand whose K is not whole chunks is a copy with zeros behind K
  if (kind != kColCol) g.K = cdiv(g.K, per16(dt)) * per16(dt);
  g.split = t.split;
  g.part = t.split > 1 ? (float*)part : nullptr;
  g.ldpart = part_ld(g.N);
  hipError_t e;
  if (t.n1 < g.N || t.m1 < g.M) {
    LinGemm r = g;  // rows m1 .. M - 1 or columns n1 .. N - 1
    const int64_t m1 = t.m1 < g.M ? t.m1 : 0, n1 = t.n1 < g.N ? t.n1 : 0;
    auto past = [&](const void* p, int64_t elems, int32_t d) { return p ? (const char*)p + elems * esize(d) : nullptr; };
    r.M = g.M - m1;
    r.N = g.N - n1;
    r.A = past(g.A, kind == kColCol ? m1 : m1 * g.lda, dt);
    r.B = past(g.B, kind == kRowRow ? n1 * g.ldb : n1, dt);
    r.bias = past(g.bias, n1, g.bias_dtype);
    r.add = past(g.add, m1 * g.ldadd + n1, g.add_dtype);
    r.Y = (void*)past(g.Y, m1 * g.ldy + n1, g.y_dtype);
    r.Z = (void*)past(g.Z, m1 * g.ldz + n1, dt);
    if (m1) g.M = m1;
    if (n1) g.N = n1;
    e = launch_linear_tiles(g, bf, kind, t.first, s);
    return e == hipSuccess ? launch_linear_tiles(r, bf, kind, t.rest, s) : e;
  }
  e = launch_linear_tiles(g, bf, kind, t.first, s);
  if (e == hipSuccess && t.split > 1) e = launch_split_finish(g, bf, s);
  return e;
}

// Few rows: weight rows per workgroup / 16 through nb, and the chunks of K;
// `us` receives the time of an fp32 product.
int few_rows(int64_t m, int64_t n, int64_t k, int32_t dtype, int& nb, double& us) {
  // Workgroups of 64 weight rows read the tokens least often; of 16, the weight
  // with the most workgroups.  Chunks of K, of two steps per wave at least,
  // make up to the 256 CUs' worth of either, and cost a second launch (4 us).
  const int64_t steps = cdiv(k * esize(dtype), 128);
  const int64_t wide = cdiv(n, 64), narrow = cdiv(n, 16);
  auto chunks = [&](int64_t wgs, int64_t most) { return std::max<int64_t>(1, std::min<int64_t>({most, 256 / wgs, steps / 16})); };
  const int64_t split4 = chunks(wide, 8), split1 = chunks(narrow, 16);
  // 64 rows: enough workgroups without a split, or, where the tokens are many
  // enough to count (more than 16, or 8 of a weight that is wide too), half a
  // chip of them with one.
  const bool many = m > 16 || (m > 8 && wide >= 80);
  nb = wide >= 192 || (many && wide * split4 >= 128) ? 4 : 1;
  if (nb == 4) {
    // a workgroup per CU; its eight waves take a step each at once, which takes
    // so many us by the blocks of 16 tokens (fp32)
    const double step[] = {2.9, 4.0, 5.5, 6.5};
    const int64_t split = wide >= 192 ? 1 : split4;
    us = 5 + (double)(cdiv(wide * split, 256) * cdiv(cdiv(steps, split), 8)) * step[(m - 1) / 16] + (split > 1 ? 4 : 0);
    return (int)split;
  }
  // A wave's time per step grows with the tokens.  A split pays where the steps
  // it saves are worth more than its launch, and the call takes longer than one
  // of two launches from Python, workspace included (13 us).
  const double per_step = 0.4 + (double)m / 40, whole = 5 + (double)steps / 8 * per_step;
  const int64_t split = whole > 16 && (whole - 5) * (1 - 1.0 / (double)split1) > 6 ? split1 : 1;
  us = 5 + (double)cdiv(steps, split * 8) * per_step + (split > 1 ? 4 : 0);
  return (int)split;
}

// fp32, 17 to 64 rows: whether the tiles are faster.  They read the weight at
// 2.4 TB/s at most with so few rows, and pad the rows to 64; the few-row kernel
// multiplies rows padded to 16, one step per wave at a time, and takes a K that
// is not whole chunks without a copy.  By the sizes alone, so that a result
// does not depend on its operands' alignment.  us, few-row kernel and tiles, at
// 24, 40 and 64 rows:
//   9472 x 2504    45 37   59 38   77 39
//   6144 x 4096    39 34   52 35   61 36
//   1024 x 8192    22 18   27 18   32 18
//   4096 x 4096    25 34   31 34   37 35
//   14336 x 4096   67 106  92 107  108 107
bool tiles_for_few(int64_t m, int64_t n, int64_t k, int32_t dtype, const Tiling& t, double few_us) {
  return dtype == MUON_F32 && m > 16 && k % per16(dtype) == 0 &&
         1.1 * std::max(t.us, (double)n * (double)k * 4 / 2.4e6) < few_us;
}

// Work of a forward call: the small kernel for few rows, else tiles.
struct LinearPlan {
  bool small;
  int nb;          // small: weight rows per workgroup / 16
  Operand x, w;
  Tiling t;
  size_t part_off, total;
};

LinearPlan plan_linear(const muon_linear_problem* q) {
  LinearPlan P{};
  P.small = q->m <= kSmallRows;
  if (q->m == 0 || q->n == 0) return P;
  P.x = operand(q->x, q->m, q->k, q->x_row_stride, q->dtype, true);
  P.w = operand(q->w, q->n, q->k, q->w_row_stride, q->dtype, true);
  if (P.small) {
    double us = 0;
    const int split = few_rows(q->m, q->n, q->k, q->dtype, P.nb, us);
    if (q->dtype == MUON_F32 && q->m > 16) {
      P.t = choose_tiling(q->m, q->n, q->k, false);
      P.small = !tiles_for_few(q->m, q->n, q->k, q->dtype, P.t, us);
    }
    if (P.small) {
      P.t.split = split;
      P.total = part_bytes(q->m, q->n, split);
      return P;
    }
  } else {
    P.t = choose_tiling(q->m, q->n, q->k, q->dtype == MUON_BF16);
  }
  size_t off = 0;
  P.x.off = off; off += pack_bytes(P.x, q->dtype);
  P.w.off = off; off += pack_bytes(P.w, q->dtype);
  P.part_off = off; off += part_bytes(q->m, q->n, P.t.split);
  P.total = off;
  return P;
}

// Work of a gradient call.  The elementwise pass runs when the gradient at the
// pre-activation differs from dy (an activation, or dy of another type than
// the operands), when dy's rows cannot be loaded in place, or when the bias
// gradient is wanted.  The split sums of dx and dw use one region in turn.
// With bf16 operands g = dy act'(z) has more bits than an operand.  A gradient
// in bf16 takes g rounded to bf16, whose error (2^-8 of each term) is the one
// that its own rounding has.  A gradient in fp32 takes two terms, the rounded g
// and what that leaves, rounded: 2^-16 of each term, at twice the products.
struct GradPlan {
  bool store_g, colsum, low;
  int64_t ldg;
  int chunks;
  int64_t rows_per;
  Operand x, w;
  Tiling tx, tw;
  size_t g_off, low_off, partial_off, part_off, total;
};

GradPlan plan_grad(const muon_linear_grad* q) {
  GradPlan P{};
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t at = off; off = align256(off + bytes); return at; };
  const bool dx = q->dx && q->m > 0 && q->k > 0, dw = q->dw && q->n > 0 && q->k > 0;
  const Operand dy = operand(q->dy, q->m, q->n, q->dy_row_stride, q->dtype, dx);
  P.store_g = q->m > 0 && q->n > 0 && (dx || dw) && (q->activation != MUON_ACT_NONE || q->dy_dtype != q->dtype || dy.pack);
  P.colsum = q->dbias && q->n > 0;
  // Rows per workgroup of the elementwise pass: enough workgroups to fill the
  // chip (256 columns each), at least the 8 rows it takes at once.
  const int64_t cols = std::max<int64_t>(1, cdiv(q->n, 256));
  const int64_t want = std::max<int64_t>(1, 2048 / cols);
  P.rows_per = std::max<int64_t>(8, cdiv(q->m, want));
  P.chunks = (int)cdiv(q->m, P.rows_per);
  P.ldg = cdiv(q->n, 8) * 8;
  if (P.store_g) P.g_off = take((size_t)(q->m * P.ldg * esize(q->dtype)));
  P.low = P.store_g && q->dtype == MUON_BF16 && (q->activation != MUON_ACT_NONE || q->dy_dtype != MUON_BF16) &&
          ((dx && q->dx_dtype == MUON_F32) || (dw && q->dw_dtype == MUON_F32));
  if (P.low) P.low_off = take((size_t)(q->m * P.ldg * 2));
  if (P.colsum) P.partial_off = take((size_t)P.chunks * (size_t)q->n * 4);
  const bool bf = q->dtype == MUON_BF16;
  size_t part = 0;
  if (dx) {
    P.w = operand(q->w, q->n, q->k, q->w_row_stride, q->dtype, false);
    if (q->n == 0) { P.w.pack = false; P.w.p = nullptr; }  // an empty sum reads nothing
    P.w.off = take(pack_bytes(P.w, q->dtype));
    P.tx = choose_tiling(q->m, q->k, q->n, bf);
    part = std::max(part, part_bytes(q->m, q->k, P.tx.split));
  }
  if (dw) {
    P.x = operand(q->x, q->m, q->k, q->x_row_stride, q->dtype, false);
    if (q->m == 0) { P.x.pack = false; P.x.p = nullptr; }
    P.x.off = take(pack_bytes(P.x, q->dtype));
    P.tw = choose_tiling(q->n, q->k, q->m, bf);
    part = std::max(part, part_bytes(q->n, q->k, P.tw.split));
  }
  P.part_off = take(part);
  P.total = off;
  return P;
}

}  // namespace

extern "C" {

int muon_linear_workspace_bytes(const muon_linear_problem* q, size_t* bytes) {
  if (!q || !bytes) return fail(MUON_ERR_INVALID_ARG, "problem or bytes is NULL");
  int rc = check_linear(q);
  if (rc) return rc;
  *bytes = plan_linear(q).total;
  return ok();
}

int muon_linear(const muon_linear_problem* q, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_linear(q);
  if (rc) return rc;
  if (q->m == 0 || q->n == 0) return ok();
  LinearPlan P = plan_linear(q);
  if ((rc = check_workspace(workspace, workspace_bytes, P.total))) return rc;
  hipStream_t s = (hipStream_t)stream;
  char* ws = (char*)workspace;
  LinGemm g{};
  g.A = q->x; g.lda = q->x_row_stride;
  g.B = q->w; g.ldb = q->w_row_stride;
  g.M = q->m; g.N = q->n; g.K = q->k;
  g.bias = q->bias; g.bias_dtype = q->bias_dtype;
  g.add = q->residual; g.add_dtype = q->residual_dtype; g.ldadd = q->residual_row_stride;
  g.Y = q->y; g.y_dtype = q->y_dtype; g.ldy = q->y_row_stride;
  g.Z = q->preact; g.ldz = q->preact_row_stride;
  g.act = q->activation;
  g.split = 1;
  hipError_t e;
  if (P.small) {
    const bool bf = q->dtype == MUON_BF16;
    g.split = P.t.split;
    g.part = g.split > 1 ? (float*)(ws + P.part_off) : nullptr;
    g.ldpart = part_ld(g.N);
    e = launch_linear_small(g, bf, P.nb, s);
    if (e == hipSuccess && g.split > 1) e = launch_split_finish(g, bf, s);
  } else {
    Operand* ops[] = {&P.x, &P.w};
    if ((e = pack_all(ops, 2, q->dtype, ws, s)) != hipSuccess) return hip_fail(e, "operand copies");
    g.A = P.x.p; g.lda = P.x.ld;
    g.B = P.w.p; g.ldb = P.w.ld;
    e = run_product(g, q->dtype, kRowRow, P.t, ws + P.part_off, s);
  }
  return e == hipSuccess ? ok() : hip_fail(e, "linear kernels");
}

int muon_linear_plan(int64_t m, int64_t n, int64_t k, int32_t dtype, int32_t kind, int32_t plan[4]) {
  if (!plan) return fail(MUON_ERR_INVALID_ARG, "plan is NULL");
  if (kind < 0 || kind > 2) return fail(MUON_ERR_INVALID_ARG, "kind %d is not in 0..2", kind);
  if (!dtype_ok(dtype)) return fail(MUON_ERR_UNSUPPORTED, "dtype %d is not MUON_F32 or MUON_BF16", dtype);
  const int rc = check_sizes(m, n, k);
  if (rc) return rc;
  const int64_t M = kind == 2 ? n : m, N = kind == 0 ? n : k, K = kind == 0 ? k : (kind == 1 ? n : m);
  for (int i = 0; i < 4; ++i) plan[i] = 0;  // an empty output runs nothing
  if (M == 0 || N == 0) return ok();
  const Tiling t = choose_tiling(M, N, K, dtype == MUON_BF16);
  if (kind == 0 && m <= kSmallRows) {
    int nb = 1;
    double us = 0;
    const int split = few_rows(m, n, k, dtype, nb, us);
    if (!tiles_for_few(m, n, k, dtype, t, us)) {
      plan[1] = 16 * nb; plan[2] = split;
      return ok();
    }
  }
  const int edge[4][2] = {{256, 256}, {256, 128}, {128, 128}, {64, 64}};
  plan[0] = edge[t.first][0]; plan[1] = edge[t.first][1]; plan[2] = t.split; plan[3] = t.m1 < M || t.n1 < N;
  return ok();
}

int muon_linear_backward_workspace_bytes(const muon_linear_grad* q, size_t* bytes) {
  if (!q || !bytes) return fail(MUON_ERR_INVALID_ARG, "problem or bytes is NULL");
  int rc = check_linear_grad(q);
  if (rc) return rc;
  *bytes = plan_grad(q).total;
  return ok();
}

int muon_linear_backward(const muon_linear_grad* q, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_linear_grad(q);
  if (rc) return rc;
  GradPlan P = plan_grad(q);
  if ((rc = check_workspace(workspace, workspace_bytes, P.total))) return rc;
  const bool bf = q->dtype == MUON_BF16;
  hipStream_t s = (hipStream_t)stream;
  char* ws = (char*)workspace;
  hipError_t e;
  // the gradient at the pre-activation; dy itself where they are the same
  const void* G = q->m && q->n ? q->dy : nullptr;
  int64_t ldg = q->m > 1 && q->n ? q->dy_row_stride : P.ldg;  // (the stride of one row, or of none, means nothing)
  if (P.store_g || (P.colsum && P.chunks > 0)) {
    ActGrad a{};
    a.dy = q->dy; a.dy_dtype = q->dy_dtype; a.lddy = q->dy_row_stride;
    a.act = q->activation;
    if (a.act != MUON_ACT_NONE) { a.z = q->preact; a.ldz = q->preact_row_stride; }
    if (P.store_g) {
      a.G = ws + P.g_off; a.ldg = P.ldg;
      G = a.G; ldg = P.ldg;
    }
    if (P.low) a.low = ws + P.low_off;
    if (P.colsum) a.partial = (float*)(ws + P.partial_off);
    a.chunks = P.chunks; a.rows_per = P.rows_per;
    a.M = q->m; a.N = q->n;
    if ((e = launch_act_grad(a, bf, s)) != hipSuccess) return hip_fail(e, "gradient at the pre-activation");
  }
  if (P.colsum) {
    e = launch_col_sum((const float*)(ws + P.partial_off), P.chunks, q->n, q->dbias, q->dbias_dtype, q->accumulate != 0, s);
    if (e != hipSuccess) return hip_fail(e, "bias gradient");
  }
  const bool dx = q->dx && q->m > 0 && q->k > 0, dw = q->dw && q->n > 0 && q->k > 0;
  Operand* ops[] = {&P.w, &P.x};
  if ((e = pack_all(ops, 2, q->dtype, ws, s)) != hipSuccess) return hip_fail(e, "operand copies");
  if (dx) {
    LinGemm g{};
    g.A = G; g.lda = ldg;
    g.B = P.w.p; g.ldb = P.w.ld;
    g.M = q->m; g.N = q->k; g.K = q->n;
    g.Y = q->dx; g.y_dtype = q->dx_dtype; g.ldy = q->dx_row_stride;
    e = run_product(g, q->dtype, kRowCol, P.tx, ws + P.part_off, s);
    if (e == hipSuccess && P.low && q->dx_dtype == MUON_F32) {
      g.A = ws + P.low_off;
      g.add = q->dx; g.add_dtype = q->dx_dtype; g.ldadd = q->dx_row_stride;
      e = run_product(g, q->dtype, kRowCol, P.tx, ws + P.part_off, s);
    }
    if (e != hipSuccess) return hip_fail(e, "input gradient");
  }
  if (dw) {
    LinGemm g{};
    g.A = G; g.lda = ldg;
    g.B = P.x.p; g.ldb = P.x.ld;
    g.M = q->n; g.N = q->k; g.K = q->m;
    g.Y = q->dw; g.y_dtype = q->dw_dtype; g.ldy = q->dw_row_stride;
    if (q->accumulate) { g.add = q->dw; g.add_dtype = q->dw_dtype; g.ldadd = q->dw_row_stride; }
    e = run_product(g, q->dtype, kColCol, P.tw, ws + P.part_off, s);
    if (e == hipSuccess && P.low && q->dw_dtype == MUON_F32) {
      g.A = ws + P.low_off;
      g.add = q->dw; g.add_dtype = q->dw_dtype; g.ldadd = q->dw_row_stride;
      e = run_product(g, q->dtype, kColCol, P.tw, ws + P.part_off, s);
    }
    if (e != hipSuccess) return hip_fail(e, "weight gradient");
  }
  return ok();
}

}  // extern "C"

namespace {

// ---- per-head norms and rotation -------------------------------------------------------

const char* kQ[2] = {"q", "k"};

// Extent of one strided [batch][token][head][dim] tensor in bytes; strides are
// not negative.
struct Span { uintptr_t lo, hi; };

// Whether n positions `stride` apart stay below 2^54 bytes in all (with at most
// four such terms, every offset fits 64 bits).
bool extent_ok(int64_t n, int64_t stride) { return n <= 1 || stride <= ((int64_t)1 << 54) / 8 / (n - 1); }

int check_heads(const char* what, int i, const muon_heads* t, int32_t dt, const muon_qk_problem* q) {
  if (!t->p) return fail(MUON_ERR_INVALID_ARG, "%s of %s is NULL", what, kQ[i]);
  if (t->batch_stride < 0 || t->token_stride < 0 || t->head_stride < 0)
    return fail(MUON_ERR_INVALID_ARG, "%s of %s has a negative stride", what, kQ[i]);
  if (!extent_ok(q->batch, t->batch_stride) || !extent_ok(q->tokens, t->token_stride) || !extent_ok(q->heads[i], t->head_stride))
    return fail(MUON_ERR_INVALID_ARG, "%s of %s reaches too far", what, kQ[i]);
  if ((uintptr_t)t->p % esize(dt)) return fail(MUON_ERR_INVALID_ARG, "%s of %s is not aligned to its element size", what, kQ[i]);
  return MUON_OK;
}

Span span_of(const muon_heads& t, int64_t heads, int32_t dt, const muon_qk_problem* q) {
  const int64_t last = (q->batch - 1) * t.batch_stride + (q->tokens - 1) * t.token_stride + (heads - 1) * t.head_stride + q->dim;
  return {(uintptr_t)t.p, (uintptr_t)t.p + (uintptr_t)(last * esize(dt))};
}

// No element of a strided tensor is another one's: sorted by stride, each
// stride reaches past everything the smaller ones cover.
bool self_disjoint(const muon_heads& t, int64_t heads, const muon_qk_problem* q) {
  struct D { int64_t stride, n; } d[3] = {{t.batch_stride, q->batch}, {t.token_stride, q->tokens}, {t.head_stride, heads}};
  std::sort(d, d + 3, [](const D& a, const D& b) { return a.stride < b.stride; });
  int64_t reach = q->dim;
  for (const D& x : d) {
    if (x.n <= 1) continue;
    if (x.stride < reach) return false;
    reach += (x.n - 1) * x.stride;
  }
  return true;
}

bool same_view(const muon_heads& a, const muon_heads& b, const muon_qk_problem* q, int64_t heads) {
  return a.p == b.p && (q->batch <= 1 || a.batch_stride == b.batch_stride) &&
         (q->tokens <= 1 || a.token_stride == b.token_stride) && (heads <= 1 || a.head_stride == b.head_stride);
}

// One index of a strided tensor: its stride in bytes and its first and last value.
struct Index { int64_t stride, lo, hi; };

// Whether `at` plus a multiple of every stride lies strictly between two
// bounds.  Largest stride first, each index is tried only where the smaller
// ones can still reach the bounds; more than `tries` of them count as a yes.
bool reaches(int64_t at, const Index* d, int n, int64_t above, int64_t below, int& tries) {
  if (n == 0) return at > above && at < below;
  int64_t lo = 0, hi = 0;  // what the smaller strides add
  for (int i = 1; i < n; ++i) { lo += d[i].lo * d[i].stride; hi += d[i].hi * d[i].stride; }
  const int64_t s = d[0].stride;
  if (s <= 0) return reaches(at, d + 1, n - 1, above, below, tries);
  auto floordiv = [](int64_t a, int64_t b) { return a / b - (a % b != 0 && a < 0); };
  const int64_t first = std::max(d[0].lo, floordiv(above - hi - at, s) + 1), last = std::min(d[0].hi, -floordiv(at + lo - below, s) - 1);
  for (int64_t k = first; k <= last; ++k) {
    if (--tries < 0) return true;
    if (reaches(at + k * s, d + 1, n - 1, above, below, tries)) return true;
  }
  return false;
}

// Whether two tensors may share a byte.  Views with the same strides, such as q
// and k in packed rows or in a heads-first buffer, are compared row by row: the
// distance of two head rows is that of the tensors plus a multiple of every
// stride.  Else views with the same token stride, each token's heads within it,
// are told apart by their place within that stride; others by their whole
// extent.
bool may_meet(const muon_heads& a, int64_t ha, const muon_heads& b, int64_t hb, int32_t dt, const muon_qk_problem* q) {
  const Span x = span_of(a, ha, dt, q), y = span_of(b, hb, dt, q);
  if (x.lo >= y.hi || y.lo >= x.hi) return false;
  const int64_t e = esize(dt);
  const struct { int64_t sa, sb, na, nb; } axes[3] = {{a.batch_stride, b.batch_stride, q->batch, q->batch},
                                                      {a.token_stride, b.token_stride, q->tokens, q->tokens},
                                                      {a.head_stride, b.head_stride, ha, hb}};
  Index ix[3];
  bool alike = true;
  for (int i = 0; i < 3; ++i) {
    alike &= axes[i].na <= 1 || axes[i].nb <= 1 || axes[i].sa == axes[i].sb;
    ix[i] = {(axes[i].na > 1 ? axes[i].sa : axes[i].sb) * e, 1 - axes[i].na, axes[i].nb - 1};
  }
  if (alike) {
    std::sort(ix, ix + 3, [](const Index& p, const Index& r) { return p.stride > r.stride; });
    int tries = 4096;
    return reaches((int64_t)(y.lo - x.lo), ix, 3, -q->dim * e, q->dim * e, tries);
  }
  // The stride between tokens; with one token per sequence, between sequences
  // (the stride of an axis of one entry means nothing).
  const bool one = q->tokens <= 1;
  const int64_t S = one ? a.batch_stride : a.token_stride, Sb = one ? b.batch_stride : b.token_stride;
  const int64_t wa = (ha - 1) * a.head_stride + q->dim, wb = (hb - 1) * b.head_stride + q->dim;
  if (S != Sb || S <= 0 || wa > S || wb > S || (one && q->batch <= 1)) return true;
  if (!one && q->batch > 1 && (a.batch_stride % S || b.batch_stride % S)) return true;
  const int64_t bytes = S * esize(dt);
  const int64_t d = (int64_t)((x.lo >= y.lo ? x.lo - y.lo : (uintptr_t)bytes - (y.lo - x.lo) % (uintptr_t)bytes) % (uintptr_t)bytes);
  return !(d >= wb * esize(dt) && d + wa * esize(dt) <= bytes);
}

// Whether a head row of `t` shares a byte with the range of `bytes` from p on.
bool meets_range(const muon_heads& t, int64_t heads, int32_t dt, const muon_qk_problem* q, const void* p, int64_t bytes) {
  if (!p || bytes <= 0 || !heads) return false;
  const int64_t e = esize(dt);
  Index d[3] = {{t.batch_stride * e, 0, q->batch - 1}, {t.token_stride * e, 0, q->tokens - 1}, {t.head_stride * e, 0, heads - 1}};
  std::sort(d, d + 3, [](const Index& a, const Index& b) { return a.stride > b.stride; });
  int tries = 4096;
  return reaches((int64_t)((uintptr_t)t.p - (uintptr_t)p), d, 3, -q->dim * e, bytes, tries);
}

// The outputs against the vectors: the weights, the positions, the frequencies,
// and, backward, the weights' gradients, which are outputs themselves.
int check_vectors(const muon_qk_problem* q, bool backward, bool norm) {
  struct Range { const char* name; const void* p; int64_t bytes; };
  const int64_t wb = q->dim * esize(q->weight_dtype), pe = q->positions_i64 ? 8 : 4;
  const int64_t pos = (q->axes - 1) * q->pos_axis_stride + (q->batch - 1) * q->pos_batch_stride + (q->tokens - 1) * q->pos_token_stride + 1;
  const bool rot = q->rotary_dim > 0;
  const Range in[] = {{"the weight of q", norm ? q->weight[0] : nullptr, wb},
                      {"the weight of k", norm ? q->weight[1] : nullptr, wb},
                      {"positions", rot ? q->positions : nullptr, pos * pe},
                      {"inv_freq", rot ? q->inv_freq : nullptr, q->rotary_dim / 2 * (int64_t)(q->inv_freq_f64 ? 8 : 4)}};
  for (int i = 0; i < 2; ++i) {
    for (const Range& r : in)
      if (meets_range(q->y[i], q->heads[i], q->dtype, q, r.p, r.bytes)) return fail(MUON_ERR_INVALID_ARG, "output of %s overlaps %s", kQ[i], r.name);
    const void* const dw = backward && norm ? q->dweight[i] : nullptr;
    if (!dw) continue;
    for (const Range& r : in)
      if (ranges_meet(dw, wb, r.p, r.bytes)) return fail(MUON_ERR_INVALID_ARG, "dweight of %s overlaps %s", kQ[i], r.name);
    for (int k = 0; k < 2; ++k)
      for (const muon_heads* t : {&q->x[k], &q->g[k], &q->y[k]})
        if (meets_range(*t, q->heads[k], q->dtype, q, dw, wb)) return fail(MUON_ERR_INVALID_ARG, "dweight of %s overlaps a tensor of %s", kQ[i], kQ[k]);
    if (i == 1 && ranges_meet(dw, wb, q->dweight[0], wb)) return fail(MUON_ERR_INVALID_ARG, "the dweights overlap");
  }
  return MUON_OK;
}

int check_qk(const muon_qk_problem* q, bool backward, bool norm) {
  if (!q) return fail(MUON_ERR_INVALID_ARG, "problem is NULL");
  if (q->batch < 0 || q->tokens < 0) return fail(MUON_ERR_INVALID_ARG, "negative batch or tokens");
  if (q->batch > kMaxSize || q->tokens > kMaxSize || q->batch * q->tokens > kMaxSize) return fail(MUON_ERR_INVALID_ARG, "more than 2^30 tokens");
  if (q->dim < 1 || q->dim > MUON_QK_MAX_DIM) return fail(MUON_ERR_INVALID_ARG, "dim %d is not in 1..%d", q->dim, MUON_QK_MAX_DIM);
  if (q->rotary_dim < 0 || q->rotary_dim % 2 || q->rotary_dim > q->dim || q->rotary_dim > 2 * kMaxPairs)
    return fail(MUON_ERR_INVALID_ARG, "rotary_dim %d must be even, at most dim %d and at most %d", q->rotary_dim, q->dim, 2 * kMaxPairs);
  if (q->axes < 1 || q->axes > kMaxAxes) return fail(MUON_ERR_INVALID_ARG, "axes must be in 1..%d", kMaxAxes);
  for (int i = 0; i < q->rotary_dim / 2; ++i)
    if (q->axis[i] >= q->axes) return fail(MUON_ERR_INVALID_ARG, "pair %d turns by axis %d of %d", i, q->axis[i], q->axes);
  if (!dtype_ok(q->dtype)) return fail(MUON_ERR_UNSUPPORTED, "dtype %d is not MUON_F32 or MUON_BF16", q->dtype);
  if (norm && !dtype_ok(q->weight_dtype)) return fail(MUON_ERR_UNSUPPORTED, "weight_dtype %d is not MUON_F32 or MUON_BF16", q->weight_dtype);
  if (!std::isfinite(q->scale)) return fail(MUON_ERR_INVALID_ARG, "scale must be finite");
  if (norm && !(std::isfinite(q->eps) && q->eps >= 0)) return fail(MUON_ERR_INVALID_ARG, "eps must be finite and >= 0");
  for (int i = 0; i < 2; ++i)
    if (q->heads[i] < 0 || q->heads[i] > 65536) return fail(MUON_ERR_INVALID_ARG, "heads must be in 0..65536");
  if (q->batch == 0 || q->tokens == 0 || (q->heads[0] == 0 && q->heads[1] == 0)) return MUON_OK;
  if (q->rotary_dim) {
    if (!q->positions) return fail(MUON_ERR_INVALID_ARG, "positions is NULL");
    if (!q->inv_freq) return fail(MUON_ERR_INVALID_ARG, "inv_freq is NULL");
    if ((uintptr_t)q->positions % (q->positions_i64 ? 8 : 4) || (uintptr_t)q->inv_freq % (q->inv_freq_f64 ? 8 : 4))
      return fail(MUON_ERR_INVALID_ARG, "positions or inv_freq is not aligned to its element size");
    if (q->pos_axis_stride < 0 || q->pos_batch_stride < 0 || q->pos_token_stride < 0) return fail(MUON_ERR_INVALID_ARG, "positions has a negative stride");
    if (!extent_ok(q->axes, q->pos_axis_stride) || !extent_ok(q->batch, q->pos_batch_stride) || !extent_ok(q->tokens, q->pos_token_stride))
      return fail(MUON_ERR_INVALID_ARG, "positions reach too far");
  }
  int rc;
  for (int i = 0; i < 2; ++i) {
    if (!q->heads[i]) continue;
    if (!(backward && !norm) && (rc = check_heads("input", i, &q->x[i], q->dtype, q))) return rc;
    if (backward && (rc = check_heads("gradient", i, &q->g[i], q->dtype, q))) return rc;
    if ((rc = check_heads("output", i, &q->y[i], q->dtype, q))) return rc;
    if (!self_disjoint(q->y[i], q->heads[i], q)) return fail(MUON_ERR_INVALID_ARG, "output of %s overlaps itself", kQ[i]);
    if (norm && q->weight[i] && (uintptr_t)q->weight[i] % esize(q->weight_dtype)) return fail(MUON_ERR_INVALID_ARG, "weight of %s is not aligned to its element size", kQ[i]);
  }
  for (int i = 0; i < 2; ++i) {
    if (!q->heads[i]) continue;
    for (int k = 0; k < 2; ++k) {
      if (!q->heads[k]) continue;
      const bool same = i == k;
      if (!(backward && !norm) && !(same && same_view(q->y[i], q->x[k], q, q->heads[i])) &&
          may_meet(q->y[i], q->heads[i], q->x[k], q->heads[k], q->dtype, q))
        return fail(MUON_ERR_INVALID_ARG, "output of %s overlaps the input of %s (only the same view is allowed)", kQ[i], kQ[k]);
      if (backward && !(same && same_view(q->y[i], q->g[k], q, q->heads[i])) &&
          may_meet(q->y[i], q->heads[i], q->g[k], q->heads[k], q->dtype, q))
        return fail(MUON_ERR_INVALID_ARG, "output of %s overlaps the gradient of %s (only the same view is allowed)", kQ[i], kQ[k]);
    }
  }
  if (q->heads[0] && q->heads[1] && may_meet(q->y[0], q->heads[0], q->y[1], q->heads[1], q->dtype, q))
    return fail(MUON_ERR_INVALID_ARG, "outputs of q and k overlap");
  return check_vectors(q, backward, norm);
}

// Launch geometry of one call: chunk size, tokens per wave item, row parts,
// workgroups.  It depends on the problem only, so results do too.
struct QkPlan { int vec, tw[2], parts[2], blocks[2]; };

QkPlan plan_qk(const muon_qk_problem* q, bool backward, bool norm) {
  QkPlan P{1, {1, 1}, {1, 1}, {0, 0}};
  const int64_t tokens = q->batch * q->tokens;
  // Largest chunk that divides the head and its rotated part in pairs and
  // whose every access is aligned (16 bytes at most per access).
  for (int vec : {8, 4, 2}) {
    if (vec * esize(q->dtype) > 16 || q->dim % (2 * vec) || q->rotary_dim % (2 * vec) || q->dim / (2 * vec) > 64) continue;
    const int64_t al = std::min<int64_t>(16, vec * esize(q->dtype));
    bool good = true;
    auto look = [&](const muon_heads& t, int64_t heads) {
      if (!heads) return;
      const int64_t e = esize(q->dtype);
      good &= (uintptr_t)t.p % al == 0 && (q->batch <= 1 || t.batch_stride * e % al == 0) &&
              (q->tokens <= 1 || t.token_stride * e % al == 0) && (heads <= 1 || t.head_stride * e % al == 0);
    };
    for (int i = 0; i < 2; ++i) {
      if (!(backward && !norm)) look(q->x[i], q->heads[i]);
      if (backward) look(q->g[i], q->heads[i]);
      look(q->y[i], q->heads[i]);
    }
    if (good) { P.vec = vec; break; }
  }
  const bool sums = backward && norm;
  // Weight sums keep one partial per workgroup: at most 1024 of them.
  for (int i = 0; i < 2; ++i) {
    if (!q->heads[i]) continue;
    if (P.vec == 1) {
      P.blocks[i] = (int)std::min<int64_t>(tokens, sums ? 1024 : 65536);
      continue;
    }
    const int nch = q->dim / (2 * P.vec);
    int lpr = 4;
    while (lpr < nch) lpr *= 2;
    const int rpw = 64 / lpr;
    // Tokens of one wave item: as many as fill four loads of the wave's lanes
    // (the token's angles are formed once per item), up to eight.
    P.tw[i] = std::max(1, std::min(8, 4 * rpw / q->heads[i]));
    if (q->rotary_dim) P.tw[i] = std::min(P.tw[i], 512 / (q->rotary_dim / 2));
    // few tokens: one each, and its heads over several waves
    while (P.tw[i] > 1 && cdiv(tokens, P.tw[i]) < 2048) P.tw[i] /= 2;
    const int64_t groups = cdiv(tokens, P.tw[i]);
    P.parts[i] = (int)std::max<int64_t>(1, std::min<int64_t>(cdiv((int64_t)P.tw[i] * q->heads[i], rpw), 2048 / groups));
    P.blocks[i] = (int)std::min<int64_t>(cdiv(groups * P.parts[i], 4), sums ? 1024 : 8192);
  }
  return P;
}

size_t qk_partial_bytes(const muon_qk_problem* q, const QkPlan& P) {
  return align256((size_t)(P.blocks[0] + P.blocks[1]) * q->dim * 4);
}

int run_qk(const muon_qk_problem* q, int mode, float sign, void* workspace, hipStream_t s) {
  const bool backward = sign < 0 || mode == 2;
  const QkPlan P = plan_qk(q, backward, mode != 0);
  QkParams p{};
  for (int i = 0; i < 2; ++i) {
    auto conv = [](const muon_heads& t) { return QkTensor{t.p, t.batch_stride, t.token_stride, t.head_stride}; };
    p.x[i] = conv(mode == 0 && backward ? q->g[i] : q->x[i]);
    p.g[i] = conv(q->g[i]);
    p.y[i] = conv(q->y[i]);
    p.heads[i] = q->heads[i];
    p.w[i] = mode ? q->weight[i] : nullptr;
  }
  p.w_dtype = q->weight_dtype;
  p.seq = q->tokens; p.tokens = q->batch * q->tokens;
  p.dim = q->dim; p.rot = q->rotary_dim;
  p.pos = q->positions; p.pos_i64 = q->positions_i64;
  p.pos_sa = q->pos_axis_stride; p.pos_sb = q->pos_batch_stride; p.pos_st = q->pos_token_stride;
  p.inv_freq = q->inv_freq; p.inv_freq_f64 = q->inv_freq_f64;
  p.scale = q->scale; p.sign = sign; p.eps = q->eps;
  p.partial = (float*)workspace;
  for (int i = 0; i < 2; ++i) { p.tw[i] = P.tw[i]; p.parts[i] = P.parts[i]; p.blocks[i] = P.blocks[i]; }
  for (int i = 0; i < q->rotary_dim / 2; ++i) p.axis[i] = q->axis[i];
  hipError_t e = launch_qk(p, mode, q->dtype == MUON_BF16, q->interleaved != 0, P.vec, s);
  if (e != hipSuccess) return hip_fail(e, "norm and rotation kernel");
  if (mode == 2 && (q->dweight[0] || q->dweight[1])) {
    e = launch_qk_weight_sum(p, q->dweight, q->weight_dtype, s);
    if (e != hipSuccess) return hip_fail(e, "norm weight gradients");
  }
  return ok();
}

bool qk_empty(const muon_qk_problem* q) {
  return q->batch == 0 || q->tokens == 0 || (q->heads[0] == 0 && q->heads[1] == 0);
}

}  // namespace

extern "C" {

int muon_qk_norm_rope(const muon_qk_problem* q, void* stream) {
  int rc = check_qk(q, false, true);
  if (rc) return rc;
  return qk_empty(q) ? ok() : run_qk(q, 1, 1.f, nullptr, (hipStream_t)stream);
}

int muon_rope(const muon_qk_problem* q, void* stream) {
  int rc = check_qk(q, false, false);
  if (rc) return rc;
  return qk_empty(q) ? ok() : run_qk(q, 0, 1.f, nullptr, (hipStream_t)stream);
}

int muon_rope_backward(const muon_qk_problem* q, void* stream) {
  int rc = check_qk(q, true, false);
  if (rc) return rc;
  return qk_empty(q) ? ok() : run_qk(q, 0, -1.f, nullptr, (hipStream_t)stream);
}

int muon_qk_norm_rope_backward_workspace_bytes(const muon_qk_problem* q, size_t* bytes) {
  if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
  int rc = check_qk(q, true, true);
  if (rc) return rc;
  *bytes = qk_empty(q) ? 0 : qk_partial_bytes(q, plan_qk(q, true, true));
  return ok();
}

int muon_qk_norm_rope_backward(const muon_qk_problem* q, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_qk(q, true, true);
  if (rc) return rc;
  for (int i = 0; i < 2; ++i)
    if (q->dweight[i] && (uintptr_t)q->dweight[i] % esize(q->weight_dtype))
      return fail(MUON_ERR_INVALID_ARG, "dweight of %s is not aligned to its element size", kQ[i]);
  if (qk_empty(q)) return ok();
  if ((rc = check_workspace(workspace, workspace_bytes, qk_partial_bytes(q, plan_qk(q, true, true))))) return rc;
  return run_qk(q, 2, -1.f, workspace, (hipStream_t)stream);
}

}  // extern "C"
