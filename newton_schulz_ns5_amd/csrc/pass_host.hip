// Host side of the operators around a layer's products: validation, workspace
// carve-up and launch sequences of the gradient norm and clipping, of the norms
// around a block and of the embedding with its gradient.  Every argument is
// checked before anything is enqueued.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "host_check.h"
#include "pass_internal.h"

using namespace muon;

namespace {

// ---- gradient norm and clipping -------------------------------------------------------
constexpr int64_t kMaxTensors = (int64_t)1 << 20;
// Workgroups of a launch.  The norm's partials are added by every workgroup of
// the clipping behind it: 1024 (3 GiB of bf16 normed in 466 us, by 512 in 456;
// clipped in 1748, and 1879 by 512 and 4096).
constexpr int kNormBlocks = 1024, kClipBlocks = 16384;

// Tensors [begin, end) of a list, one launch's: at most kListMax that are not
// empty, and 2^30 items.
struct ListPart { int64_t begin, end, items; };

int blocks_of(int64_t items, int most) { return (int)std::min<int64_t>(cdiv(items, 4), most); }

// Calls f(part) for every launch of a list.
template <class F>
int each_part(int64_t n, const int64_t* numel, F&& f) {
  ListPart part{0, 0, 0};
  int held = 0;
  auto flush = [&](int64_t at) {
    part.end = at;
    const int rc = part.items ? f(part) : MUON_OK;
    part = {at, at, 0};
    held = 0;
    return rc;
  };
  for (int64_t i = 0; i < n; ++i) {
    const int64_t items = cdiv(numel[i], kListItem);
    if (!items) continue;
    if (held == kListMax || part.items + items > ((int64_t)1 << 30)) {
      const int rc = flush(i);
      if (rc) return rc;
    }
    part.items += items;
    ++held;
  }
  return flush(n);
}

struct ListPlan { int64_t parts = 0, partials = 0; };
ListPlan plan_list(int64_t n, const int64_t* numel) {
  ListPlan P;
  each_part(n, numel, [&](const ListPart& part) {
    ++P.parts;
    P.partials += blocks_of(part.items, kNormBlocks);
    return MUON_OK;
  });
  return P;
}
// The partials, and their sum behind them.
size_t list_bytes(const ListPlan& P) { return align256((size_t)(P.partials + 1) * 8); }

int check_list(int64_t n, const int64_t* numel) {
  if (n < 0 || n > kMaxTensors) return fail(MUON_ERR_INVALID_ARG, "a list has 0 to 2^20 tensors, not %lld", (long long)n);
  if (n && !numel) return fail(MUON_ERR_INVALID_ARG, "numel is NULL");
  for (int64_t i = 0; i < n; ++i) {
    if (numel[i] < 0) return fail(MUON_ERR_INVALID_ARG, "tensor %lld has a negative size", (long long)i);
    if (numel[i] > ((int64_t)1 << 40)) return fail(MUON_ERR_INVALID_ARG, "tensor %lld has more than 2^40 elements", (long long)i);
  }
  return MUON_OK;
}

int check_tensors(const char* name, int64_t n, const void* const* p, const int32_t* dtype, const int64_t* numel) {
  if (n && (!p || !dtype)) return fail(MUON_ERR_INVALID_ARG, "the pointers or types of every %s are NULL", name);
  for (int64_t i = 0; i < n; ++i) {
    if (!dtype_ok(dtype[i])) return fail(MUON_ERR_UNSUPPORTED, "%s %lld: dtype %d is not MUON_F32 or MUON_BF16", name, (long long)i, dtype[i]);
    if (!numel[i]) continue;
    if (!p[i]) return fail(MUON_ERR_INVALID_ARG, "%s %lld is NULL", name, (long long)i);
    if ((uintptr_t)p[i] % esize(dtype[i])) return fail(MUON_ERR_INVALID_ARG, "%s %lld is not aligned to its element size", name, (long long)i);
  }
  return MUON_OK;
}

// No output shares a byte with another tensor or the scalars, but with its own
// input as a whole.
int check_apart(int64_t n, const void* const* x, const int32_t* xt, const int64_t* numel, void* const* y, const int32_t* yt,
                const void* total, int64_t total_bytes, const void* norm) {
  struct Span { uintptr_t lo, hi; int64_t tensor; bool out; };
  std::vector<Span> spans;
  spans.reserve((size_t)(2 * n + 2));
  auto add = [&](const void* p, int64_t bytes, int64_t i, bool out) {
    if (p && bytes) spans.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, i, out});
  };
  for (int64_t i = 0; i < n; ++i) {
    add(y[i], numel[i] * esize(yt[i]), i, true);
    if (!(x[i] == y[i] && xt[i] == yt[i])) add(x[i], numel[i] * esize(xt[i]), i, false);
  }
  add(total, total_bytes, -1, false);
  add(norm, 4, -2, true);
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  uintptr_t all = 0, outs = 0;  // ends of what came before
  for (const Span& s : spans) {
    if (s.lo < outs || (s.out && s.lo < all)) {
      if (s.tensor < 0) return fail(MUON_ERR_INVALID_ARG, "%s overlaps a tensor of the call", s.tensor == -1 ? "the given total" : "norm");
      return fail(MUON_ERR_INVALID_ARG, "%s %lld overlaps another tensor of the call", s.out ? "output" : "gradient", (long long)s.tensor);
    }
    all = std::max(all, s.hi);
    if (s.out) outs = std::max(outs, s.hi);
  }
  return MUON_OK;
}

void fill_list(TensorList& l, const ListPart& part, const void* const* x, const int32_t* xt, void* const* y, const int32_t* yt,
               const int64_t* numel) {
  l = TensorList{};
  int64_t items = 0;
  for (int64_t i = part.begin; i < part.end; ++i) {
    if (!numel[i]) continue;
    const int k = l.n++;
    l.x[k] = x[i];
    l.numel[k] = numel[i];
    if (xt[i] == MUON_BF16) l.x_bf16[k >> 6] |= (uint64_t)1 << (k & 63);
    if (y) {
      l.y[k] = y[i];
      if (yt[i] == MUON_BF16) l.y_bf16[k >> 6] |= (uint64_t)1 << (k & 63);
    }
    items += cdiv(numel[i], kListItem);
    l.end[k] = (int32_t)items;
  }
  l.items = (int32_t)items;
}

int check_kind(int32_t kind) {
  if (kind != MUON_NORM_2 && kind != MUON_NORM_MAX) return fail(MUON_ERR_UNSUPPORTED, "norm kind %d is not MUON_NORM_2 or MUON_NORM_MAX", kind);
  return MUON_OK;
}

// The partials of a list into the workspace.
int run_partials(int64_t n, const void* const* x, const int32_t* xt, const int64_t* numel, int32_t kind, uint64_t* partial, hipStream_t s) {
  return each_part(n, numel, [&](const ListPart& part) {
    NormPartial p;
    fill_list(p.list, part, x, xt, nullptr, nullptr, numel);
    const int blocks = blocks_of(part.items, kNormBlocks);
    p.partial = partial;
    p.max_norm_kind = kind == MUON_NORM_MAX;
    partial += blocks;
    const hipError_t e = launch_norm_partial(p, blocks, s);
    return e == hipSuccess ? MUON_OK : hip_fail(e, "gradient norm");
  });
}

int clip(int64_t n, const void* const* x, const int32_t* xt, const int64_t* numel, void* const* y, const int32_t* yt, int32_t kind,
         double max_norm, double eps, const void* total, int32_t total_f64, float* norm, void* workspace, size_t workspace_bytes, hipStream_t s) {
  int rc;
  if ((rc = check_list(n, numel)) || (rc = check_kind(kind)) || (rc = check_tensors("gradient", n, x, xt, numel)) ||
      (rc = check_tensors("output", n, (const void* const*)y, yt, numel)))
    return rc;
  if (!(max_norm >= 0)) return fail(MUON_ERR_INVALID_ARG, "max_norm must be >= 0");
  if (!(eps >= 0) || std::isinf(eps)) return fail(MUON_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (total_f64 != 0 && total_f64 != 1) return fail(MUON_ERR_INVALID_ARG, "total_f64 must be 0 or 1");
  if (total && total_f64 && kind != MUON_NORM_2) return fail(MUON_ERR_INVALID_ARG, "an fp64 total is a sum of squares, which MUON_NORM_MAX has not");
  if ((total && (uintptr_t)total % (total_f64 ? 8 : 4)) || (uintptr_t)norm % 4) return fail(MUON_ERR_INVALID_ARG, "norm or total is not aligned to its element size");
  if ((rc = check_apart(n, x, xt, numel, y, yt, total, total_f64 ? 8 : 4, norm))) return rc;
  const ListPlan P = plan_list(n, numel);
  NormTotal t{};
  t.total = total; t.total_f64 = total_f64;
  t.max_norm_kind = kind == MUON_NORM_MAX;
  t.norm = norm;
  if (!total && P.parts) {
    if ((rc = check_workspace(workspace, workspace_bytes, list_bytes(P)))) return rc;
    uint64_t* const partial = (uint64_t*)workspace;
    if ((rc = run_partials(n, x, xt, numel, kind, partial, s))) return rc;
    t.partial = partial; t.count = P.partials;
    // The partials of one launch are added by every workgroup of the next one
    // (one launch less); those of several once, in between.
    if (P.parts > 1) t.store = partial + P.partials;
  }
  if ((t.store || !P.parts) && (t.store || norm)) {
    const hipError_t e = launch_norm_total(t, s);
    if (e != hipSuccess) return hip_fail(e, "gradient norm");
    t.partial = t.store; t.count = 1;
    t.store = nullptr; t.norm = nullptr;
  }
  return each_part(n, numel, [&](const ListPart& part) {
    ClipParams p{};
    fill_list(p.list, part, x, xt, y, yt, numel);
    p.total = t;
    t.norm = nullptr;  // written once
    p.max_norm = max_norm; p.eps = eps;
    p.in_place = 1;
    for (int i = 0; i < p.list.n; ++i) p.in_place &= p.list.x[i] == p.list.y[i];
    const hipError_t e = launch_clip(p, blocks_of(part.items, kClipBlocks), s);
    return e == hipSuccess ? MUON_OK : hip_fail(e, "clipping");
  });
}

}  // namespace

extern "C" {

int muon_grad_norm_workspace_bytes(int64_t n, const int64_t* numel, size_t* bytes) {
  if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
  const int rc = check_list(n, numel);
  if (rc) return rc;
  const ListPlan P = plan_list(n, numel);
  *bytes = P.parts ? list_bytes(P) : 0;
  return ok();
}

int muon_grad_norm(int64_t n, const void* const* x, const int32_t* x_dtype, const int64_t* numel, int32_t kind, float* norm,
                   double* square, void* workspace, size_t workspace_bytes, void* stream) {
  int rc;
  if ((rc = check_list(n, numel)) || (rc = check_kind(kind)) || (rc = check_tensors("gradient", n, x, x_dtype, numel))) return rc;
  if (!norm && !square) return fail(MUON_ERR_INVALID_ARG, "norm and square are both NULL");
  if (square && kind != MUON_NORM_2) return fail(MUON_ERR_INVALID_ARG, "MUON_NORM_MAX has no sum of squares");
  if ((uintptr_t)norm % 4 || (uintptr_t)square % 8) return fail(MUON_ERR_INVALID_ARG, "norm or square is not aligned to its element size");
  if (ranges_meet(norm, 4, square, 8)) return fail(MUON_ERR_INVALID_ARG, "norm overlaps square");
  for (int64_t i = 0; i < n; ++i)
    if (ranges_meet(norm, 4, x[i], numel[i] * esize(x_dtype[i])) || ranges_meet(square, 8, x[i], numel[i] * esize(x_dtype[i])))
      return fail(MUON_ERR_INVALID_ARG, "norm or square overlaps gradient %lld", (long long)i);
  const ListPlan P = plan_list(n, numel);
  if (P.parts && (rc = check_workspace(workspace, workspace_bytes, list_bytes(P)))) return rc;
  if ((rc = run_partials(n, x, x_dtype, numel, kind, (uint64_t*)workspace, (hipStream_t)stream))) return rc;
  NormTotal t{};
  t.partial = (const uint64_t*)workspace; t.count = P.partials;
  t.max_norm_kind = kind == MUON_NORM_MAX;
  t.norm = norm; t.square = square;
  const hipError_t e = launch_norm_total(t, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "gradient norm");
}

int muon_clip_grad_norm(int64_t n, const void* const* x, const int32_t* x_dtype, const int64_t* numel, void* const* y,
                        const int32_t* y_dtype, int32_t kind, double max_norm, double eps, const void* total, int32_t total_f64,
                        float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  try {
    const int rc = clip(n, x, x_dtype, numel, y, y_dtype, kind, max_norm, eps, total, total_f64, norm, workspace, workspace_bytes,
                        (hipStream_t)stream);
    return rc ? rc : ok();
  } catch (const std::bad_alloc&) {
    return fail(MUON_ERR_INVALID_ARG, "out of host memory");
  }
}

}  // extern "C"

namespace {

// ---- norms around a block ----------------------------------------------------------------
constexpr int64_t kMaxNormRows = (int64_t)1 << 30;

int check_rows(const char* name, const void* p, int32_t dt, int64_t rows, int64_t cols, int64_t ld) {
  if (!p) return fail(MUON_ERR_INVALID_ARG, "%s is NULL", name);
  if (rows > 1 && ld < cols) return fail(MUON_ERR_INVALID_ARG, "%s row stride %lld is smaller than its %lld columns", name, (long long)ld, (long long)cols);
  if (rows > 1 && ld > ((int64_t)1 << 54) / 8 / (rows - 1)) return fail(MUON_ERR_INVALID_ARG, "%s reaches too far", name);
  if ((uintptr_t)p % esize(dt)) return fail(MUON_ERR_INVALID_ARG, "%s is not aligned to its element size", name);
  return MUON_OK;
}

// Gate rows are read gate_each rows long; 1 stands for one for all rows.
int64_t gate_each(const muon_residual_norm_problem* q) { return q->gate_rows > 1 ? q->rows / q->gate_rows : q->rows; }

int check_norms(const muon_residual_norm_problem* q, bool backward) {
  if (!q) return fail(MUON_ERR_INVALID_ARG, "problem is NULL");
  if (q->rows < 0 || q->cols < 0) return fail(MUON_ERR_INVALID_ARG, "negative rows or cols");
  if (q->rows > kMaxNormRows) return fail(MUON_ERR_INVALID_ARG, "rows must be at most 2^30");
  if (q->cols > kNormMaxCols) return fail(MUON_ERR_INVALID_ARG, "cols must be at most %d", kNormMaxCols);
  if (!dtype_ok(q->dtype) || !dtype_ok(q->stream_dtype)) return fail(MUON_ERR_UNSUPPORTED, "dtype and stream_dtype must be MUON_F32 or MUON_BF16");
  const bool weights = q->weight || q->post_weight || (backward && (q->dweight || q->dpost_weight));
  if (weights && !dtype_ok(q->weight_dtype)) return fail(MUON_ERR_UNSUPPORTED, "weight_dtype %d is not MUON_F32 or MUON_BF16", q->weight_dtype);
  if (q->gate && !dtype_ok(q->gate_dtype)) return fail(MUON_ERR_UNSUPPORTED, "gate_dtype %d is not MUON_F32 or MUON_BF16", q->gate_dtype);
  if ((q->norm != 0 && q->norm != 1) || (q->post_norm != 0 && q->post_norm != 1)) return fail(MUON_ERR_INVALID_ARG, "norm and post_norm must be 0 or 1");
  if (q->reserved) return fail(MUON_ERR_INVALID_ARG, "reserved must be 0");
  if (!std::isfinite(q->scale) || !std::isfinite(q->residual_scale) || !std::isfinite(q->weight_offset))
    return fail(MUON_ERR_INVALID_ARG, "scale, residual_scale and weight_offset must be finite");
  if (!(std::isfinite(q->eps) && q->eps >= 0)) return fail(MUON_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (q->gate && (q->gate_rows < 1 || q->rows % q->gate_rows)) return fail(MUON_ERR_INVALID_ARG, "gate_rows must divide the rows");
  if (q->weight && !q->norm) return fail(MUON_ERR_INVALID_ARG, "weight goes with norm");
  if (q->post_weight && !q->post_norm) return fail(MUON_ERR_INVALID_ARG, "post_weight goes with post_norm");
  if (backward) {
    if (!q->norm && !q->dstream) return fail(MUON_ERR_INVALID_ARG, "without a norm there is no gradient but dstream");
    if (q->dweight && !q->norm) return fail(MUON_ERR_INVALID_ARG, "dweight goes with norm");
    if (q->dpost_weight && !q->post_norm) return fail(MUON_ERR_INVALID_ARG, "dpost_weight goes with post_norm");
    if (q->dgate && !q->gate) return fail(MUON_ERR_INVALID_ARG, "dgate goes with a gate");
  }
  if (!q->rows || !q->cols) return MUON_OK;
  // Row tensors first, the vectors behind them.
  struct Tensor { const char* name; const void* p; int32_t dt; int64_t rows, ld; bool needed; };
  const int64_t R = q->rows;
  const bool need_b = q->post_norm || q->gate;
  const Tensor fin[] = {{"block", q->block, q->dtype, R, q->block_row_stride, true},
                        {"residual", q->residual, q->stream_dtype, R, q->residual_row_stride, false}};
  const Tensor fout[] = {{"stream", q->stream, q->stream_dtype, R, q->stream_row_stride, !q->norm},
                         {"y", q->norm ? q->y : nullptr, q->dtype, R, q->y_row_stride, q->norm != 0}};
  const Tensor bin[] = {{"block", need_b ? q->block : nullptr, q->dtype, R, q->block_row_stride, need_b},
                        {"stream", q->norm ? q->stream : nullptr, q->stream_dtype, R, q->stream_row_stride, q->norm != 0},
                        {"dy", q->norm ? q->dy : nullptr, q->dtype, R, q->dy_row_stride, q->norm != 0},
                        {"dstream", q->dstream, q->stream_dtype, R, q->dstream_row_stride, false}};
  const Tensor bout[] = {{"dblock", q->dblock, q->dtype, R, q->dblock_row_stride, false},
                         {"dresidual", q->dresidual, q->stream_dtype, R, q->dresidual_row_stride, false}};
  const Tensor vin[] = {{"weight", q->weight, q->weight_dtype, 1, q->cols, false},
                        {"post_weight", q->post_weight, q->weight_dtype, 1, q->cols, false},
                        {"gate", q->gate, q->gate_dtype, q->gate_rows, q->gate_row_stride, false}};
  const Tensor vout[] = {{"dweight", q->dweight, q->weight_dtype, 1, q->cols, false},
                         {"dpost_weight", q->dpost_weight, q->weight_dtype, 1, q->cols, false},
                         {"dgate", q->dgate, q->gate_dtype, q->gate_rows, q->dgate_row_stride, false}};
  const Tensor* const in = backward ? bin : fin;
  const Tensor* const out = backward ? bout : fout;
  const int nin = backward ? 4 : 2, nv = backward ? 3 : 0;
  int rc;
  auto look = [&](const Tensor& t) { return !t.p && !t.needed ? MUON_OK : check_rows(t.name, t.p, t.dt, t.rows, q->cols, t.ld); };
  for (int i = 0; i < nin; ++i)
    if ((rc = look(in[i]))) return rc;
  for (int i = 0; i < 2; ++i)
    if ((rc = look(out[i]))) return rc;
  for (const Tensor& t : vin)
    if ((rc = look(t))) return rc;
  for (int i = 0; i < nv; ++i)
    if ((rc = look(vout[i]))) return rc;
  auto span = [&](const Tensor& t) { return rows_of(t.name, t.p, t.dt, t.p ? t.rows : 0, q->cols, t.ld); };
  auto apart = [&](const Tensor& a, const Tensor& b, bool same_ok) {
    if (!a.p || !b.p) return MUON_OK;
    if (same_ok && a.p == b.p && a.dt == b.dt && (R <= 1 || a.ld == b.ld)) return MUON_OK;
    if (meet(span(a), span(b))) return fail(MUON_ERR_INVALID_ARG, "%s overlaps %s", a.name, b.name);
    return MUON_OK;
  };
  for (int o = 0; o < 2; ++o) {
    for (int i = 0; i < nin; ++i)
      if ((rc = apart(out[o], in[i], true))) return rc;
    for (const Tensor& t : vin)
      if ((rc = apart(out[o], t, false))) return rc;
  }
  if ((rc = apart(out[0], out[1], false))) return rc;
  for (int o = 0; o < nv; ++o) {
    for (int i = 0; i < nin; ++i)
      if ((rc = apart(vout[o], in[i], false))) return rc;
    for (int i = 0; i < 2; ++i)
      if ((rc = apart(vout[o], out[i], false))) return rc;
    for (const Tensor& t : vin)
      if ((rc = apart(vout[o], t, false))) return rc;
    for (int i = 0; i < o; ++i)
      if ((rc = apart(vout[o], vout[i], false))) return rc;
  }
  return MUON_OK;
}

// Workgroups of the gradients' kernels that a CU holds: four waves per SIMD,
// and a workgroup's waves are dealt out to the four SIMDs in turn.
int norm_resident(int threads) {
  const int waves = threads / 64;
  return waves < 4 ? 16 / waves : 4 / (int)cdiv(waves, 4);
}

// Launch geometry of the gradients; it depends on the sizes only.  A unit of rows
// belongs to one row of the gate, so gates of many sequences share the card out
// unevenly, and their partials are added by a workgroup for every 32 columns of
// every sequence.  8192 x 4096 in bf16 takes 96 us with a gate for all rows, 99 as
// 5 sequences, 166 as 256 (two partials each: 74 us of it in their sums), 127 as 300
// (one workgroup each, 212 of 512 idle), 96 as 512, 117 as 513 (one workgroup has
// two), 96 as 1024.
struct NormPlan {
  int blocks = 0;
  int64_t units = 0, unit_rows = 0, span = 0, gates = 0;
  int chunks = 1;
  size_t off[3] = {0, 0, 0}, bytes = 0;
  bool part[3] = {false, false, false};
};

NormPlan plan_norm_grad(const muon_residual_norm_problem* q) {
  NormPlan P;
  const NormShape shape = norm_shape(q->cols);
  const int threads = norm_threads(shape), rpw = norm_rows(shape);
  const int target = 256 * norm_resident(threads);
  const int64_t each = gate_each(q);
  const bool gate_sum = q->gate && (each > 1 || q->rows == 1);
  P.gates = gate_sum ? q->rows / each : 1;
  P.span = q->rows / P.gates;
  const int64_t chunks = std::min<int64_t>(cdiv(P.span, rpw), std::max<int64_t>(1, target / P.gates));
  P.unit_rows = cdiv(cdiv(P.span, chunks), rpw) * rpw;
  P.chunks = (int)cdiv(P.span, P.unit_rows);
  P.units = P.gates * P.chunks;
  P.blocks = (int)std::min<int64_t>(P.units, target);
  P.part[0] = q->dweight != nullptr;
  P.part[1] = q->dpost_weight != nullptr;
  P.part[2] = q->dgate && gate_sum && P.chunks > 1;
  for (int i = 0; i < 3; ++i) {
    if (!P.part[i]) continue;
    P.off[i] = P.bytes;
    P.bytes += align256((size_t)(i < 2 ? P.blocks : P.units) * q->cols * 4);
  }
  return P;
}

// groups: of threads, over all workgroups.
ResidualNorm norm_params(const muon_residual_norm_problem* q, bool backward, int64_t groups) {
  ResidualNorm p{};
  p.rows = q->rows; p.cols = (int32_t)q->cols;
  p.post = q->post_norm; p.norm = q->norm;
  p.block = q->block; p.ldb = q->block_row_stride;
  p.residual = q->residual; p.ldr = q->residual_row_stride;
  p.stream = q->stream; p.lds = q->stream_row_stride;
  p.y = q->y; p.ldy = q->y_row_stride;
  p.weight = q->weight; p.post_weight = q->post_weight; p.weight_bf16 = q->weight_dtype == MUON_BF16;
  p.gate = q->gate; p.ldg = q->gate_row_stride; p.gate_bf16 = q->gate_dtype == MUON_BF16;
  p.gate_each = gate_each(q);
  p.scale = q->scale; p.residual_scale = q->residual_scale; p.eps = q->eps; p.offset = q->weight_offset;
  // The vectors of every row in LDS where groups have several rows and those of
  // the workgroups that a CU holds fit its 160 KiB, beside what a workgroup has
  // for its sums.  8192 x 4096 in bf16 with three vectors: forward 49 us, read
  // again for every row 57; backward 97 and 110; with one 57 and 61.  Forward with
  // one: 43 and 42, but beside an fp32 stream (5105 x 2056) 26 and 28.  1024 rows,
  // one to a workgroup, forward with two: 10.3 us and 9.2.  The backward pass holds
  // the gate of a sequence too while it goes through its rows (5 of 1021 x 2050: 63
  // and 75).  All of calls behind each other on six sets of inputs in turn, whose
  // outputs share memory and stay in the caches in part: the forward pass into
  // memory of its own takes 54 us, a copy's rate.
  const NormShape shape = norm_shape(q->cols);
  const int64_t width = (int64_t)shape.group * shape.columns;
  const int vectors = (q->norm && q->weight) + (q->post_norm && q->post_weight) + (q->gate && (p.gate_each >= q->rows || (backward && p.gate_each > 1)));
  const int64_t held = 4 * width * vectors;
  if (backward && shape.columns == 16 && q->post_norm && q->gate) p.sums = (int32_t)(8 * width);
  const bool fits = (held + p.sums + (shape.group < 64 ? 8192 : 1024)) * norm_resident(norm_threads(shape)) <= 163840;
  p.held = fits && q->rows > groups && vectors > (backward || q->dtype != q->stream_dtype ? 0 : 1) ? (int32_t)held : 0;
  return p;
}

}  // namespace

extern "C" {

int muon_residual_norm(const muon_residual_norm_problem* q, void* stream) {
  const int rc = check_norms(q, false);
  if (rc) return rc;
  if (!q->rows || !q->cols) return ok();
  const NormShape shape = norm_shape(q->cols);
  const int threads = norm_threads(shape), rpw = norm_rows(shape);
  const int blocks = (int)std::min<int64_t>(cdiv(q->rows, rpw), 256 * (2048 / threads));
  const hipError_t e = launch_residual_norm(norm_params(q, false, (int64_t)blocks * rpw), q->dtype == MUON_BF16, q->stream_dtype == MUON_BF16, blocks, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "norms around a block");
}

int muon_residual_norm_backward_workspace_bytes(const muon_residual_norm_problem* q, size_t* bytes) {
  if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
  const int rc = check_norms(q, true);
  if (rc) return rc;
  *bytes = q->rows && q->cols ? plan_norm_grad(q).bytes : 0;
  return ok();
}

int muon_residual_norm_backward(const muon_residual_norm_problem* q, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_norms(q, true);
  if (rc) return rc;
  if (!q->rows || !q->cols) return ok();
  const NormPlan P = plan_norm_grad(q);
  if ((rc = check_workspace(workspace, workspace_bytes, P.bytes))) return rc;
  ResidualNorm p = norm_params(q, true, (int64_t)P.blocks * norm_rows(norm_shape(q->cols)));
  p.dy = q->dy; p.lddy = q->dy_row_stride;
  p.dstream = q->dstream; p.ldds = q->dstream_row_stride;
  p.dblock = q->dblock; p.lddb = q->dblock_row_stride;
  p.dresidual = q->dresidual; p.lddr = q->dresidual_row_stride;
  p.dgate = q->dgate; p.lddg = q->dgate_row_stride;
  for (int i = 0; i < 3; ++i) p.part[i] = P.part[i] ? (float*)((char*)workspace + P.off[i]) : nullptr;
  p.units = P.units; p.unit_rows = P.unit_rows; p.span = P.span; p.gate_chunks = P.chunks;
  hipError_t e = launch_residual_norm_grad(p, q->dtype == MUON_BF16, q->stream_dtype == MUON_BF16, P.blocks, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "gradients of the norms around a block");
  NormSums n{};
  void* const outs[3] = {q->dweight, q->dpost_weight, q->dgate};
  for (int i = 0; i < 3; ++i) {
    n.part[i] = p.part[i];
    n.out[i] = outs[i];
    n.ld[i] = i == 2 ? q->dgate_row_stride : 0;
    n.count[i] = i == 2 ? P.chunks : P.blocks;
    n.groups[i] = P.part[i] ? (i == 2 ? (int)P.gates : 1) : 0;
    n.bf16[i] = (i == 2 ? q->gate_dtype : q->weight_dtype) == MUON_BF16;
  }
  n.cols = (int32_t)q->cols;
  e = launch_norm_sums(n, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "gradients of the norms' vectors");
}

}  // extern "C"

namespace {

// ---- embedding ----------------------------------------------------------------------------
constexpr int64_t kMaxTokens = (int64_t)1 << 26, kMaxVocab = (int64_t)1 << 26, kMaxWidth = 65536;
constexpr int64_t kMaxGrid = (int64_t)1 << 24;  // workgroups of 256 threads: fewer than 2^32 in all

int check_embedding(const muon_embedding_problem* q, bool backward) {
  if (!q) return fail(MUON_ERR_INVALID_ARG, "problem is NULL");
  if (q->tokens < 0 || q->rows < 0 || q->dim < 0) return fail(MUON_ERR_INVALID_ARG, "negative tokens, rows or dim");
  if (q->tokens > kMaxTokens || q->rows > kMaxVocab) return fail(MUON_ERR_INVALID_ARG, "tokens and rows must be at most 2^26");
  if (q->dim > kMaxWidth) return fail(MUON_ERR_INVALID_ARG, "dim must be at most %lld", (long long)kMaxWidth);
  if (!dtype_ok(q->y_dtype) || !dtype_ok(q->w_dtype)) return fail(MUON_ERR_UNSUPPORTED, "w_dtype and y_dtype must be MUON_F32 or MUON_BF16");
  if (!std::isfinite(q->scale)) return fail(MUON_ERR_INVALID_ARG, "scale must be finite");
  for (int32_t f : {q->ids_i64, q->has_padding, q->accumulate})
    if (f != 0 && f != 1) return fail(MUON_ERR_INVALID_ARG, "ids_i64, has_padding and accumulate must be 0 or 1");
  if (q->reserved) return fail(MUON_ERR_INVALID_ARG, "reserved must be 0");
  int rc;
  if (q->tokens && q->dim) {
    if (!q->ids) return fail(MUON_ERR_INVALID_ARG, "ids is NULL");
    if ((uintptr_t)q->ids % (q->ids_i64 ? 8 : 4)) return fail(MUON_ERR_INVALID_ARG, "ids is not aligned to its element size");
    if ((rc = check_rows(backward ? "dy" : "y", q->y, q->y_dtype, q->tokens, q->dim, q->y_row_stride))) return rc;
  }
  if (backward && cdiv(q->tokens, kPieceMost) * cdiv(q->dim, kJoinCols) + cdiv(q->rows, kClearRows) >= kMaxGrid)
    return fail(MUON_ERR_INVALID_ARG, "tokens, rows and dim are too many together");
  const bool table = q->rows && q->dim && (backward || q->tokens);
  if (table && (rc = check_rows(backward ? "dw" : "w", q->w, q->w_dtype, q->rows, q->dim, q->w_row_stride))) return rc;
  if (!q->dim || !q->tokens) return MUON_OK;
  const Rows y = rows_of("y", q->y, q->y_dtype, q->tokens, q->dim, q->y_row_stride);
  const Rows w = rows_of("w", q->w, q->w_dtype, table ? q->rows : 0, q->dim, q->w_row_stride);
  Rows ids = rows_of("ids", q->ids, MUON_F32, 1, q->tokens, q->tokens);
  ids.width = ids.stride = q->tokens * (q->ids_i64 ? 8 : 4);
  if (meet(y, w)) return fail(MUON_ERR_INVALID_ARG, backward ? "dw overlaps dy" : "y overlaps w");
  if (meet(backward ? w : y, ids)) return fail(MUON_ERR_INVALID_ARG, backward ? "dw overlaps ids" : "y overlaps ids");
  return MUON_OK;
}

EmbedIds ids_of(const muon_embedding_problem* q) {
  return EmbedIds{q->ids, q->ids_i64, q->first, q->rows, q->padding, q->has_padding};
}

// How the gradient's tokens are sorted and summed; it depends on the sizes only.
struct EmbedPlan {
  bool ranked = false;
  int passes = 0, bits = 0, tiles = 0, scanned = 0;
  int piece = 0, sum_blocks = 0, col_blocks = 0;
  int64_t pieces = 0;
  size_t key[2] = {0, 0}, tok[2] = {0, 0}, hist = 0, totals = 0, slots = 0, bytes = 0;
};

EmbedPlan plan_embed(const muon_embedding_problem* q) {
  EmbedPlan P;
  const int64_t n = q->tokens;
  if (!n || !q->rows || !q->dim) return P;
  P.ranked = n <= kRankMost;
  int width = 1;  // bits of the largest key, which is `rows`
  while ((q->rows >> width) != 0) ++width;
  P.passes = (width + kSortBits - 1) / kSortBits;
  P.bits = (width + P.passes - 1) / P.passes;
  P.tiles = (int)cdiv(n, kSortTile);
  P.scanned = P.tiles > 64;
  const int chunk = embed_chunk(q->y_dtype == MUON_BF16, q->w_dtype == MUON_BF16);
  const int group = embed_group(q->dim, chunk), per = 256 / group;
  P.col_blocks = (int)cdiv(q->dim, chunk * group);
  // Long pieces leave few slots to join, short ones many workgroups.  32 tokens
  // where a row fills waves and there are many (8192 tokens of 4096: 218 us, by
  // 16: 223, by 64 of 65537: 89 for 75); rows that share a wave wait for each
  // other's stores, so theirs stay short (48435 tokens of 27: 12 us, by 32: 21).
  // Many is more than 4096, where the two do not cross: 4096 tokens of 512 over 1000
  // rows take 17.4 us, 4097 take 21.0.
  P.piece = group >= 64 && n > 4096 ? 2 * kPieceLeast : kPieceLeast;
  while (P.piece < kPieceMost && cdiv(cdiv(n, P.piece), per) * P.col_blocks > 4096) P.piece *= 2;
  P.pieces = cdiv(n, P.piece);
  P.sum_blocks = (int)(cdiv(P.pieces, per) * P.col_blocks);
  auto take = [&](size_t bytes) {
    const size_t at = P.bytes;
    P.bytes += align256(bytes);
    return at;
  };
  for (int i = 0; i < (P.ranked ? 1 : 2); ++i) {
    P.key[i] = take((size_t)n * 4);
    P.tok[i] = take((size_t)n * 4);
  }
  if (!P.ranked) {
    P.hist = take((size_t)P.tiles * kSortBins * 4);
    P.totals = take((size_t)kSortBins * 4);
  }
  P.slots = take((size_t)P.pieces * 2 * q->dim * 4);
  return P;
}

}  // namespace

extern "C" {

int muon_embedding(const muon_embedding_problem* q, void* stream) {
  const int rc = check_embedding(q, false);
  if (rc) return rc;
  if (!q->tokens || !q->dim) return ok();
  const Embed p{ids_of(q), q->tokens, (int32_t)q->dim, q->w, q->w_row_stride, q->y, q->y_row_stride, q->scale};
  const hipError_t e = launch_embed(p, q->w_dtype == MUON_BF16, q->y_dtype == MUON_BF16, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "embedding");
}

int muon_embedding_backward_workspace_bytes(const muon_embedding_problem* q, size_t* bytes) {
  if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
  const int rc = check_embedding(q, true);
  if (rc) return rc;
  *bytes = plan_embed(q).bytes;
  return ok();
}

int muon_embedding_backward(const muon_embedding_problem* q, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_embedding(q, true);
  if (rc) return rc;
  if (!q->rows || !q->dim || (!q->tokens && q->accumulate)) return ok();
  const EmbedPlan P = plan_embed(q);
  if ((rc = check_workspace(workspace, workspace_bytes, P.bytes))) return rc;
  const hipStream_t s = (hipStream_t)stream;
  char* const ws = (char*)workspace;
  hipError_t e;
  int from = 1;
  if (P.ranked) {
    EmbedSort p{};
    p.ids = ids_of(q);
    p.key_out = (uint32_t*)(ws + P.key[0]); p.tok_out = (uint32_t*)(ws + P.tok[0]);
    p.first_pass = 1;
    p.n = q->tokens;
    if ((e = launch_sort_rank(p, s)) != hipSuccess) return hip_fail(e, "token sort");
    from = 0;
  }
  for (int pass = 0; !P.ranked && pass < P.passes; ++pass) {
    EmbedSort p{};
    p.ids = ids_of(q);
    p.key_in = (const uint32_t*)(ws + P.key[from]); p.tok_in = (const uint32_t*)(ws + P.tok[from]);
    p.key_out = (uint32_t*)(ws + P.key[from ^ 1]); p.tok_out = (uint32_t*)(ws + P.tok[from ^ 1]);
    p.hist = (uint32_t*)(ws + P.hist); p.totals = (uint32_t*)(ws + P.totals);
    p.first_pass = pass == 0; p.shift = pass * P.bits; p.bits = P.bits; p.scanned = P.scanned;
    p.n = q->tokens;
    if ((e = launch_sort_hist(p, P.tiles, s)) != hipSuccess) return hip_fail(e, "token counts");
    if (P.scanned && (e = launch_sort_scan(p, P.tiles, s)) != hipSuccess) return hip_fail(e, "token counts");
    if ((e = launch_sort_scatter(p, P.tiles, s)) != hipSuccess) return hip_fail(e, "token sort");
    from ^= 1;
  }
  EmbedGrad g{};
  g.key = (const uint32_t*)(ws + P.key[from]); g.tok = (const uint32_t*)(ws + P.tok[from]);
  g.n = q->tokens; g.rows = q->rows; g.dim = (int32_t)q->dim; g.piece = P.piece ? P.piece : 1;
  g.dy = q->y; g.lddy = q->y_row_stride;
  g.dw = q->w; g.lddw = q->w_row_stride;
  g.scale = q->scale; g.accumulate = q->accumulate;
  g.slots = (float*)(ws + P.slots);
  g.sum_blocks = P.sum_blocks; g.col_blocks = P.col_blocks;
  const int clear = q->accumulate ? 0 : (int)cdiv(q->rows, kClearRows);
  e = launch_embed_grad(g, q->y_dtype == MUON_BF16, q->w_dtype == MUON_BF16, P.sum_blocks + clear, s);
  if (e != hipSuccess) return hip_fail(e, "embedding gradient");
  if (P.pieces > 1 && (e = launch_embed_join(g, q->w_dtype == MUON_BF16, s)) != hipSuccess) return hip_fail(e, "embedding gradient");
  return ok();
}

}  // extern "C"
