"""The operators around a layer's products in a pass: the embedding with its
gradient, the norms before and after a block with its gate and its residual,
the norm over all gradients and their clipping.

Marshalling like :mod:`layer_ops`, whose rules hold here too: raw pointers to
the library, work enqueued on the current stream of the tensors' device,
workspaces from torch's allocator for the one call, given outputs written in
place with their autograd version counters moved, tracers and forward-mode
inputs refused.
"""
import array
import ctypes
import functools
import math
import operator
import struct

import torch

from . import MuonError, _lib, _written
from ._lib import MUON_NORM_2, MUON_NORM_MAX
from .layer_ops import (_CODE, _NO_WORKSPACE, _Uneven, _bad, _call, _current_device, _dt, _dual, _given, _raw_stream,
                        _refuse_capture, _refuse_tangents, _rows, _same_device, _vector, _wants_grad)

__all__ = ["embedding", "embedding_backward", "residual_norm", "residual_norm_backward", "grad_norm", "clip_grad_norm"]


def _unsupported(text):
    raise MuonError(_lib.MUON_ERR_UNSUPPORTED, text)


def _on(dev, fn):
    """fn() with the device current."""
    if dev != _current_device():
        with torch.cuda.device(dev):
            return fn()
    return fn()


# ---- the embedding and its gradient ------------------------------------------------------
_EMBED = struct.Struct("@qqq P qq Pq Pq iiiiif q")


def _embed_pack(tokens, rows, dim, ids, first, padding, table, values, wcode, ycode, accumulate, scale):
    try:
        return _EMBED.pack(tokens, rows, dim, ids.data_ptr(), operator.index(first), operator.index(padding if padding is not None else 0),
                           *table, *values, wcode, ycode, ids.dtype is torch.int64, padding is not None, bool(accumulate), scale, 0)
    except (OverflowError, struct.error, TypeError):  # every other field is a size or an address
        _bad(f"first and padding_idx must be 64-bit integers and scale a number that fp32 holds, not {first!r}, {padding!r} and {scale!r}")


def _token_ids(ids):
    if ids.dtype not in (torch.int32, torch.int64):
        _unsupported(f"ids are {ids.dtype}, not int32 or int64")
    return ids if ids.is_contiguous() else ids.contiguous()


def embedding(ids, weight, *, scale=1.0, first=0, padding_idx=None, dtype=None, out=None):
    """``scale * weight[ids - first]``, and zeros for ids outside [first, first + rows) (see muon_embedding).

    ``ids`` is int32 or int64 of any shape, ``weight`` [rows, dim] in fp32 or bf16; the result [..., dim] has
    weight's type unless ``dtype`` or ``out`` says otherwise.  ``first`` is the first id of a shard of a vocabulary.
    ``padding_idx`` is an id that gives weight no gradient.
    """
    if _wants_grad(weight):
        if out is not None:
            _bad("out cannot be given when weight requires a gradient")
        _refuse_capture()
        return _Embedding.apply(ids, weight, scale, first, padding_idx, dtype)
    return _embedding(ids, weight, scale, first, padding_idx, dtype, out)


def _embedding(ids, weight, scale, first, padding_idx, dtype, out=None):
    given = () if out is None else _given(out)
    dev = _same_device(weight, ids, out)
    if weight.dim() != 2:
        _bad("weight must be [rows, dim]")
    wcode = _dt(weight)
    rows, dim = weight.shape
    ids = _token_ids(ids)
    weight, wp, ldw = _input_rows(weight, "weight", weight.shape)
    shape = ids.shape + (dim,)
    if out is None:
        out = weight.new_empty(shape) if dtype is None else torch.empty(shape, dtype=dtype, device=weight.device)
        y = out.data_ptr(), dim
    else:
        y = _output_rows(out, "out", shape, dtype or out.dtype)
    prob = _embed_pack(ids.numel(), rows, dim, ids, first, padding_idx, (wp, ldw), y, wcode, _dt(out), False, scale)
    _call(dev, _lib.lib().muon_embedding, prob, None)
    if given:
        _written(*given)
    return out


def embedding_backward(dy, ids, rows, *, scale=1.0, first=0, padding_idx=None, dw_dtype=None, dw=None, accumulate=False):
    """dw [rows, dim] of :func:`embedding` for the gradient ``dy`` of its result (see muon_embedding_backward).

    ``dw_dtype`` defaults to dy's type.  A given ``dw`` is written in place, and added to with ``accumulate``
    (rows without a token are then not touched).  No atomics: the same call gives the same bits.
    """
    _refuse_tangents(dy, dw)
    given = () if dw is None else _given(dw)
    dev = _same_device(dy, ids, dw)
    code = _dt(dy)
    if dy.dim() < 1 or dy.shape[:-1] != ids.shape:
        _bad(f"dy {tuple(dy.shape)} does not go with ids {tuple(ids.shape)}")
    if accumulate and dw is None:
        _bad("accumulate needs the tensor to add to")
    try:
        rows = operator.index(rows)
    except TypeError:
        _bad(f"rows must be an integer, not {rows!r}")
    if rows < 0:
        _bad("rows must not be negative")
    dim = dy.shape[-1]
    ids = _token_ids(ids)
    dy, dyp, lddy = _input_rows(dy, "dy", dy.shape)
    if dw is None:
        dw = torch.empty((rows, dim), dtype=dw_dtype or dy.dtype, device=dy.device)
    w = _output_rows(dw, "dw", (rows, dim), dw_dtype or dw.dtype)
    prob = _embed_pack(ids.numel(), rows, dim, ids, first, padding_idx, w, (dyp, lddy), _dt(dw), code, accumulate, scale)
    L = _lib.lib()
    _call(dev, L.muon_embedding_backward, prob, L.muon_embedding_backward_workspace_bytes, True)
    if given:
        _written(*given)
    return dw


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, weight, scale, first, padding_idx, dtype):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.dtype = weight.shape[0] if weight.dim() else 0, weight.dtype
        ctx.how = dict(scale=scale, first=first, padding_idx=padding_idx)
        return _embedding(ids, weight, scale, first, padding_idx, dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        _refuse_capture()
        ids, = ctx.saved_tensors
        return None, embedding_backward(_row_grad(dy), ids, ctx.rows, dw_dtype=ctx.dtype, **ctx.how), None, None, None, None


# ---- the norms before and after a block, its gate and its residual ---------------------
_NORM = struct.Struct("@qq iiiiii Pq Pq Pq Pq PP Pqq ffff Pq Pq Pq Pq PP Pq q")


def _input_rows(t, name, shape):
    """(tensor, pointer, row stride) of an input of this shape, copied where its rows are not evenly spaced or share
    elements."""
    if t.shape != shape:
        _bad(f"{name} is {tuple(t.shape)}, not {tuple(shape)}")
    if t.is_contiguous():
        return t, t.data_ptr(), shape[-1]
    if t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1 and t.numel():
        _bad(f"{name} needs unit column stride")
    try:
        p, r, c, ld = _rows(t, name)
        if r <= 1 or ld >= c:
            return t, p, ld
    except _Uneven:
        pass
    t = t.contiguous()
    p, _, _, ld = _rows(t, name)
    return t, p, ld


def _output_rows(t, name, shape, dtype):
    if t.shape != shape:
        _bad(f"{name} is {tuple(t.shape)}, not {tuple(shape)}")
    if t.dtype != dtype:
        _unsupported(f"{name} is {t.dtype}, not {dtype}")
    if t.is_contiguous():
        return t.data_ptr(), shape[-1]
    p, _, _, ld = _rows(t, name)
    return p, ld


def _gate_rows(gate, shape):
    """(tensor, pointer, rows, row stride) of a gate for rows of this shape: [cols], or as many dimensions as the
    rows have, of which the leading ones agree and the others are 1."""
    lead, own = shape[:-1], gate.shape[:-1]
    if gate.dim() < 1 or gate.shape[-1] != shape[-1]:
        _bad(f"gate {tuple(gate.shape)} does not go with rows {tuple(shape)}")
    if len(own):
        same = 0
        while same < len(lead) and same < len(own) and own[same] == lead[same]:
            same += 1
        if len(own) != len(lead) or any(n != 1 for n in own[same:]):
            _bad(f"gate {tuple(gate.shape)} does not go with rows {tuple(shape)}: its leading dimensions are theirs, then 1")
    t, p, ld = _input_rows(gate, "gate", gate.shape)
    return t, p, max(own.numel(), 1), ld


def _norm_vectors(weight, post_weight, cols):
    if weight is not None and post_weight is not None and weight.dtype != post_weight.dtype:
        _unsupported(f"weight is {weight.dtype} and post_weight {post_weight.dtype}: one type is needed")
    first = weight if weight is not None else post_weight
    return (_dt(first) if first is not None else 0, _vector(weight, "weight", cols) if weight is not None else 0,
            _vector(post_weight, "post_weight", cols) if post_weight is not None else 0)


def _pack_norm(*fields):
    try:
        return _NORM.pack(*fields)
    except (OverflowError, struct.error, TypeError):  # every other field is a size or an address
        _bad("scale, residual_scale, eps and weight_offset must be numbers that fp32 holds")


def _norm_flags(norm, post_norm, weight, post_weight):
    post = post_weight is not None if post_norm is None else bool(post_norm)
    if weight is not None and not norm:
        _bad("weight goes with norm")
    if post_weight is not None and not post:
        _bad("post_weight goes with post_norm")
    return bool(norm), post


def residual_norm(block, residual=None, *, weight=None, post_weight=None, gate=None, norm=True, post_norm=None,
                  scale=1.0, residual_scale=1.0, eps=1e-6, weight_offset=0.0, stream=None, out=None):
    """The join of a block with its residual stream and the norm before the next block (see muon_residual_norm):

    ``u = block``, or with ``post_norm`` (on when ``post_weight`` is given) its RMS norm times
    ``post_weight + weight_offset``; ``s = residual_scale * residual + scale * gate * u``; with ``norm``
    ``y = `` the RMS norm of ``s`` times ``weight + weight_offset``.  Returns (s, y); y is None without ``norm``.

    ``block`` is [..., cols] in fp32 or bf16 (y has its type), ``residual`` of the same shape, whose type, fp32 or
    bf16, the stream keeps.  Weights are [cols] (None: ones), ``gate`` is [cols], or has block's dimensions with
    trailing leading ones of 1 ([batch, 1, cols]: one per sequence; block's shape: one per row).  Columns are
    contiguous, rows of any stride; rows that share elements or are not evenly spaced are copied first.  Without
    a residual, a norm after the block, a gate and a scale the stream is ``block`` itself: the first norm of a
    model.  ``stream`` and ``out`` may be given, and be the inputs themselves; where ``out`` is written over such
    a block the stream is a copy of it.
    """
    if _wants_grad(block, residual, weight, post_weight, gate):
        if stream is not None or out is not None:
            _bad("stream and out cannot be given when an input requires a gradient")
        _refuse_capture()
        how = dict(norm=norm, post_norm=post_norm, scale=scale, residual_scale=residual_scale, eps=eps,
                   weight_offset=weight_offset)
        s, y = _ResidualNorm.apply(block, residual, weight, post_weight, gate, how)
        return (block if s is None else s), y
    return _residual_norm(block, residual, weight, post_weight, gate, norm, post_norm, scale, residual_scale, eps,
                          weight_offset, stream, out)


def _is_block(residual, gate, post, scale, stream):
    """Whether the stream is the block's output itself."""
    return residual is None and gate is None and not post and scale == 1 and stream is None


def _extent(t):
    """The addresses from the first to behind the last byte of t."""
    at = t.data_ptr()
    return at, at + (1 + sum((n - 1) * st for n, st in zip(t.shape, t.stride()))) * t.element_size() if t.numel() else at


def _written_over(out, source, read):
    """Whether writing out changes source, of which the library reads `read`: source itself, beside which it
    refuses every output that shares elements other than as a whole, or a copy, about which it knows nothing."""
    if read is source:
        return out.data_ptr() == source.data_ptr()
    (a, b), (c, d) = _extent(out), _extent(source)
    return a < d and c < b


def _residual_norm(block, residual, weight, post_weight, gate, norm, post_norm, scale, residual_scale, eps,
                   weight_offset, stream=None, out=None):
    norm, post = _norm_flags(norm, post_norm, weight, post_weight)
    given = () if stream is None and out is None else _given(stream, out)
    dev = _same_device(block, residual, weight, post_weight, gate, stream, out)
    code, shape = _dt(block), block.shape
    if not shape:
        _bad("block needs at least one dimension")
    cols = shape[-1]
    source = block
    block, bp, ldb = _input_rows(block, "block", shape)
    rp = ldr = gp = grows = ldg = gcode = wcode = wp = pwp = sp = lds = yp = ldy = 0
    if weight is not None or post_weight is not None:
        wcode, wp, pwp = _norm_vectors(weight, post_weight, cols)
    kept = residual
    if residual is not None:
        kept, rp, ldr = _input_rows(residual, "residual", shape)
    if gate is not None:
        gate, gp, grows, ldg = _gate_rows(gate, shape)
        gcode = _dt(gate)
    same = residual is None and _is_block(residual, gate, post, scale, stream)
    if same and out is not None and _written_over(out, source, block):
        same = False
    if same:
        stream, scode = source, code
    else:
        if stream is None:
            stream = (kept if residual is not None else block).new_empty(shape)
            sp, lds = stream.data_ptr(), cols
        else:
            sp, lds = _output_rows(stream, "stream", shape, residual.dtype if residual is not None else stream.dtype)
        scode = _dt(stream)
    if norm:
        if out is None:
            out = block.new_empty(shape)
            yp, ldy = out.data_ptr(), cols
        else:
            yp, ldy = _output_rows(out, "out", shape, block.dtype)
    elif out is not None:
        _bad("out goes with norm")
    if norm or not same:
        prob = _pack_norm(shape[:-1].numel(), cols, code, scode, wcode, gcode, post, norm, bp, ldb, rp, ldr, sp, lds,
                          yp, ldy, wp, pwp, gp, grows, ldg, scale, residual_scale, eps, weight_offset,
                          0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
        _call(dev, _lib.lib().muon_residual_norm, prob, None)
    if given:
        _written(*given)
    return stream, out


def residual_norm_backward(dy, dstream, stream, block, *, weight=None, post_weight=None, gate=None, norm=True,
                           post_norm=None, scale=1.0, residual_scale=1.0, eps=1e-6, weight_offset=0.0,
                           need_dblock=True, need_dresidual=True, need_dweight=None, need_dpost_weight=None,
                           need_dgate=None, dblock=None, dresidual=None):
    """(dblock, dresidual, dweight, dpost_weight, dgate) of :func:`residual_norm` for the gradients ``dy`` of y and
    ``dstream`` of the stream (either may be None); None for those not asked for.

    ``stream`` is what the forward pass returned (read where ``dy`` is), ``block`` its input (read with a norm
    after the block or a gate; may be None else).  The vectors' gradients are asked for by default where
    there is a vector.  Where dblock and dresidual are equal (no norm after the block, no gate, equal scales,
    one type) and neither is given, both are the same tensor.  Given outputs are written in place, and may be
    the input gradients themselves.
    """
    _refuse_tangents(dy, dstream, stream, block, weight, post_weight, gate)
    _, post = _norm_flags(norm, post_norm, weight, post_weight)
    if not norm and dy is not None:
        _bad("without norm there is no dy")
    norm = dy is not None  # a result that nothing depends on
    if dy is None and dstream is None:
        _bad("dy and dstream are both None")
    need_b = post or gate is not None
    if norm and stream is None:
        _bad("a gradient of the norm needs stream")
    if need_b and block is None:
        _bad("a norm after the block and a gate need block")
    given = () if dblock is None and dresidual is None else _given(dblock, dresidual)
    first = dy if dy is not None else dstream
    dev = _same_device(first, dstream, stream, block, weight, post_weight, gate, dblock, dresidual)
    shape, cols = first.shape, first.shape[-1] if first.dim() else _bad("gradients need at least one dimension")
    t = block.dtype if block is not None else dy.dtype if dy is not None else dblock.dtype if dblock is not None else dstream.dtype
    st = dstream.dtype if dstream is not None else stream.dtype
    for x, name, want in ((dy, "dy", t), (block, "block", t), (stream if norm else None, "stream", st)):
        if x is not None and x.dtype != want:
            _unsupported(f"{name} is {x.dtype}, not {want}")
    wcode, wp, pwp = _norm_vectors(weight, post_weight, cols)
    keep = []

    def rows(x, name, read):
        if x is None or not read:
            return 0, 0
        x, p, ld = _input_rows(x, name, shape)
        keep.append(x)
        return p, ld
    dyp, dsp, sp, bp = rows(dy, "dy", norm), rows(dstream, "dstream", True), rows(stream, "stream", norm), rows(block, "block", need_b)
    gp = grows = ldg = gcode = 0
    if gate is not None:
        gate_shape = gate.shape
        gate, gp, grows, ldg = _gate_rows(gate, shape)
        gcode = _dt(gate)
    device = first.device
    shared = (need_dblock and need_dresidual and not need_b and scale == residual_scale and t == st and dblock is None
              and dresidual is None)
    if dblock is None and need_dblock and not shared:
        dblock = torch.empty(shape, dtype=t, device=device)
    if dresidual is None and need_dresidual:
        dresidual = torch.empty(shape, dtype=st, device=device)
    dbp = _output_rows(dblock, "dblock", shape, t) if dblock is not None else (0, 0)
    drp = _output_rows(dresidual, "dresidual", shape, st) if dresidual is not None else (0, 0)
    dw = torch.empty_like(weight) if weight is not None and need_dweight is not False else None
    dpw = torch.empty_like(post_weight) if post_weight is not None and need_dpost_weight is not False else None
    dg = torch.empty(gate_shape, dtype=gate.dtype, device=device) if gate is not None and need_dgate is not False else None
    if (need_dweight and weight is None) or (need_dpost_weight and post_weight is None) or (need_dgate and gate is None):
        _bad("there is no vector to give the gradient of")
    dgp, lddg = _output_rows(dg, "dgate", gate_shape, gate.dtype) if dg is not None else (0, 0)
    if not norm and dw is not None:
        dw.zero_()
    nrows = shape[:-1].numel()
    if not nrows or not cols:  # empty sums, which the library has no work for
        for v in (dw, dpw, dg):
            if v is not None:
                v.zero_()
    prob = _pack_norm(nrows, cols, _CODE.get(t, -1), _CODE.get(st, -1), wcode, gcode, post, norm, *bp, 0, 0, *sp, 0, 0,
                      wp if norm else 0, pwp, gp, grows, ldg, scale, residual_scale, eps, weight_offset, *dyp, *dsp, *dbp,
                      *drp, dw.data_ptr() if dw is not None and norm else 0, dpw.data_ptr() if dpw is not None else 0,
                      dgp, lddg, 0)
    L = _lib.lib()
    _call(dev, L.muon_residual_norm_backward, prob, L.muon_residual_norm_backward_workspace_bytes, True)
    if given:
        _written(*given)
    return (dresidual if shared else dblock), dresidual, dw, dpw, dg


def _row_grad(g):
    """A gradient whose columns are contiguous (autograd may hand over expanded or transposed ones)."""
    return g if g is None or g.shape[-1] <= 1 or g.stride(-1) == 1 else g.contiguous()


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, block, residual, weight, post_weight, gate, how):
        s, y = _residual_norm(block, residual, weight, post_weight, gate, how["norm"], how["post_norm"], how["scale"],
                              how["residual_scale"], how["eps"], how["weight_offset"])
        same = s is block
        post = post_weight is not None if how["post_norm"] is None else bool(how["post_norm"])
        ctx.save_for_backward(block if post or gate is not None else None, s if how["norm"] else None, weight, post_weight, gate)
        ctx.how = how
        ctx.block_dtype = block.dtype
        ctx.set_materialize_grads(False)
        return (None if same else s), y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, ds, dy):
        if ds is None and dy is None:
            return (None,) * 6
        _refuse_capture()
        block, s, weight, post_weight, gate = ctx.saved_tensors
        need = ctx.needs_input_grad
        dblock = None
        if dy is None and block is None and need[0]:
            # only the stream's gradient: its type need not be the block's
            dblock = torch.empty(ds.shape, dtype=ctx.block_dtype, device=ds.device)
        got = residual_norm_backward(_row_grad(dy), _row_grad(ds), s, block, weight=weight, post_weight=post_weight, gate=gate,
                                     need_dblock=need[0], need_dresidual=need[1], need_dweight=need[2],
                                     need_dpost_weight=need[3], need_dgate=need[4], dblock=dblock, **ctx.how)
        return got + (None,)


# ---- the norm over all gradients, and clipping ---------------------------------------
def _norm_kind(norm_type):
    if norm_type == 2:
        return MUON_NORM_2
    if norm_type == math.inf or norm_type == "inf":
        return MUON_NORM_MAX
    _unsupported(f"norm_type {norm_type!r} is not 2 or inf")


_is_none = functools.partial(operator.is_, None)


def _tensors(grads):
    if isinstance(grads, torch.Tensor):
        return [grads]
    ts = list(grads)
    return [t for t in ts if t is not None] if any(map(_is_none, ts)) else ts


def _dense(t):
    """Whether t's elements lie side by side in memory, in whatever order of its dimensions."""
    if t.layout is not torch.strided:
        _unsupported(f"a tensor is {t.layout}, not strided")
    if t.is_contiguous():
        return True
    n = 1
    for stride, size in sorted((st, sz) for st, sz in zip(t.stride(), t.shape) if sz != 1):
        if stride != n:
            return False
        n *= size
    return True


# What is asked of every tensor of a list, without an attribute lookup for each.
_data_ptr, _numel, _get_device, _is_contiguous = (torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.get_device,
                                                  torch.Tensor.is_contiguous)
_dtype, _shape, _needs_grad = (operator.attrgetter(n) for n in ("dtype", "shape", "requires_grad"))


def _list_device(*lists):
    """The index of the one GPU that holds every tensor of the lists (the first is not empty)."""
    first = lists[0][0]
    dev = _same_device(first)
    for ts in lists:
        if set(map(_get_device, ts)) - {dev}:
            _same_device(first, *ts)
    return dev


def _table(ts, sizes=True):
    """(count, pointers, types, sizes) of a list as the library takes them."""
    n = len(ts)
    codes = list(map(_CODE.get, map(_dtype, ts)))
    if None in codes:
        _unsupported(f"dtype {ts[codes.index(None)].dtype} is not float32 or bfloat16")
    try:
        pointers = array.array("Q", map(_data_ptr, ts)).tobytes()
    except (RuntimeError, NotImplementedError):
        _unsupported("tensors must be strided (dense in memory)")
    return n, pointers, array.array("i", codes).tobytes(), array.array("q", map(_numel, ts)).tobytes() if sizes else None


# Bytes that the partials of a list of one launch fit (up to 128 tensors).
_ONE_LAUNCH, _ONE_LAUNCH_BYTES = 128, 8448


def _norm_workspace(n, sizes, device):
    if n <= _ONE_LAUNCH:
        return torch.empty(_ONE_LAUNCH_BYTES, dtype=torch.uint8, device=device)
    need = ctypes.c_size_t(0)
    _lib.check(_lib.lib().muon_grad_norm_workspace_bytes(n, sizes, ctypes.byref(need)))
    return torch.empty(max(need.value, 1), dtype=torch.uint8, device=device)


def _no_gradients(dtype=torch.float32):
    return torch.zeros((), dtype=dtype, device="cuda" if torch.cuda.is_available() else "cpu")


def grad_norm(grads, *, norm_type=2, squared=False):
    """The norm over all tensors of ``grads`` as one vector, a 0-dim fp32 tensor on their device (see muon_grad_norm).

    ``grads`` is a tensor or an iterable of fp32 and bf16 tensors of any shapes on one device (None entries
    are skipped).  ``norm_type`` is 2 or inf (the largest magnitude).  ``squared=True`` gives the sum of squares
    instead, in fp64: what ranks that hold different gradients add up (``all_reduce``) before
    :func:`clip_grad_norm` takes it as its ``total``.  Nothing synchronizes.  The result carries no gradient:
    tensors that require one are refused while gradients are recorded.
    """
    kind = _norm_kind(norm_type)
    if squared and kind != MUON_NORM_2:
        _bad("squared goes with norm_type 2")
    ts = _tensors(grads)
    if not ts:
        return _no_gradients(torch.float64 if squared else torch.float32)
    dev = _list_device(ts)
    if _dual["_current_level"] >= 0:
        _refuse_tangents(*ts)
    if torch.is_grad_enabled() and any(map(_needs_grad, ts)):
        _unsupported("the norm carries no gradient: detach the tensors")
    if not all(map(_is_contiguous, ts)):
        ts = [t if _dense(t) else t.contiguous() for t in ts]
    n, ptrs, codes, sizes = _table(ts)
    out = torch.empty((), dtype=torch.float64 if squared else torch.float32, device=ts[0].device)
    at = (None, out.data_ptr()) if squared else (out.data_ptr(), None)

    def call():
        ws = _norm_workspace(n, sizes, out.device)
        _lib.check(_lib.lib().muon_grad_norm(n, ptrs, codes, sizes, kind, *at, ws.data_ptr(), ws.numel(), _raw_stream(dev)))
    _on(dev, call)
    return out


def clip_grad_norm(grads, max_norm, *, norm_type=2, eps=1e-6, total=None, out=None):
    """Scales every tensor of ``grads`` by ``max_norm / (norm + eps)`` where their norm plus eps is above
    ``max_norm``, and returns the norm, a 0-dim fp32 tensor (see muon_clip_grad_norm).

    In place, or into the tensors of ``out`` (one for each of ``grads``, of its shape and memory order, fp32 or
    bf16).  ``norm_type`` as for :func:`grad_norm`.  ``total``, a 0-dim tensor on the device, stands for the
    norm of the tensors given: an fp32 one is the norm itself, an fp64 one the sum of squares, e.g. of all
    ranks.  Nothing synchronizes: a NaN norm makes the gradients NaN, an infinite one zero (NaN where they are
    infinite).  The same tensor twice, or tensors that overlap, are refused.
    """
    kind = _norm_kind(norm_type)
    if out is not None:
        grads, out = _pair(grads, out)
    ts = _tensors(grads)
    outs = ts if out is None else out
    if total is not None:
        if total.numel() != 1 or total.dtype not in (torch.float32, torch.float64):
            _bad("total must be one fp32 or fp64 value")
        if total.dtype is torch.float64 and kind != MUON_NORM_2:
            _bad("an fp64 total is a sum of squares, which goes with norm_type 2")
    try:
        max_norm, eps = float(max_norm), float(eps)
    except (TypeError, ValueError):
        _bad(f"max_norm and eps must be numbers, not {max_norm!r} and {eps!r}")
    if not ts:
        return _no_gradients() if total is None else (total.sqrt().float() if total.dtype is torch.float64 else total.clone()).reshape(())
    dev = _list_device(ts, outs) if total is None else _list_device(ts, outs, [total])
    if _dual["_current_level"] >= 0:
        _refuse_tangents(*ts, *outs, total)
    if torch.is_grad_enabled() and any(map(_needs_grad, ts)):
        if out is None:
            _bad("a gradient to be written requires a gradient itself: detach it")
        _unsupported("clipped gradients carry no gradient: detach the tensors")
    whole = all(map(_is_contiguous, ts))
    if not whole and not all(map(_dense, ts)):
        _bad("a gradient's elements do not lie side by side: it cannot be scaled as a whole")
    if out is not None:
        _given(*outs)
        if list(map(_shape, ts)) != list(map(_shape, outs)):
            _bad("an output has not its gradient's shape")
        if not (whole and all(map(_is_contiguous, outs))):
            for t, o in zip(ts, outs):
                if not (t.is_contiguous() and o.is_contiguous()) and t.stride() != o.stride():
                    _bad("an output's memory order is not its gradient's")
    n, ptrs, codes, sizes = _table(ts)
    optrs, ocodes = (ptrs, codes) if out is None else _table(outs, False)[1:3]
    norm = torch.empty((), dtype=torch.float32, device=ts[0].device)

    def call():
        ws = _norm_workspace(n, sizes, norm.device) if total is None else None
        _lib.check(_lib.lib().muon_clip_grad_norm(
            n, ptrs, codes, sizes, optrs, ocodes, kind, max_norm, eps, total.data_ptr() if total is not None else None,
            int(total is not None and total.dtype is torch.float64), norm.data_ptr(),
            ws.data_ptr() if ws is not None else _NO_WORKSPACE, ws.numel() if ws is not None else 0, _raw_stream(dev)))
    _on(dev, call)
    _written(*outs)
    return norm


def _pair(grads, out):
    grads, out = ([t] if isinstance(t, torch.Tensor) else list(t) for t in (grads, out))
    if len(grads) != len(out):
        _bad(f"{len(out)} outputs for {len(grads)} gradients")
    if any(map(_is_none, grads)):
        out = [o for g, o in zip(grads, out) if g is not None]
    if any(map(_is_none, out)):
        _bad("a gradient has no output")
    return grads, out
