"""Layer operators: the linear product with bias, activation and residual, the
per-head norms of queries and keys with the position rotation, the rotation
alone, and the gradients of each.

Thin marshalling like the rest of the binding: shapes and strides in, raw
pointers to the library, work enqueued on the current stream.  ``linear``,
``qk_norm_rope`` and ``rope`` record themselves for autograd when an input
requires a gradient; the ``*_backward`` entry points are the same gradients
called directly, and their results carry no gradient of their own.  Inputs of
forward-mode differentiation are refused.
"""
import ctypes
import operator
import struct

import torch
from torch.autograd import forward_ad as _forward_ad

from . import MuonError, _lib, _written
from ._lib import MUON_BF16, MUON_F32

__all__ = ["linear", "linear_backward", "qk_norm_rope", "qk_norm_rope_backward", "rope", "rope_backward",
           "ACTIVATIONS"]

ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "relu2": 2, "silu": 3, "gelu": 4, "gelu_tanh": 5}


def _bad(text):
    raise MuonError(_lib.MUON_ERR_INVALID_ARG, text)


def _act(name):
    try:
        return ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise MuonError(_lib.MUON_ERR_UNSUPPORTED, f"activation {name!r} is not one of {sorted(filter(None, ACTIVATIONS))}")


_CODE = {torch.float32: MUON_F32, torch.bfloat16: MUON_BF16}

# The problem structures of the C ABI, packed in one call each (setting a
# ctypes structure field by field costs more than the kernel of a small call).
_LINEAR = struct.Struct("@qqq ii Pq Pq P Pq Pq Pq iiii")
_GRAD = struct.Struct("@qqq ii Pq Pq Pq Pq Pq Pq P iiiiii")
_QK = struct.Struct("@qq iiiiii " + "Pqqq" * 6 + " PPPP Pqqq P iiii ff 256s")


def _dt(t):
    code = _CODE.get(t.dtype)
    if code is None:
        raise MuonError(_lib.MUON_ERR_UNSUPPORTED, f"dtype {t.dtype} is not float32 or bfloat16")
    return code


_tracing_state = torch._C._get_tracing_state
_dispatch_modes = torch._C._len_torch_dispatch_stack


def _refuse_tracing():
    """A tracer records the allocation of a result but not the launch that writes
    it: its replays would return memory that nobody wrote."""
    if _tracing_state() is not None:
        raise MuonError(_lib.MUON_ERR_UNSUPPORTED, "torch.jit.trace cannot record this operator")
    from torch.fx.experimental.proxy_tensor import get_proxy_mode
    if get_proxy_mode() is not None:
        raise MuonError(_lib.MUON_ERR_UNSUPPORTED, "torch.fx tracing cannot record this operator")


def _same_device(first, *others):
    """The index of the one GPU that holds every tensor."""
    if _tracing_state() is not None or _dispatch_modes():
        _refuse_tracing()
    dev = first.get_device()
    if dev < 0:
        _bad(f"tensors must be on a GPU, got {first.device}")
    for t in others:
        if t is not None and t.get_device() != dev:
            _bad(f"tensors are on {t.device} and {first.device}")
    return dev


# The raw handle of a device's current stream (what current_stream().cuda_stream
# gives, without making a Stream object).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)  # tensors on a GPU: it is initialised


def _call(dev, fn, problem, need, likely=False):
    """Run fn(problem[, workspace]) on the device's current stream.  The device
    is made current for the launch when another one is.  likely: the call will
    want a workspace."""
    if dev != _current_device():
        with torch.cuda.device(dev):
            return _call_here(dev, fn, problem, need, likely)
    return _call_here(dev, fn, problem, need, likely)


_NO_WORKSPACE = 256  # an aligned address that stands for an empty workspace


def _call_here(dev, fn, problem, need, likely):
    if need is None:
        return _lib.check(fn(problem, _raw_stream(dev)))
    if not likely:
        # Most small calls need no workspace: an empty one is offered first, and the
        # library, which enqueues nothing without what it needs, says if it is too small.
        status = fn(problem, _NO_WORKSPACE, 0, _raw_stream(dev))
        if status != _lib.MUON_ERR_WORKSPACE:
            return _lib.check(status)
    size = ctypes.c_size_t(0)
    _lib.check(need(problem, ctypes.byref(size)))
    # Taken from torch's allocator for this call: it goes back to the stream that
    # runs the call, and one taken under capture belongs to that graph alone.
    ws = torch.empty(max(size.value, 1), dtype=torch.uint8, device=torch.device("cuda", dev))
    return _lib.check(fn(problem, ws.data_ptr(), size.value, _raw_stream(dev)))


# ---- the linear product ---------------------------------------------------------------
class _Uneven(MuonError):
    """Rows that are not one stride apart."""


def _rows(t, name, cols=None):
    """(pointer, rows, columns, row stride) of a [..., columns] tensor seen as rows."""
    if t.dim() < 1:
        _bad(f"{name} needs at least one dimension")
    if t.dim() != 2:
        try:
            t = t.view(-1, t.shape[-1]) if t.numel() else t.reshape(-1, t.shape[-1]) if t.shape[-1] else \
                t.new_empty((t.shape[:-1].numel(), 0))
        except RuntimeError:
            raise _Uneven(_lib.MUON_ERR_INVALID_ARG, f"the leading dimensions of {name} cannot be seen as one")
    (r, c), (row, col) = t.shape, t.stride()
    if cols is not None and c != cols:
        _bad(f"{name} has {c} columns, not {cols}")
    if col != 1 and r and c > 1:
        _bad(f"{name} needs unit column stride")
    return t.data_ptr(), r, c, (row if r > 1 and c else c)


# Elements that rows may be apart for the library (2^23 - 32 bytes).
_FAR = {MUON_F32: (2 ** 23 - 32) // 4, MUON_BF16: (2 ** 23 - 32) // 2}


def _input(t, name, cols=None):
    """(tensor, pointer, rows, columns, row stride) of an input seen as rows.  The
    tensor is t, or a copy where the library cannot take its rows: leading
    dimensions that are not one, rows that share elements (expanded), rows too
    far apart (one token of every long sequence, h[:, -1]).  The caller holds it
    until the launch."""
    try:
        p, r, c, ld = _rows(t, name, cols)
        if r <= 1 or (c <= ld and (ld <= 1 << 20 or ld <= _FAR[_dt(t)])):
            return t, p, r, c, ld
    except _Uneven:
        if t.stride(-1) != 1:
            _bad(f"{name} needs unit column stride")
    t = t.contiguous()
    return (t, *_rows(t, name, cols))


def _input_matrix(t, name, rows, cols):
    t, p, r, c, ld = _input(t, name)
    if (r, c) != (rows, cols):
        _bad(f"{name} is [{r}, {c}], not [{rows}, {cols}]")
    return t, p, ld


def _vector(t, name, n):
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        _bad(f"{name} must be a contiguous [{n}] tensor")
    return t.data_ptr()


def _check_matrix(t, name, rows, cols):
    p, r, c, ld = _rows(t, name)
    if (r, c) != (rows, cols):
        _bad(f"{name} is [{r}, {c}], not [{rows}, {cols}]")
    return p, ld


def _refuse_capture():
    if torch.cuda.is_current_stream_capturing():
        raise MuonError(_lib.MUON_ERR_UNSUPPORTED,
                        "autograd is not recorded under stream capture: call the *_backward entry point there")


# Where the level of forward-mode differentiation stands (below 0: none is open).
_dual = vars(_forward_ad) if "_current_level" in vars(_forward_ad) else {"_current_level": 0}


def _refuse_tangents(*ts):
    """These operators have no forward-mode derivative: a result would silently come without its tangent."""
    if _dual["_current_level"] >= 0:
        for t in ts:
            if t is not None and _forward_ad.unpack_dual(t).tangent is not None:
                raise MuonError(_lib.MUON_ERR_UNSUPPORTED, "forward-mode automatic differentiation is not supported")


def _wants_grad(*ts):
    """Whether to record the call for autograd."""
    if _dual["_current_level"] >= 0:
        _refuse_tangents(*ts)
    if torch.is_grad_enabled():
        for t in ts:
            if t is not None and t.requires_grad:
                return True
    return False


def _refuse_frequency_gradient(inv_freq):
    """The frequencies are constants of the rotation."""
    if inv_freq.requires_grad:
        raise MuonError(_lib.MUON_ERR_UNSUPPORTED, "inv_freq has no gradient here: detach it")


def _given(*outs):
    """The outputs that the caller gave.  Writing into one that is part of an
    autograd graph would leave its old history on it."""
    outs = [t for t in outs if t is not None]
    for t in outs:
        if t.requires_grad and torch.is_grad_enabled():
            _bad("a given output requires a gradient: detach it")
    return outs


def linear(x, w, bias=None, residual=None, *, activation=None, return_preact=False, out=None, preact=None):
    """``activation(x @ w.T + bias) + residual`` for x [..., k] and w [n, k] (see muon_linear).

    Columns are contiguous, rows of any stride.  Inputs whose rows share elements (expanded), are 8 MiB or
    more apart, or are not evenly spaced are copied first.

    ``activation`` is None, "relu", "relu2", "silu", "gelu" or "gelu_tanh".
    The result has the residual's type, or x's without one, unless ``out`` is
    given (``out`` may be the residual).  ``return_preact=True`` returns
    (y, x @ w.T + bias), the second in x's type, which
    :func:`linear_backward` takes when there is an activation.  Both carry
    gradients.
    """
    if _wants_grad(x, w, bias, residual):
        if out is not None or preact is not None:
            _bad("out and preact cannot be given when an input requires a gradient")
        _refuse_capture()
        y, z = _Linear.apply(x, w, bias, residual, activation, return_preact)
        return (y, z) if return_preact else y
    return _linear(x, w, bias, residual, activation, return_preact, out, preact)


def _linear(x, w, bias, residual, activation, return_preact, out=None, preact=None):
    act = _act(activation)
    given = () if out is None and preact is None else _given(out, preact)
    dev = _same_device(x, w, bias, residual, out, preact)
    code = _dt(x)
    if w.dtype != x.dtype:
        raise MuonError(_lib.MUON_ERR_UNSUPPORTED, f"x is {x.dtype} and w {w.dtype}: one type is needed")
    if w.dim() != 2:
        _bad("w must be [n, k]")
    w, wp, n, k, ldw = _input(w, "w")
    x, xp, m, _, ldx = _input(x, "x", k)
    shape = x.shape[:-1] + (n,)
    if out is None:
        out = (x if residual is None else residual).new_empty(shape)
    if (return_preact or preact is not None):
        if preact is None:
            preact = x.new_empty(shape)
        elif preact.dtype != x.dtype:
            raise MuonError(_lib.MUON_ERR_UNSUPPORTED, f"preact must be {x.dtype} like x")
    yp, ldy = _check_matrix(out, "out", m, n)
    zp, ldz = _check_matrix(preact, "preact", m, n) if preact is not None else (0, 0)
    rp, ldr = 0, 0
    if residual is out and out is not None:
        rp, ldr = yp, ldy
    elif residual is not None:
        residual, rp, ldr = _input_matrix(residual, "residual", m, n)
    bp = _vector(bias, "bias", n) if bias is not None else 0
    prob = _LINEAR.pack(m, n, k, code, act, xp, ldx, wp, ldw, bp, rp, ldr, yp, ldy, zp, ldz,
                        _dt(bias) if bias is not None else 0, _dt(residual) if residual is not None else 0, _dt(out), 0)
    L = _lib.lib()
    _call(dev, L.muon_linear, prob, L.muon_linear_workspace_bytes, m > 64)  # copies, or a divided sum
    if given:
        _written(*given)
    return (out, preact) if return_preact else out


def linear_backward(dy, x, w, *, activation=None, preact=None, need_dx=True, need_dw=True, need_dbias=False,
                    dw_dtype=None, dbias_dtype=None, dx=None, dw=None, dbias=None, accumulate=False):
    """(dx, dw, dbias) of :func:`linear` for the gradient ``dy`` of its result (see
    muon_linear_backward); None for those not asked for.  The residual's
    gradient is dy itself.

    ``preact`` is the pre-activation that linear returned (needed with an
    activation).  ``dw_dtype`` and ``dbias_dtype`` default to w's type;
    bf16 and fp32 are both what a step takes as a gradient; in fp32 they have
    its precision, which with bf16 operands behind an activation takes a second
    product.  Given outputs are asked for by being given, and written in place;
    with ``accumulate`` dw and dbias are added to.
    """
    _refuse_tangents(dy, x, w, preact)
    act = _act(activation)
    given = _given(dx, dw, dbias)
    dev = _same_device(dy, x, w, preact, dx, dw, dbias)
    code = _dt(x)
    if w.dtype != x.dtype:
        raise MuonError(_lib.MUON_ERR_UNSUPPORTED, f"x is {x.dtype} and w {w.dtype}: one type is needed")
    if w.dim() != 2:
        _bad("w must be [n, k]")
    w, wp, n, k, ldw = _input(w, "w")
    x, xp, m, _, ldx = _input(x, "x", k)
    dy, gp, ldg = _input_matrix(dy, "dy", m, n)
    zp, ldz = 0, 0
    if act:
        if preact is None:
            _bad("an activation's gradient needs preact")
        if preact.dtype != x.dtype:
            raise MuonError(_lib.MUON_ERR_UNSUPPORTED, f"preact must be {x.dtype} like x")
        preact, zp, ldz = _input_matrix(preact, "preact", m, n)
    if accumulate and ((need_dw and dw is None) or (need_dbias and dbias is None)):
        _bad("accumulate needs the tensors to add to")
    if dx is None and need_dx:
        dx = torch.empty_like(x, memory_format=torch.contiguous_format)
    if dw is None and need_dw:
        dw = torch.empty((n, k), dtype=dw_dtype or w.dtype, device=x.device)
    if dbias is None and need_dbias:
        dbias = torch.empty((n,), dtype=dbias_dtype or w.dtype, device=x.device)
    dxp, lddx = _check_matrix(dx, "dx", m, k) if dx is not None else (0, 0)
    dwp, lddw = _check_matrix(dw, "dw", n, k) if dw is not None else (0, 0)
    dbp = _vector(dbias, "dbias", n) if dbias is not None else 0
    prob = _GRAD.pack(m, n, k, code, act, gp, ldg, xp, ldx, wp, ldw, zp, ldz, dxp, lddx, dwp, lddw, dbp,
                      _dt(dy), _dt(dx) if dx is not None else 0, _dt(dw) if dw is not None else 0,
                      _dt(dbias) if dbias is not None else 0, int(bool(accumulate)), 0)
    L = _lib.lib()
    _call(dev, L.muon_linear_backward, prob, L.muon_linear_backward_workspace_bytes, act != 0 or dbias is not None)
    if given:
        _written(*given)
    return dx, dw, dbias


def _rowable(t):
    """t as rows of unit column stride (autograd may hand over expanded or transposed gradients)."""
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1]:
        return t
    return t.contiguous()


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, residual, activation, return_preact):
        keep = _act(activation) != 0
        r = _linear(x, w, bias, residual, activation, keep or return_preact)
        y, z = r if keep or return_preact else (r, None)
        ctx.save_for_backward(x, w, z if keep else None)
        ctx.activation = activation
        ctx.bias_dtype = bias.dtype if bias is not None else None
        ctx.residual_shape = residual.shape if residual is not None else None
        ctx.set_materialize_grads(False)
        if z is not None and not return_preact:
            ctx.mark_non_differentiable(z)
        return y, z

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dz):
        if dy is None and dz is None:
            return (None,) * 6
        _refuse_capture()
        x, w, z = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx = dw = db = None
        if need[0] or need[1] or need[2]:
            how = dict(need_dx=need[0], need_dw=need[1], need_dbias=need[2], dbias_dtype=ctx.bias_dtype)
            if dy is not None:
                dx, dw, db = linear_backward(_rowable(dy), x, w, activation=ctx.activation, preact=z, **how)
            if dz is not None:  # the returned pre-activation's own gradient, added onto y's
                more, dw, db = linear_backward(_rowable(dz), x, w, dw=dw, dbias=db, accumulate=dy is not None, **how)
                dx = more if dx is None else dx.add_(more) if need[0] else None
        # the residual may have other leading dimensions than x, of as many rows
        dr = dy.reshape(ctx.residual_shape) if need[3] and dy is not None else None
        return dx, dw, db, dr, None, None


# ---- per-head norms and rotation ----------------------------------------------------------
_NO_HEADS = (0, 0, 0, 0)
_NO_PAIR = _NO_HEADS * 2


def _heads_of(t, name, shape):
    """(pointer, batch, token, head stride) of a [tokens, heads, dim] or [batch, tokens, heads, dim] tensor
    of this shape (None: it is where the shape comes from)."""
    if shape is not None and t.shape != shape:
        _bad(f"{name} is {tuple(t.shape)}, not {tuple(shape)}")
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1 and t.numel():
        _bad(f"{name} needs unit stride in its last dimension")
    return (t.data_ptr(), 0, *st[:2]) if len(st) == 3 else (t.data_ptr(), *st[:3])


def _integers(name, values):
    try:
        return [operator.index(v) for v in values]
    except TypeError:
        _bad(f"{name} must be a sequence of integers, not {values!r}")


def _qk_problem(q, k, positions, inv_freq, sections, axes, interleaved, scale, x, g, y, weight, dweight, eps):
    """The problem of one call; q and k (either may be None) give the shapes, x,
    g and y are pairs of tensors or None."""
    first = q if q is not None else k
    if first is None:
        _bad("q and k are both None")
    qs, ks = q.shape if q is not None else None, k.shape if k is not None else None
    if q is not None and k is not None:
        if len(qs) != len(ks) or qs[:-2] != ks[:-2] or qs[-1] != ks[-1]:
            _bad(f"q {tuple(qs)} and k {tuple(ks)} differ in more than their heads")
        if q.dtype != k.dtype:
            raise MuonError(_lib.MUON_ERR_UNSUPPORTED, f"q is {q.dtype} and k {k.dtype}: one type is needed")
    fs = qs if qs is not None else ks
    if len(fs) not in (3, 4):
        _bad("q and k must be [tokens, heads, dim] or [batch, tokens, heads, dim]")
    dtype = first.dtype
    fields = []
    for pair in (x, g, y):
        if pair is None:
            fields += _NO_PAIR
            continue
        for t, like, shape, name in ((pair[0], q, qs, "q"), (pair[1], k, ks, "k")):
            if t is None or like is None:
                if t is not like:
                    _bad("q and k must both be given, or both be left out, in every pair of tensors")
                fields += _NO_HEADS
                continue
            if t.dtype != dtype:
                raise MuonError(_lib.MUON_ERR_UNSUPPORTED, f"head tensors are {t.dtype} and {dtype}: one type is needed")
            fields += _heads_of(t, name, shape if t is not like else None)
    dev = _same_device(positions, inv_freq, *(x or ()), *(g or ()), *(y or ()), *weight, *dweight)
    batch, tokens = (fs[0], fs[1]) if len(fs) == 4 else (1, fs[0])
    dim = fs[-1]
    wtype = None
    for t in weight + dweight:
        if t is None:
            fields.append(0)
            continue
        if wtype is not None and t.dtype != wtype:
            raise MuonError(_lib.MUON_ERR_UNSUPPORTED, "the norm weights and their gradients need one type")
        wtype = t.dtype
        wcode = _dt(t)
        fields.append(_vector(t, "a norm weight", dim))
    if inv_freq.dim() != 1 or inv_freq.dtype not in (torch.float32, torch.float64) or not inv_freq.is_contiguous():
        _bad("inv_freq must be a contiguous fp32 or fp64 vector of one frequency per pair")
    pairs = inv_freq.shape[0]
    if 2 * pairs > dim or pairs > _lib.QK_MAX_PAIRS:
        _bad(f"{pairs} pairs do not fit heads of {dim} (at most {_lib.QK_MAX_PAIRS})")
    if positions.dtype not in (torch.int32, torch.int64):
        raise MuonError(_lib.MUON_ERR_UNSUPPORTED, f"positions are {positions.dtype}, not int32 or int64")
    lead, shape, st = fs[:-2], positions.shape, positions.stride()
    naxes, axis_st, batch_st = 1, 0, 0
    if shape == lead:
        token_st = st[-1]
        batch_st = st[0] if len(lead) == 2 else 0
    elif shape[1:] == lead:
        naxes, axis_st, token_st = shape[0], st[0], st[-1]
        batch_st = st[1] if len(lead) == 2 else 0
    elif len(lead) == 2 and shape == lead[1:]:
        token_st = st[0]
    else:
        _bad(f"positions {tuple(shape)} do not go with tokens {tuple(lead)}")
    turns = b""
    if sections is not None:
        if axes is not None:
            _bad("give sections or axes, not both")
        sections = _integers("sections", sections)
        if len(sections) != naxes or sum(sections) != pairs or any(n < 0 for n in sections):
            _bad(f"sections {sections} do not split {pairs} pairs over {naxes} axes")
        if naxes > 1:
            turns = b"".join([bytes((i,)) * n for i, n in enumerate(sections)])
    elif axes is not None:
        axes = _integers("axes", axes)
        if len(axes) != pairs or not all(0 <= a < naxes for a in axes):
            _bad(f"axes must name one of {naxes} axes for each of {pairs} pairs")
        turns = bytes(axes)
    elif naxes > 1:
        _bad("positions with several axes need sections or axes")
    try:
        return dev, _QK.pack(batch, tokens, qs[-2] if qs is not None else 0, ks[-2] if ks is not None else 0, dim,
                             2 * pairs, _dt(first), wcode if wtype is not None else 0, *fields, positions.data_ptr(),
                             axis_st, batch_st, token_st, inv_freq.data_ptr(), positions.dtype is torch.int64,
                             inv_freq.dtype is torch.float64, bool(interleaved), naxes, scale, eps, turns)
    except (OverflowError, struct.error, TypeError):  # every other field is a size or an address
        _bad(f"scale and eps must be numbers that fp32 holds, not {scale!r} and {eps!r}")


def _like(t, out):
    if out is not None:
        return out
    return None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format)


def qk_norm_rope(q, k, positions, inv_freq, *, q_weight=None, k_weight=None, eps=1e-6, sections=None, axes=None,
                 interleaved=False, scale=1.0, q_out=None, k_out=None):
    """RMS norm of every head of q and k, times its weight, then the position rotation (see muon_qk_norm_rope).

    q and k are [tokens, heads, dim] or [batch, tokens, heads, dim] of any
    strides with a contiguous head (views of packed q/k/v rows, heads-first
    layouts); either may be None.  ``positions`` is [tokens] / [batch, tokens]
    (int32 or int64), or has a leading dimension of up to four axes, and then
    ``sections`` (pairs per axis, in order) or ``axes`` (one axis per pair)
    says which pair turns by which.  ``inv_freq`` [rotary pairs] is fp32 or
    fp64, and has no gradient.  Returns (q_out, k_out); an output may be its own input.
    """
    if _wants_grad(q, k, q_weight, k_weight, inv_freq):
        _refuse_frequency_gradient(inv_freq)
        if q_out is not None or k_out is not None:
            _bad("q_out and k_out cannot be given when an input requires a gradient")
        _refuse_capture()
        how = dict(eps=eps, sections=sections, axes=axes, interleaved=interleaved, scale=scale)
        return _QkNormRope.apply(q, k, q_weight, k_weight, positions, inv_freq, how)
    given = () if q_out is None and k_out is None else _given(q_out, k_out)
    y = (_like(q, q_out), _like(k, k_out))
    dev, p = _qk_problem(q, k, positions, inv_freq, sections, axes, interleaved, scale, (q, k), None, y,
                         (q_weight, k_weight), (None, None), eps)
    _call(dev, _lib.lib().muon_qk_norm_rope, p, None)
    if given:
        _written(*given)
    return y


def qk_norm_rope_backward(dq_out, dk_out, q, k, positions, inv_freq, *, q_weight=None, k_weight=None, eps=1e-6,
                          sections=None, axes=None, interleaved=False, scale=1.0, dq=None, dk=None):
    """(dq, dk, dq_weight, dk_weight) of :func:`qk_norm_rope` for the gradients of its outputs; None for what
    was not given.  dq may be dq_out, and dk dk_out."""
    _refuse_tangents(dq_out, dk_out, q, k, q_weight, k_weight)
    given = () if dq is None and dk is None else _given(dq, dk)
    y = (_like(q, dq), _like(k, dk))
    dwt = (_like(q_weight, None), _like(k_weight, None))
    dev, p = _qk_problem(q, k, positions, inv_freq, sections, axes, interleaved, scale, (q, k), (dq_out, dk_out), y,
                         (q_weight, k_weight), dwt, eps)
    if all(t is None or not t.numel() for t in (q, k)):  # an empty sum, which the library has no work for
        for t in dwt:
            if t is not None:
                t.zero_()
    L = _lib.lib()
    _call(dev, L.muon_qk_norm_rope_backward, p, L.muon_qk_norm_rope_backward_workspace_bytes, True)
    if given:
        _written(*given)
    return y + dwt


def rope(q, k, positions, inv_freq, *, sections=None, axes=None, interleaved=False, scale=1.0, q_out=None, k_out=None):
    """The position rotation of :func:`qk_norm_rope` without its norm (see muon_rope)."""
    if _wants_grad(q, k, inv_freq):
        _refuse_frequency_gradient(inv_freq)
        if q_out is not None or k_out is not None:
            _bad("q_out and k_out cannot be given when an input requires a gradient")
        _refuse_capture()
        how = dict(sections=sections, axes=axes, interleaved=interleaved, scale=scale)
        return _Rope.apply(q, k, positions, inv_freq, how)
    given = () if q_out is None and k_out is None else _given(q_out, k_out)
    y = (_like(q, q_out), _like(k, k_out))
    dev, p = _qk_problem(q, k, positions, inv_freq, sections, axes, interleaved, scale, (q, k), None, y,
                         (None, None), (None, None), 0.0)
    _call(dev, _lib.lib().muon_rope, p, None)
    if given:
        _written(*given)
    return y


def rope_backward(dq_out, dk_out, positions, inv_freq, *, sections=None, axes=None, interleaved=False, scale=1.0,
                  dq=None, dk=None):
    """(dq, dk) of :func:`rope`: the rotation by the opposite angles.  dq may be dq_out, and dk dk_out."""
    _refuse_tangents(dq_out, dk_out)
    given = () if dq is None and dk is None else _given(dq, dk)
    y = (_like(dq_out, dq), _like(dk_out, dk))
    dev, p = _qk_problem(dq_out, dk_out, positions, inv_freq, sections, axes, interleaved, scale, None,
                         (dq_out, dk_out), y, (None, None), (None, None), 0.0)
    _call(dev, _lib.lib().muon_rope_backward, p, None)
    if given:
        _written(*given)
    return y


def _head_grad(g, like):
    """A gradient of a head tensor, zeros where autograd has none."""
    if like is None:
        return None
    if g is None:
        return torch.zeros(like.shape, dtype=like.dtype, device=like.device)
    return g if g.shape[-1] <= 1 or g.stride(-1) == 1 else g.contiguous()


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, inv_freq, how):
        y = qk_norm_rope(q, k, positions, inv_freq, q_weight=q_weight, k_weight=k_weight, **how)
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, inv_freq)
        ctx.how = how
        ctx.set_materialize_grads(False)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gq, gk):
        if gq is None and gk is None:
            return (None,) * 7
        _refuse_capture()
        q, k, wq, wk, positions, inv_freq = ctx.saved_tensors
        grads = qk_norm_rope_backward(_head_grad(gq, q), _head_grad(gk, k), q, k, positions, inv_freq, q_weight=wq,
                                      k_weight=wk, **ctx.how)
        return tuple(t if n else None for t, n in zip(grads, ctx.needs_input_grad)) + (None, None, None)


class _Rope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, how):
        y = rope(q, k, positions, inv_freq, **how)
        ctx.save_for_backward(positions, inv_freq)
        ctx.how = how
        ctx.set_materialize_grads(False)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gq, gk):
        _refuse_capture()
        positions, inv_freq = ctx.saved_tensors
        # a gradient that autograd does not have is left out of the call
        gs = [None if g is None else (g if g.shape[-1] <= 1 or g.stride(-1) == 1 else g.contiguous()) for g in (gq, gk)]
        if gs[0] is None and gs[1] is None:
            return (None,) * 5
        dq, dk = rope_backward(gs[0], gs[1], positions, inv_freq, **ctx.how)
        return dq, dk, None, None, None
