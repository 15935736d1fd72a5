"""The operators around a layer's products in a pass: the norm over all
gradients and their clipping.

Marshalling like :mod:`layer_ops`, whose rules hold here too: raw pointers to
the library, work enqueued on the current stream of the tensors' device,
workspaces from torch's allocator for the one call, given outputs written in
place with their autograd version counters moved, tracers and forward-mode
inputs refused.
"""
import ctypes
import math
import struct

import torch

from . import MuonError, _lib, _written
from ._lib import MUON_NORM_2, MUON_NORM_MAX
from .layer_ops import (_CODE, _NO_WORKSPACE, _bad, _current_device, _dual, _given, _raw_stream, _refuse_tangents,
                        _same_device)

__all__ = ["grad_norm", "clip_grad_norm"]


def _unsupported(text):
    raise MuonError(_lib.MUON_ERR_UNSUPPORTED, text)


def _on(dev, fn):
    """fn() with the device current."""
    if dev != _current_device():
        with torch.cuda.device(dev):
            return fn()
    return fn()


# ---- the norm over all gradients, and clipping ---------------------------------------
def _norm_kind(norm_type):
    if norm_type == 2:
        return MUON_NORM_2
    if norm_type == math.inf or norm_type == "inf":
        return MUON_NORM_MAX
    _unsupported(f"norm_type {norm_type!r} is not 2 or inf")


def _tensors(grads):
    return [grads] if isinstance(grads, torch.Tensor) else [t for t in grads if t is not None]


def _dense(t):
    """Whether t's elements lie side by side in memory, in whatever order of its dimensions."""
    if t.is_contiguous():
        return True
    n = 1
    for stride, size in sorted((st, sz) for st, sz in zip(t.stride(), t.shape) if sz != 1):
        if stride != n:
            return False
        n *= size
    return True


def _codes(ts):
    codes = [_CODE.get(t.dtype) for t in ts]
    if None in codes:
        _unsupported(f"dtype {ts[codes.index(None)].dtype} is not float32 or bfloat16")
    return codes


def _table(ts):
    """(count, pointers, types, sizes) as the library takes them, and the packed sizes' own count."""
    n = len(ts)
    return (n, struct.pack(f"{n}Q", *[t.data_ptr() for t in ts]), struct.pack(f"{n}i", *_codes(ts)),
            struct.pack(f"{n}q", *[t.numel() for t in ts]))


def _norm_workspace(n, sizes, device):
    need = ctypes.c_size_t(0)
    _lib.check(_lib.lib().muon_grad_norm_workspace_bytes(n, sizes, ctypes.byref(need)))
    return torch.empty(need.value, dtype=torch.uint8, device=device) if need.value else None


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
    dev = _same_device(*ts)
    if _dual["_current_level"] >= 0:
        _refuse_tangents(*ts)
    if torch.is_grad_enabled() and any(t.requires_grad for t in ts):
        _unsupported("the norm carries no gradient: detach the tensors")
    ts = [t if _dense(t) else t.contiguous() for t in ts]
    n, ptrs, codes, sizes = _table(ts)
    out = torch.empty((), dtype=torch.float64 if squared else torch.float32, device=ts[0].device)
    at = (None, out.data_ptr()) if squared else (out.data_ptr(), None)

    def call():
        ws = _norm_workspace(n, sizes, out.device)
        _lib.check(_lib.lib().muon_grad_norm(n, ptrs, codes, sizes, kind, *at, ws.data_ptr() if ws is not None else _NO_WORKSPACE,
                                             ws.numel() if ws is not None else 0, _raw_stream(dev)))
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
    outs = ts if out is None else [o for o in out if o is not None]
    if len(outs) != len(ts):
        _bad(f"{len(outs)} outputs for {len(ts)} gradients")
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
    dev = _same_device(*ts, *(outs if out is not None else ()), total)
    if _dual["_current_level"] >= 0:
        _refuse_tangents(*ts, *outs, total)
    _given(*outs)
    for t in ts:
        if not _dense(t):
            _bad("a gradient's elements do not lie side by side: it cannot be scaled as a whole")
    if out is not None:
        if torch.is_grad_enabled() and any(t.requires_grad for t in ts):
            _unsupported("clipped gradients carry no gradient: detach the tensors")
        for t, o in zip(ts, outs):
            if o.shape != t.shape:
                _bad(f"an output is {tuple(o.shape)}, not {tuple(t.shape)}")
            if not (t.is_contiguous() and o.is_contiguous()) and t.stride() != o.stride():
                _bad("an output's memory order is not its gradient's")
    n, ptrs, codes, sizes = _table(ts)
    optrs, ocodes = (ptrs, codes) if out is None else _table(outs)[1:3]
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
    keep = [(g, o) for g, o in zip(grads, out) if g is not None]
    if any(o is None for _, o in keep):
        _bad("a gradient has no output")
    return [g for g, _ in keep], [o for _, o in keep]
