"""The operators around a layer's products without a GPU: every refusal,
reported before anything is enqueued."""
import ctypes
import math
import struct

import pytest
import torch

import newton_schulz_ns5_amd as ns
from newton_schulz_ns5_amd import _lib

FAKE = 1 << 30  # a non-null, aligned address that is never dereferenced
MIB = 1 << 20


# ---- gradient norm and clipping -------------------------------------------------------
def arrays(ptrs, sizes, types):
    n = len(ptrs)
    return n, struct.pack(f"{n}Q", *ptrs), struct.pack(f"{n}i", *types), struct.pack(f"{n}q", *sizes)


def norm_call(ptrs=(FAKE, FAKE + MIB), sizes=(100, 7), types=(1, 0), kind=0, norm=FAKE + 2 * MIB, square=None,
              ws=FAKE + 3 * MIB, room=1 << 20):
    n, p, t, s = arrays(ptrs, sizes, types)
    return _lib.lib().muon_grad_norm(n, p, t, s, kind, norm, square, ws, room, None)


def clip_call(ptrs=(FAKE, FAKE + MIB), sizes=(100, 7), types=(1, 0), outs=None, otypes=None, kind=0, max_norm=1.0,
              eps=1e-6, total=None, f64=0, norm=FAKE + 2 * MIB, ws=FAKE + 3 * MIB, room=1 << 20):
    n, p, t, s = arrays(ptrs, sizes, types)
    outs, otypes = outs or ptrs, otypes or types
    _, o, ot, _ = arrays(outs, sizes, otypes)
    return _lib.lib().muon_clip_grad_norm(n, p, t, s, o, ot, kind, max_norm, eps, total, f64, norm, ws, room, None)


@pytest.mark.parametrize("over,code", [
    (dict(sizes=(-1, 7)), -1), (dict(sizes=(100, (1 << 40) + 1)), -1), (dict(ptrs=(FAKE, 0)), -1), (dict(types=(2, 0)), -2),
    (dict(ptrs=(FAKE + 1, FAKE + MIB)), -1), (dict(ptrs=(FAKE, FAKE + MIB + 2)), -1), (dict(kind=2), -2),
    (dict(ws=None), -1), (dict(ws=FAKE + 3 * MIB + 8), -1), (dict(room=8), -3),
])
def test_norm_and_clip_refusals(over, code):
    assert norm_call(**over) == code
    assert _lib.lib().muon_last_error()
    assert clip_call(**over) == code


@pytest.mark.parametrize("over", [
    dict(norm=None), dict(kind=1, square=FAKE + 2 * MIB + 8), dict(norm=FAKE + 2 * MIB + 2), dict(square=FAKE + 2 * MIB + 4),
    dict(square=FAKE + 2 * MIB), dict(norm=FAKE + 4), dict(norm=None, square=FAKE + MIB + 24),
])
def test_norm_outputs_refused(over):
    assert norm_call(**over) == -1


@pytest.mark.parametrize("over,code", [
    (dict(max_norm=-1.0), -1), (dict(max_norm=math.nan), -1), (dict(eps=-1e-9), -1), (dict(eps=math.inf), -1),
    (dict(eps=math.nan), -1), (dict(f64=2), -1), (dict(total=FAKE + 4 * MIB + 4, f64=1), -1), (dict(total=FAKE + 4 * MIB + 2), -1),
    (dict(total=FAKE + 4 * MIB, f64=1, kind=1), -1), (dict(norm=FAKE + 2 * MIB + 1), -1),
    # the same tensor twice, tensors that overlap, an output over another's input, a total or norm inside a tensor
    (dict(ptrs=(FAKE, FAKE), types=(1, 1)), -1), (dict(ptrs=(FAKE, FAKE + 196)), -1), (dict(outs=(FAKE + MIB, FAKE)), -1),
    (dict(outs=(FAKE + 2, FAKE + MIB)), -1), (dict(outs=(FAKE, FAKE + MIB), otypes=(0, 0)), -1), (dict(total=FAKE + 8), -1),
    (dict(norm=FAKE + 8), -1), (dict(total=FAKE + 2 * MIB), -1), (dict(outs=(FAKE + 5 * MIB, 0)), -1),
    (dict(outs=(FAKE + 5 * MIB, FAKE + 6 * MIB), otypes=(1, 3)), -2), (dict(outs=(FAKE + 5 * MIB, FAKE + 5 * MIB + 100)), -1),
])
def test_clip_refusals(over, code):
    assert clip_call(**over) == code
    assert _lib.lib().muon_last_error()


def test_norm_workspace():
    L = _lib.lib()
    need = ctypes.c_size_t()
    assert L.muon_grad_norm_workspace_bytes(0, None, ctypes.byref(need)) == 0 and need.value == 0
    assert L.muon_grad_norm_workspace_bytes(2, struct.pack("2q", 0, 0), ctypes.byref(need)) == 0 and need.value == 0
    assert L.muon_grad_norm_workspace_bytes(1, struct.pack("q", 1 << 36), ctypes.byref(need)) == 0
    assert 2048 * 8 < need.value <= 2049 * 8 + 256  # one launch's workgroups and their sum
    assert L.muon_grad_norm_workspace_bytes(1, None, ctypes.byref(need)) == -1
    assert L.muon_grad_norm_workspace_bytes(-1, None, ctypes.byref(need)) == -1
    assert L.muon_grad_norm_workspace_bytes(1, struct.pack("q", 1), None) == -1


def refused(fn, *a, code, **kw):
    with pytest.raises(ns.MuonError) as e:
        fn(*a, **kw)
    assert e.value.status == code


def test_norm_and_clip_bindings_refuse():
    t = torch.ones(3)
    refused(ns.grad_norm, [t], code=-1)  # not on a GPU
    refused(ns.clip_grad_norm, [t], 1.0, code=-1)
    refused(ns.grad_norm, [t], norm_type=1, code=-2)
    refused(ns.clip_grad_norm, [t], 1.0, norm_type=3, code=-2)
    refused(ns.grad_norm, [t], norm_type="inf", squared=True, code=-1)
    refused(ns.clip_grad_norm, [t], 1.0, out=[t, t], code=-1)
    refused(ns.clip_grad_norm, [t], 1.0, out=[None], code=-1)
    refused(ns.clip_grad_norm, [t], None, code=-1)
    refused(ns.clip_grad_norm, [t], 1.0, total=torch.ones(2), code=-1)
    refused(ns.clip_grad_norm, [t], 1.0, total=torch.ones((), dtype=torch.int64), code=-1)
    refused(ns.clip_grad_norm, [t], 1.0, norm_type=math.inf, total=torch.ones((), dtype=torch.float64), code=-1)


def test_no_gradients_have_the_norm_zero():
    if torch.cuda.is_available():
        pytest.skip("this is the case of a machine without a GPU")
    assert ns.grad_norm([]).item() == 0 and ns.clip_grad_norm([None], 1.0).item() == 0
    assert ns.grad_norm([None], squared=True).dtype is torch.float64
    assert ns.clip_grad_norm([], 1.0, total=torch.tensor(9.0, dtype=torch.float64)).item() == 3
