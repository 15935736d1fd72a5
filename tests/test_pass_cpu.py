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
    assert 1024 * 8 < need.value <= 1025 * 8 + 256  # one launch's workgroups and their sum
    from newton_schulz_ns5_amd import pass_ops
    sizes = struct.pack("128q", *[1 << 23] * 128)
    assert L.muon_grad_norm_workspace_bytes(pass_ops._ONE_LAUNCH, sizes, ctypes.byref(need)) == 0
    assert need.value <= pass_ops._ONE_LAUNCH_BYTES
    assert L.muon_grad_norm_workspace_bytes(1, None, ctypes.byref(need)) == -1
    assert L.muon_grad_norm_workspace_bytes(-1, None, ctypes.byref(need)) == -1
    assert L.muon_grad_norm_workspace_bytes(1, struct.pack("q", 1), None) == -1


# ---- norms around a block ----------------------------------------------------------------
def test_ctypes_struct_matches_c_layout():
    import os
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    lines = []
    structs = [("muon_residual_norm_problem", _lib.ResidualNormProblem), ("muon_embedding_problem", _lib.EmbeddingProblem)]
    for c, py in structs:
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "muon_mi355x.h"\nint main(void) {' + "\n".join(lines) + "return 0; }"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(root, "include"), c, "-o", exe], check=True)
        lay = dict(x.split() for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines())
    for c, py in structs:
        assert ctypes.sizeof(py) == int(lay[c]), c
        for f, _ in py._fields_:
            assert getattr(py, f).offset == int(lay[f"{c}.{f}"]), (c, f)


def test_packed_problems_match_the_structs():
    from newton_schulz_ns5_amd import pass_ops
    assert pass_ops._NORM.size == ctypes.sizeof(_lib.ResidualNormProblem)
    fields = [f for f, _ in _lib.ResidualNormProblem._fields_]
    p = _lib.ResidualNormProblem.from_buffer_copy(pass_ops._NORM.pack(*range(1, len(fields) + 1)))
    assert [getattr(p, f) for f in fields] == list(range(1, len(fields) + 1))
    assert pass_ops._EMBED.size == ctypes.sizeof(_lib.EmbeddingProblem)
    fields = [f for f, _ in _lib.EmbeddingProblem._fields_]
    p = _lib.EmbeddingProblem.from_buffer_copy(pass_ops._EMBED.pack(*range(1, len(fields) + 1)))
    assert [getattr(p, f) for f in fields] == list(range(1, len(fields) + 1))


def norm_problem(**over):
    a = dict(rows=6, cols=64, dtype=1, stream_dtype=0, weight_dtype=1, gate_dtype=1, post_norm=1, norm=1, block=FAKE,
             block_row_stride=64, residual=FAKE + MIB, residual_row_stride=64, stream=FAKE + 2 * MIB, stream_row_stride=64,
             y=FAKE + 3 * MIB, y_row_stride=64, weight=FAKE + 4 * MIB, post_weight=FAKE + 5 * MIB, gate=FAKE + 6 * MIB,
             gate_rows=2, gate_row_stride=64, scale=1.0, residual_scale=1.0, eps=1e-6, weight_offset=0.0,
             dy=FAKE + 7 * MIB, dy_row_stride=64, dstream=FAKE + 8 * MIB, dstream_row_stride=64, dblock=FAKE + 9 * MIB,
             dblock_row_stride=64, dresidual=FAKE + 10 * MIB, dresidual_row_stride=64, dweight=FAKE + 11 * MIB,
             dpost_weight=FAKE + 12 * MIB, dgate=FAKE + 13 * MIB, dgate_row_stride=64, reserved=0)
    a.update(over)
    p = _lib.ResidualNormProblem()
    for k, v in a.items():
        setattr(p, k, v)
    return p


BOTH = [
    (dict(rows=-1), -1), (dict(cols=-1), -1), (dict(rows=(1 << 30) + 1, gate=None), -1), (dict(cols=16385), -1),
    (dict(dtype=2), -2), (dict(stream_dtype=-1), -2), (dict(weight_dtype=4), -2), (dict(gate_dtype=5), -2),
    (dict(norm=2), -1), (dict(post_norm=3), -1), (dict(reserved=1), -1), (dict(scale=math.inf), -1),
    (dict(residual_scale=math.nan), -1), (dict(eps=-1.0), -1), (dict(eps=math.nan), -1), (dict(weight_offset=math.inf), -1),
    (dict(gate_rows=4), -1), (dict(gate_rows=0), -1), (dict(norm=0), -1), (dict(post_norm=0), -1), (dict(block=None), -1),
    (dict(block_row_stride=63), -1), (dict(gate_row_stride=63), -1), (dict(block=FAKE + 1), -1), (dict(stream=FAKE + 2 * MIB + 2), -1),
    (dict(weight=FAKE + 4 * MIB + 1), -1), (dict(stream_row_stride=1 << 60), -1), (dict(gate=FAKE + 1), -1),
]


@pytest.mark.parametrize("over,code", BOTH + [
    (dict(y=None), -1), (dict(y=FAKE + 2), -1), (dict(y=FAKE, y_row_stride=65), -1), (dict(stream=FAKE), -1),
    (dict(stream=FAKE + MIB, stream_row_stride=80), -1), (dict(y=FAKE + 2 * MIB), -1), (dict(y=FAKE + 4 * MIB), -1),
    (dict(stream=FAKE + 5 * MIB), -1), (dict(y=FAKE + 6 * MIB), -1), (dict(y_row_stride=8), -1), (dict(y=FAKE + MIB), -1),
    (dict(norm=0, weight=None, stream=None), -1), (dict(residual=FAKE + MIB + 2), -1),
])
def test_residual_norm_refusals(over, code):
    assert _lib.lib().muon_residual_norm(ctypes.byref(norm_problem(**over)), None) == code
    assert _lib.lib().muon_last_error()


@pytest.mark.parametrize("over,code", BOTH + [
    (dict(dy=None), -1), (dict(stream=None), -1), (dict(dy_row_stride=1), -1), (dict(norm=0, weight=None), -1),
    (dict(norm=0, weight=None, dweight=None, dstream=None), -1), (dict(post_norm=0, post_weight=None), -1),
    (dict(gate=None), -1), (dict(dblock=FAKE + 2), -1), (dict(dblock=FAKE + 8 * MIB), -1), (dict(dresidual=FAKE + 7 * MIB), -1),
    (dict(dresidual=FAKE + 9 * MIB), -1), (dict(dweight=FAKE), -1), (dict(dweight=FAKE + 4 * MIB), -1),
    (dict(dpost_weight=FAKE + 11 * MIB), -1), (dict(dgate=FAKE + 6 * MIB), -1), (dict(dgate=FAKE + 12 * MIB), -1),
    (dict(dgate=FAKE + 10 * MIB), -1), (dict(dgate_row_stride=3), -1), (dict(dweight=FAKE + 11 * MIB + 1), -1),
    (dict(dblock=FAKE + 4 * MIB), -1), (dict(dstream=FAKE + 8 * MIB + 2), -1),
])
def test_residual_norm_backward_refusals(over, code):
    assert _lib.lib().muon_residual_norm_backward(ctypes.byref(norm_problem(**over)), FAKE + 20 * MIB, 1 << 40, None) == code
    assert _lib.lib().muon_last_error()


def test_residual_norm_empty_calls_and_workspace():
    L = _lib.lib()
    need = ctypes.c_size_t(7)
    for over in (dict(rows=0, gate_rows=1), dict(cols=0)):
        p = norm_problem(**over)
        assert L.muon_residual_norm(ctypes.byref(p), None) == 0
        assert L.muon_residual_norm_backward(ctypes.byref(p), None, 0, None) == 0
        assert L.muon_residual_norm_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(need)) == 0 and need.value == 0
    p = norm_problem()
    assert L.muon_residual_norm_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(need)) == 0 and need.value > 0
    assert L.muon_residual_norm_backward(ctypes.byref(p), FAKE + 20 * MIB, need.value - 1, None) == -3
    assert L.muon_residual_norm_backward(ctypes.byref(p), FAKE + 20 * MIB + 16, need.value, None) == -1
    assert L.muon_residual_norm(None, None) == -1
    assert L.muon_residual_norm_backward(None, None, 0, None) == -1


def test_residual_norm_bindings_refuse():
    b, w = torch.ones(2, 3, 8), torch.ones(8)
    refused(ns.residual_norm, b, code=-1)  # not on a GPU
    refused(ns.residual_norm, b, weight=w, norm=False, code=-1)
    refused(ns.residual_norm, b, post_weight=w, post_norm=False, code=-1)
    refused(ns.residual_norm_backward, None, None, None, b, code=-1)
    refused(ns.residual_norm_backward, b, None, None, b, code=-1)
    refused(ns.residual_norm_backward, b, None, b, b, norm=False, code=-1)
    refused(ns.residual_norm_backward, b, None, b, None, gate=w, code=-1)


# ---- embedding ------------------------------------------------------------------------------
def embed_problem(**over):
    a = dict(tokens=10, rows=20, dim=16, ids=FAKE, first=0, padding=0, w=FAKE + MIB, w_row_stride=16, y=FAKE + 2 * MIB,
             y_row_stride=16, w_dtype=1, y_dtype=1, ids_i64=1, has_padding=0, accumulate=0, scale=1.0, reserved=0)
    a.update(over)
    p = _lib.EmbeddingProblem()
    for k, v in a.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,code", [
    (dict(tokens=-1), -1), (dict(rows=-1), -1), (dict(dim=-1), -1), (dict(tokens=(1 << 26) + 1), -1), (dict(rows=(1 << 26) + 1), -1),
    (dict(dim=65537), -1), (dict(w_dtype=2), -2), (dict(y_dtype=-1), -2), (dict(scale=math.nan), -1), (dict(ids_i64=2), -1),
    (dict(has_padding=-1), -1), (dict(accumulate=2), -1), (dict(reserved=1), -1), (dict(ids=None), -1), (dict(ids=FAKE + 4), -1),
    (dict(ids_i64=0, ids=FAKE + 2), -1), (dict(w=None), -1), (dict(y=None), -1), (dict(w=FAKE + MIB + 1), -1), (dict(y=FAKE + 1), -1),
    (dict(w_row_stride=15), -1), (dict(y_row_stride=15), -1), (dict(y_row_stride=1 << 58), -1), (dict(y=FAKE + MIB + 32), -1),
])
def test_embedding_refusals(over, code):
    L = _lib.lib()
    assert L.muon_embedding(ctypes.byref(embed_problem(**over)), None) == code
    assert L.muon_last_error()
    assert L.muon_embedding_backward(ctypes.byref(embed_problem(**over)), FAKE + 20 * MIB, 1 << 40, None) == code


def test_embedding_gradients_of_too_many_workgroups_refused():
    p = embed_problem(tokens=1 << 26, dim=4096, w_row_stride=4096, y_row_stride=4096, w=1 << 50, rows=4)
    assert _lib.lib().muon_embedding_backward(ctypes.byref(p), FAKE + 20 * MIB, 1 << 60, None) == -1
    assert b"together" in _lib.lib().muon_last_error()


def test_embedding_outputs_over_the_ids():
    L = _lib.lib()
    assert L.muon_embedding(ctypes.byref(embed_problem(y=FAKE + 72)), None) == -1
    assert L.muon_embedding_backward(ctypes.byref(embed_problem(w=FAKE + 72)), FAKE + 20 * MIB, 1 << 40, None) == -1


def test_embedding_empty_calls_and_workspace():
    L = _lib.lib()
    need = ctypes.c_size_t(7)
    assert L.muon_embedding(None, None) == -1 and L.muon_embedding_backward(None, None, 0, None) == -1
    for over in (dict(tokens=0, ids=None, y=None), dict(dim=0)):
        assert L.muon_embedding(ctypes.byref(embed_problem(**over)), None) == 0
    for over in (dict(tokens=0, ids=None, y=None, accumulate=1), dict(dim=0), dict(rows=0, w=None)):
        p = embed_problem(**over)
        assert L.muon_embedding_backward(ctypes.byref(p), None, 0, None) == 0
        assert L.muon_embedding_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(need)) == 0 and need.value == 0
    p = embed_problem()
    assert L.muon_embedding_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(need)) == 0 and need.value > 0
    assert L.muon_embedding_backward(ctypes.byref(p), FAKE + 20 * MIB, need.value - 1, None) == -3
    assert L.muon_embedding_backward(ctypes.byref(p), FAKE + 20 * MIB + 16, need.value, None) == -1
    assert L.muon_embedding_backward_workspace_bytes(ctypes.byref(p), None) == -1


def test_embedding_bindings_refuse():
    ids, w = torch.zeros(3, dtype=torch.int64), torch.ones(4, 8)
    refused(ns.embedding, ids, w, code=-1)  # not on a GPU
    refused(ns.embedding_backward, torch.ones(3, 8), ids, 4, code=-1)


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
