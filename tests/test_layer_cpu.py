"""Layer operators without a GPU: the C structures, and every refusal reported
before anything is enqueued."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

import newton_schulz_ns5_amd as ns
from newton_schulz_ns5_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 30  # a non-null, aligned address that is never dereferenced
MIB = 1 << 20

STRUCTS = [("muon_linear_problem", _lib.LinearProblem), ("muon_linear_grad", _lib.LinearGrad),
           ("muon_heads", _lib.Heads), ("muon_qk_problem", _lib.QkProblem)]


def test_ctypes_structs_match_c_layout():
    lines = []
    for c, py in STRUCTS:
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "muon_mi355x.h"\nint main(void) {' + "\n".join(lines) + "return 0; }"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        lay = dict(x.split() for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines())
    for c, py in STRUCTS:
        assert ctypes.sizeof(py) == int(lay[c]), c
        for f, _ in py._fields_:
            assert getattr(py, f).offset == int(lay[f"{c}.{f}"]), (c, f)


def test_packed_problems_match_the_structs():
    from newton_schulz_ns5_amd import layer_ops
    for packed, py in [(layer_ops._LINEAR, _lib.LinearProblem), (layer_ops._GRAD, _lib.LinearGrad), (layer_ops._QK, _lib.QkProblem)]:
        assert packed.size == ctypes.sizeof(py)
    # every field its own number, read back through the structure
    p = _lib.LinearProblem.from_buffer_copy(layer_ops._LINEAR.pack(*range(1, 21)))
    assert [getattr(p, f) for f, _ in p._fields_] == list(range(1, 21))
    p = _lib.LinearGrad.from_buffer_copy(layer_ops._GRAD.pack(*range(1, 25)))
    assert [getattr(p, f) for f, _ in p._fields_] == list(range(1, 25))
    nums = list(range(1, 9)) + list(range(100, 124)) + list(range(200, 213)) + [1.5, 2.5, bytes(range(256))]
    q = _lib.QkProblem.from_buffer_copy(layer_ops._QK.pack(*nums))
    assert (q.batch, q.tokens, list(q.heads), q.dim, q.rotary_dim, q.dtype, q.weight_dtype) == (1, 2, [3, 4], 5, 6, 7, 8)
    flat = [v for pair in (q.x, q.g, q.y) for h in pair for v in (h.p, h.batch_stride, h.token_stride, h.head_stride)]
    assert flat == list(range(100, 124)) and list(q.weight) + list(q.dweight) == [200, 201, 202, 203]
    assert (q.positions, q.pos_axis_stride, q.pos_batch_stride, q.pos_token_stride, q.inv_freq) == (204, 205, 206, 207, 208)
    assert (q.positions_i64, q.inv_freq_f64, q.interleaved, q.axes, q.scale, q.eps) == (209, 210, 211, 212, 1.5, 2.5)
    assert bytes(q.axis) == bytes(range(256))


def linear_problem(**over):
    a = dict(m=8, n=16, k=32, dtype=1, activation=0, x=FAKE, x_row_stride=32, w=FAKE + MIB, w_row_stride=32, bias=None,
             residual=None, residual_row_stride=16, y=FAKE + 2 * MIB, y_row_stride=16, preact=None, preact_row_stride=16,
             bias_dtype=1, residual_dtype=1, y_dtype=1, reserved=0)
    a.update(over)
    p = _lib.LinearProblem()
    for k, v in a.items():
        setattr(p, k, v)
    return p


Y = FAKE + 2 * MIB


@pytest.mark.parametrize("over,code", [
    (dict(m=-1), -1), (dict(n=-1), -1), (dict(k=-1), -1), (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1),
    (dict(x_row_stride=31), -1), (dict(w_row_stride=31), -1), (dict(y_row_stride=15), -1),
    (dict(dtype=2), -2), (dict(y_dtype=7), -2), (dict(bias=FAKE + 3 * MIB, bias_dtype=5), -2),
    (dict(residual=FAKE + 3 * MIB, residual_dtype=-1), -2), (dict(activation=6), -2), (dict(activation=-1), -2),
    (dict(x=FAKE + 1), -1), (dict(y=FAKE + 2 * MIB + 2, y_dtype=0), -1), (dict(m=(1 << 30) + 1), -1),
    (dict(x_row_stride=1 << 22), -1), (dict(reserved=1), -1),
    (dict(y=FAKE), -1), (dict(y=FAKE + MIB), -1), (dict(preact=Y), -1), (dict(preact=FAKE), -1),
    (dict(residual=Y + 2), -1), (dict(residual=Y, residual_dtype=0), -1), (dict(residual=Y, residual_row_stride=32), -1),
    (dict(preact=FAKE + 3 * MIB, residual=FAKE + 3 * MIB), -1),
])
def test_linear_refusals(over, code):
    L = _lib.lib()
    p = linear_problem(**over)
    assert L.muon_linear(ctypes.byref(p), FAKE, 1 << 40, None) == code
    assert L.muon_last_error()


def test_linear_null_problem_and_empty_calls():
    L = _lib.lib()
    assert L.muon_linear(None, FAKE, 0, None) == -1
    assert L.muon_linear_workspace_bytes(None, None) == -1
    for over in (dict(m=0, x=None, y=None), dict(n=0, w=None, y=None)):
        p = linear_problem(**over)
        assert L.muon_linear(ctypes.byref(p), None, 0, None) == 0  # nothing to enqueue


def grad_problem(**over):
    a = dict(m=8, n=16, k=32, dtype=1, activation=3, dy=FAKE, dy_row_stride=16, x=FAKE + MIB, x_row_stride=32,
             w=FAKE + 2 * MIB, w_row_stride=32, preact=FAKE + 3 * MIB, preact_row_stride=16, dx=FAKE + 4 * MIB,
             dx_row_stride=32, dw=FAKE + 5 * MIB, dw_row_stride=32, dbias=FAKE + 6 * MIB, dy_dtype=1, dx_dtype=1,
             dw_dtype=0, dbias_dtype=0, accumulate=0, reserved=0)
    a.update(over)
    p = _lib.LinearGrad()
    for k, v in a.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,code", [
    (dict(m=-1), -1), (dict(dy=None), -1), (dict(x=None), -1), (dict(w=None), -1), (dict(preact=None), -1),
    (dict(dy_row_stride=3), -1), (dict(dw_row_stride=31), -1), (dict(dtype=4), -2), (dict(dw_dtype=9), -2),
    (dict(dy_dtype=3), -2), (dict(activation=17), -2), (dict(accumulate=2), -1), (dict(reserved=3), -1),
    (dict(dx=FAKE), -1), (dict(dw=FAKE + MIB), -1), (dict(dbias=FAKE + 5 * MIB), -1), (dict(dx=FAKE + 3 * MIB), -1),
    (dict(dx=FAKE + 2 * MIB), -1),
    # bf16 gradients whose fp32 copy would have rows of 2^23 bytes
    (dict(dtype=0, activation=0, n=1 << 21, dy_row_stride=1 << 21, dx_dtype=0, dw=None, dbias=None), -1),
])
def test_linear_backward_refusals(over, code):
    L = _lib.lib()
    p = grad_problem(**over)
    assert L.muon_linear_backward(ctypes.byref(p), FAKE, 1 << 40, None) == code
    assert L.muon_last_error()


def test_linear_backward_workspace():
    L = _lib.lib()
    p = grad_problem()
    need = ctypes.c_size_t()
    assert L.muon_linear_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(need)) == 0 and need.value > 0
    assert L.muon_linear_backward(ctypes.byref(p), FAKE, need.value - 1, None) == -3
    assert L.muon_linear_backward(ctypes.byref(p), FAKE + 16, need.value, None) == -1
    assert L.muon_linear_backward(ctypes.byref(p), None, need.value, None) == -1


def qk_problem(**over):
    p = _lib.QkProblem()
    a = dict(batch=1, tokens=5, dim=64, rotary_dim=64, dtype=1, weight_dtype=1, positions=FAKE, pos_token_stride=1,
             inv_freq=FAKE + MIB, positions_i64=1, inv_freq_f64=1, axes=1, scale=1.0, eps=1e-6)
    hq, hk = over.pop("heads", (4, 2))
    p.heads[0], p.heads[1] = hq, hk
    # packed rows of q, k and v heads
    row = (hq + 2 * hk) * 64
    x = over.pop("x", (FAKE + 2 * MIB, FAKE + 2 * MIB + hq * 128))
    y = over.pop("y", x)
    for i in range(2):
        p.x[i] = p.g[i] = _lib.Heads(x[i], 0, row, 64)
        p.y[i] = _lib.Heads(y[i], 0, row, 64)
    a.update(over)
    for k, v in a.items():
        setattr(p, k, v)
    return p


QKV = FAKE + 2 * MIB


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), -1), (dict(tokens=-2), -1), (dict(dim=0), -1), (dict(dim=1025), -1), (dict(rotary_dim=63), -1),
    (dict(rotary_dim=66), -1), (dict(axes=0), -1), (dict(axes=5), -1), (dict(dtype=2), -2), (dict(weight_dtype=3), -2),
    (dict(scale=float("inf")), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(heads=(-1, 2)), -1),
    (dict(positions=None), -1), (dict(inv_freq=None), -1), (dict(inv_freq=FAKE + 4), -1), (dict(pos_token_stride=-1), -1),
    (dict(x=(None, QKV)), -1), (dict(x=(QKV + 1, QKV + 512)), -1),
    (dict(y=(QKV, QKV)), -1),              # k's output over q's input
    (dict(y=(QKV + 2, QKV + 512)), -1),    # shifted in place
    (dict(y=(QKV + MIB, QKV + MIB)), -1),  # both outputs in one place
    (dict(tokens=(1 << 30) + 1), -1),
])
def test_qk_refusals(over, code):
    L = _lib.lib()
    p = qk_problem(**over)
    assert L.muon_qk_norm_rope(ctypes.byref(p), None) == code
    assert L.muon_last_error()
    assert L.muon_qk_norm_rope_backward(ctypes.byref(p), FAKE, 1 << 40, None) == code


def test_qk_axis_out_of_range_and_null():
    L = _lib.lib()
    p = qk_problem(axes=2)
    p.axis[31] = 2
    assert L.muon_rope(ctypes.byref(p), None) == -1 and b"pair 31" in L.muon_last_error()
    assert L.muon_qk_norm_rope(None, None) == -1 and L.muon_rope_backward(None, None) == -1


def test_qk_empty_calls_and_workspace():
    L = _lib.lib()
    for over in (dict(tokens=0), dict(batch=0), dict(heads=(0, 0))):
        p = qk_problem(**over)
        assert L.muon_qk_norm_rope(ctypes.byref(p), None) == 0
        assert L.muon_rope(ctypes.byref(p), None) == 0
    p = qk_problem()
    need = ctypes.c_size_t()
    assert L.muon_qk_norm_rope_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(need)) == 0 and need.value
    assert L.muon_qk_norm_rope_backward(ctypes.byref(p), FAKE, need.value - 1, None) == -3


def test_qk_output_that_overlaps_itself():
    L = _lib.lib()
    p = qk_problem()
    p.y[0] = _lib.Heads(FAKE + 8 * MIB, 0, 64, 64)  # every token's heads run into the next token's
    assert L.muon_qk_norm_rope(ctypes.byref(p), None) == -1 and b"itself" in L.muon_last_error()


def code_of(f):
    with pytest.raises(ns.MuonError) as e:
        f()
    return e.value.status


def test_python_refusals():
    x, w = torch.zeros(4, 8), torch.zeros(16, 8)
    assert code_of(lambda: ns.linear(x, w)) == -1                          # not on a GPU
    assert code_of(lambda: ns.linear(x, w, activation="swish")) == -2
    q = torch.zeros(4, 2, 8)
    pos, f = torch.zeros(4, dtype=torch.int64), torch.ones(4)
    assert code_of(lambda: ns.qk_norm_rope(q, q, pos, f)) == -1
    assert code_of(lambda: ns.rope(None, None, pos, f)) == -1


# ---- calls that would lose what their caller asked for, refused before the device is looked at ----
def heads_call():
    q = torch.randn(4, 2, 8)
    return q, torch.arange(4), torch.ones(4)


def test_forward_mode_is_refused():
    """The result would come without its tangent."""
    from torch.autograd import forward_ad as fwd
    x, w, b, r = torch.randn(4, 8), torch.randn(16, 8), torch.randn(16), torch.randn(4, 16)
    q, pos, f = heads_call()
    with fwd.dual_level():
        def dual(t):
            return fwd.make_dual(t, torch.ones_like(t))
        for args in ((dual(x), w, b, r), (x, dual(w), b, r), (x, w, dual(b), r), (x, w, b, dual(r))):
            assert code_of(lambda: ns.linear(*args)) == -2
        assert code_of(lambda: ns.linear_backward(dual(r), x, w)) == -2
        assert code_of(lambda: ns.rope(dual(q), None, pos, f)) == -2
        assert code_of(lambda: ns.rope(q, q, pos, dual(f))) == -2
        assert code_of(lambda: ns.rope_backward(None, dual(q), pos, f)) == -2
        assert code_of(lambda: ns.qk_norm_rope(q, dual(q), pos, f)) == -2
        assert code_of(lambda: ns.qk_norm_rope(q, None, pos, f, q_weight=dual(torch.ones(8)))) == -2
        assert code_of(lambda: ns.qk_norm_rope_backward(q, None, dual(q), None, pos, f)) == -2
        with torch.no_grad():
            assert code_of(lambda: ns.linear(dual(x), w)) == -2
        assert code_of(lambda: ns.linear(x, w)) == -1  # no dual tensor: only the device is wrong


def test_tracing_is_refused():
    """A trace would hold the result's allocation without the launch that writes it."""
    from torch.fx.experimental.proxy_tensor import make_fx
    x, w = torch.randn(4, 8), torch.randn(16, 8)
    q, pos, f = heads_call()
    calls = [(lambda a: ns.linear(a, w), x), (lambda a: ns.linear_backward(torch.ones(4, 16), a, w)[0], x),
             (lambda a: ns.rope(a, None, pos, f)[0], q), (lambda a: ns.rope_backward(a, None, pos, f)[0], q),
             (lambda a: ns.qk_norm_rope(a, None, pos, f)[0], q),
             (lambda a: ns.qk_norm_rope_backward(a, None, a, None, pos, f)[0], q)]
    for call, a in calls:
        assert code_of(lambda: torch.jit.trace(call, (a,), check_trace=False)) == -2
        assert code_of(lambda: make_fx(call)(a)) == -2
        assert code_of(lambda: call(a)) == -1  # not traced: only the device is wrong


def test_frequencies_that_require_a_gradient_are_refused():
    """The rotation has none for them; it would be dropped."""
    q, pos, f = heads_call()
    g = f.clone().requires_grad_()
    for fn in (ns.rope, ns.qk_norm_rope):
        assert code_of(lambda: fn(q, None, pos, g)) == -2
        assert code_of(lambda: fn(q.clone().requires_grad_(), None, pos, g)) == -2
        assert code_of(lambda: fn(q, None, pos, g.detach())) == -1  # only the device is wrong
        with torch.no_grad():
            assert code_of(lambda: fn(q, None, pos, g)) == -1


def test_given_outputs_that_require_a_gradient_are_refused():
    """They would keep a history that their new values do not have."""
    def msg(f):
        with pytest.raises(ns.MuonError) as e:
            f()
        return "given output requires a gradient" in str(e.value)

    x, w, dy = torch.randn(4, 8), torch.randn(16, 8), torch.randn(4, 16)
    q, pos, f = heads_call()

    def leaf(t):
        return torch.empty_like(t).requires_grad_()

    calls = [lambda o: ns.linear(x, w, out=o(dy)), lambda o: ns.linear(x, w, preact=o(dy)),
             lambda o: ns.linear_backward(dy, x, w, dx=o(x)), lambda o: ns.linear_backward(dy, x, w, dw=o(w)),
             lambda o: ns.linear_backward(dy, x, w, dbias=o(dy[0])), lambda o: ns.rope(q, q, pos, f, q_out=o(q)),
             lambda o: ns.rope_backward(q, q, pos, f, dk=o(q)), lambda o: ns.qk_norm_rope(q, q, pos, f, k_out=o(q)),
             lambda o: ns.qk_norm_rope_backward(q, q, q, q, pos, f, dq=o(q))]
    for call in calls:
        assert msg(lambda: call(leaf)) and not msg(lambda: call(torch.empty_like))
        with torch.no_grad():
            assert not msg(lambda: call(leaf))


# ---- overlaps ---------------------------------------------------------------------------
ROW = (4 + 2 * 2) * 64 * 2  # bytes of a packed row of qk_problem


def with_vectors(**over):
    """qk_problem with weights, and their gradients, of their own."""
    p = qk_problem(**{k: v for k, v in over.items() if k not in ("weight", "dweight")})
    for i in range(2):
        p.weight[i] = over.get("weight", (FAKE + 3 * MIB, FAKE + 4 * MIB))[i]
        p.dweight[i] = over.get("dweight", (FAKE + 5 * MIB, FAKE + 6 * MIB))[i]
    return p


@pytest.mark.parametrize("over", [
    dict(weight=(QKV, FAKE + 4 * MIB)),                     # q's weight is q's first head
    dict(weight=(FAKE + 4 * MIB, QKV + 2 * ROW + 100)),     # k's weight is in q's heads of the third token
    dict(weight=(QKV - 126, None)),                         # its last value is q's first
    dict(positions=QKV + 8), dict(positions=QKV - 32), dict(inv_freq=QKV + 4 * ROW), dict(inv_freq=QKV - 248),
])
def test_qk_outputs_over_the_vectors_are_refused(over):
    L = _lib.lib()
    p = with_vectors(**over)
    assert L.muon_qk_norm_rope(ctypes.byref(p), None) == -1 and b"overlaps" in L.muon_last_error()
    if "weight" not in over:
        assert L.muon_rope(ctypes.byref(p), None) == -1 and b"overlaps" in L.muon_last_error()
    assert L.muon_qk_norm_rope_backward(ctypes.byref(p), FAKE + 64 * MIB, 1 << 30, None) == -1


@pytest.mark.parametrize("over", [
    dict(dweight=(FAKE + 3 * MIB, None)), dict(dweight=(None, FAKE + 3 * MIB)),     # a weight
    dict(dweight=(FAKE + 5 * MIB, FAKE + 5 * MIB + 126)),                           # each other
    dict(dweight=(QKV, None)), dict(dweight=(None, QKV + 4 * ROW + 640)),           # head rows
    dict(dweight=(FAKE, None)), dict(dweight=(FAKE + MIB + 8, None)),               # positions, inv_freq
])
def test_qk_weight_gradients_over_other_tensors_are_refused(over):
    L = _lib.lib()
    p = with_vectors(**over)
    need = ctypes.c_size_t()
    assert L.muon_qk_norm_rope_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(need)) == -1
    assert L.muon_qk_norm_rope_backward(ctypes.byref(p), FAKE + 64 * MIB, 1 << 30, None) == -1
    assert b"overlap" in L.muon_last_error()


def test_qk_vectors_beside_and_between_the_rows_are_taken():
    """Up to the first and from the last byte on, and in the v heads between the rows of q and k."""
    L = _lib.lib()
    need = ctypes.c_size_t()
    for over in (dict(weight=(QKV - 128, QKV + 5 * ROW)), dict(positions=QKV - 40), dict(inv_freq=QKV + 5 * ROW),
                 dict(weight=(QKV + 6 * 128, QKV + ROW + 6 * 128)), dict(dweight=(QKV + 7 * 128, QKV + 4 * ROW + 6 * 128)),
                 dict(positions=QKV + 2 * ROW + 6 * 128)):
        p = with_vectors(**over)
        assert L.muon_qk_norm_rope_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(need)) == 0, (over, L.muon_last_error())


def packed_problem(B, S, hq, hk, dim, heads_first, at=(0, 0)):
    """q and k of one buffer, in place, k's output `at` values off its input."""
    p = qk_problem(heads=(hq, hk), batch=B, tokens=S, dim=dim, rotary_dim=0)
    n = hq + 2 * hk
    st = (n * S * dim, dim, S * dim) if heads_first else (n * S * dim, n * dim, dim)
    for i, h0 in enumerate((0, hq)):
        first = QKV + 2 * h0 * st[2]
        p.x[i] = p.g[i] = _lib.Heads(first, *st)
        p.y[i] = _lib.Heads(first + 2 * at[i], *st)
    return p


@pytest.mark.parametrize("heads_first", [False, True])
def test_qk_in_place_views_of_one_buffer_are_told_apart(heads_first):
    """q and k of packed rows ([B, S, heads, D]) and of a heads-first buffer
    ([B, heads, S, D]) are disjoint, for any number of sequences; moved by a
    value, by a head or by a row they are not."""
    L = _lib.lib()
    need = ctypes.c_size_t()

    def status(*a, **k):
        p = packed_problem(*a, **k)
        return L.muon_qk_norm_rope_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(need))

    for B, S, hq, hk, dim in [(1, 7, 4, 2, 64), (3, 7, 4, 2, 64), (5, 1, 8, 2, 128), (4, 9, 1, 1, 63), (2, 1000, 32, 8, 128), (1, 1, 2, 1, 8)]:
        assert status(B, S, hq, hk, dim, heads_first) == 0, L.muon_last_error()
        step = S * dim if heads_first else dim
        assert status(B, S, hq, hk, dim, heads_first, at=(0, 1)) == -1       # by one value, over its own input
        assert status(B, S, hq, hk, dim, heads_first, at=(0, -step)) == -1   # onto q's last head
        assert status(B, S, hq, hk, dim, heads_first, at=(step * hq, 0)) == -1


def test_qk_overlap_agrees_with_the_sets_of_elements():
    """Against the elements written down, for small tensors of random strides: nothing that
    shares an element is taken; where the strides are the same, nothing else is refused."""
    import random
    L, rng, need = _lib.lib(), random.Random(5), ctypes.c_size_t()
    seen = set()
    for _ in range(4000):
        B, S, hq, hk, dim = (rng.randint(1, 3) for _ in range(5))
        p = qk_problem(heads=(hq, hk), batch=B, tokens=S, dim=dim, rotary_dim=0)

        def strides():
            order, st, reach = rng.sample(range(3), 3), [0] * 3, dim
            for i in order:
                st[i] = reach + rng.randint(0, 6)
                reach += (max(B, S, hq, hk) - 1) * st[i]
            return st

        st = strides()
        same = rng.random() < 0.7
        offs = [0, rng.randint(0, 60)]
        all_st = [st, st if same else strides()]
        for i in range(2):
            p.y[i] = _lib.Heads(QKV + 2 * offs[i], *all_st[i])
            p.x[i] = p.g[i] = _lib.Heads(FAKE + (9 + i) * MIB, S * hq * hk * 8, hq * hk * 8, 8)
        sets = [{offs[i] + b * all_st[i][0] + s * all_st[i][1] + h * all_st[i][2] + e for b in range(B) for s in range(S)
                 for h in range((hq, hk)[i]) for e in range(dim)} for i in range(2)]
        rc = L.muon_qk_norm_rope_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(need))
        meets = bool(sets[0] & sets[1])
        assert rc == (-1 if meets else 0) or (rc == -1 and not same), (B, S, hq, hk, dim, all_st, offs, rc, L.muon_last_error())
        seen.add((same, meets, rc))
    assert {(True, True, -1), (True, False, 0), (False, True, -1), (False, False, 0)} <= seen


def test_qk_strides_that_pass_64_bits_are_refused():
    """Their offsets wrapped round, and the overlap checks with them."""
    L = _lib.lib()
    for st in ((1 << 61, 512, 64), (0, 1 << 62, 64), (0, 512, 1 << 62), (0, 1 << 54, 64)):
        p = qk_problem(batch=8 if st[0] else 1)
        for t in (*p.x, *p.y):
            t.batch_stride = 5 * 512
        p.x[1] = _lib.Heads(FAKE + 8 * MIB, *st)
        assert L.muon_qk_norm_rope(ctypes.byref(p), None) == -1 and b"too far" in L.muon_last_error()
    for over in (dict(pos_token_stride=1 << 61), dict(pos_batch_stride=1 << 61, batch=8), dict(pos_axis_stride=1 << 62, axes=4)):
        p = qk_problem(**over)
        assert L.muon_rope(ctypes.byref(p), None) == -1 and b"too far" in L.muon_last_error()


# ---- how products are divided: the workspace holds split products of m x n, one per chunk ----
def split_of(m, n, k, dtype):
    """Chunks that the sum of aligned operands is divided into."""
    L, need = _lib.lib(), ctypes.c_size_t()
    p = linear_problem(m=m, n=n, k=k, dtype=dtype, y_dtype=dtype, x_row_stride=k, w_row_stride=k, y_row_stride=n,
                       w=FAKE + (1 << 38), y=FAKE + (1 << 39))
    assert L.muon_linear_workspace_bytes(ctypes.byref(p), ctypes.byref(need)) == 0, L.muon_last_error()
    return max(1, need.value // (m * -(-n // 8) * 8 * 4))


def test_fp32_products_with_half_empty_rounds_are_split():
    """Where the tiles fill the CUs unevenly, chunks of the sum even them out (474 to 297 us and
    238 to 197 us at the first two); where they fill whole rounds they are not split."""
    assert split_of(260, 4096, 14336, 0) >= 3 and split_of(227, 9174, 4920, 0) >= 3 and split_of(87, 8584, 4288, 0) >= 4
    assert split_of(4096, 4096, 4096, 0) == 1 and split_of(1024, 4096, 4096, 0) == 1


def test_few_rows_times_narrow_weights_are_split():
    """A weight with few rows leaves most CUs without a workgroup unless its K is divided
    (123 to 23 us and 64 to 15 us at the first two); few steps, or a full chip, are not split."""
    assert split_of(62, 384, 13972, 0) >= 8 and split_of(64, 512, 14336, 1) >= 8 and split_of(38, 5920, 10392, 1) >= 2
    assert split_of(1, 1024, 16384, 1) >= 2
    for m, n, k, t in ((1, 6144, 4096, 1), (48, 14336, 4096, 1), (4, 576, 3456, 0), (16, 1024, 1024, 0), (64, 1024, 1024, 1)):
        assert split_of(m, n, k, t) == 1


def test_the_gpu_tests_reach_every_kernel_of_the_products():
    """Each type, layout, tile, with and without a divided sum and a last round of smaller tiles;
    for few rows each number of token and weight blocks: by the plan of the sizes that the GPU tests run."""
    import test_gpu_layer as old
    import test_gpu_layer_mends as new
    L = _lib.lib()

    def plan(m, n, k, dtype, kind):
        p = (ctypes.c_int32 * 4)()
        assert L.muon_linear_plan(m, n, k, dtype, kind, ctypes.byref(p)) == 0
        return tuple(p)

    code = {torch.float32: 0, torch.bfloat16: 1}
    runs = [(code[t], m, k, n) for t in code for m, k, n in old.SIZES + new.TILE_SIZES[t] + new.FEW_ROWS + new.FEW_ROWS_WHOLE]
    tiles, few = set(), set()
    for dtype, m, k, n in runs:
        for kind in range(3):
            rows, cols, split, last = plan(m, n, k, dtype, kind)
            if rows:
                tiles.add((dtype, kind, rows, cols, split > 1, last))
            else:
                few.add((dtype, -(-m // 16), cols, split > 1))
    every = {(t, mb, cols, split) for t in (0, 1) for mb in (1, 2, 3, 4) for cols in (16, 64) for split in (False, True)}
    assert few == every, sorted(every - few)
    want = {(0, kind, rows, cols, split, 0) for kind in range(3) for rows, cols in ((64, 64), (256, 128)) for split in (False, True)}
    want |= {(1, kind, rows, cols, split, 0) for kind in range(3) for rows, cols in ((64, 64), (256, 128)) for split in (False, True)}
    want |= {(1, kind, rows, rows, False, last) for kind in range(3) for rows, last in ((128, 0), (256, 0), (256, 1))}
    assert not want - tiles, sorted(want - tiles)


def test_plan_refusals():
    L, p = _lib.lib(), (ctypes.c_int32 * 4)()
    assert L.muon_linear_plan(1, 1, 1, 0, 0, None) == -1
    assert L.muon_linear_plan(1, 1, 1, 0, 3, ctypes.byref(p)) == -1 and L.muon_linear_plan(1, 1, 1, 0, -1, ctypes.byref(p)) == -1
    assert L.muon_linear_plan(1, 1, 1, 2, 0, ctypes.byref(p)) == -2 and L.muon_linear_plan(-1, 1, 1, 0, 0, ctypes.byref(p)) == -1


def test_plan_of_empty_and_largest_sizes():
    L, p = _lib.lib(), (ctypes.c_int32 * 4)()
    for dtype in (0, 1):
        for kind in range(3):
            for m, n, k in ((0, 5, 5), (5, 0, 5), (5, 5, 0), (0, 0, 0), (100, 0, 7), (100, 7, 0), (0, 100, 100)):
                assert L.muon_linear_plan(m, n, k, dtype, kind, ctypes.byref(p)) == 0
                empty = {0: m and n, 1: m and k, 2: n and k}[kind] == 0
                assert (tuple(p) == (0, 0, 0, 0)) == empty
            for m, n, k in ((1 << 30, 64, 64), (64, 1 << 22, 64), (1 << 20, 1 << 15, 1 << 20), (1, 1, 1 << 30)):
                assert L.muon_linear_plan(m, n, k, dtype, kind, ctypes.byref(p)) == 0 and p[2] >= 1


def test_no_grid_passes_2_32_threads():
    """An fp32 product of 2^30 rows by 8 columns (34 GB) chose more 64-edge tiles than a launch has threads."""
    L, p = _lib.lib(), (ctypes.c_int32 * 4)()
    threads = {(256, 256): 512, (256, 128): 512, (128, 128): 256, (64, 64): 256}
    for dtype in (0, 1):
        for kind in range(3):
            for m in ((1 << 30), (1 << 30) - 64, 1 << 29, (1 << 28) + 1):
                for n in (1, 8, 64):
                    a, b, c = (m, n, 8) if kind != 2 else (8, m, n)
                    if L.muon_linear_plan(a, b, c, dtype, kind, ctypes.byref(p)) or not p[0]:
                        continue
                    M, N = {0: (a, b), 1: (a, c), 2: (b, c)}[kind]
                    tiles = -(-M // p[0]) * -(-N // p[1]) * p[2]
                    assert tiles * threads[p[0], p[1]] < 1 << 32, (dtype, kind, m, n, tuple(p))


def test_fp32_few_rows_take_the_faster_kernel():
    """Both measured, few-row kernel and tiles: 59 and 38 us, 52 and 35 us, 32 and 18 us, 92 and 107 us at the first four."""
    L, p = _lib.lib(), (ctypes.c_int32 * 4)()
    for m, n, k, tiles in ((40, 9472, 2504, True), (40, 6144, 4096, True), (64, 1024, 8192, True), (40, 14336, 4096, False),
                           (24, 4096, 4096, False), (16, 9472, 2504, False), (40, 9472, 2501, False)):
        assert L.muon_linear_plan(m, n, k, 0, 0, ctypes.byref(p)) == 0
        assert (p[0] > 0) == tiles, (m, n, k, tuple(p))
    assert L.muon_linear_plan(40, 9472, 2504, 1, 0, ctypes.byref(p)) == 0 and p[0] == 0  # bf16 as before
