"""The layer operators on the GPU where a careful user goes: gradients kept in
fp32, buffers that autograd has saved, recorded and traced calls, tails of the
activations, far positions, layouts.

Tolerances as in test_gpu_layer: u(t) = eps(t) / 2 per rounding, a product
summed over K terms in fp32 off by at most (K + 8) 2^-23 of the sum of its
terms' magnitudes."""
import math

import pytest
import torch

import newton_schulz_ns5_amd as ns
from gpu_util import torch_cuda
from test_gpu_layer import ACTS, BF, F32, U, act64, check_backward, check_forward, close, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dy_dtype", [BF, F32], ids=["dy_bf16", "dy_f32"])
@pytest.mark.parametrize("m,k,n", [(150, 72, 200), (300, 264, 520), (2, 33, 65), (700, 512, 1040)])
def test_fp32_gradients_of_bf16_operands(m, k, n, dy_dtype, act):
    """A gradient asked for in fp32 holds g to 2^-16, not to bf16's 2^-8."""
    torch_cuda()
    x, w, dy, z = rand((m, k), BF, 1), rand((n, k), BF, 2), rand((m, n), dy_dtype, 3), rand((m, n), BF, 4, 2)
    base = rand((n, k), F32, 5)
    dx, dw, acc = torch.empty((m, k), dtype=F32, device="cuda"), None, base.clone()
    dx, dw, _ = ns.linear_backward(dy, x, w, activation=act, preact=z if act else None, dx=dx, dw_dtype=F32)
    ns.linear_backward(dy, x, w, activation=act, preact=z if act else None, need_dx=False, dw=acc, accumulate=True)
    g, err = dy.double(), 0 * dy.double()
    if act:
        _, slope, _, serr = act64(z.double(), act)
        g, err = g * slope, g.abs() * serr
    err = err + g.abs() * (2.0 ** -16 + 2.0 ** -22)  # two bf16 terms, and the fp32 arithmetic that forms them
    for got, a, b, terms, more in ((dx, g, w.double(), n, 0), (dw, g.t(), x.double(), m, 0), (acc, g.t(), x.double(), m, base.double())):
        e = err if a is g else err.t()
        want = a @ b + more
        # the second term's product is added onto the first's, which is stored in fp32
        tol = e @ b.abs() + (2 * terms + 16) * 2.0 ** -23 * (a.abs() @ b.abs()) + 4 * U[F32] * want.abs() + 2.0 ** -22
        close(got, want, tol, (act, terms))


def test_fp32_gradients_behind_an_infinite_one():
    """An infinite g stays one: its second term is left out, not infinity less infinity."""
    torch_cuda()
    x, w, dy, z = rand((80, 40), BF, 1), rand((96, 40), BF, 2), rand((80, 96), BF, 3), rand((80, 96), BF, 4).abs() + 1
    dy[7, 5] = float("inf")
    _, dw, _ = ns.linear_backward(dy, x, w, activation="relu", preact=z, need_dx=False, dw_dtype=F32)
    assert torch.isinf(dw[5]).all() and torch.equal(dw[5] > 0, x[7] > 0)
    assert torch.isfinite(dw[:5]).all() and torch.isfinite(dw[6:]).all()


# ---- buffers written through their pointers ------------------------------------------
def versions(ts, call):
    """call() and which of ts it moved on."""
    before = [t._version for t in ts]
    call()
    return [t._version > b for t, b in zip(ts, before)]


def test_written_outputs_move_their_version_counters():
    torch_cuda()
    x, w, dy, z = rand((20, 64), BF, 1), rand((48, 64), BF, 2), rand((20, 48), BF, 3), rand((20, 48), BF, 4)
    out, pre = torch.empty_like(dy), torch.empty_like(dy)
    assert versions([out, pre, x, w], lambda: ns.linear(x, w, activation="silu", out=out, preact=pre, return_preact=True)) == \
        [True, True, False, False]
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(48, dtype=BF, device="cuda")
    assert all(versions([dx, dw, db], lambda: ns.linear_backward(dy, x, w, dx=dx, dw=dw, dbias=db, need_dbias=True)))
    assert versions([dw, dy], lambda: ns.linear_backward(dy, x, w, need_dx=False, dw=dw, accumulate=True)) == [True, False]
    q, k, gq, gk = (rand((6, h, 64), BF, i) for i, h in enumerate((4, 2, 4, 2)))
    pos, f = torch.arange(6, device="cuda"), torch.rand(32, device="cuda")
    for fn in (ns.rope, ns.qk_norm_rope):
        assert versions([q, k], lambda: fn(q, k, pos, f, q_out=q)) == [True, False]
        assert all(versions([q, k], lambda: fn(q, k, pos, f, q_out=q, k_out=k)))
    assert versions([gq, gk], lambda: ns.rope_backward(gq, gk, pos, f, dk=gk)) == [False, True]
    assert versions([gq, gk, q], lambda: ns.qk_norm_rope_backward(gq, gk, q, k, pos, f, dq=gq, dk=gk)) == [True, True, False]
    buf = rand((6, 8 * 64), BF, 5)  # a view's buffer with it
    assert versions([buf], lambda: ns.rope(buf[:, :256].view(6, 4, 64), None, pos, f, q_out=buf[:, :256].view(6, 4, 64))) == [True]


def test_backward_after_a_saved_buffer_was_written_raises():
    torch_cuda()
    x, w = rand((6, 128), BF, 1), rand((32, 128), BF, 2).requires_grad_()
    pos, f = torch.arange(6, device="cuda"), torch.rand(32, device="cuda")
    h = ns.linear(x, w)
    ns.rope(x.view(6, 2, 64), None, pos, f, q_out=x.view(6, 2, 64))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        h.sum().backward()
    with torch.inference_mode():  # tensors without a counter are written like any other
        y = rand((6, 32), BF, 3)
        ns.linear(x, w.detach(), out=y)
    assert torch.equal(y, ns.linear(x, w.detach()))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_backward_after_the_step_raises(dtype):
    """The step writes the weight that linear saved."""
    torch_cuda()
    x, w = rand((8, 64), dtype, 1).requires_grad_(), rand((32, 64), dtype, 2).requires_grad_()
    opt = ns.MuonNS5([w], lr=0.05)
    h = ns.linear(x, w)
    h.sum().backward(retain_graph=True)
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        h.sum().backward()


def test_step_and_newton_schulz_outputs_move_their_version_counters():
    torch_cuda()
    shape = (64, 96)
    w, g, m, v, wm = rand(shape, F32, 1), rand(shape, BF, 2), rand(shape, BF, 3), torch.ones(64, device="cuda"), rand(shape, BF, 4)
    ts = [w, m, v, wm, g]
    assert versions(ts, lambda: ns.step_group([w], [g], [m], [v], [wm], normuon=True)) == [True] * 4 + [False]
    one = {"w_master": [w], "grads": [g], "moms": [m], "variances": [v], "w_model": [wm]}
    assert versions(ts, lambda: ns.step_groups([one], normuon=True)) == [True] * 4 + [False]
    out = torch.empty_like(g)
    assert versions([out, g], lambda: ns.ns_batched(g, out)) == [True, False]
    assert versions([out, g], lambda: ns.ns_batched_noalloc(g, out)) == [True, False]
    assert versions([out, g], lambda: ns.ns_groups([g], [out])) == [True, False]
    assert versions([out, v], lambda: ns.normuon_normalize(out, v)) == [True, True]


# ---- autograd --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act", [None, "silu", "gelu"])
def test_the_returned_preactivation_carries_its_gradient(act, dtype):
    """A loss on y and on z, on z alone and on y alone, against the sum of the two
    gradients called directly: bf16 sums of two bf16 gradients, one more rounding."""
    torch_cuda()
    x, w, b, r = rand((2, 33, 48), dtype, 1), rand((80, 48), dtype, 2), rand((80,), F32, 3), rand((2, 33, 80), F32, 4)
    gy, gz = rand((2, 33, 80), F32, 5), rand((2, 33, 80), dtype, 6)
    _, z = ns.linear(x, w, b, r, activation=act, return_preact=True)
    of_y = ns.linear_backward(gy, x, w, activation=act, preact=z if act else None, need_dbias=True, dbias_dtype=F32)
    of_z = ns.linear_backward(gz, x, w, need_dbias=True, dbias_dtype=F32)
    for on in ((gy, gz), (None, gz), (gy, None)):
        leaves = [t.clone().requires_grad_() for t in (x, w, b, r)]
        y, z = ns.linear(*leaves, activation=act, return_preact=True)
        assert z.requires_grad
        torch.autograd.backward([t for t, g in zip((y, z), on) if g is not None], [g for g in on if g is not None])
        for leaf, p, q in zip(leaves, of_y, of_z):
            parts = [t.double().view(leaf.shape) for t, g in ((p, on[0]), (q, on[1])) if g is not None]
            size = sum(t.abs() for t in parts)
            close(leaf.grad, sum(parts), 2 * U[leaf.dtype] * size + 2.0 ** -20 * size, (act, on[0] is None, on[1] is None))
        assert (leaves[3].grad is None) if on[0] is None else torch.equal(leaves[3].grad, gy)


def test_gradient_through_the_preactivation_against_fp64():
    torch_cuda()
    x, w, b = rand((40, 64), F32, 1), rand((72, 64), F32, 2, 1 / 8), rand((72,), F32, 3)
    gy, gz = rand((40, 72), F32, 4), rand((40, 72), F32, 5)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    y, z = ns.linear(*leaves, activation="silu", return_preact=True)
    torch.autograd.backward([y, z], [gy, gz])
    exact = [t.double().requires_grad_() for t in (x, w, b)]
    z = exact[0] @ exact[1].t() + exact[2]
    torch.autograd.backward([z * torch.sigmoid(z), z], [gy.double(), gz.double()])
    for a, e in zip(leaves, exact):
        # sums of at most 72 fp32 terms, twice, and the activation's slope: well under 200 units
        assert float((a.grad.double() - e.grad).norm() / e.grad.norm()) <= 200 * 2.0 ** -24


def test_residual_of_other_leading_dimensions():
    """The residual's rows are x's, its leading dimensions need not be."""
    torch_cuda()
    x, w = rand((2, 33, 48), BF, 1), rand((80, 48), BF, 2)
    gy = rand((2, 33, 80), F32, 4)
    for shape in ((66, 80), (2, 33, 80), (6, 11, 80), (1, 66, 80)):
        r = rand(shape, F32, 3).requires_grad_()
        y = ns.linear(x, w, None, r)
        assert torch.equal(y, ns.linear(x, w, None, r.detach().view(2, 33, 80)))
        y.backward(gy)
        assert torch.equal(r.grad, gy.view(shape))
    r = rand((80,), F32, 5).requires_grad_()
    ns.linear(x[0, :1], w, None, r).backward(gy[0, :1])
    assert torch.equal(r.grad, gy[0, 0])


# ---- the activations' values and slopes, in their tails too -----------------------------
def exact_act(z, name):
    """Value and slope in fp64, and the magnitudes that the slope is a sum of."""
    if name == "gelu":
        cdf, zp = 0.5 * torch.erfc(-z / math.sqrt(2)), z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return z * cdf, cdf + zp, cdf + zp.abs(), 0 * z
    t, dt = z, torch.ones_like(z)
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        t, dt = c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z)
    s, r = torch.sigmoid(t), torch.sigmoid(-t)
    # 1 - s is off by 2^-24 where s is near one
    return z * s, s + z * s * r * dt, s + (z * s * r * dt).abs(), (z * s * dt).abs() * 2.0 ** -23


# silu and gelu: the fp32 functions and three roundings beside them, under 16 units of 2^-24; bf16 operands:
# exponentials whose argument a is rounded, |a| 2^-23 of the result, and |a| <= 104 here.  gelu_tanh: its argument
# is a product of fp32 numbers, each rounding of it |2 u| 2^-24 of the result, three of them, and 2 u >= -87 here.
TAILS = [("gelu", -12, 12, 2.0 ** -20), ("silu", -80, 80, 2.0 ** -20), ("gelu_tanh", -9.5, 9.5, 2.0 ** -15)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act,lo,hi,rel", TAILS)
def test_activation_values_in_their_tails(act, lo, hi, rel, dtype):
    """The bias alone, in fp32, is the pre-activation: values relative to themselves."""
    torch_cuda()
    z = torch.cat([torch.linspace(lo, hi, 60001, device="cuda"), torch.linspace(-1e-2, 1e-2, 2001, device="cuda")])
    x, w = torch.zeros((1, 8), dtype=dtype, device="cuda"), torch.zeros((z.numel(), 8), dtype=dtype, device="cuda")
    y = ns.linear(x, w, z, activation=act, out=torch.empty((1, z.numel()), device="cuda"))
    want = exact_act(z.double(), act)[0][None]
    close(y, want, want.abs() * max(rel, 2.0 ** -17 if dtype == BF else 0), (act, "value"))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act,lo,hi,rel", TAILS)
def test_activation_slopes_in_their_tails(act, lo, hi, rel, dtype):
    """The bias gradient of one row of ones is the slope at its pre-activation."""
    torch_cuda()
    z = torch.linspace(lo, hi, 60001, device="cuda").to(dtype)[None]
    x, w = torch.zeros((1, 8), dtype=dtype, device="cuda"), torch.zeros((z.numel(), 8), dtype=dtype, device="cuda")
    _, _, db = ns.linear_backward(torch.ones_like(z), x, w, activation=act, preact=z, need_dx=False, need_dw=False,
                                  need_dbias=True, dbias_dtype=F32)
    _, want, size, more = exact_act(z.double(), act)
    close(db[None], want, size * 2 * max(rel, 2.0 ** -17 if dtype == BF else 0) + more, (act, "slope"))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_slopes_far_out_are_zero_and_one(act, dtype):
    torch_cuda()
    z = torch.tensor([[-float("inf"), -1e30, -300.0, -120.0, 120.0, 1e30, float("inf")]], device="cuda").to(dtype)
    x, w = torch.zeros((1, 8), dtype=dtype, device="cuda"), torch.zeros((7, 8), dtype=dtype, device="cuda")
    _, _, db = ns.linear_backward(torch.ones_like(z), x, w, activation=act, preact=z, need_dx=False, need_dw=False,
                                  need_dbias=True, dbias_dtype=F32)
    assert (db[:4].abs() <= 2.0 ** -126).all() and torch.equal(db[4:], torch.ones(3, device="cuda"))
    s = torch.tensor([[-40.0]], device="cuda", dtype=dtype)  # between: silu's slope there is -1.66e-16
    _, _, db = ns.linear_backward(torch.ones_like(s), x, w[:1], activation=act, preact=s, need_dx=False, need_dw=False,
                                  need_dbias=True, dbias_dtype=F32)
    assert abs(float(db[0]) - (-40 * math.exp(-40) if act == "silu" else 0.0)) <= 1e-17


# ---- far positions ---------------------------------------------------------------------
def turn_of(pos, f):
    """cos and sin of pos * f, the angle reduced in exact rational arithmetic."""
    from fractions import Fraction
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
    turns = Fraction(pos) * Fraction(f) / (2 * pi)
    a = 2 * math.pi * float(turns - round(turns))
    return math.cos(a), math.sin(a)


def test_angles_of_far_positions():
    """Rotations of (1, 0) are the cosine and sine themselves: within two units of 2^-23
    (the library's sine and cosine of a reduced angle, and the last rounding) at any position
    that fp64 holds, against angles from rational arithmetic."""
    torch_cuda()
    pos = [0, 1, -1, 12345, 10 ** 7 + 3, 2 ** 28 - 1, 2 ** 30 + 7, 10 ** 9 + 1, 2 ** 34 + 5, 2 ** 40 + 11, -(2 ** 45) - 9, 2 ** 53]
    for dtype in (torch.float64, F32):
        f = torch.pow(10000.0, -torch.arange(64, device="cuda", dtype=torch.float64) / 64).to(dtype)
        q = torch.zeros((len(pos), 1, 128), device="cuda")
        q[..., :64] = 1
        y, _ = ns.rope(q, None, torch.tensor(pos, device="cuda"), f)
        want = torch.tensor([[turn_of(p, g) for g in f.tolist()] for p in pos], dtype=torch.float64, device="cuda")
        close(y[:, 0, :64], want[..., 0], torch.full_like(want[..., 0], 2.0 ** -22), "cos")
        close(y[:, 0, 64:], want[..., 1], torch.full_like(want[..., 0], 2.0 ** -22), "sin")


@pytest.mark.parametrize("B,S", [(1, 9), (3, 9), (4, 1)])
def test_qk_in_place_in_a_heads_first_buffer(B, S):
    torch_cuda()
    hq, hk, d = 4, 2, 64
    buf = rand((B, hq + 2 * hk, S, d), BF, 1)
    f, pos = torch.rand(d // 2, device="cuda"), torch.arange(S, device="cuda")
    want = ns.qk_norm_rope(buf[:, :hq].transpose(1, 2), buf[:, hq:hq + hk].transpose(1, 2), pos, f)
    rest = buf[:, hq + hk:].clone()
    q, k = buf[:, :hq].transpose(1, 2), buf[:, hq:hq + hk].transpose(1, 2)
    ns.qk_norm_rope(q, k, pos, f, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(buf[:, hq + hk:], rest)
    with pytest.raises(ns.MuonError):
        ns.rope(q, k, pos, f, k_out=buf[:, hq - 1:hq - 1 + hk].transpose(1, 2))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_rows_far_apart(dtype):
    """The last token of every long sequence, 8 MiB and more apart; every input so, and their gradients."""
    torch_cuda()

    def spread(rows, cols, seed):
        gap = 2 ** 23 // (2 if dtype == BF else 4)
        buf = torch.empty(rows * gap, dtype=dtype, device="cuda")
        view = buf.as_strided((rows, cols), (gap, 1))
        view.copy_(rand((rows, cols), dtype, seed))
        return view

    for m, k, n in ((4, 72, 40), (70, 72, 40)):
        x, w, r, z = spread(m, k, 1), spread(n, k, 2), spread(m, n, 3), spread(m, n, 4)
        want = ns.linear(x.contiguous(), w.contiguous(), None, r.contiguous(), activation="silu")
        assert torch.equal(ns.linear(x, w, None, r, activation="silu"), want)
        assert torch.equal(ns.linear(x, w.contiguous()), ns.linear(x.contiguous(), w.contiguous()))
        want = ns.linear_backward(r.contiguous(), x.contiguous(), w.contiguous(), activation="gelu", preact=z.contiguous())
        got = ns.linear_backward(r, x, w, activation="gelu", preact=z)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    h = rand((4, 1024, 4096), dtype, 5)
    w = rand((96, 4096), dtype, 6)
    assert torch.equal(ns.linear(h[:, -1], w), ns.linear(h[:, -1].contiguous(), w))
    leaf = h.clone().requires_grad_()
    ns.linear(leaf[:, -1], w).sum().backward()
    assert not leaf.grad[:, :-1].any() and leaf.grad[:, -1].any()
    with pytest.raises(ns.MuonError):  # an output is not copied
        ns.linear(h[:, -1].contiguous(), w, out=torch.empty(4 * 2 ** 22, dtype=dtype, device="cuda").as_strided((4, 96), (2 ** 22, 1)))


def test_axes_sections_and_numbers_that_are_not():
    torch_cuda()
    q, f = rand((4, 2, 16), BF, 1), torch.ones(8, device="cuda")
    pos = torch.zeros((2, 4), dtype=torch.int64, device="cuda")

    def status(**how):
        with pytest.raises(ns.MuonError) as e:
            ns.rope(q, None, pos, f, **how)
        return e.value.status

    for axes in (8, [0] * 7, [0] * 7 + [2], [0] * 7 + [256], [0] * 7 + [-1], [0.0] * 8, ["0"] * 8, "00000000", torch.ones(8)):
        assert status(axes=axes) == -1
    for sections in (8, [8], [4, 5], [9, -1], [4.0, 4.0], "44", [4, 4, 0], None, []):
        assert status(sections=sections) == -1
    for number in (float("nan"), float("inf"), 1e39, "1", None, [1.0]):
        assert status(axes=[0] * 8, scale=number) == -1
        with pytest.raises(ns.MuonError):
            ns.qk_norm_rope(q, None, pos[0], f, eps=number)
    want = ns.rope(q, None, pos, f, axes=[0, 1] * 4)[0]
    for axes in ((0, 1) * 4, torch.tensor([0, 1] * 4), bytes([0, 1] * 4)):
        assert torch.equal(ns.rope(q, None, pos, f, axes=axes)[0], want)
    assert torch.equal(ns.rope(q, None, pos, f, sections=torch.tensor([3, 5]), scale=2)[0], ns.rope(q, None, pos, f, sections=(3, 5), scale=2.0)[0])


# ---- few rows times narrow weights: 16 or 64 weight rows per workgroup, K divided over workgroups --------
FEW_ROWS = [(m, k, n) for m in (1, 5, 16, 17, 33, 40, 49, 64)
            for k, n in ((8200, 70), (14336, 512), (13973, 37), (6016, 2051), (4160, 5100), (4161, 5100), (12300, 100))]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,k,n", FEW_ROWS)
def test_few_rows_divided_sums(m, k, n, dtype):
    torch_cuda()
    x, w = rand((m, k), dtype, 1), rand((n, k), dtype, 2, 1 / math.sqrt(k))
    b, r = rand((n,), dtype, 3), rand((m, n), dtype, 4)
    check_forward(x, w, None, None, None, ns.linear(x, w), None, "plain")
    y, z = ns.linear(x, w, b, r, activation="gelu", return_preact=True)
    check_forward(x, w, b, r, "gelu", y, z, "bias, gelu, residual")
    assert torch.equal(ns.linear(x, w), ns.linear(x, w))


# ---- every kernel that a call can choose (test_layer_cpu says which sizes reach which) ---------------------
TILE_SIZES = {
    F32: [(69, 360, 72), (67, 62, 358), (355, 81, 65), (3150, 229, 2241), (2549, 2766, 897), (2226, 3299, 226), (1239, 1868, 2771),
          (231, 2572, 2790), (2387, 1102, 2303)],
    BF: [(67, 1001, 66), (71, 63, 992), (1005, 83, 69), (3176, 65, 2465), (1876, 4160, 67), (66, 3318, 2334), (774, 60, 3617),
         (2527, 1155, 65), (65, 910, 3010), (2386, 3965, 67), (2588, 67, 3612), (2505, 66, 3988), (2576, 60, 3123), (3370, 2374, 65),
         (65, 3417, 2324), (4134, 63, 4181), (4153, 4079, 73), (66, 4100, 4124), (65, 4096, 6144)],
}
FEW_ROWS_WHOLE = [(m, k, n) for m in (3, 23, 42, 60) for k, n in ((72, 12300), (1030, 16400), (200, 99))]


@pytest.mark.parametrize("dtype,m,k,n", [(t, *s) for t in (BF, F32) for s in TILE_SIZES[t]])
def test_every_tile(dtype, m, k, n):
    torch_cuda()
    x, w, b, r = rand((m, k), dtype, 1), rand((n, k), dtype, 2, 1 / math.sqrt(k)), rand((n,), F32, 3), rand((m, n), dtype, 4)
    y, z = ns.linear(x, w, b, r, activation="silu", return_preact=True)
    check_forward(x, w, b, r, "silu", y, z, "forward")
    check_forward(x, w, None, None, None, ns.linear(x, w), None, "plain")
    dy, base = rand((m, n), dtype, 5), rand((n, k), F32, 6)
    dx, dw, db = ns.linear_backward(dy, x, w, activation="silu", preact=z, need_dbias=True)
    check_backward(dy, x, w, z, "silu", dx, dw, db, "backward")
    dw = base.clone()
    dx, _, _ = ns.linear_backward(dy, x, w, dw=dw, accumulate=True)
    check_backward(dy, x, w, None, None, dx, dw, None, "accumulated", base)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,k,n", FEW_ROWS_WHOLE)
def test_few_rows_undivided_sums(m, k, n, dtype):
    torch_cuda()
    x, w, b, r = rand((m, k), dtype, 1), rand((n, k), dtype, 2, 1 / math.sqrt(k)), rand((n,), dtype, 3), rand((m, n), F32, 4)
    y, z = ns.linear(x, w, b, r, activation="relu2", return_preact=True)
    check_forward(x, w, b, r, "relu2", y, z, "undivided")


@pytest.mark.filterwarnings("ignore")
def test_inside_torch_compile():
    """A compiled function breaks its graph at these calls: every call with new tensors gives what the plain call gives."""
    torch_cuda()
    w = rand((96, 64), BF, 1)
    pos, f = torch.arange(40, device="cuda"), torch.rand(32, device="cuda")

    def fn(x, w, q):
        y = ns.linear(x * 2, w, activation="silu") + 1
        a, _ = ns.rope(q, None, pos, f)
        return y.float().sum(-1) + a.float().sum((1, 2))

    compiled = torch.compile(fn, backend="eager")
    for i in range(3):
        for grad in (False, True):
            x, q = rand((40, 64), BF, 10 + i), rand((40, 2, 64), BF, 20 + i)
            a, b = [t.clone().requires_grad_(grad) for t in (x, w, q)], [t.clone().requires_grad_(grad) for t in (x, w, q)]
            got, want = compiled(*a), fn(*b)
            assert torch.equal(got, want)
            if grad:
                got.sum().backward()
                want.sum().backward()
                assert all(torch.equal(s.grad, t.grad) for s, t in zip(a, b))


def test_inputs_that_share_rows_or_are_unevenly_spaced():
    torch_cuda()
    x, w, z = rand((5, 7, 64), BF, 1), rand((48, 64), BF, 2), rand((5, 7, 48), BF, 3)
    t, u = x.transpose(0, 1), z.transpose(0, 1)  # [S, B, E] in [B, S, E] memory
    want = ns.linear(t.contiguous(), w, None, u.contiguous(), activation="silu")
    assert torch.equal(ns.linear(t, w, None, u, activation="silu"), want)
    want = ns.linear_backward(u.contiguous(), t.contiguous(), w, activation="gelu", preact=u.contiguous())
    got = ns.linear_backward(u, t, w, activation="gelu", preact=u)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for m in (5, 100):
        row, line = rand((1, 64), BF, 4), rand((1, 48), F32, 5)
        got = ns.linear(row.expand(m, 64), w, None, line.expand(m, 48))
        assert torch.equal(got, ns.linear(row.repeat(m, 1), w, None, line.repeat(m, 1)))
        got = ns.linear_backward(line.expand(m, 48), row.expand(m, 64), w)
        want = ns.linear_backward(line.repeat(m, 1), row.repeat(m, 1), w)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    leaf = x.clone().requires_grad_()
    ns.linear(leaf.transpose(0, 1), w).sum().backward()
    want = ns.linear_backward(torch.ones(35, 48, dtype=BF, device="cuda"), x.view(35, 64), w)[0]
    assert torch.equal(leaf.grad, want.view(5, 7, 64))
    for bad in (lambda: ns.linear(x.transpose(1, 2), rand((48, 7), BF, 6)),           # columns are not contiguous
                lambda: ns.linear(x, w, out=u.transpose(0, 1).transpose(0, 1)),       # an output is not copied
                lambda: ns.linear(x.view(35, 64), w, out=torch.empty(48, dtype=BF, device="cuda").expand(35, 48))):
        with pytest.raises(ns.MuonError) as e:
            bad()
        assert e.value.status == -1


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_bits_do_not_depend_on_alignment(dtype):
    """Views of odd strides and addresses give the bits of dense operands, whichever kernel their sizes choose."""
    torch_cuda()

    def odd(t):
        buf = torch.zeros(t.shape[0], t.shape[1] + 3, dtype=t.dtype, device="cuda")
        buf[:, 1:1 + t.shape[1]] = t
        return buf[:, 1:1 + t.shape[1]]

    for m, k, n in ((3, 256, 200), (24, 2504, 9472), (40, 4096, 1100), (64, 8192, 1024), (70, 264, 520), (300, 1000, 2000)):
        x, w, dy = rand((m, k), dtype, 1), rand((n, k), dtype, 2), rand((m, n), dtype, 3)
        want = ns.linear(x, w)
        assert torch.equal(ns.linear(odd(x), w), want) and torch.equal(ns.linear(x, odd(w)), want)
        a, b = ns.linear_backward(dy, x, w), ns.linear_backward(odd(dy), odd(x), odd(w))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
