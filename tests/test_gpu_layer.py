"""The layer operators on the GPU against their definitions in fp64.

Tolerances are derived element by element.  u(t) = eps(t) / 2 is the largest
relative rounding of type t.  A product summed over K terms in fp32 is off by
at most (K + 8) 2^-23 of the sum of its terms' magnitudes (2^-23 covers a
matrix unit that truncates); an operand that the operator rounds to bf16 first
(the gradient behind an activation) adds 2^-8 of that sum."""
import math

import pytest
import torch

import newton_schulz_ns5_amd as ns
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}
ACTS = [None, "relu", "relu2", "silu", "gelu", "gelu_tanh"]


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def act64(z, name):
    """The activation, its derivative, and a bound of what fp32 does to each (absolute)."""
    a = z.abs()
    if name is None:
        return z, torch.ones_like(z), 0 * z, 0 * z
    if name == "relu":
        return z.clamp(min=0), (z > 0).double(), 0 * z, 0 * z
    if name == "relu2":
        p = z.clamp(min=0)
        return p * p, 2 * p, p * p * 2.0 ** -23, p * 2.0 ** -22
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        pdf = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        # erf to a few units of 2^-24; exp's argument -z^2/2 is rounded before it is raised
        return z * cdf, cdf + z * pdf, a * 2.0 ** -21, 2.0 ** -21 + a * pdf * (z * z + 4) * 2.0 ** -22
    if name == "silu":
        t, dt = z, torch.ones_like(z)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        t, dt = c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(t)
    # logistic: its argument is rounded a few times, exp and the reciprocal are off by a unit each
    rel = (4 * t.abs() + 6) * 2.0 ** -23
    slope = s + z * s * (1 - s) * dt
    return z * s, slope, (z * s).abs() * rel, (s + a * s * dt) * (2 * rel)


def close(got, want, tol, what):
    assert got.shape == want.shape, what
    off = (got.double() - want).abs() - tol
    assert not torch.isnan(got).any(), what
    worst = int(off.argmax()) if off.numel() else 0
    assert off.numel() == 0 or float(off.max()) <= 0, (what, "at", worst, float(got.flatten()[worst]), float(want.flatten()[worst]),
                                                       float(tol.flatten()[worst]))


def slope_bound(name, z, room):
    """The largest |act'| within `room` of z."""
    if name == "relu2":
        return 2 * (z.abs() + room)
    return torch.full_like(z, 1.0 if name in (None, "relu") else 1.2)


def check_forward(x, w, b, r, act, y, z, what):
    x64, w64 = x.double(), w.double()
    k = x.shape[-1]
    pre = x64 @ w64.t()
    mag = x64.abs() @ w64.abs().t()
    if b is not None:
        pre, mag = pre + b.double(), mag + b.double().abs()
    off = (k + 8) * 2.0 ** -23 * mag
    if z is not None:
        close(z, pre, off * (1 + U[z.dtype]) + U[z.dtype] * pre.abs(), (what, "preact"))
    val, _, aerr, _ = act64(pre, act)
    tol = off * slope_bound(act, pre, off) + aerr + val.abs() * 2.0 ** -22
    if r is not None:
        val = val + r.double()
        tol = tol + val.abs() * 2.0 ** -23
    close(y, val, tol * (1 + U[y.dtype]) + U[y.dtype] * val.abs(), what)


SIZES = [(1, 1, 1), (1, 4096, 640), (2, 33, 65), (5, 130, 7), (16, 512, 1000), (17, 64, 64), (31, 1001, 129),
         (48, 768, 256), (65, 200, 513), (127, 127, 127), (128, 256, 384), (130, 64, 300), (257, 320, 260), (300, 8, 1040),
         (512, 1024, 512), (9, 8200, 3200), (24, 4096, 4100), (64, 2050, 12300)]
# Outputs of a little more than whole rounds of the largest tile: columns, rows.
BIG = [(4096, 128, 4400), (4400, 128, 4096), (4104, 72, 4104)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,k,n", SIZES)
def test_linear_sizes(m, k, n, dtype):
    torch_cuda()
    x, w = rand((m, k), dtype, 1), rand((n, k), dtype, 2, 1 / math.sqrt(k))
    b, r = rand((n,), dtype, 3), rand((m, n), dtype, 4)
    check_forward(x, w, None, None, None, ns.linear(x, w), None, "plain")
    y, z = ns.linear(x, w, b, r, activation="silu", return_preact=True)
    check_forward(x, w, b, r, "silu", y, z, "bias, silu, residual")


@pytest.mark.parametrize("m,k,n", BIG)
def test_linear_big_outputs(m, k, n):
    torch_cuda()
    x, w = rand((m, k), BF, 1), rand((n, k), BF, 2, 1 / math.sqrt(k))
    b, r = rand((n,), BF, 3), rand((m, n), F32, 4)
    y, z = ns.linear(x, w, b, r, activation="gelu_tanh", return_preact=True)
    check_forward(x, w, b, r, "gelu_tanh", y, z, "forward")
    dy = rand((m, n), BF, 5)
    dx, dw, _ = ns.linear_backward(dy, x, w)
    check_backward(dy, x, w, None, None, dx, dw, None, "backward")
    # the input gradient of an m x n output over few columns, and the weight gradient of one over few rows
    x, w, dy = rand((m, n), BF, 6), rand((k, n), BF, 7), rand((m, k), BF, 8)
    dx, dw, _ = ns.linear_backward(dy, x, w, dw_dtype=F32)
    check_backward(dy, x, w, None, None, dx, dw, None, "backward, wide")
    x, w, dy = rand((k, n), BF, 9), rand((m, n), BF, 10), rand((k, m), BF, 11)
    dw = rand((m, n), BF, 12)
    base = dw.clone()
    ns.linear_backward(dy, x, w, need_dx=False, dw=dw, accumulate=True)
    check_backward(dy, x, w, None, None, None, dw, None, "weight gradient", base)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,k,n", [(3, 96, 80), (96, 96, 80), (256, 128, 512)])
def test_linear_activations(m, k, n, act, dtype):
    torch_cuda()
    x, w, b = rand((m, k), dtype, 5), rand((n, k), dtype, 6, 2 / math.sqrt(k)), rand((n,), F32, 7)
    for r in (None, rand((m, n), F32, 8), rand((m, n), BF, 9)):
        y, z = ns.linear(x, w, b, r, activation=act, return_preact=True)
        assert y.dtype == (dtype if r is None else r.dtype) and z.dtype == dtype
        check_forward(x, w, b, r, act, y, z, (act, None if r is None else r.dtype))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,k,n,at", [(1, 96, 200, 1), (20, 100, 72, 3), (70, 100, 72, 1), (140, 136, 264, 8), (300, 65, 130, 5)])
def test_linear_strided_views_keep_their_surroundings(m, k, n, at, dtype):
    """x, w, the residual and the outputs are columns of wider buffers whose other
    values are NaN: none of them may reach a result or be written over."""
    torch_cuda()

    def inside(rows, cols, seed):
        buf = torch.full((rows, cols + 2 * at + 3), float("nan"), dtype=dtype, device="cuda")
        view = buf[:, at:at + cols]
        view.copy_(rand((rows, cols), dtype, seed))
        return buf, view

    (_, x), (_, w), (_, r) = inside(m, k, 11), inside(n, k, 12), inside(m, n, 13)
    ybuf, y = inside(m, n, 14)
    zbuf, z = inside(m, n, 15)
    ns.linear(x, w, None, r, activation="relu", out=y, preact=z)
    check_forward(x, w, None, r, "relu", y, z, "views")
    for buf in (ybuf, zbuf):
        assert torch.isnan(buf[:, :at]).all() and torch.isnan(buf[:, at + n:]).all()


def test_linear_adds_onto_its_residual_in_place():
    torch_cuda()
    x, w, r = rand((200, 96), BF, 21), rand((136, 96), BF, 22), rand((200, 136), F32, 23)
    want = ns.linear(x, w, None, r, activation="gelu")
    again = r.clone()
    assert ns.linear(x, w, None, again, activation="gelu", out=again) is again
    assert torch.equal(again, want)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_linear_rows_are_independent(m):
    """A row with NaN and infinities leaves the other rows' bits alone, and gives
    what IEEE sums give."""
    torch_cuda()
    x, w = rand((m, 160), BF, 31), rand((320, 160), BF, 32)
    want = ns.linear(x, w, activation="relu")
    bad = x.clone()
    bad[m // 2, 5] = float("nan")
    got = ns.linear(bad, w, activation="relu")
    assert torch.isnan(got[m // 2]).all()
    keep = [i for i in range(m) if i != m // 2]
    assert torch.equal(got[keep], want[keep])
    bad[m // 2, 5] = float("inf")
    got = ns.linear(bad, w)
    assert torch.isinf(got[m // 2]).all()


def test_linear_empty_sizes():
    torch_cuda()
    b, r = rand((24,), BF, 1), rand((10, 24), BF, 2)
    x, w = rand((10, 0), BF, 3), rand((24, 0), BF, 4)
    y = ns.linear(x, w, b, r, activation="relu")  # no columns: relu(bias) + residual
    want = b.double().clamp(min=0) + r.double()
    close(y, want, want.abs() * (U[BF] + 2.0 ** -20), "k = 0")
    x = rand((100, 0), BF, 3)
    y = ns.linear(x, w, b, None)
    assert torch.equal(y, b.expand(100, 24))
    assert ns.linear(rand((0, 8), BF, 5), rand((24, 8), BF, 6)).shape == (0, 24)
    assert ns.linear(rand((4, 8), BF, 5), rand((0, 8), BF, 6)).shape == (4, 0)
    dx, dw, db = ns.linear_backward(rand((0, 24), BF, 1), rand((0, 8), BF, 2), rand((24, 8), BF, 3), need_dbias=True)
    assert dx.shape == (0, 8) and not dw.any() and not db.any()
    dx, dw, _ = ns.linear_backward(rand((5, 0), BF, 1), rand((5, 8), BF, 2), rand((0, 8), BF, 3))
    assert not dx.any() and dw.shape == (0, 8)


def test_empty_sum_ignores_its_operands_strides():
    """The C entry point with n = 0: dx is zero whatever the strides of the empty dy and w."""
    torch_cuda()
    import ctypes
    from newton_schulz_ns5_amd import _lib
    dx = torch.full((70, 24), 7.0, dtype=BF, device="cuda")
    p = _lib.LinearGrad(m=70, n=0, k=24, dtype=1, dy_dtype=1, dx_dtype=1, dy_row_stride=5, w_row_stride=3,
                        dx=dx.data_ptr(), dx_row_stride=24)
    need = ctypes.c_size_t()
    _lib.check(_lib.lib().muon_linear_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(need)))
    ws = torch.empty(max(need.value, 256), dtype=torch.uint8, device="cuda")
    _lib.check(_lib.lib().muon_linear_backward(ctypes.byref(p), ws.data_ptr(), ws.numel(),
                                               torch.cuda.current_stream().cuda_stream))
    assert not dx.any()


def test_linear_beyond_32_bit_offsets():
    """Operands of more than 2^32 bytes: rows at the end of x, and sums over all of them."""
    torch_cuda()
    m, k, n = 70000, 32768, 72
    x = torch.empty((m, k), dtype=BF, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    w, dy = rand((n, k), BF, 2, 1 / math.sqrt(k)), rand((m, n), BF, 3)
    y = ns.linear(x, w)
    tail = slice(m - 300, m)
    check_forward(x[tail], w, None, None, None, y[tail], None, "last rows")
    dx, dw, _ = ns.linear_backward(dy, x, w)
    check_backward(dy[tail], x[tail], w, None, None, dx[tail], None, None, "last rows")
    cols = slice(k - 64, k)
    want, size = dy.double().t() @ x[:, cols].double(), dy.double().abs().t() @ x[:, cols].double().abs()
    close(dw[:, cols], want, size * (m + 8) * 2.0 ** -23 + U[BF] * want.abs(), "dw")


def test_linear_leading_dimensions():
    torch_cuda()
    x, w = rand((3, 5, 64), BF, 1), rand((40, 64), BF, 2)
    assert torch.equal(ns.linear(x, w).view(15, 40), ns.linear(x.view(15, 64), w))
    assert ns.linear(x[0, 0], w).shape == (40,)


def check_backward(dy, x, w, z, act, dx, dw, db, what, base_w=None, base_b=None):
    g = dy.double()
    gerr = 0 * g
    if act is not None:
        _, slope, _, serr = act64(z.double(), act)
        gerr = g.abs() * serr
        g = g * slope
        gerr = gerr + g.abs() * 2.0 ** -23
    fine = gerr.clone()
    if x.dtype == BF and (act is not None or dy.dtype != BF):
        gerr = gerr + g.abs() * 2.0 ** -8
    ga = g.abs()
    m, n = g.shape
    if dx is not None:
        want = g @ w.double()
        tol = gerr @ w.double().abs() + (n + 8) * 2.0 ** -23 * (ga @ w.double().abs())
        close(dx, want, tol * 1.01 + U[dx.dtype] * want.abs(), (what, "dx"))
    if dw is not None:
        want = g.t() @ x.double()
        tol = gerr.t() @ x.double().abs() + (m + 8) * 2.0 ** -23 * (ga.t() @ x.double().abs())
        if base_w is not None:
            want = want + base_w.double()
            tol = tol + want.abs() * 2.0 ** -23
        close(dw, want, tol * 1.01 + U[dw.dtype] * want.abs(), (what, "dw"))
    if db is not None:
        want, tol = g.sum(0), fine.sum(0) + (m + 8) * 2.0 ** -24 * ga.sum(0)
        if base_b is not None:
            want = want + base_b.double()
            tol = tol + want.abs() * 2.0 ** -23
        close(db, want, tol * 1.01 + U[db.dtype] * want.abs(), (what, "db"))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,k,n", SIZES)
def test_linear_backward_sizes(m, k, n, dtype):
    torch_cuda()
    x, w, dy = rand((m, k), dtype, 1), rand((n, k), dtype, 2), rand((m, n), dtype, 3)
    dx, dw, db = ns.linear_backward(dy, x, w, need_dbias=True, dw_dtype=F32)
    check_backward(dy, x, w, None, None, dx, dw, db, "no activation")
    z = rand((m, n), dtype, 4)
    dx, dw, db = ns.linear_backward(dy, x, w, activation="gelu", preact=z, need_dbias=True, dbias_dtype=F32)
    check_backward(dy, x, w, z, "gelu", dx, dw, db, "gelu")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dy_dtype", [BF, F32], ids=["dy_bf16", "dy_f32"])
def test_linear_backward_activations(act, dtype, dy_dtype):
    torch_cuda()
    m, k, n = 150, 72, 200
    x, w, dy, z = rand((m, k), dtype, 1), rand((n, k), dtype, 2), rand((m, n), dy_dtype, 3), rand((m, n), dtype, 4, 3)
    z[0, :4] = torch.tensor([0.0, -0.0, 200.0, -200.0], dtype=dtype)
    z[1, :2] = torch.tensor([float("inf"), float("-inf")], dtype=dtype)
    dx, dw, db = ns.linear_backward(dy, x, w, activation=act, preact=z if act else None, need_dbias=True)
    zz = z.clone()
    if act == "relu2":  # its slope has no limit at infinity
        zz[1, :2] = 1.0
        dx, dw, db = ns.linear_backward(dy, x, w, activation=act, preact=zz, need_dbias=True)
    elif act:
        zz[1, :2] = torch.tensor([100.0, -100.0], dtype=dtype)  # every slope is 1 or 0 from here on
    check_backward(dy, x, w, zz if act else None, act, dx, dw, db, act)


def test_linear_backward_accumulates_and_leaves_out():
    torch_cuda()
    m, k, n = 90, 130, 68
    x, w, dy = rand((m, k), BF, 1), rand((n, k), BF, 2), rand((m, n), BF, 3)
    for t in (F32, BF):
        dw, db = rand((n, k), t, 4), rand((n,), t, 5)
        bw, bb = dw.clone(), db.clone()
        r = ns.linear_backward(dy, x, w, need_dx=False, need_dbias=True, dw=dw, dbias=db, accumulate=True)
        assert r[0] is None and r[1] is dw and r[2] is db
        check_backward(dy, x, w, None, None, None, dw, db, t, bw, bb)
    r = ns.linear_backward(dy, x, w, need_dx=False, need_dw=False, need_dbias=True)
    assert r[0] is None and r[1] is None
    check_backward(dy, x, w, None, None, None, None, r[2], "bias only")
    whole = ns.linear_backward(dy, x, w)
    assert torch.equal(ns.linear_backward(dy, x, w, need_dw=False)[0], whole[0])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,k,n,at", [(20, 100, 72, 3), (150, 136, 264, 8), (260, 65, 130, 1)])
def test_linear_backward_strided_views(m, k, n, at, dtype):
    torch_cuda()

    def inside(rows, cols, seed):
        buf = torch.full((rows, cols + 2 * at + 1), float("nan"), dtype=dtype, device="cuda")
        buf[:, at:at + cols] = rand((rows, cols), dtype, seed)
        return buf, buf[:, at:at + cols]

    (_, x), (_, w), (_, dy), (_, z) = inside(m, k, 1), inside(n, k, 2), inside(m, n, 3), inside(m, n, 4)
    (bx, dx), (bw, dw) = inside(m, k, 5), inside(n, k, 6)
    _, _, db = ns.linear_backward(dy, x, w, activation="silu", preact=z, dx=dx, dw=dw, need_dbias=True)
    check_backward(dy, x, w, z, "silu", dx, dw, db, "views")
    for buf in (bx, bw):
        assert torch.isnan(buf[:, :at]).all() and torch.isnan(buf[:, buf.shape[1] - at - 1:]).all()


@pytest.mark.parametrize("act", ACTS)
def test_linear_gradient_against_differences(act):
    """<dL/dp, d> against (L(p + h d) - L(p - h d)) / 2 h in fp64 of the definition:
    the difference quotient is off by h^2 times a third derivative of order one."""
    torch_cuda()
    m, k, n, h = 24, 40, 56, 1e-4
    x, w, b, dy = (rand(s, F32, i) for i, s in enumerate([(m, k), (n, k), (n,), (m, n)]))
    w = w / math.sqrt(k)
    _, z = ns.linear(x, w, b, activation=act, return_preact=True)
    grads = ns.linear_backward(dy, x, w, activation=act, preact=z if act else None, need_dbias=True)

    def loss(*p):
        return (act64(p[0] @ p[1].t() + p[2], act)[0] * dy.double()).sum()

    p = [t.double() for t in (x, w, b)]
    for i, g in enumerate(grads):
        d = rand(p[i].shape, F32, 50 + i).double()
        up, down = list(p), list(p)
        up[i], down[i] = p[i] + h * d, p[i] - h * d
        quotient = float((loss(*up) - loss(*down)) / (2 * h))
        size = float((g.double().abs() * d.abs()).sum())
        # fp32 sums, and for relu a kink within h of at most a few of the 1344 pre-activations
        assert abs(float((g.double() * d).sum()) - quotient) <= size * (2e-4 if act == "relu" else 2e-6) + 1e-6, (act, i)


def test_linear_is_deterministic_and_batch_free():
    torch_cuda()
    x, w, dy, z = rand((300, 256), BF, 1), rand((520, 256), BF, 2), rand((300, 520), BF, 3), rand((300, 520), BF, 4)
    a = ns.linear_backward(dy, x, w, activation="silu", preact=z, need_dbias=True)
    b = ns.linear_backward(dy, x, w, activation="silu", preact=z, need_dbias=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert torch.equal(ns.linear(x, w), ns.linear(x, w))


def test_linear_autograd():
    torch_cuda()
    x, w, b, r = rand((2, 33, 48), BF, 1), rand((80, 48), BF, 2), rand((80,), F32, 3), rand((2, 33, 80), F32, 4)
    leaves = [t.clone().requires_grad_() for t in (x, w, b, r)]
    y = ns.linear(*leaves, activation="gelu_tanh")
    y.sum().backward()  # an expanded gradient
    _, z = ns.linear(x, w, b, r, activation="gelu_tanh", return_preact=True)
    dy = torch.ones_like(y)
    dx, dw, db = ns.linear_backward(dy.view(66, 80), x, w, activation="gelu_tanh", preact=z, need_dbias=True, dbias_dtype=F32)
    for leaf, want in zip(leaves, (dx, dw, db, dy)):
        assert leaf.grad.dtype == leaf.dtype and torch.equal(leaf.grad, want.view(leaf.shape))
    with pytest.raises(ns.MuonError):
        ns.linear(leaves[0], w, out=torch.empty(2, 33, 80, dtype=BF, device="cuda"))


# ---- per-head norms and rotation --------------------------------------------------------
def ref_qk(x, w, pos, f, axes, rot, inter, scale, eps):
    """u, y and the turn's pieces in fp64; pos [axes, ...tokens]."""
    x = x.double()
    d = x.shape[-1]
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) if eps is not None else torch.ones_like(x[..., :1])
    u = x * r * (w.double() if w is not None else 1)
    p = torch.arange(rot // 2, device=x.device)
    theta = pos.double()[axes].movedim(0, -1) * f.double()
    a, b = (2 * p, 2 * p + 1) if inter else (p, p + rot // 2)
    return u, r, scale * torch.cos(theta)[..., None, :], scale * torch.sin(theta)[..., None, :], a, b


def turn(u, c, s, a, b):
    y = u.clone()
    y[..., a], y[..., b] = u[..., a] * c - u[..., b] * s, u[..., b] * c + u[..., a] * s
    return y


def spread(u, a, b):
    """Per value the magnitudes that its turned value is made of."""
    m = u.abs().clone()
    m[..., a] = m[..., b] = u[..., a].abs() + u[..., b].abs()
    return m


def check_qk(x, w, pos, f, axes, inter, scale, eps, y, what):
    rot = 2 * f.shape[0]
    u, _, c, s, a, b = ref_qk(x, w, pos, f, axes, rot, inter, scale, eps)
    want = turn(u, c, s, a, b)
    # the row's sum of squares, its root and the weight: under 40 units of 2^-24; cos and sin within 2^-21
    tol = spread(u, a, b) * max(1.0, abs(scale)) * 2.0 ** -19
    close(y, want, tol + U[y.dtype] * want.abs(), what)


def check_qk_backward(g, x, w, pos, f, axes, inter, scale, eps, dx, dw, what):
    rot = 2 * f.shape[0]
    _, r, c, s, a, b = ref_qk(x, w, pos, f, axes, rot, inter, scale, eps)
    n = x.double() * r
    h = turn(g.double(), c, -s, a, b)
    hm = spread(g.double(), a, b) * max(1.0, abs(scale))
    wt = w.double() if w is not None else torch.ones(x.shape[-1], dtype=torch.float64, device=x.device)
    gw, gm = h * wt, hm * wt.abs()
    mean = (gw * n).mean(-1, keepdim=True)
    want = r * (gw - n * mean)
    tol = r * (gm + n.abs() * (gm * n.abs()).mean(-1, keepdim=True)) * 2.0 ** -18
    close(dx, want, tol + U[dx.dtype] * want.abs(), (what, "dx"))
    if dw is not None:
        dims = tuple(range(x.dim() - 1))
        want = (h * n).sum(dims)
        size = (hm * n.abs()).sum(dims)
        rows = x.numel() // x.shape[-1]
        close(dw, want, size * (2.0 ** -18 + rows * 2.0 ** -24) + U[dw.dtype] * want.abs(), (what, "dw"))


def packed(t, hq, hk, d, dtype, seed, pad=0):
    buf = rand((t, (hq + 2 * hk) * d + pad), dtype, seed)
    return buf, buf[:, :hq * d].view(t, hq, d), buf[:, hq * d:(hq + hk) * d].view(t, hk, d)


HEADS = [  # tokens, q heads, k heads, dim, rotary
    (1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (3, 4, 2, 128, 64), (70, 28, 4, 128, 128), (33, 16, 16, 80, 80),
    (19, 3, 1, 72, 72), (5, 5, 5, 96, 48), (40, 7, 1, 112, 112), (9, 2, 2, 192, 96), (21, 8, 1, 256, 256), (6, 3, 2, 512, 512),
    (7, 2, 1, 20, 8), (11, 3, 2, 63, 30), (4, 2, 2, 1, 0), (13, 2, 1, 1000, 500), (600, 2, 1, 64, 64), (5, 1, 2, 130, 2)]


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("t,hq,hk,d,rot", HEADS)
def test_qk_norm_rope(t, hq, hk, d, rot, dtype, inter):
    torch_cuda()
    _, q, k = packed(t, hq, hk, d, dtype, 1)
    wq, wk = 1 + rand((d,), F32, 2, 0.2), 1 + rand((d,), F32, 3, 0.2)
    wq, wk = wq.to(dtype), wk.to(dtype)
    pos = torch.randint(0, 1 << 20, (t,), device="cuda")
    f = torch.pow(10000.0, -torch.arange(rot // 2, device="cuda", dtype=torch.float64) / max(1, rot // 2))
    how = dict(interleaved=inter, eps=1e-5)
    yq, yk = ns.qk_norm_rope(q, k, pos, f, q_weight=wq, k_weight=wk, **how)
    axes = torch.zeros(rot // 2, dtype=torch.int64, device="cuda")
    for x, w, y in ((q, wq, yq), (k, wk, yk)):
        check_qk(x, w, pos[None], f, axes, inter, 1.0, 1e-5, y, "forward")
    gq, gk = rand((t, hq, d), dtype, 5), rand((t, hk, d), dtype, 6)
    dq, dk, dwq, dwk = ns.qk_norm_rope_backward(gq, gk, q, k, pos, f, q_weight=wq, k_weight=wk, **how)
    for g, x, w, dx, dw in ((gq, q, wq, dq, dwq), (gk, k, wk, dk, dwk)):
        check_qk_backward(g, x, w, pos[None], f, axes, inter, 1.0, 1e-5, dx, dw, "backward")


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("axes_n,sections,d", [(3, [16, 24, 24], 128), (2, [20, 20], 80), (4, [1, 0, 7, 8], 64), (3, [5, 5, 5], 63)])
def test_rope_axes(axes_n, sections, d, dtype, inter):
    torch_cuda()
    t, hq, hk = 45, 6, 2
    pairs = sum(sections)
    _, q, k = packed(t, hq, hk, d, dtype, 1)
    pos = torch.randint(0, 5000, (axes_n, t), device="cuda", dtype=torch.int32)
    f = torch.rand(pairs, device="cuda")
    axes = torch.repeat_interleave(torch.arange(axes_n, device="cuda"), torch.tensor(sections, device="cuda"))
    yq, yk = ns.rope(q, k, pos, f, sections=sections, interleaved=inter, scale=1.25)
    for x, y in ((q, yq), (k, yk)):
        check_qk(x, None, pos, f, axes, inter, 1.25, None, y, "rope")
    shuffled = axes[torch.randperm(pairs, device="cuda")]
    yq, _ = ns.rope(q, k, pos, f, axes=shuffled.tolist(), interleaved=inter)
    check_qk(q, None, pos, f, shuffled, inter, 1.0, None, yq, "one axis per pair")
    gq, gk = rand((t, hq, d), dtype, 5), rand((t, hk, d), dtype, 6)
    dq, dk = ns.rope_backward(gq, gk, pos, f, sections=sections, interleaved=inter, scale=1.25)
    for g, dx in ((gq, dq), (gk, dk)):  # the opposite angles
        check_qk(g, None, -pos.long(), f, axes, inter, 1.25, None, dx, "rope backward")


def test_qk_batched_layouts_and_positions():
    torch_cuda()
    B, S, hq, hk, d = 3, 10, 4, 2, 64
    wq = 1 + rand((d,), BF, 2, 0.1)
    f = torch.rand(d // 2, device="cuda", dtype=torch.float64)
    q, k = rand((B, hq, S, d), BF, 1).transpose(1, 2), rand((B, hk, S, d), BF, 3).transpose(1, 2)  # heads first in memory
    pos = torch.randint(0, 100000, (B, S), device="cuda")
    flat = ns.qk_norm_rope(q.reshape(B * S, hq, d), k.reshape(B * S, hk, d), pos.view(-1), f, q_weight=wq)
    got = ns.qk_norm_rope(q, k, pos, f, q_weight=wq)
    assert all(torch.equal(a, b.view(a.shape)) for a, b in zip(got, flat))
    one = ns.qk_norm_rope(q, k, pos[0], f, q_weight=wq)  # one row of positions for every sequence
    two = ns.qk_norm_rope(q, k, pos[:1].expand(B, S), f, q_weight=wq)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    out = torch.empty(B, hq, S, d, dtype=BF, device="cuda").transpose(1, 2)
    ns.qk_norm_rope(q, None, pos, f, q_weight=wq, q_out=out)
    assert torch.equal(out, got[0])
    only_k = ns.qk_norm_rope(None, k, pos, f)
    assert only_k[0] is None and torch.equal(only_k[1], got[1])


@pytest.mark.parametrize("d,pad", [(128, 0), (80, 0), (64, 3), (63, 1)])
def test_qk_in_place_on_packed_rows(d, pad):
    torch_cuda()
    t, hq, hk = 50, 6, 2
    buf, q, k = packed(t, hq, hk, d, BF, 1, pad)
    rot = d // 2 * 2
    f, pos = torch.rand(rot // 2, device="cuda"), torch.arange(t, device="cuda") - 7  # positions below zero too
    want = ns.qk_norm_rope(q, k, pos, f)
    rest = buf[:, (hq + hk) * d:].clone()
    got = ns.qk_norm_rope(q, k, pos, f, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(buf[:, (hq + hk) * d:], rest)
    gq, gk = rand((t, hq, d), BF, 5), rand((t, hk, d), BF, 6)
    want = ns.qk_norm_rope_backward(gq, gk, q, k, pos, f)
    ns.qk_norm_rope_backward(gq, gk, q, k, pos, f, dq=gq, dk=gk)
    assert torch.equal(gq, want[0]) and torch.equal(gk, want[1])


def test_qk_single_token_rows_in_place():
    """Decoding: one token per sequence, q and k views of the packed rows, in place, in both shapes."""
    torch_cuda()
    B, hq, hk, d = 9, 8, 2, 128
    buf, q, k = packed(B, hq, hk, d, BF, 1)
    f, pos = torch.rand(d // 2, device="cuda"), torch.randint(0, 100000, (B,), device="cuda")
    wq, wk = 1 + rand((d,), F32, 2, 0.1), 1 + rand((d,), F32, 3, 0.1)  # fp32 weights on bf16 heads
    want = ns.qk_norm_rope(q, k, pos, f, q_weight=wq, k_weight=wk)
    axes = torch.zeros(d // 2, dtype=torch.int64, device="cuda")
    check_qk(q, wq, pos[None], f, axes, False, 1.0, 1e-6, want[0], "fp32 weight")
    again = buf.clone()
    qv, kv = again[:, :hq * d].view(B, 1, hq, d), again[:, hq * d:(hq + hk) * d].view(B, 1, hk, d)
    ns.qk_norm_rope(qv, kv, pos.view(B, 1), f, q_weight=wq, k_weight=wk, q_out=qv, k_out=kv)
    assert torch.equal(qv.reshape(B, hq, d), want[0]) and torch.equal(kv.reshape(B, hk, d), want[1])
    assert torch.equal(again[:, (hq + hk) * d:], buf[:, (hq + hk) * d:])
    one = buf[:1].clone()
    qv, kv = one[:, :hq * d].view(1, hq, d), one[:, hq * d:(hq + hk) * d].view(1, hk, d)
    ns.qk_norm_rope(qv, kv, pos[:1], f, q_weight=wq, k_weight=wk, q_out=qv, k_out=kv)
    assert torch.equal(qv, want[0][:1]) and torch.equal(kv, want[1][:1])


def test_qk_beyond_32_bit_offsets():
    torch_cuda()
    t, h, d = 140000, 128, 128
    q = torch.empty((t, h, d), dtype=BF, device="cuda")
    q.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    f, pos = torch.rand(d // 2, device="cuda"), torch.arange(t, device="cuda")
    axes = torch.zeros(d // 2, dtype=torch.int64, device="cuda")
    y, _ = ns.qk_norm_rope(q, None, pos, f)
    check_qk(q[-50:], None, pos[None, -50:], f, axes, False, 1.0, 1e-6, y[-50:], "last tokens")
    ns.qk_norm_rope_backward(y, None, q, None, pos, f, dq=y)
    assert torch.isfinite(y[-50:]).all()


def test_qk_far_positions():
    """Angles keep fp32's full precision at positions where an fp32 product would not."""
    torch_cuda()
    q = rand((6, 2, 128), F32, 1)
    pos = torch.tensor([0, 1, 10 ** 6, 10 ** 9, 2 ** 40, -(10 ** 9)], device="cuda")
    f = torch.pow(10000.0, -torch.arange(64, device="cuda", dtype=torch.float64) / 64)
    y, _ = ns.rope(q, None, pos, f)
    axes = torch.zeros(64, dtype=torch.int64, device="cuda")
    # a product of 2^40 in fp64 is itself off by 2^-13 radians, in the oracle as in the kernel
    u, _, c, s, a, b = ref_qk(q, None, pos[None], f, axes, 128, False, 1.0, None)
    tol = spread(u, a, b) * (2.0 ** -19 + pos.abs().double()[:, None, None] * 2.0 ** -51)
    close(y, turn(u, c, s, a, b), tol + U[F32] * y.double().abs(), "far")


def test_qk_rows_of_zeros_and_nan():
    torch_cuda()
    q = rand((8, 4, 128), BF, 1)
    f, pos = torch.rand(64, device="cuda"), torch.arange(8, device="cuda")
    want, _ = ns.qk_norm_rope(q, None, pos, f)
    bad = q.clone()
    bad[3, 1] = 0
    bad[5, 2, 7] = float("nan")
    got, _ = ns.qk_norm_rope(bad, None, pos, f)
    assert not got[3, 1].any() and torch.isnan(got[5, 2]).all()
    keep = torch.ones(8, 4, dtype=torch.bool, device="cuda")
    keep[3, 1] = keep[5, 2] = False
    assert torch.equal(got[keep], want[keep])
    g = rand((8, 4, 128), BF, 2)
    dq, _, _, _ = ns.qk_norm_rope_backward(g, None, bad, None, pos, f, eps=1e-6)
    assert torch.isfinite(dq[keep]).all() and torch.isfinite(dq[3, 1]).all()


def test_qk_gradient_against_differences():
    torch_cuda()
    t, hq, hk, d, h = 6, 3, 2, 64, 1e-4
    _, q, k = packed(t, hq, hk, d, F32, 1)
    wq, wk = 1 + rand((d,), F32, 2, 0.2), 1 + rand((d,), F32, 3, 0.2)
    f, pos = torch.rand(32, device="cuda", dtype=torch.float64), torch.randint(0, 1000, (t,), device="cuda")
    gq, gk = rand((t, hq, d), F32, 4), rand((t, hk, d), F32, 5)
    grads = ns.qk_norm_rope_backward(gq, gk, q, k, pos, f, q_weight=wq, k_weight=wk, eps=1e-6)
    axes = torch.zeros(32, dtype=torch.int64, device="cuda")

    def loss(q, k, wq, wk):
        out = 0
        for x, w, g in ((q, wq, gq), (k, wk, gk)):
            u, _, c, s, a, b = ref_qk(x, w, pos[None], f, axes, 64, False, 1.0, 1e-6)
            out = out + (turn(u, c, s, a, b) * g.double()).sum()
        return out

    p = [x.double() for x in (q, k, wq, wk)]
    for i, g in enumerate(grads):
        e = rand(p[i].shape, F32, 60 + i).double()
        up, down = list(p), list(p)
        up[i], down[i] = p[i] + h * e, p[i] - h * e
        quotient = float((loss(*up) - loss(*down)) / (2 * h))
        size = float((g.double().abs() * e.abs()).sum())
        assert abs(float((g.double() * e).sum()) - quotient) <= size * 2e-6 + 1e-6, i


def test_qk_autograd():
    torch_cuda()
    t, hq, hk, d = 20, 4, 2, 64
    _, q, k = packed(t, hq, hk, d, BF, 1)
    leaves = [x.clone().requires_grad_() for x in (q, k, 1 + rand((d,), BF, 2, 0.1), 1 + rand((d,), BF, 3, 0.1))]
    f, pos = torch.rand(32, device="cuda"), torch.arange(t, device="cuda")
    yq, yk = ns.qk_norm_rope(leaves[0], leaves[1], pos, f, q_weight=leaves[2], k_weight=leaves[3])
    gq, gk = rand((t, hq, d), BF, 4), rand((t, hk, d), BF, 5)
    torch.autograd.backward([yq, yk], [gq, gk])
    want = ns.qk_norm_rope_backward(gq, gk, q, k, pos, f, q_weight=leaves[2].detach(), k_weight=leaves[3].detach())
    assert all(torch.equal(a.grad, b) for a, b in zip(leaves, want))
    x = q.clone().requires_grad_()
    y, none = ns.rope(x, None, pos, f)
    y.backward(gq)
    assert none is None and torch.equal(x.grad, ns.rope_backward(gq, None, pos, f)[0])
    # only one of the two outputs is used
    a, b = q.clone().requires_grad_(), k.clone().requires_grad_()
    ns.rope(a, b, pos, f)[1].backward(gk)
    assert a.grad is None and torch.equal(b.grad, ns.rope_backward(None, gk, pos, f)[1])


# ---- together, as a layer uses them -----------------------------------------------------
def block(x, wqkv, bqkv, wo, nq, nk, pos, f, hq, hk, d, ops):
    """A projection of packed q, k and v rows, norms and rotation of q and k, a
    stand-in for what follows them (each key head's rows scaled onto the query
    heads that share it), and the output projection onto the residual."""
    t = x.shape[0]
    qkv = ops["linear"](x, wqkv, bqkv, None)
    q, k, v = qkv.split([hq * d, hk * d, hk * d], 1)
    q, k = ops["qk"](q.reshape(t, hq, d), k.reshape(t, hk, d), pos, f, nq, nk)
    mixed = q.reshape(t, hk, hq // hk, d) * k[:, :, None] + v.reshape(t, hk, 1, d)
    return ops["linear"](mixed.reshape(t, hq * d), wo, None, x)


def test_layer_forward_backward_and_step():
    """Forward, backward and the optimizer step together: gradients against fp64
    autograd of the definition, then a Muon step of the fused weight by row
    blocks that equals the step from the same gradients given directly."""
    torch_cuda()
    t, hq, hk, d, e = 96, 4, 2, 64, 256
    x = rand((t, e), F32, 1)
    params = [rand(((hq + 2 * hk) * d, e), F32, 2, 1 / 16), rand(((hq + 2 * hk) * d,), F32, 3, 0.1),
              rand((e, hq * d), F32, 4, 1 / 16), 1 + rand((d,), F32, 5, 0.1), 1 + rand((d,), F32, 6, 0.1)]
    pos = torch.arange(t, device="cuda")
    f = torch.pow(10000.0, -torch.arange(d // 2, device="cuda", dtype=torch.float64) / (d // 2))
    dy = rand((t, e), F32, 7)

    def plain_qk(q, k, pos, f, nq, nk):
        axes = torch.zeros(d // 2, dtype=torch.int64, device="cuda")
        out = []
        for a, w in ((q, nq), (k, nk)):
            u = a / torch.sqrt((a * a).mean(-1, keepdim=True) + 1e-6) * w
            th = pos.double()[:, None, None] * f
            c, s, h = torch.cos(th), torch.sin(th), d // 2
            out.append(torch.cat([u[..., :h] * c - u[..., h:] * s, u[..., h:] * c + u[..., :h] * s], -1))
        return out

    plain = {"linear": lambda x, w, b, r: x @ w.t() + (0 if b is None else b) + (0 if r is None else r), "qk": plain_qk}
    mine = {"linear": ns.linear, "qk": lambda q, k, pos, f, nq, nk: ns.qk_norm_rope(q, k, pos, f, q_weight=nq, k_weight=nk)}
    got, want = [], []
    for ops, t64, into in ((mine, False, got), (plain, True, want)):
        leaves = [(p.double() if t64 else p.clone()).requires_grad_() for p in [x] + params]
        y = block(leaves[0], leaves[1], leaves[2], leaves[3], leaves[4], leaves[5], pos, f, hq, hk, d, ops)
        y.backward(dy.double() if t64 else dy)
        into += [y.detach()] + [p.grad for p in leaves]
    for i, (a, b) in enumerate(zip(got, want)):
        # fp32 throughout: sums of up to 512 terms through four products, 2^-24 * (512 + 256 + 256) * 4 at most in norm
        assert float((a.double() - b).norm() / b.norm()) <= 2.0 ** -24 * 4096, i
    grad = got[2]  # of the fused weight
    heads = [hq * d, hk * d, hk * d]
    p = params[0].clone().requires_grad_()
    p.grad = grad
    ns.MuonNS5([p], lr=0.05, normuon=True, split_rows={id(p): heads}).step()
    w, m, v = params[0].clone(), torch.zeros_like(grad), torch.zeros(grad.shape[0], device="cuda")
    ns.step_group([w], [grad.contiguous()], [m], [v], split_rows=heads, lr=0.05, normuon=True)
    assert torch.equal(p.detach(), w) and not torch.equal(w, params[0])


# ---- graphs, streams --------------------------------------------------------------------
def test_captured_calls_replay_like_eager_ones():
    """Forward and gradients captured twice, into two graphs, replayed in turn
    with the program's own eager calls and synchronizations between."""
    torch_cuda()
    x, w, b, dy = rand((300, 264), BF, 1), rand((520, 264), BF, 2), rand((520,), BF, 3), rand((300, 520), BF, 4)
    _, q, k = packed(64, 4, 2, 128, BF, 5)
    wq = 1 + rand((128,), BF, 6, 0.1)
    gq, gk = rand((64, 4, 128), BF, 7), rand((64, 2, 128), BF, 8)
    pos, f = torch.arange(64, device="cuda"), torch.rand(64, device="cuda")

    def both():
        y, z = ns.linear(x, w, b, activation="silu", return_preact=True)
        grads = ns.linear_backward(dy, x, w, activation="silu", preact=z, need_dbias=True)
        heads = ns.qk_norm_rope(q, k, pos, f, q_weight=wq)
        back = ns.qk_norm_rope_backward(gq, gk, q, k, pos, f, q_weight=wq)
        return [y, z, *grads, *heads, *back[:3]]

    both()
    graphs = []
    for _ in range(2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            out = both()
        torch.cuda.current_stream().wait_stream(side)
        graphs.append((g, out))
    for i in range(4):
        x.copy_(rand(x.shape, BF, 100 + i))
        q.copy_(rand(q.shape, BF, 200 + i))
        want = both()
        torch.cuda.synchronize()
        for g, out in (graphs if i % 2 else graphs[::-1]):
            for t in out:
                t.fill_(7)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, r) for p, r in zip(out, want)), i


def test_autograd_refuses_capture():
    torch_cuda()
    x, w = rand((8, 64), BF, 1).requires_grad_(), rand((32, 64), BF, 2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    kept = torch.zeros(8, device="cuda")
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        kept.add_(1)
        with pytest.raises(ns.MuonError) as e:
            ns.linear(x, w)
    assert e.value.status == -2


def test_other_streams_at_once():
    torch_cuda()
    x, w, dy, z = rand((260, 512), BF, 1), rand((768, 512), BF, 2), rand((260, 768), BF, 3), rand((260, 768), BF, 4)
    want = ns.linear_backward(dy, x, w, activation="gelu", preact=z, need_dbias=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 3]):
            got.append(ns.linear_backward(dy, x, w, activation="gelu", preact=z, need_dbias=True))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))


def test_python_refusals_on_the_gpu():
    torch_cuda()
    x, w = rand((8, 64), BF, 1), rand((32, 64), BF, 2)

    def status(f):
        with pytest.raises(ns.MuonError) as e:
            f()
        return e.value.status

    assert status(lambda: ns.linear(x, w.float())) == -2
    assert status(lambda: ns.linear(x.half(), w.half())) == -2
    assert status(lambda: ns.linear(x, rand((32, 63), BF, 3))) == -1
    assert status(lambda: ns.linear(x.t().contiguous().t(), w)) == -1
    assert status(lambda: ns.linear(x, w, rand((31,), BF, 3))) == -1
    assert status(lambda: ns.linear(x, w, activation="tanh")) == -2
    assert status(lambda: ns.linear(x, w, out=x)) == -1
    assert status(lambda: ns.linear(x, w.cpu())) == -1
    dy = rand((8, 32), BF, 4)
    assert status(lambda: ns.linear_backward(dy, x, w, activation="silu")) == -1
    assert status(lambda: ns.linear_backward(dy, x, w, accumulate=True)) == -1
    assert status(lambda: ns.linear_backward(dy, x, w, dx=x)) == -1
    q, pos, f = rand((4, 2, 64), BF, 1), torch.arange(4, device="cuda"), torch.ones(32, device="cuda")
    assert status(lambda: ns.rope(q, None, pos.float(), f)) == -2
    assert status(lambda: ns.rope(q, None, pos[:3], f)) == -1
    assert status(lambda: ns.rope(q, None, pos, torch.ones(33, device="cuda"))) == -1
    assert status(lambda: ns.rope(q, None, torch.stack([pos, pos]), f)) == -1
    assert status(lambda: ns.rope(q, None, torch.stack([pos, pos]), f, sections=[16, 15])) == -1
    assert status(lambda: ns.rope(q, q, pos, f, q_out=q, k_out=q)) == -1
    assert status(lambda: ns.qk_norm_rope(q, None, pos, f, q_weight=torch.ones(63, device="cuda"))) == -1
    assert status(lambda: ns.qk_norm_rope(q, rand((4, 2, 64), F32, 2), pos, f)) == -2
