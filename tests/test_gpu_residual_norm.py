"""The norms before and after a block with its gate and its residual, and their
gradients, against the formulas in 64 bits.

Tolerances, element by element.  E = 2^-19 covers what fp32 does to a row: a
mean over the columns (each thread adds at most 16 squares, then up to 10 levels
of pairs: 30 roundings of 2^-24, halved by the root), the root, and the chain
of products behind it.  A term that is a sum of several is E times the sum of
their magnitudes off; a row sum carries its terms' errors into every element of
the row.  A vector's gradient adds at most rows / 256 + 100 rounded terms.
U(t) = eps(t) / 2 is the rounding of a result to its type."""
import math

import pytest
import torch

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}
E = 2.0 ** -19


@pytest.fixture(scope="module")
def ns():
    torch_cuda()
    import newton_schulz_ns5_amd as m
    return m


def rand(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)


def close(got, want, tol, what):
    assert got.shape == want.shape, what
    tol = (tol + U[got.dtype] * (want.abs() + tol) + 1e-37).expand(want.shape)
    off = (got.double() - want).abs() - tol
    assert not bool(got.isnan().any()), what
    if off.numel():
        i = int(off.flatten().argmax())
        assert float(off.max()) <= 0, (what, i, float(got.flatten()[i]), float(want.flatten()[i]), float(tol.flatten()[i]))


def wide(v, off=0.0):
    return None if v is None else v.double() + off


def forward64(b, x, w, pw, g, norm, post, scale, rscale, eps, offset):
    """(s, its error before rounding, y, its error)."""
    u = b.double()
    err = 0.0
    if post:
        u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps)
        u = u * (wide(pw, offset) if pw is not None else 1.0)
        err = E
    if g is not None:
        u = u * g.double()
    u = scale * u
    s = u if x is None else rscale * x.double() + u
    ds = u.abs() * (err + 2.0 ** -22) + s.abs() * 2.0 ** -23
    if not norm:
        return s, ds, None, None
    mean = (s * s).mean(-1, keepdim=True) + eps
    r = 1 / torch.sqrt(mean)
    rel = E + (s.abs() * ds).mean(-1, keepdim=True) / mean
    wt = wide(w, offset) if w is not None else torch.ones((), device=s.device, dtype=torch.float64)
    return s, ds, s * r * wt, (ds + s.abs() * rel) * r * wt.abs()


def check_forward(ns, b, x, w, pw, g, *, norm=True, post=False, scale=1.0, rscale=1.0, eps=1e-6, offset=0.0, what=None, **how):
    s, y = ns.residual_norm(b, x, weight=w, post_weight=pw, gate=g, norm=norm, post_norm=post, scale=scale,
                            residual_scale=rscale, eps=eps, weight_offset=offset, **how)
    s64, ds, y64, dy = forward64(b, x, w, pw, g, norm, post, scale, rscale, eps, offset)
    assert s.dtype is (b.dtype if x is None else x.dtype)
    close(s, s64, ds, (what, "stream"))
    if norm:
        assert y.dtype is b.dtype
        close(y, y64, dy, (what, "y"))
    else:
        assert y is None
    return s, y


def backward64(dy, dst, st, b, w, pw, g, post, scale, rscale, eps, offset):
    """{name: (value, error)} of every gradient; dgate as if every row had a gate."""
    d, err, out = (dst.double() if dst is not None else 0.0), 0.0, {}
    one = torch.ones((), device="cuda", dtype=torch.float64)
    if dy is not None:
        s, h = st.double(), dy.double() * (wide(w, offset) if w is not None else one)
        r = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
        n = s * r
        out["dweight"] = (dy.double() * n, (dy.double() * n).abs() * E)
        mag = r * (h.abs() + n.abs() * (h * n).abs().mean(-1, keepdim=True))
        d = d + r * (h - n * (h * n).mean(-1, keepdim=True))
        err = E * mag
    err = err + 2.0 ** -22 * (d.abs() + err)
    out["dresidual"] = (rscale * d, abs(rscale) * err)
    t, terr = scale * d, abs(scale) * err
    m, rb = (b.double() if b is not None else None), 1.0
    if post:
        rb = 1 / torch.sqrt((m * m).mean(-1, keepdim=True) + eps)
        m = m * rb
    pwt = wide(pw, offset) if pw is not None else one
    if g is not None:
        u = m * (pwt if post else one)
        out["dgate"] = (t * u, terr * u.abs() + (t * u).abs() * E)
        t, terr = t * g.double(), terr * g.double().abs()
    if post:
        out["dpost_weight"] = (t * m, terr * m.abs() + (t * m).abs() * E)
        k, kerr = t * pwt, terr * pwt.abs()
        mean = lambda v: v.mean(-1, keepdim=True)  # noqa: E731
        t = rb * (k - m * mean(k * m))
        terr = rb * (kerr + m.abs() * mean(kerr * m.abs()) + E * (k.abs() + m.abs() * mean((k * m).abs())))
    out["dblock"] = (t, terr + 2.0 ** -22 * (t.abs() if torch.is_tensor(t) else 0))
    return out


def summed(pair, dims, keepdim=False):
    v, err = pair
    n = 1
    for d in dims:
        n *= v.shape[d]
    s = lambda t: t.sum(dims, keepdim=keepdim) if dims else t  # noqa: E731
    return s(v), s(err) + (n / 256 + 100) * 2.0 ** -24 * s(v.abs())


def check_backward(ns, dy, dst, st, b, w, pw, g, *, post=False, scale=1.0, rscale=1.0, eps=1e-6, offset=0.0, what=None, **how):
    got = ns.residual_norm_backward(dy, dst, st, b, weight=w, post_weight=pw, gate=g, post_norm=post, scale=scale,
                                    residual_scale=rscale, eps=eps, weight_offset=offset, **how)
    want = backward64(dy, dst, st, b, w, pw, g, post, scale, rscale, eps, offset)
    shape = (dy if dy is not None else dst).shape
    for name, t in zip(("dblock", "dresidual", "dweight", "dpost_weight", "dgate"), got):
        if t is None:
            continue
        if name not in want:  # the weight of a norm that nothing depends on
            assert name == "dweight" and dy is None and float(t.abs().max()) == 0
            continue
        pair = want[name]
        lead = tuple(range(len(shape) - 1))
        if name in ("dweight", "dpost_weight"):
            pair = summed(pair, lead)
        elif name == "dgate":
            dims = lead if g.dim() == 1 else tuple(i for i in lead if g.shape[i] != shape[i])
            pair = summed(pair, dims, keepdim=g.dim() > 1)
        close(t, pair[0], pair[1], (what, name))
    return got


COLS = [1, 7, 8, 64, 65, 100, 128, 250, 256, 500, 512, 1001, 1024, 2048, 2050, 4096, 5000, 8192, 8200, 16384, 16379]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype,stream", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_widths(ns, cols, dtype, stream):
    """Every width's kernel with everything on, gate per column, and with all of it off."""
    rows = 37 if cols < 4096 else 5
    b, x = rand((rows, cols), dtype, 1), rand((rows, cols), stream, 2, 2.0)
    w, pw, g = (rand((cols,), dtype, 3 + i, 0.2, 1.0) for i in range(3))
    dy, dst = rand((rows, cols), dtype, 6, 0.1), rand((rows, cols), stream, 7, 0.1)
    how = dict(post=True, scale=0.75, rscale=0.5)
    s, _ = check_forward(ns, b, x, w, pw, g, what="all", **how)
    check_backward(ns, dy, dst, s, b, w, pw, g, what="all", **how)
    s, _ = check_forward(ns, b, x, w, None, None, what="plain")
    check_backward(ns, dy, dst, s, None, w, None, None, what="plain")


@pytest.mark.parametrize("cols", [40, 200, 512, 1024, 8192, 16384])
def test_two_vectors(ns, cols):
    """Vectors that the kernel holds where three would not fit, in fp32 and bf16."""
    b, x, dy = rand((7, cols), BF, 8), rand((7, cols), F32, 9, 2.0), rand((7, cols), BF, 10, 0.1)
    for dt in (F32, BF):
        w, pw = rand((cols,), dt, 3, 0.2, 1.0), rand((cols,), dt, 4, 0.2, 1.0)
        s, _ = check_forward(ns, b, x, w, pw, None, post=True, what=cols)
        check_backward(ns, dy, x, s, b, w, pw, None, post=True, what=cols)
        s, _ = check_forward(ns, b, x, w, None, pw, what=cols)
        check_backward(ns, dy, x, s, b, w, None, pw, what=cols)


@pytest.mark.parametrize("gate", ["none", "cols", "one", "batch", "rows"])
@pytest.mark.parametrize("post,norm,weights", [(True, True, True), (True, False, True), (False, True, True), (False, False, True),
                                               (True, True, False), (False, True, False)])
def test_every_form(ns, gate, post, norm, weights):
    for shape, dtype, stream in (((3, 17, 136), BF, F32), ((2, 5, 3, 72), F32, F32), ((1, 1, 520), BF, BF)):
        lead, cols = shape[:-1], shape[-1]
        gshape = {"none": None, "cols": (cols,), "one": (1,) * len(lead) + (cols,), "batch": lead[:1] + (1,) * (len(lead) - 1) + (cols,),
                  "rows": shape}[gate]
        b, x = rand(shape, dtype, 11), rand(shape, stream, 12, 2.0)
        w = rand((cols,), F32, 13, 0.2) if weights and norm else None
        pw = rand((cols,), F32, 14, 0.2) if weights and post else None
        g = rand(gshape, BF, 15, 0.5) if gshape is not None else None
        how = dict(post=post, scale=-1.25, rscale=0.3, eps=1e-3, offset=1.0)
        for res in (x, None):
            s, _ = check_forward(ns, b, res, w, pw, g, norm=norm, what=(shape, res is None), **how)
        s, _ = check_forward(ns, b, x, w, pw, g, norm=norm, **how)
        dy, dst = rand(shape, dtype, 16, 0.1), rand(shape, stream, 17, 0.1)
        cases = [(dy, dst), (dy, None)] if norm else []
        for a, c in cases + [(None, dst)]:
            got = check_backward(ns, a, c, s if a is not None else None, b, w, pw, g, what=(shape, a is None, c is None), **how)
            assert got[2] is None or a is not None or float(got[2].abs().max()) == 0


@pytest.mark.parametrize("rows", [1, 2, 255, 1023, 1025, 4099])
@pytest.mark.parametrize("cols,seqs", [(32, 1), (640, 1), (24, 41), (2048, 3), (96, 2000), (264, 1025)])
def test_row_counts_and_sequences(ns, rows, cols, seqs):
    """Rows that do and do not fill the workgroups, gates of few and of many sequences."""
    per = max(1, rows // seqs) if seqs > 1 else rows
    shape = (seqs, per, cols)
    if seqs * per * cols > 1 << 23:
        return
    b, st = rand(shape, BF, 21), rand(shape, F32, 22, 2.0)
    w, pw = rand((cols,), BF, 23, 0.2, 1.0), rand((cols,), BF, 24, 0.2, 1.0)
    g = rand((seqs, 1, cols), F32, 25, 0.5)
    dy, dst = rand(shape, BF, 26, 0.1), rand(shape, F32, 27, 0.1)
    check_forward(ns, b, st, w, pw, g, post=True, what=shape)
    check_backward(ns, dy, dst, st, b, w, pw, g, post=True, what=shape)


def test_the_first_norm_of_a_model(ns):
    b, w = rand((5, 300), BF, 31), rand((300,), BF, 32, 0.2, 1.0)
    s, y = ns.residual_norm(b, weight=w)
    assert s is b
    close(y, *forward64(b, None, w, None, None, True, False, 1.0, 1.0, 1e-6, 0.0)[2:], "y")
    s, y = ns.residual_norm(b, norm=False)
    assert s is b and y is None
    leaf = b.clone().requires_grad_()
    s, y = ns.residual_norm(leaf, weight=w)
    assert s is leaf
    dy = rand((5, 300), BF, 33)
    y.backward(dy)
    close(leaf.grad, *backward64(dy, None, b, None, w, None, None, False, 1.0, 1.0, 1e-6, 0.0)["dblock"], "gradient")


def test_equal_gradients_are_one_tensor(ns):
    dy, dst, st = (rand((9, 128), BF, 41 + i) for i in range(3))
    got = check_backward(ns, dy, dst, st, None, None, None, None, scale=0.5, rscale=0.5)
    assert got[0] is got[1]
    got = check_backward(ns, dy, dst, st, None, None, None, None, scale=0.5, rscale=0.25)
    assert got[0] is not got[1]
    got = ns.residual_norm_backward(dy, dst, st, None, need_dblock=False)
    assert got[0] is None and got[1] is not None
    got = ns.residual_norm_backward(dy, dst, st, None, need_dresidual=False)
    assert got[1] is None
    close(got[0], *backward64(dy, dst, st, None, None, None, None, False, 1.0, 1.0, 1e-6, 0.0)["dblock"], "dblock")


def test_in_place(ns):
    shape = (33, 264)
    for dtype in (BF, F32):
        b, x = rand(shape, dtype, 51), rand(shape, dtype, 52)
        w, pw = rand((264,), dtype, 53, 0.2, 1.0), rand((264,), dtype, 54, 0.2, 1.0)
        s, y = ns.residual_norm(b, x, weight=w, post_weight=pw)
        for into in (dict(stream=1, out=0), dict(stream=0, out=1)):
            bufs = [b.clone(), x.clone()]
            versions = [t._version for t in bufs]
            s2, y2 = ns.residual_norm(bufs[0], bufs[1], weight=w, post_weight=pw, **{k: bufs[i] for k, i in into.items()})
            assert torch.equal(s, s2) and torch.equal(y, y2) and s2 is bufs[into["stream"]] and y2 is bufs[into["out"]]
            assert all(t._version > v for t, v in zip(bufs, versions))
        dy, dst = rand(shape, dtype, 55), rand(shape, dtype, 56)
        want = ns.residual_norm_backward(dy, dst, s, b, weight=w, post_weight=pw)
        a, c = dy.clone(), dst.clone()
        got = ns.residual_norm_backward(a, c, s, b, weight=w, post_weight=pw, dblock=a, dresidual=c)
        assert got[0] is a and got[1] is c and all(torch.equal(p, q) for p, q in zip(want[:4], got[:4]))


def test_strides_and_alignments(ns):
    rows, cols = 21, 130
    for start, ld in ((0, 200), (1, 131), (3, 137), (8, 136)):
        for dtype in (BF, F32):
            def view(seed):
                return rand((rows * ld + 16,), dtype, seed)[start:start + rows * ld].view(rows, ld)[:, :cols]
            b, x, dy, dst = (view(60 + i) for i in range(4))
            w, g = rand((cols + start,), dtype, 65, 0.2, 1.0)[start:], rand((cols + start,), dtype, 66)[start:]
            buf = torch.full((rows, ld + start), 7.0, dtype=dtype, device="cuda")
            s, y = check_forward(ns, b, x, w, w, g, post=True, stream=buf[:, start:start + cols])
            assert bool((buf[:, start + cols:] == 7).all()) and bool((buf[:, :start] == 7).all())
            s = s.clone()
            check_backward(ns, dy, dst, s, b, w, w, g, post=True, dresidual=buf[:, start:start + cols])
            assert bool((buf[:, start + cols:] == 7).all()) and bool((buf[:, :start] == 7).all())
    # rows that share elements, leading dimensions that are not one stride
    b = rand((cols,), BF, 71).expand(4, cols)
    check_forward(ns, b, b, None, None, None)
    x = rand((4, 3, 2, cols), F32, 72)[:, :, 0]
    x = x.transpose(0, 1)
    check_forward(ns, x, x, None, None, None)
    with pytest.raises(ns.MuonError):
        ns.residual_norm(rand((8, 8), BF, 73).t())
    # one row far from the next
    far = torch.zeros((2, (1 << 31) + 64), dtype=BF, device="cuda")
    far[:, :cols] = rand((2, cols), BF, 74)
    check_forward(ns, far[:, :cols], far[:, :cols], None, None, None)


def test_zero_rows_columns_and_values(ns):
    w = torch.ones(16, device="cuda")
    g = torch.ones(16, device="cuda")
    e = torch.empty((0, 16), device="cuda")
    s, y = ns.residual_norm(e, e, weight=w, gate=g)
    assert s.shape == y.shape == (0, 16)
    got = ns.residual_norm_backward(e, e, e, e, weight=w, post_weight=w, gate=g)
    assert got[0].shape == (0, 16) and all(float(t.abs().max()) == 0 for t in got[2:])
    e = torch.empty((4, 0), device="cuda")
    assert ns.residual_norm(e, e)[1].shape == (4, 0)
    assert ns.residual_norm(torch.empty((0, 3, 16), device="cuda"), gate=torch.empty((0, 1, 16), device="cuda"))[0].shape == (0, 3, 16)
    z = torch.zeros((3, 16), device="cuda")
    s, y = ns.residual_norm(z, z, post_norm=True)
    assert float(s.abs().max()) == 0 and float(y.abs().max()) == 0  # eps keeps a row of zeros
    got = ns.residual_norm_backward(z + 1, z, z, z, post_norm=True)
    assert all(bool(t.isfinite().all()) for t in got[:2])


def test_nan_and_infinity_stay_in_their_rows(ns):
    b, x = rand((6, 520), BF, 81), rand((6, 520), BF, 82)
    clean = ns.residual_norm(b, x, post_norm=True)
    b[2, 7], b[4, 519] = math.nan, math.inf
    bad = ns.residual_norm(b, x, post_norm=True)
    for p, q in zip(clean, bad):
        assert torch.equal(p[[0, 1, 3, 5]], q[[0, 1, 3, 5]]) and bool(q[2].isnan().all()) and bool(q[4, 519].isnan())


def test_offsets_past_32_bits(ns):
    rows, cols = (1 << 31) // 4096 + 3, 4096
    b = torch.zeros((rows, cols), dtype=BF, device="cuda")
    b[-3:] = rand((3, cols), BF, 83)
    s, y = ns.residual_norm(b, b, stream=b, scale=0.5)
    want = forward64(b[-3:], None, None, None, None, True, False, 1.0, 1.0, 1e-6, 0.0)
    close(y[-3:], want[2], want[3] + 2.0 ** -8 * want[2].abs(), "y")  # b has been rounded to bf16 since
    assert float(y[:-3].abs().max()) == 0
    dy = torch.zeros_like(b)
    dy[-3:] = rand((3, cols), BF, 84)
    got = ns.residual_norm_backward(dy, None, s, None, dresidual=dy, need_dblock=False)
    assert float(got[1][:-3].abs().max()) == 0 and float(got[1][-3:].abs().max()) > 0


def test_gradients_against_differences(ns):
    """The directional derivative of a loss of both results, in fp32 with a step that the tolerance counts:
    a central difference of step h of results rounded to 2^-22 is 2^-22 |loss terms| / h + O(h^2) off."""
    shape, cols = (2, 3, 40), 40
    ts = [rand(shape, F32, 91), rand(shape, F32, 92), rand((cols,), F32, 93, 0.2, 1.0), rand((cols,), F32, 94, 0.2, 1.0),
          rand((2, 1, cols), F32, 95)]
    cs, cy = rand(shape, F32, 96).double(), rand(shape, F32, 97).double()
    how = dict(scale=0.7, residual_scale=1.3, eps=1e-2, weight_offset=0.1)

    def loss(b, x, w, pw, g):
        s, y = ns.residual_norm(b, x, weight=w, post_weight=pw, gate=g, **how)
        return s, y

    leaves = [t.clone().requires_grad_() for t in ts]
    s, y = loss(*leaves)
    torch.autograd.backward([s, y], [cs.float(), cy.float()])
    for i, leaf in enumerate(leaves):
        v = rand(ts[i].shape, F32, 98 + i)
        h = 2.0 ** -8
        ends = []
        for sign in (1, -1):
            moved = list(ts)
            moved[i] = ts[i] + sign * h * v
            a, b = loss(*moved)
            ends.append(float((a.double() * cs).sum() + (b.double() * cy).sum()))
        difference = (ends[0] - ends[1]) / (2 * h)
        exact = float((leaf.grad.double() * v.double()).sum())
        size = float((s.detach().double() * cs).abs().sum() + (y.detach().double() * cy).abs().sum())
        # the third derivative's term: values of order one with h^2 / 6 and v up to 4 (v^3 up to 64)
        assert abs(difference - exact) <= 2.0 ** -21 * size / h + 64 * h * h * size / 6, (i, difference, exact)


def test_autograd(ns):
    shape, cols = (2, 19, 264), 264
    b, x, w, pw, g = (rand(shape, BF, 101), rand(shape, F32, 102), rand((cols,), BF, 103, 0.2, 1.0), rand((cols,), BF, 104, 0.2, 1.0),
                      rand((2, 1, cols), BF, 105))
    cs, cy = rand(shape, F32, 106), rand(shape, BF, 107)
    how = dict(scale=0.7, residual_scale=0.9)
    leaves = [t.clone().requires_grad_() for t in (b, x, w, pw, g)]
    s, y = ns.residual_norm(leaves[0], leaves[1], weight=leaves[2], post_weight=leaves[3], gate=leaves[4], **how)
    torch.autograd.backward([s, y], [cs, cy])
    want = ns.residual_norm_backward(cy, cs, s.detach(), b, weight=w, post_weight=pw, gate=g, **how)
    assert all(torch.equal(p.grad, q) for p, q in zip(leaves, want))
    # only one result used, only one input recorded
    for use in (0, 1):
        leaf = x.clone().requires_grad_()
        out = ns.residual_norm(b, leaf, weight=w, post_weight=pw, gate=g, **how)
        out[use].sum().backward()  # an expanded gradient
        ones = torch.ones(shape, device="cuda", dtype=out[use].dtype)
        q = ns.residual_norm_backward(ones if use else None, None if use else ones, out[0].detach(), b, weight=w, post_weight=pw, gate=g, **how)
        assert torch.equal(leaf.grad, q[1])
    # the block and the residual are one tensor
    leaf = b.clone().requires_grad_()
    s, y = ns.residual_norm(leaf, leaf, weight=w)
    y.backward(cy)
    one = ns.residual_norm_backward(cy, None, s.detach(), None, weight=w)[0]
    assert torch.equal(leaf.grad, one + one)
    # a stream of another type than the block, and only the stream used: the block's gradient has its type
    leaf = b.clone().requires_grad_()
    s, _ = ns.residual_norm(leaf, x, norm=False)
    s.backward(cs)
    assert leaf.grad.dtype is BF and torch.equal(leaf.grad, cs.to(BF))
    # a saved tensor that was written since
    s, y = ns.residual_norm(b.clone().requires_grad_(), x, weight=w)
    with torch.no_grad():
        s.add_(1)
    with pytest.raises(RuntimeError):
        y.backward(cy)
    with pytest.raises(ns.MuonError):
        ns.residual_norm(leaf, x, stream=torch.empty_like(x))
    with pytest.raises(ns.MuonError):
        ns.residual_norm(b, x, stream=x.clone().requires_grad_())


def test_bindings_refuse(ns):
    b, x, w = rand((4, 64), BF, 111), rand((4, 64), F32, 112), rand((64,), BF, 113)
    for bad, code in [
        (lambda: ns.residual_norm(b, x[:3]), -1), (lambda: ns.residual_norm(b, x.half()), -2), (lambda: ns.residual_norm(b.double()), -2),
        (lambda: ns.residual_norm(b, x, weight=w[:63]), -1), (lambda: ns.residual_norm(b, x, weight=w, post_weight=w.float()), -2),
        (lambda: ns.residual_norm(b, x, gate=b[:2]), -1), (lambda: ns.residual_norm(b.view(2, 2, 64), gate=b[:2]), -1),
        (lambda: ns.residual_norm(b, x, out=b.float()), -2), (lambda: ns.residual_norm(b, x, stream=torch.empty_like(b)), -2),
        (lambda: ns.residual_norm(b, x, stream=x[:, :32]), -1), (lambda: ns.residual_norm(b, x, scale="a"), -1),
        (lambda: ns.residual_norm(b, x, eps=1e39), -1), (lambda: ns.residual_norm(b, x, scale=math.nan), -1),
        (lambda: ns.residual_norm(b, x.cpu()), -1), (lambda: ns.residual_norm(b, x, norm=False, out=b), -1),
        (lambda: ns.residual_norm(b, b, stream=b, out=b), -1), (lambda: ns.residual_norm_backward(b, x[:3], x, b), -1),
        (lambda: ns.residual_norm_backward(b, x, b, b), -2), (lambda: ns.residual_norm_backward(b, x, x, b, need_dgate=True), -1),
        (lambda: ns.residual_norm(torch.empty(1, 16385, device="cuda")), -1),
    ]:
        with pytest.raises(ns.MuonError) as e:
            bad()
        assert e.value.status == code
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises(ns.MuonError):
            ns.residual_norm(torch.autograd.forward_ad.make_dual(b, b), x)


def test_streams_bits_and_graphs(ns):
    shape, cols = (700, 1024), 1024
    b, x, w, pw, g = (rand(shape, BF, 121), rand(shape, F32, 122), rand((cols,), BF, 123, 0.2, 1.0), rand((cols,), BF, 124, 0.2, 1.0),
                      rand((cols,), BF, 125))
    dy, dst = rand(shape, BF, 126), rand(shape, F32, 127)

    def both():
        s, y = ns.residual_norm(b, x, weight=w, post_weight=pw, gate=g)
        return (s, y) + ns.residual_norm_backward(dy, dst, s, b, weight=w, post_weight=pw, gate=g)
    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = both()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, other))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = both()
        graphs.append((graph, out))
    for i in range(4):
        for t, seed in ((b, 130), (dy, 140), (x, 150)):
            t.copy_(rand(shape, t.dtype, seed + i))
        for graph, out in (graphs if i % 2 else graphs[::-1]):
            graph.replay()
        want = both()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(p, q) for p, q in zip(out, want))
    leaf = b.clone().requires_grad_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ns.MuonError):
            ns.residual_norm(leaf, x)


@pytest.mark.parametrize("cols", [8200, 12296, 16379, 16384])
@pytest.mark.parametrize("shape", [(3, 100), (300, 2), (2, 1), (41, 1)])
def test_wide_rows_of_sequences(ns, cols, shape):
    """More than 8192 columns with both the norm after the block and a gate of each sequence: workgroups
    that go through rows of one sequence, and through several sequences."""
    for dtype, stream in ((BF, BF), (F32, F32)) if cols == 8200 else ((BF, F32),):
        b, st = rand(shape + (cols,), dtype, 81), rand(shape + (cols,), stream, 82, 2.0)
        w, pw = rand((cols,), dtype, 83, 0.2, 1.0), rand((cols,), dtype, 84, 0.2, 1.0)
        g = rand((shape[0], 1, cols), dtype, 85, 0.5)
        dy, dst = rand(shape + (cols,), dtype, 86, 0.1), rand(shape + (cols,), stream, 87, 0.1)
        check_backward(ns, dy, dst, st, b, w, pw, g, post=True, what=(cols, shape))


@pytest.mark.parametrize("shape", [(1100, 40, 24), (1500, 10, 96), (1100, 2, 2048), (1100, 3, 2050)])
@pytest.mark.parametrize("post", [True, False])
def test_more_sequences_than_workgroups(ns, shape, post):
    """Workgroups that go through one sequence with its gate and then through another one."""
    cols = shape[-1]
    b, st = rand(shape, BF, 91), rand(shape, F32, 92, 2.0)
    w, pw = rand((cols,), BF, 93, 0.2, 1.0), rand((cols,), BF, 94, 0.2, 1.0) if post else None
    dy, dst = rand(shape, BF, 96, 0.1), rand(shape, F32, 97, 0.1)
    for dt in (BF, F32):
        g = rand((shape[0], 1, cols), dt, 95, 0.5)
        check_backward(ns, dy, dst, st, b, w, pw, g, post=post, what=shape)
