"""The operators of a training pass run together, as they are used: token ids
through the embedding, the norms around a block, the block's products, the loss
by a product with the embedding, the gradients of all, their clipping and the
step, against the same pass in 64 bits."""
import math

import pytest
import torch

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ns():
    torch_cuda()
    import newton_schulz_ns5_amd as m
    return m


VOCAB, WIDE, MLP, BATCH, TOKENS, LAYERS = 211, 96, 160, 3, 17, 2
SCALE = math.sqrt(WIDE)


def rand(shape, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * scale + shift


def parameters():
    ps = {"embed": rand((VOCAB, WIDE), 1, 0.05), "first": rand((WIDE,), 2, 0.1, 1.0)}
    for i in range(LAYERS):
        ps[f"up{i}"] = rand((MLP, WIDE), 10 + i, 1 / math.sqrt(WIDE))
        ps[f"down{i}"] = rand((WIDE, MLP), 20 + i, 1 / math.sqrt(MLP))
        ps[f"post{i}"] = rand((WIDE,), 30 + i, 0.1, 1.0)
        ps[f"next{i}"] = rand((WIDE,), 40 + i, 0.1, 1.0)
        ps[f"gate{i}"] = rand((BATCH, 1, WIDE), 50 + i, 0.2, 0.5)
    return ps


def ids():
    g = torch.Generator(device="cuda").manual_seed(3)
    t = torch.randint(0, VOCAB, (BATCH, TOKENS), generator=g, device="cuda")
    t[:, -3:] = torch.tensor([-1, 7, 7], device="cuda")  # padding, and a token that repeats
    return t


def forward(ns, ps, t):
    x = ns.embedding(t, ps["embed"], scale=SCALE)
    stream, y = ns.residual_norm(x, weight=ps["first"])
    for i in range(LAYERS):
        h = ns.linear(y, ps[f"up{i}"], activation="silu")
        h = ns.linear(h, ps[f"down{i}"])
        stream, y = ns.residual_norm(h, stream, weight=ps[f"next{i}"], post_weight=ps[f"post{i}"], gate=ps[f"gate{i}"],
                                     scale=0.5, residual_scale=0.9)
    return ns.linear(y, ps["embed"])  # tied: its gradient is the sum of both uses


def forward64(ps, t):
    def norm(v, w):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w
    inside = (t >= 0)[..., None]
    stream = ps["embed"][t.clamp(min=0)] * SCALE * inside
    y = norm(stream, ps["first"])
    for i in range(LAYERS):
        h = y @ ps[f"up{i}"].t()
        h = (h * torch.sigmoid(h)) @ ps[f"down{i}"].t()
        stream = 0.9 * stream + 0.5 * ps[f"gate{i}"] * norm(h, ps[f"post{i}"])
        y = norm(stream, ps[f"next{i}"])
    return y @ ps["embed"].t()


def test_a_training_pass(ns):
    t, c = ids(), rand((BATCH, TOKENS, VOCAB), 4, 0.1)
    leaves = {k: v.clone().requires_grad_() for k, v in parameters().items()}
    logits = forward(ns, leaves, t)
    logits.backward(c)
    exact = {k: v.double().requires_grad_() for k, v in parameters().items()}
    want = forward64(exact, t)
    want.backward(c.double())
    # fp32 throughout.  Roundings of either sign leave a sum of K terms off by about sqrt(K) 2^-24 of its size: up to
    # 211 terms, 2^-20; 2^-17 for every operator leaves a factor of eight.  A dozen of them follow each other,
    # and as many backward.
    want = want.detach()
    assert float((logits.detach().double() - want).norm() / want.norm()) <= 12 * 2.0 ** -17
    for k in leaves:
        err = float((leaves[k].grad.double() - exact[k].grad).norm() / exact[k].grad.norm())
        assert err <= 24 * 2.0 ** -17, (k, err)
    # clip what the matrices' optimizer steps together with all others, then step
    matrices = [leaves[k] for k in leaves if k[:2] in ("up", "do")]
    others = [p.grad for k, p in leaves.items() if k[:2] not in ("up", "do")]
    opt = ns.MuonNS5(matrices, lr=0.05, normuon=True)
    total = math.sqrt(sum(float(p.grad.square().sum()) for p in exact.values()))
    norm = opt.clip_grad_norm(0.5 * total, extra=others)
    assert abs(float(norm) - total) <= 24 * 2.0 ** -17 * total
    after = ns.grad_norm([p.grad for p in leaves.values()])
    assert abs(float(after) - 0.5 * total) <= 25 * 2.0 ** -17 * total
    before = [p.detach().clone() for p in matrices]
    opt.step()
    assert all(bool(p.isfinite().all()) and not torch.equal(p, b) for p, b in zip(matrices, before))


def test_gradients_called_directly_are_autograds(ns):
    """The same pass through the *_backward entry points, captured into a graph and replayed on new data."""
    ps, t = parameters(), ids()
    c = rand((BATCH, TOKENS, VOCAB), 5, 0.1)

    def whole():
        x = ns.embedding(t, ps["embed"], scale=SCALE)
        s0, y0 = ns.residual_norm(x, weight=ps["first"])
        h, z = ns.linear(y0, ps["up0"], activation="silu", return_preact=True)
        b = ns.linear(h, ps["down0"])
        how = dict(weight=ps["next0"], post_weight=ps["post0"], gate=ps["gate0"], scale=0.5, residual_scale=0.9)
        s1, y1 = ns.residual_norm(b, s0, **how)
        logits = ns.linear(y1, ps["embed"])
        dy1, dwe, _ = ns.linear_backward(c, y1, ps["embed"])
        db, ds0, dn, dp, dg = ns.residual_norm_backward(dy1, None, s1, b, **how)
        dh, dd, _ = ns.linear_backward(db, h, ps["down0"])
        dy0, du, _ = ns.linear_backward(dh, y0, ps["up0"], activation="silu", preact=z)
        dx, _, df, _, _ = ns.residual_norm_backward(dy0, ds0, s0, None, weight=ps["first"], need_dresidual=False)
        ns.embedding_backward(dx, t, VOCAB, scale=SCALE, dw=dwe, accumulate=True)
        out = [dwe, df, du, dd, dp, dn, dg]
        norm = ns.clip_grad_norm(out, 1e-3)
        return [logits, norm] + out

    whole()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = whole()
    for rep in range(3):
        c.copy_(rand(c.shape, 60 + rep, 0.1))
        t.copy_(ids().roll(rep, 1))
        ps["embed"].add_(0.01)
        graph.replay()
        eager = whole()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))
        leaves = {k: ps[k].clone().requires_grad_() for k in ("embed", "first", "up0", "down0", "post0", "next0", "gate0")}
        x = ns.embedding(t, leaves["embed"], scale=SCALE)
        s, y = ns.residual_norm(x, weight=leaves["first"])
        b = ns.linear(ns.linear(y, leaves["up0"], activation="silu"), leaves["down0"])
        _, y = ns.residual_norm(b, s, weight=leaves["next0"], post_weight=leaves["post0"], gate=leaves["gate0"], scale=0.5, residual_scale=0.9)
        ns.linear(y, leaves["embed"]).backward(c)
        own = [leaves[k].grad for k in ("embed", "first", "up0", "down0", "post0", "next0", "gate0")]
        total = float(ns.grad_norm(own))
        assert abs(float(captured[1]) - total) <= 2.0 ** -20 * total
        for a, b in zip(captured[2:], own):
            # the embedding's gradient is the sum of two, rounded once more or less
            assert float((a / (1e-3 / (total + 1e-6)) - b).norm()) <= 2.0 ** -19 * float(b.norm())


def test_streams_of_their_own(ns):
    """Tensors used on a stream of their own, the results awaited there."""
    t, ps = ids(), parameters()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = forward(ns, ps, t)
    b = forward(ns, ps, t)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b)
    with pytest.raises(ns.MuonError):
        ns.residual_norm(a, b.cpu())


def test_inside_torch_compile(ns):
    """A compiled function breaks its graph at these calls: every call with new tensors gives what the plain call gives."""
    w, n, g = rand((50, 64), 1), rand((64,), 2, 0.1, 1.0), rand((64,), 3)

    def fn(t, table, x, norm):
        e = ns.embedding(t, table, scale=2.0) * 2
        s, y = ns.residual_norm(e, x, weight=norm, gate=g, scale=0.5)
        return s.sum(-1) + y.sum(-1)

    def clip(a, b):
        return ns.clip_grad_norm([a, b], 1.0), a + ns.grad_norm(b)

    compiled, compiled_clip = torch.compile(fn, backend="eager"), torch.compile(clip, backend="eager")
    for i in range(3):
        t = torch.randint(0, 50, (30 + i,), device="cuda")
        for grad in (False, True):
            x = rand((30 + i, 64), 10 + i)
            a, b = [v.clone().requires_grad_(grad) for v in (w, x, n)], [v.clone().requires_grad_(grad) for v in (w, x, n)]
            got, want = compiled(t, *a), fn(t, *b)
            assert torch.equal(got, want)
            if grad:
                got.sum().backward()
                want.sum().backward()
                assert all(torch.equal(p.grad, q.grad) for p, q in zip(a, b))
        a, b = [[rand((77 + i,), 20), rand((5, 3), 21)] for _ in range(2)]
        assert all(torch.equal(p, q) for p, q in zip(compiled_clip(*a), clip(*b)))
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_tracers_are_refused(ns):
    from torch.fx.experimental.proxy_tensor import make_fx
    t, w = torch.arange(5, device="cuda"), rand((9, 16), 1)
    for fn in (lambda v: ns.embedding(t, v), lambda v: ns.residual_norm(v)[1], lambda v: ns.grad_norm([v]),
               lambda v: ns.clip_grad_norm([v], 1.0), lambda v: ns.embedding_backward(v[:5], t, 9),
               lambda v: ns.residual_norm_backward(v, None, v, None)[0]):
        for trace in (lambda f: torch.jit.trace(f, (w,)), lambda f: make_fx(f)(w)):
            with pytest.raises(Exception) as e:
                trace(fn)
            assert "tracing" in str(e.value) or "trace" in str(e.value)


def test_two_streams_at_once(ns):
    """Calls of every operator in flight on two streams, each with its own workspace."""
    t, w = torch.randint(0, 900, (5000,), device="cuda"), rand((900, 264), 1)
    dy, n = rand((5000, 264), 2), rand((264,), 3, 0.1, 1.0)

    def work():
        e = ns.embedding(t, w)
        dw = ns.embedding_backward(dy, t, 900)
        s, y = ns.residual_norm(e, dy, weight=n, post_weight=n, gate=n)
        grads = ns.residual_norm_backward(y, dy, s, e, weight=n, post_weight=n, gate=n)
        out = [torch.empty_like(g) for g in grads]
        return [dw, s, y, ns.clip_grad_norm(grads, 0.5, out=out), ns.grad_norm(out, squared=True)] + out
    want = work()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(work())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for runs in got for run in runs for a, b in zip(run, want))
