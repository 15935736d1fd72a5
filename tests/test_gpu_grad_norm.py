"""The norm over all gradients and their clipping against plain formulas in
64 bits.

Tolerances.  Squares are formed and added in fp64, n of them: at most
n 2^-53 off, below 2^-26 for every size here.  The norm is rounded to fp32
once (2^-24): 2^-23 in all.  A clipped value is x times the factor, which is
rounded to fp32, and the product is rounded once more in fp32 and then to its
own type: 2 * 2^-24 and half a step of the type, or half of the smallest
subnormal.
"""
import math

import pytest
import torch

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134}
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ns():
    torch_cuda()
    import newton_schulz_ns5_amd as m
    return m


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def exact_norm(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def check_norm(got, want):
    assert got.dtype is torch.float32 and got.shape == ()
    assert abs(float(got) - want) <= 2.0 ** -23 * want, (float(got), want)


def check_clipped(got, x, factor):
    want = x.double() * factor
    err = (got.double() - want).abs()
    assert bool((err <= want.abs() * (HALF[got.dtype] + 2.0 ** -23) + TINY[got.dtype]).all()), float(err.max())


LISTS = [
    [((1,), F32)], [((1,), BF)], [((4096,), BF)], [((4095,), F32)], [((4097,), BF)],
    [((3, 5, 7), F32), ((0,), BF), ((), F32), ((1000, 333), BF), ((0, 4), F32), ((8192,), BF)],
    [((17, 31), BF)] * 300,                       # three launches
    [((1,), F32)] * 128, [((2,), BF)] * 129,      # one launch's tensors, and one more
    [((2999, 4001), BF), ((129,), F32)],          # more items than waves
    [((1 << 20,), F32), ((1 << 20,), BF)],
]


@pytest.mark.parametrize("case", range(len(LISTS)))
def test_norm_and_clip(ns, case):
    xs = [randn(shape, dt, 100 * case + i) for i, (shape, dt) in enumerate(LISTS[case])]
    want = exact_norm(xs)
    check_norm(ns.grad_norm(xs), want)
    square = ns.grad_norm(xs, squared=True)
    assert square.dtype is torch.float64 and abs(float(square) - want * want) <= 2.0 ** -26 * want * want
    top = max([float(x.abs().max()) for x in xs if x.numel()])
    assert float(ns.grad_norm(xs, norm_type="inf")) == top
    keep = [x.clone() for x in xs]
    # below: nothing changes
    check_norm(ns.clip_grad_norm(xs, 1.01 * want), want)
    assert all(torch.equal(a, b) for a, b in zip(xs, keep))
    # into others of both types, the gradients as they were
    for types in ([x.dtype for x in xs], [F32] * len(xs), [BF] * len(xs)):
        outs = [torch.full(x.shape, 7.0, dtype=t, device="cuda") for x, t in zip(xs, types)]
        check_norm(ns.clip_grad_norm(xs, 0.37 * want, out=outs), want)
        for o, x in zip(outs, keep):
            check_clipped(o, x, 0.37 * want / (want + 1e-6))
        assert all(torch.equal(a, b) for a, b in zip(xs, keep))
        # nothing to clip: a copy
        ns.clip_grad_norm(xs, math.inf, out=outs)
        assert all(torch.equal(o, x.to(o.dtype)) for o, x in zip(outs, keep))
    # in place
    check_norm(ns.clip_grad_norm(xs, 0.37 * want, eps=0.0), want)
    for x, k in zip(xs, keep):
        check_clipped(x, k, 0.37)
    # by the largest magnitude
    got = ns.clip_grad_norm(keep, top / 3, norm_type=math.inf, eps=0.0, out=xs)
    assert float(got) == top
    for x, k in zip(xs, keep):
        check_clipped(x, k, (top / 3) / top)


def test_values_whose_squares_leave_fp32(ns):
    for scale in (1e-30, 1e30):
        xs = [randn((5000,), BF, 1, scale), randn((333,), F32, 2, scale)]
        want = exact_norm(xs)
        check_norm(ns.grad_norm(xs), want)
        keep = [x.clone() for x in xs]
        ns.clip_grad_norm(xs, 0.25 * want, eps=0.0)
        for x, k in zip(xs, keep):
            check_clipped(x, k, 0.25)


def test_a_long_sum_keeps_small_values(ns):
    # one large value and millions that an fp32 sum would lose beside it
    x = torch.full((1 << 24,), 2.0 ** -13, dtype=BF, device="cuda")
    x[5] = 1.0
    want = exact_norm([x])
    check_norm(ns.grad_norm(x), want)
    assert want > 1.1


def test_infinities_and_nans(ns):
    inf, nan = math.inf, math.nan
    for dt in (F32, BF):
        x = randn((9001,), dt, 3)
        for at in (0, 4095, 4096, 9000):
            for bad in (inf, -inf, nan):
                y = x.clone()
                y[at] = bad
                for kind in (2, inf):
                    n = float(ns.grad_norm([x, y], norm_type=kind))
                    assert math.isnan(n) if math.isnan(bad) else n == inf
        y = x.clone()
        y[77] = inf
        assert float(ns.clip_grad_norm([y], 1.0)) == inf
        assert bool(y[77].isnan()) and float(y[:77].abs().max()) == 0 and float(y[78:].abs().max()) == 0
        y = x.clone()
        y[77] = nan
        assert math.isnan(float(ns.clip_grad_norm([y], 1.0))) and bool(y.isnan().all())
        # an infinite bound leaves an infinite norm's gradients alone
        y = x.clone()
        y[77] = inf
        k = y.clone()
        ns.clip_grad_norm([y], inf)
        assert torch.equal(y, k)


def test_subnormal_values(ns):
    for dt, tiny in ((F32, 2.0 ** -149), (BF, 2.0 ** -133)):
        x = (torch.arange(-300, 300, device="cuda", dtype=torch.float64) * tiny).to(dt)
        want = exact_norm([x])
        assert want > 0
        check_norm(ns.grad_norm([x]), want) if want > 2.0 ** -126 else None
        outs = [torch.empty_like(x)]
        ns.clip_grad_norm([x], 1.0, out=outs)
        assert torch.equal(outs[0], x)  # a copy keeps them
        ns.clip_grad_norm([x], want / 2, eps=0.0, out=outs)
        assert bool(((outs[0].double() - x.double() / 2).abs() <= tiny / 2).all())


def test_sparse_gradients_are_refused(ns):
    x = torch.eye(4, device="cuda").to_sparse()
    for call in (lambda: ns.grad_norm([x]), lambda: ns.clip_grad_norm([x], 1.0)):
        with pytest.raises(ns.MuonError) as e:
            call()
        assert e.value.status == -2


def test_zero_gradients_and_a_zero_bound(ns):
    z = torch.zeros(100, device="cuda")
    for max_norm in (0.0, 1.0):
        for eps in (0.0, 1e-6):
            assert float(ns.clip_grad_norm([z], max_norm, eps=eps)) == 0
            assert float(z.abs().max()) == 0
    x = randn((100,), F32, 4)
    ns.clip_grad_norm([x], 0.0)
    assert float(x.abs().max()) == 0


def test_views_and_memory_orders(ns):
    buf = randn((100003,), BF, 5)
    for start in (0, 1, 3, 8):  # any alignment to the element
        for size in (1, 4097, 90001):
            x = buf[start:start + size]
            check_norm(ns.grad_norm([x]), exact_norm([x]))
            before, k = buf.clone(), x.clone()
            ns.clip_grad_norm([x], 0.5, eps=0.0)
            check_clipped(x, k, min(1.0, 0.5 / exact_norm([k])))
            assert torch.equal(buf[:start], before[:start]) and torch.equal(buf[start + size:], before[start + size:])
            buf.copy_(before)
    for x in (randn((8, 3, 5, 7), F32, 6).to(memory_format=torch.channels_last), randn((33, 65), BF, 7).t()):
        k, want = x.clone(), exact_norm([x])
        o = torch.empty_like(x, dtype=F32)
        assert o.stride() == x.stride()
        check_norm(ns.clip_grad_norm([x], 0.3, eps=0.0, out=[o]), want)
        check_clipped(o, k, 0.3 / want)
        with pytest.raises(ns.MuonError):
            ns.clip_grad_norm([x], 0.3, out=[torch.empty(x.shape, device="cuda")])
        ns.clip_grad_norm([x], 0.3, eps=0.0)
        check_clipped(x, k, 0.3 / want)
    # columns of a wider buffer: their norm is that of a copy, but they are not scaled
    x = randn((50, 64), F32, 8)[:, :20]
    check_norm(ns.grad_norm([x]), exact_norm([x]))
    with pytest.raises(ns.MuonError):
        ns.clip_grad_norm([x], 1.0)
    with pytest.raises(ns.MuonError):
        ns.clip_grad_norm([x[0].expand(4, 20)], 1.0)


def test_more_than_two_to_the_31_elements(ns):
    x = torch.zeros((1 << 31) + 4097, dtype=BF, device="cuda")
    x[-1], x[1 << 31], x[7] = 3.0, -4.0, 12.0
    assert float(ns.clip_grad_norm([x], 6.5, eps=0.0)) == 13
    assert [float(x[i]) for i in (-1, 1 << 31, 7)] == [1.5, -2.0, 6.0]
    assert float(ns.grad_norm([x])) == 6.5


def test_a_given_total(ns):
    xs = [randn((1000,), F32, 9), randn((77, 13), BF, 10)]
    other = [randn((555,), F32, 11)]
    both = exact_norm(xs + other)
    square = ns.grad_norm(xs, squared=True) + ns.grad_norm(other, squared=True)  # as ranks add them up
    for total in (square, square.sqrt().float(), square.reshape(1)):
        outs = [torch.empty_like(x) for x in xs]
        n = ns.clip_grad_norm(xs, 2.0, eps=0.0, total=total, out=outs)
        check_norm(n, both)
        for o, x in zip(outs, xs):
            # a factor from an fp32 norm is half a step of it further off
            err = (o.double() - x.double() * (2.0 / both)).abs()
            assert bool((err <= x.double().abs() * (2.0 / both) * (HALF[o.dtype] + 2.0 ** -22)).all())
    top = torch.tensor(50.0, device="cuda")
    k = xs[0].clone()
    assert float(ns.clip_grad_norm(xs[:1], 25.0, eps=0.0, norm_type="inf", total=top)) == 50
    assert torch.equal(xs[0], k * 0.5)


def test_refusals_on_the_gpu(ns):
    x, y = randn((100,), F32, 12), randn((100,), F32, 13)
    for bad, code in [
        (lambda: ns.clip_grad_norm([x, x], 1.0), -1), (lambda: ns.clip_grad_norm([x, x[50:]], 1.0), -1),
        (lambda: ns.clip_grad_norm([x, y], 1.0, out=[y, x]), -1), (lambda: ns.clip_grad_norm([x], 1.0, out=[x[:50]]), -1),
        (lambda: ns.clip_grad_norm([x], 1.0, total=x[:1]), -1), (lambda: ns.grad_norm([x.half()]), -2),
        (lambda: ns.clip_grad_norm([x], 1.0, out=[x.half()]), -2), (lambda: ns.clip_grad_norm([x.double()], 1.0), -2),
        (lambda: ns.grad_norm([x, y.cpu()]), -1), (lambda: ns.clip_grad_norm([x], -1.0), -1),
        (lambda: ns.grad_norm([x.clone().requires_grad_()]), -2),
        (lambda: ns.clip_grad_norm([x.clone().requires_grad_()], 1.0), -1),
        (lambda: ns.clip_grad_norm([x.clone().requires_grad_()], 1.0, out=[y]), -2),
    ]:
        kx, ky = x.clone(), y.clone()
        with pytest.raises(ns.MuonError) as e:
            bad()
        assert e.value.status == code
        assert torch.equal(x, kx) and torch.equal(y, ky)
    assert float(ns.grad_norm([x, x])) > 0  # a norm may count a tensor twice
    # an output written through its pointer moves its version counter
    v = x._version
    ns.clip_grad_norm([x], 1.0)
    assert x._version > v


def test_the_same_bits_every_time(ns):
    xs = [randn((1237, 2011), BF, 14), randn((4001,), F32, 15)]
    first = ns.grad_norm(xs, squared=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        assert torch.equal(ns.grad_norm(xs, squared=True), first)
        with torch.cuda.stream(side):
            other = ns.grad_norm(xs, squared=True)
        side.synchronize()
        assert torch.equal(other, first)


def test_captured_and_replayed(ns):
    xs = [randn((700, 513), BF, 16), randn((3001,), F32, 17)]
    ys = [torch.zeros_like(x) for x in xs]
    many = [randn((9,), F32, 300 + i) for i in range(200)]
    ns.clip_grad_norm(xs, 1.0, out=ys)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        n1 = ns.clip_grad_norm(xs, 5.0, out=ys)
    with torch.cuda.graph(g2):
        n2 = ns.clip_grad_norm(many, 2.0)
        s2 = ns.grad_norm(many, squared=True)
    for rep in range(4):
        for i, x in enumerate(xs):
            x.copy_(randn(x.shape, x.dtype, 40 + 10 * rep + i, 1 + rep))
        for i, x in enumerate(many):
            x.copy_(randn(x.shape, x.dtype, 900 + 1000 * rep + i))
        keep = [x.clone() for x in many]
        g1.replay()
        g2.replay()
        g1.replay()
        torch.cuda.synchronize()
        check_norm(n1, exact_norm(xs))
        for x, y in zip(xs, ys):
            check_clipped(y, x, 5.0 / (exact_norm(xs) + 1e-6))
        want = exact_norm(keep)
        check_norm(n2, want)
        for x, k in zip(many, keep):
            check_clipped(x, k, 2.0 / (want + 1e-6))
        assert abs(float(s2) - exact_norm(many) ** 2) <= 2.0 ** -26 * float(s2)
        eager = [torch.empty_like(x) for x in xs]
        ns.clip_grad_norm(xs, 5.0, out=eager)
        assert all(torch.equal(a, b) for a, b in zip(ys, eager))


def test_an_optimizers_gradients(ns):
    ps = [torch.nn.Parameter(randn(s, t, 20 + i, 0.02)) for i, (s, t) in enumerate([((64, 96), F32), ((128, 64), BF), ((64, 96), F32)])]
    emb = torch.nn.Parameter(randn((100, 8), BF, 30))
    for p in ps[:2] + [emb]:
        p.grad = randn(p.shape, p.dtype, 31)
    opt = ns.MuonNS5(ps, lr=0.05)
    keep = [p.grad.clone() for p in ps[:2] + [emb]]
    want = exact_norm(keep)
    check_norm(opt.clip_grad_norm(0.5, extra=[emb.grad, None], eps=0.0), want)
    for p, k in zip(ps[:2] + [emb], keep):
        check_clipped(p.grad, k, 0.5 / want)
    before = [p.detach().clone() for p in ps]
    opt.step()
    assert not torch.equal(ps[0], before[0]) and torch.equal(ps[2], before[2])
    assert float(ns.MuonNS5([]).clip_grad_norm(1.0)) == 0
