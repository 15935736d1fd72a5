"""The embedding and its gradient by sorted tokens against the formulas in 64 bits.

Tolerances.  A looked-up value is one fp32 product (2^-24) and one rounding to
its type, U(t) = eps(t) / 2.  A row's gradient is the sum of its k tokens, in
whatever order: k roundings of at most 2^-24 of the sum of magnitudes, one more
for the scale and one for what it is added to."""
import math

import pytest
import torch

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}
BIG = 2 ** 63 - 1


@pytest.fixture(scope="module")
def ns():
    torch_cuda()
    import newton_schulz_ns5_amd as m
    return m


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def make_ids(kind, tokens, rows, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.rand((tokens,), generator=g, device="cuda", dtype=torch.float64)
    if kind == "zipf":
        return (torch.exp(u * math.log(rows + 1)) - 1).long().clamp_(0, rows - 1)
    if kind == "same":
        return torch.full((tokens,), rows // 2, device="cuda")
    if kind == "rising":
        return torch.arange(tokens, device="cuda") % rows
    if kind == "falling":
        return rows - 1 - torch.arange(tokens, device="cuda") * rows // max(tokens, 1) % rows
    if kind == "two":  # two rows that alternate
        return (torch.arange(tokens, device="cuda") % 2) * (rows - 1)
    return (u * rows).long().clamp_(0, rows - 1)


def close(got, want, tol, what):
    assert got.shape == want.shape, what
    tol = tol + U[got.dtype] * (want.abs() + tol) + 1e-40
    off = (got.double() - want).abs() - tol
    assert not bool(got.isnan().any()), what
    if off.numel():
        i = int(off.flatten().argmax())
        assert float(off.max()) <= 0, (what, i, float(got.flatten()[i]), float(want.flatten()[i]), float(tol.flatten()[i]))


def rows_of(ids, first, rows, padding=None):
    """(positions that have a row, their rows), computed on the host, where ids of any size subtract."""
    flat = [int(i) for i in ids.flatten().tolist()]
    have = [(t, i - first) for t, i in enumerate(flat) if 0 <= i - first < rows and i != padding]
    return (torch.tensor([t for t, _ in have], dtype=torch.int64, device="cuda"),
            torch.tensor([r for _, r in have], dtype=torch.int64, device="cuda"))


def check_forward(ns, ids, w, *, scale=1.0, first=0, what=None, **how):
    y = ns.embedding(ids, w, scale=scale, first=first, **how)
    at, rows = rows_of(ids, first, w.shape[0])
    want = torch.zeros((ids.numel(), w.shape[1]), device="cuda", dtype=torch.float64)
    want[at] = w[rows].double() * scale
    want = want.view(ids.shape + (w.shape[1],))
    close(y, want, want.abs() * 2.0 ** -24, what)
    return y


def check_backward(ns, dy, ids, rows, *, scale=1.0, first=0, padding=None, start=None, what=None, **how):
    if start is not None:
        how.update(dw=start.clone(), accumulate=True)
    dw = ns.embedding_backward(dy, ids, rows, scale=scale, first=first, padding_idx=padding, **how)
    at, v = rows_of(ids, first, rows, padding)
    flat = dy.reshape(-1, dy.shape[-1])[at].double()
    zero = torch.zeros((rows, dy.shape[-1]), device="cuda", dtype=torch.float64)
    want, mag = zero.clone().index_add_(0, v, flat * scale), zero.clone().index_add_(0, v, flat.abs() * abs(scale))
    count = torch.zeros((rows, 1), device="cuda", dtype=torch.float64).index_add_(0, v, torch.ones((len(v), 1), device="cuda", dtype=torch.float64))
    tol = mag * (count + 2) * 2.0 ** -24
    if start is not None:
        want = want + start.double()
        tol = tol + want.abs() * 2.0 ** -24
        assert torch.equal(dw[count[:, 0] == 0], start[count[:, 0] == 0]), what
    close(dw, want, tol, what)
    if start is None:
        assert not bool(dw[count[:, 0] == 0].any()), what
    return dw


TOKENS = [1, 2, 16, 17, 255, 2048, 2049, 5000]
ROWS = [1, 2, 511, 512, 1000, 50021]
DIMS = [1, 8, 100, 520]
KINDS = ["zipf", "same", "rising", "falling", "two", "uniform"]


@pytest.mark.parametrize("tokens", TOKENS)
@pytest.mark.parametrize("rows", ROWS)
def test_tokens_and_rows(ns, tokens, rows):
    for n, kind in enumerate(KINDS):
        dim = DIMS[(n + tokens) % len(DIMS)]
        ids = make_ids(kind, tokens, rows, n)
        check_forward(ns, ids, rand((rows, dim), BF, 1), scale=3.5, what=kind)
        check_backward(ns, rand((tokens, dim), BF, 2), ids, rows, scale=3.5, what=kind)


@pytest.mark.parametrize("dim", [1, 3, 7, 8, 9, 63, 64, 65, 128, 250, 256, 512, 1000, 1024, 1025, 2048, 2049, 2056, 4096, 5003])
@pytest.mark.parametrize("a,b", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
def test_widths_and_types(ns, dim, a, b):
    tokens, rows = 300, 77
    ids = make_ids("zipf", tokens, rows, dim)
    check_forward(ns, ids, rand((rows, dim), a, 3), scale=0.7, dtype=b, what=dim)
    check_backward(ns, rand((tokens, dim), a, 4), ids, rows, scale=0.7, dw_dtype=b, what=dim)
    check_backward(ns, rand((tokens, dim), a, 5), ids, rows, scale=0.7, start=rand((rows, dim), b, 6), what=dim)


@pytest.mark.parametrize("tokens,rows,dim", [(20000, 262144, 16), (70000, 300, 24), (131072, 1 << 19, 8), (140001, 32003, 40),
                                             (600000, 100, 8), (1 << 20, 1 << 20, 4)])
def test_many_tokens(ns, tokens, rows, dim):
    for kind in ("zipf", "same", "uniform"):
        ids = make_ids(kind, tokens, rows, 7)
        # whole numbers, whose sums are exact in any order
        dy = torch.randint(-3, 4, (tokens, dim), device="cuda").to(BF)
        order = ids.argsort()  # sums of runs as differences of a running sum, exact too
        total = torch.cat([torch.zeros((1, dim), device="cuda", dtype=torch.float64), dy[order].double().cumsum(0)])
        ends = torch.bincount(ids, minlength=rows).cumsum(0)
        want = total[ends] - total[torch.cat([ends.new_zeros(1), ends[:-1]])]
        assert float(want.abs().max()) < 2 ** 24
        assert torch.equal(ns.embedding_backward(dy, ids, rows, dw_dtype=F32).double(), want), kind


def test_a_token_among_more_rows_than_18_bits(ns):
    rows = (1 << 22) + 5
    ids = torch.tensor([rows - 1, 0, 1 << 21, rows - 1, (1 << 18) + 1, -1, rows], device="cuda")
    check_backward(ns, rand((7, 8), F32, 8), ids, rows)
    check_forward(ns, ids, rand((rows, 8), BF, 9))


def test_shards_masks_and_padding(ns):
    rows, dim = 50, 72
    ids = torch.tensor([[-1, 0, 99, 100, 149, 150, 10 ** 12], [120, 120, -100, 149, BIG, -BIG - 1, 100]], device="cuda")
    for kind in (torch.int64, torch.int32):
        i = ids if kind is torch.int64 else ids.clamp(-2 ** 31, 2 ** 31 - 1).to(kind)
        for first in (100, 0, -120, 2 ** 31 - 60, -BIG - 1, BIG - 20):
            check_forward(ns, i, rand((rows, dim), BF, 11), first=first, what=first)
            dy = rand(i.shape + (dim,), F32, 12)
            check_backward(ns, dy, i, rows, first=first, what=first)
            check_backward(ns, dy, i, rows, first=first, padding=120, what=first)
            check_backward(ns, dy, i, rows, first=first, padding=120, start=rand((rows, dim), BF, 13), what=first)
    # a whole vocabulary's gradient is its shards'
    w = 400
    ids = make_ids("zipf", 3000, w, 14)
    dy = rand((3000, dim), BF, 15)
    whole = ns.embedding_backward(dy, ids, w)
    for first in range(0, w, 100):
        check_backward(ns, dy, ids, 100, first=first)
    table = rand((w, dim), BF, 16)
    parts = [ns.embedding(ids, table[f:f + 100], first=f) for f in range(0, w, 100)]
    assert torch.equal(sum(parts), ns.embedding(ids, table)) and whole.shape == (w, dim)


def test_empty_calls(ns):
    w = rand((10, 24), BF, 21)
    none = torch.empty((0,), dtype=torch.int64, device="cuda")
    assert ns.embedding(none, w).shape == (0, 24)
    assert ns.embedding(none.view(0, 3), w).shape == (0, 3, 24)
    assert float(ns.embedding_backward(none.new_empty((0, 24), dtype=BF), none, 10).abs().max()) == 0
    keep = w.clone()
    ns.embedding_backward(none.new_empty((0, 24), dtype=BF), none, 10, dw=w, accumulate=True)
    assert torch.equal(w, keep)
    ids = torch.zeros((3,), dtype=torch.int64, device="cuda")
    assert float(ns.embedding(ids, w[:0]).abs().max()) == 0
    assert ns.embedding_backward(rand((3, 24), BF, 22), ids, 0).shape == (0, 24)
    assert ns.embedding(ids, w[:, :0]).shape == (3, 0)
    assert ns.embedding_backward(rand((3, 0), BF, 22), ids, 5).shape == (5, 0)
    one = torch.tensor(4, device="cuda")
    check_forward(ns, one, w)
    check_backward(ns, rand((24,), BF, 23), one, 10)
    check_backward(ns, rand((3, 24), BF, 24), ids - 1, 10)  # no token has a row


def test_strides_and_alignments(ns):
    rows, dim, tokens = 40, 130, 333
    ids = make_ids("zipf", tokens, rows, 31)
    for start, ld in ((0, 200), (1, 131), (3, 137), (8, 136)):
        for dt in (BF, F32):
            def view(n, seed):
                return rand((n * ld + 16,), dt, seed)[start:start + n * ld].view(n, ld)[:, :dim]
            buf = torch.full((tokens, ld + start), 7.0, dtype=dt, device="cuda")
            check_forward(ns, ids, view(rows, 32), out=buf[:, start:start + dim])
            assert bool((buf[:, start + dim:] == 7).all()) and bool((buf[:, :start] == 7).all())
            buf = torch.full((rows, ld + start), 7.0, dtype=dt, device="cuda")
            check_backward(ns, view(tokens, 33), ids, rows, dw=buf[:, start:start + dim])
            assert bool((buf[:, start + dim:] == 7).all()) and bool((buf[:, :start] == 7).all())
    wide = torch.stack([ids, ids], 1)[:, 0]
    assert not wide.is_contiguous()
    check_forward(ns, wide, rand((rows, dim), BF, 34))
    check_backward(ns, rand((dim,), BF, 35).expand(tokens, dim), wide, rows)
    # a table past 2^31 elements
    big = torch.zeros(((1 << 31) // 64 + 9, 64), dtype=BF, device="cuda")
    big[-5:] = rand((5, 64), BF, 36)
    n = big.shape[0]
    at = torch.tensor([n - 1, n - 5, 3, n], device="cuda")
    y = ns.embedding(at, big)
    assert torch.equal(y[0], big[-1]) and torch.equal(y[1], big[-5]) and not bool(y[2:].any())
    dy = rand((4, 64), BF, 37)
    ns.embedding_backward(dy, at, n, dw=big)
    assert torch.equal(big[-1], dy[0]) and torch.equal(big[-5], dy[1]) and torch.equal(big[3], dy[2])
    assert int(big.ne(0).any(1).sum()) == 3


def test_infinities_stay_in_their_rows(ns):
    ids = make_ids("zipf", 500, 20, 41)
    dy = rand((500, 64), BF, 42)
    clean = ns.embedding_backward(dy, ids, 20)
    dy[100, 5] = math.nan
    bad = ns.embedding_backward(dy, ids, 20)
    row = int(ids[100])
    others = [r for r in range(20) if r != row]
    assert torch.equal(clean[others], bad[others]) and bool(bad[row, 5].isnan())
    # an id without a row hides whatever its gradient is
    ids[100] = -1
    assert bool(ns.embedding_backward(dy, ids, 20).isfinite().all())


def test_autograd(ns):
    ids = make_ids("zipf", 240, 50, 51).view(12, 20)
    w = rand((50, 96), BF, 52)
    leaf = w.clone().requires_grad_()
    y = ns.embedding(ids, leaf, scale=2.0, padding_idx=int(ids[0, 0]), dtype=F32)
    assert y.dtype is F32
    dy = rand(y.shape, F32, 53)
    y.backward(dy)
    assert leaf.grad.dtype is BF
    assert torch.equal(leaf.grad, ns.embedding_backward(dy, ids, 50, scale=2.0, padding_idx=int(ids[0, 0]), dw_dtype=BF))
    leaf.grad = None
    ns.embedding(ids, leaf).sum().backward()  # an expanded gradient
    count = torch.bincount(ids.flatten(), minlength=50)
    assert torch.equal(leaf.grad, count[:, None].expand(50, 96).to(BF))
    with pytest.raises(ns.MuonError):
        ns.embedding(ids, leaf, out=torch.empty(ids.shape + (96,), device="cuda"))
    y = ns.embedding(ids, leaf)
    saved = y.grad_fn.saved_tensors[0]
    saved.add_(1)
    with pytest.raises(RuntimeError):
        y.sum().backward()


def test_a_lookups_gradient_against_differences(ns):
    """The lookup is linear in its table: a difference is exact but for roundings."""
    ids = make_ids("uniform", 60, 30, 61)
    w, v, c = rand((30, 24), F32, 62), rand((30, 24), F32, 63), rand((60, 24), F32, 64)
    leaf = w.clone().requires_grad_()
    ns.embedding(ids, leaf, scale=1.5).backward(c)
    ends = [float((ns.embedding(ids, w + s * v, scale=1.5).double() * c.double()).sum()) for s in (1, -1)]
    size = float((c.double().abs() * 1.5 * (w.abs() + v.abs())[ids].double()).sum())
    assert abs((ends[0] - ends[1]) / 2 - float((leaf.grad.double() * v.double()).sum())) <= size * 2.0 ** -20


def test_refusals(ns):
    ids, w, dy = make_ids("zipf", 10, 20, 71), rand((20, 16), BF, 72), rand((10, 16), BF, 73)
    for bad, code in [
        (lambda: ns.embedding(ids.float(), w), -2), (lambda: ns.embedding(ids, w.half()), -2), (lambda: ns.embedding(ids, w[0]), -1),
        (lambda: ns.embedding(ids.cpu(), w), -1), (lambda: ns.embedding(ids, w, out=w[:10]), -1), (lambda: ns.embedding(ids, w.t()), -1),
        (lambda: ns.embedding(ids, w, scale=math.inf), -1), (lambda: ns.embedding(ids, w, scale="x"), -1), (lambda: ns.embedding(ids, w, first=1.5), -1),
        (lambda: ns.embedding(ids, w, first=2 ** 63), -1), (lambda: ns.embedding(ids, w, dtype=torch.float16), -2),
        (lambda: ns.embedding_backward(dy[:9], ids, 20), -1), (lambda: ns.embedding_backward(dy, ids, 20, accumulate=True), -1),
        (lambda: ns.embedding_backward(dy, ids, -1), -1), (lambda: ns.embedding_backward(dy, ids, 20, dw=w[:, :8]), -1),
        (lambda: ns.embedding_backward(dy, ids, 10, dw=dy), -1), (lambda: ns.embedding_backward(dy, ids, "a"), -1),
        (lambda: ns.embedding_backward(dy, ids, 20, dw=w, dw_dtype=F32), -2), (lambda: ns.embedding_backward(dy, ids, 20, padding_idx=0.5), -1),
        (lambda: ns.embedding_backward(dy, ids, 20, dw=w.clone().requires_grad_()), -1),
    ]:
        with pytest.raises(ns.MuonError) as e:
            bad()
        assert e.value.status == code


def test_streams_bits_and_graphs(ns):
    tokens, rows, dim = 3000, 5000, 264
    ids, w, dy = make_ids("zipf", tokens, rows, 81), rand((rows, dim), BF, 82), rand((tokens, dim), BF, 83)

    def both():
        return ns.embedding(ids, w, scale=2.0), ns.embedding_backward(dy, ids, rows, scale=2.0), ns.embedding_backward(dy, ids, rows, dw_dtype=F32)
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
        ids.copy_(make_ids(KINDS[i], tokens, rows, 90 + i))
        dy.copy_(rand(dy.shape, BF, 95 + i))
        for graph, _ in (graphs if i % 2 else graphs[::-1]):
            graph.replay()
        want = both()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(p, q) for p, q in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    leaf = w.clone().requires_grad_()
    with torch.cuda.graph(graph):
        torch.zeros(1, device="cuda")
        with pytest.raises(ns.MuonError):
            ns.embedding(ids, leaf)
