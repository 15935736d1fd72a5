"""Paths of the operators of a training pass that only larger calls take: the
embedding gradient's digit sort with tokens that have no row, its longest pieces
and the count of many tiles; the norms' gradients with few and with very many
sequences; rows past 2^31 elements.

Embedding gradients here are of whole numbers whose sums stay below 2^24, so
fp32 holds every sum exactly in any order, and results have to be equal.
Tolerances of the norms' gradients: those of test_gpu_residual_norm.py but for
the terms of a sum over rows.  There a workgroup adds its rows, whose number is
at most twice an even share of the rows over the 256 workgroups or more that the
card holds (a whole number of workgroups for every sequence, or of sequences for
every workgroup), then groups of threads join by up to 6 additions, and of up
to 4096 partials each of 32 parts adds 128, the parts joining by 5: rows / 128
+ 160 terms.  A gate's sum over the n rows of a sequence has fewer than n + 20
roundings in whatever order."""
import math

import pytest
import torch

import test_gpu_residual_norm as norms
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
rand = norms.rand


@pytest.fixture(scope="module")
def ns():
    torch_cuda()
    import newton_schulz_ns5_amd as m
    return m


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def whole(shape, dtype, seed):
    return torch.randint(-3, 4, shape, generator=generator(seed), device="cuda").to(dtype)


def frequent(tokens, rows, seed):
    """Row numbers whose frequency falls with their rank."""
    u = torch.rand((tokens,), generator=generator(seed), device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(rows + 1)) - 1).long().clamp_(0, rows - 1)


def exact(dy, ids, first, rows, padding=None):
    """(gradient, which rows have a token), in 64 bits: sums of runs as differences of a running sum, exact too."""
    ids = ids.long()
    mine = (ids >= first) & (ids < first + rows)
    if padding is not None:
        mine &= ids != padding
    v = ids[mine] - first
    count = torch.bincount(v, minlength=rows)
    total = torch.cat([torch.zeros((1, dy.shape[-1]), device="cuda", dtype=torch.float64),
                       dy[mine][v.argsort()].double().cumsum(0)])
    ends = count.cumsum(0)
    want = total[ends] - total[ends - count]
    assert float(want.abs().max()) < 2 ** 24
    return want, count > 0


@pytest.mark.parametrize("tokens", [8193, 20011, 131073, 1100003])
@pytest.mark.parametrize("rows,dim", [(1, 8), (512, 20), (1000, 72), (1 << 18, 8)])
@pytest.mark.parametrize("kind", [torch.int64, torch.int32])
def test_digit_sort_of_a_shard(ns, tokens, rows, dim, kind):
    """More tokens than ranks are counted for, a third of them before the shard and behind it; rows of 2^9 and
    2^18, whose number, the key of a token without a row, takes one bit more than theirs; up to 538 tiles."""
    for first in (0, rows + 7, -rows):
        ids = frequent(tokens, rows, 1) + first
        away = torch.randint(0, 6, (tokens,), generator=generator(2), device="cuda")
        ids = torch.where(away == 0, ids + rows, torch.where(away == 1, ids - rows, ids)).to(kind)
        dy = whole((tokens, dim), BF, 3)
        for padding in (None, first):  # the most frequent one
            want, has = exact(dy, ids, first, rows, padding)
            how = dict(first=first, padding_idx=padding)
            assert torch.equal(ns.embedding_backward(dy, ids, rows, dw_dtype=F32, **how).double(), want), (first, padding)
            start = whole((rows, dim), F32, 4) + 0.5
            dw = start.clone()
            ns.embedding_backward(dy, ids, rows, dw=dw, accumulate=True, scale=2.0, **how)
            assert float(want.abs().max()) < 2 ** 21
            assert torch.equal(dw.double(), 2 * want + start.double()), (first, padding)
            assert torch.equal(dw[~has], start[~has])


def test_digit_sort_without_any_row(ns):
    ids = torch.full((9000,), -100, device="cuda")
    dy = whole((9000, 16), F32, 5)
    dw = torch.full((300, 16), 7.0, device="cuda")
    ns.embedding_backward(dy, ids, 300, dw=dw, accumulate=True)
    assert bool((dw == 7).all())
    ns.embedding_backward(dy, ids, 300, dw=dw)
    assert not bool(dw.any())


LONG_PIECES = [(40000, 1000, 4096, F32), (140001, 3, 1001, F32), (140001, 40000, 520, F32), (4300001, 100, 8, BF)]


@pytest.mark.parametrize("tokens,rows,dim,dtype", LONG_PIECES)
def test_the_longest_pieces(ns, tokens, rows, dim, dtype):
    """Pieces of 64 tokens (test_pass_mends_cpu.py holds the sizes to it)."""
    dy = whole((tokens, dim), dtype, 6)
    for kind in ("frequent", "same", "even", "halves"):
        ids = {"frequent": lambda: frequent(tokens, rows, 7), "same": lambda: torch.full((tokens,), rows - 1, device="cuda"),
               "even": lambda: torch.randint(0, rows, (tokens,), generator=generator(8), device="cuda"),
               "halves": lambda: (torch.arange(tokens, device="cuda") % 2) * (rows - 1)}[kind]()
        want, _ = exact(dy, ids, 0, rows)
        assert torch.equal(ns.embedding_backward(dy, ids, rows, dw_dtype=F32).double(), want), kind
        del want


@pytest.mark.parametrize("seqs,per,cols", [(3, 1366, 2048), (129, 20, 16384), (257, 9, 16384), (300, 27, 4096), (513, 9, 4096),
                                           (2, 5000, 24), (31, 300, 64), (5, 2000, 200), (600, 100, 520), (1, 9000, 512)])
@pytest.mark.parametrize("post", [True, False])
def test_sequences_of_uneven_shares(ns, seqs, per, cols, post):
    """Sequences that fill the card badly: workgroups of many rows, of several sequences, groups without a row."""
    shape = (seqs, per, cols)
    b, st = rand(shape, BF, 11), rand(shape, F32, 12, 2.0)
    w, pw = rand((cols,), F32, 13, 0.2, 1.0), rand((cols,), F32, 14, 0.2, 1.0) if post else None
    g = rand((seqs, 1, cols), F32, 15, 0.5)
    dy, dst = rand(shape, BF, 16, 0.1), rand(shape, F32, 17, 0.1)
    got = ns.residual_norm_backward(dy, dst, st, b, weight=w, post_weight=pw, gate=g, scale=0.75, residual_scale=0.5)
    want = norms.backward64(dy, dst, st, b, w, pw, g, post, 0.75, 0.5, 1e-6, 0.0)
    for name, t in zip(("dblock", "dresidual", "dweight", "dpost_weight", "dgate"), got):
        if t is None:
            assert name == "dpost_weight" and not post
            continue
        v, err = want[name]
        if name in ("dweight", "dpost_weight"):
            v, err = v.sum((0, 1)), err.sum((0, 1)) + (seqs * per / 128 + 160) * 2.0 ** -24 * v.abs().sum((0, 1))
        elif name == "dgate":
            v, err = v.sum(1, keepdim=True), err.sum(1, keepdim=True) + (per + 20) * 2.0 ** -24 * v.abs().sum(1, keepdim=True)
        norms.close(t, v, err, name)


def test_gradients_past_32_bits(ns):
    """The last rows of more than 2^31 elements have their own gradients, written over those that came in."""
    rows, cols = (1 << 31) // 4096 + 3, 4096
    s, dy = (torch.zeros((rows, cols), dtype=BF, device="cuda") for _ in range(2))
    s[-3:], dy[-3:] = rand((3, cols), BF, 21, 2.0), rand((3, cols), BF, 22)
    keep, w = dy[-3:].clone(), rand((cols,), BF, 23, 0.2, 1.0)
    got = ns.residual_norm_backward(dy, None, s, None, weight=w, dresidual=dy, need_dblock=False, residual_scale=0.5)
    assert got[1] is dy
    want = norms.backward64(keep, None, s[-3:], None, w, None, None, False, 1.0, 0.5, 1e-6, 0.0)
    norms.close(dy[-3:], *want["dresidual"], "dresidual")
    norms.close(got[2], *norms.summed(want["dweight"], (0,)), "dweight")
    assert not bool(dy[:-3].any())


def test_equal_gradients_of_two_leaves_are_theirs(ns):
    """The block's and the residual's gradient are one tensor inside the backward pass; two leaves do not share it."""
    a, b = (rand((9, 128), BF, 31 + i).requires_grad_() for i in range(2))
    dy = rand((9, 128), BF, 33)
    for _ in range(2):  # the second time onto gradients that are there
        ns.residual_norm(a, b)[1].backward(dy)
        assert torch.equal(a.grad, b.grad) and a.grad.data_ptr() != b.grad.data_ptr()
    keep = b.grad.clone()
    ns.clip_grad_norm([a.grad], 0.01)
    assert torch.equal(b.grad, keep) and not torch.equal(a.grad, keep)


@pytest.mark.parametrize("reentrant", [True, False])
def test_under_checkpointing(ns, reentrant):
    from torch.utils.checkpoint import checkpoint
    ids = frequent(60, 40, 41)
    ts = [rand((40, 72), BF, 42), rand((72,), BF, 43, 0.2, 1.0), rand((72,), BF, 44, 0.2, 1.0), rand((72,), BF, 45)]

    def fn(table, w, pw, g):
        x = ns.embedding(ids, table, scale=2.0)
        s, y = ns.residual_norm(x, weight=w)
        s, y = ns.residual_norm(y, s, weight=w, post_weight=pw, gate=g, scale=0.5)
        return s + y
    grads = []
    for run in (fn, lambda *a: checkpoint(fn, *a, use_reentrant=reentrant)):
        leaves = [t.clone().requires_grad_() for t in ts]
        run(*leaves).backward(rand((60, 72), BF, 46))
        grads.append([t.grad for t in leaves])
    assert all(torch.equal(p, q) for p, q in zip(*grads))


def test_lists_of_nothing_and_of_several_launches(ns):
    none = torch.empty((0, 5), device="cuda")
    for kind in (2, math.inf):
        assert float(ns.grad_norm([none], norm_type=kind)) == 0
        assert float(ns.clip_grad_norm([none, none], 1.0, norm_type=kind)) == 0
        assert float(ns.clip_grad_norm([none], 1.0, norm_type=kind, total=torch.tensor(3.0, device="cuda"))) == 3
    assert float(ns.clip_grad_norm([none], 1.0, total=torch.tensor(9.0, device="cuda", dtype=torch.float64))) == 3
    # a given total, the largest magnitude and a NaN over three launches
    xs = [rand((37,), F32, 50 + i) for i in range(300)]
    keep = [x.clone() for x in xs]
    assert float(ns.clip_grad_norm(xs, 1.0, eps=0.0, total=torch.tensor(4.0, device="cuda"))) == 4
    assert all(torch.equal(x, k / 4) for x, k in zip(xs, keep))
    top = max(float(x.abs().max()) for x in xs)
    assert float(ns.clip_grad_norm(xs, top / 2, eps=0.0, norm_type="inf")) == top
    assert all(torch.equal(x, k / 8) for x, k in zip(xs, keep))
    xs[299][5] = math.nan
    for kind in (2, math.inf):
        outs = [torch.zeros_like(x) for x in xs]
        assert math.isnan(float(ns.clip_grad_norm(xs, 1.0, norm_type=kind, out=outs)))
        assert all(bool(o.isnan().all()) for o in outs)


def test_inference_mode(ns):
    ids, table, w = frequent(20, 30, 61), rand((30, 40), BF, 62).requires_grad_(), rand((40,), BF, 63, 0.2, 1.0).requires_grad_()
    with torch.no_grad():
        x = ns.embedding(ids, table)
        want = (x.clone(),) + ns.residual_norm(x, x, weight=w)
    with torch.inference_mode():
        x = ns.embedding(ids, table, out=torch.empty((20, 40), dtype=BF, device="cuda"))
        got = (x.clone(),) + ns.residual_norm(x, x, weight=w, out=torch.empty_like(x))
        grads = [x.clone()]
        assert float(ns.clip_grad_norm(grads, 1e9)) == float(ns.grad_norm(grads))
    assert all(torch.equal(p, q) for p, q in zip(got, want))
