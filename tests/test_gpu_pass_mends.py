"""Calls of the operators of a training pass that once gave something else than
documented."""
import pytest
import torch

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ns():
    torch_cuda()
    import newton_schulz_ns5_amd as m
    return m


def rand(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)


@pytest.mark.parametrize("cols", [64, 264, 2050, 16384])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_first_norm_written_over_its_block_returns_the_stream(ns, cols, dtype):
    """Where the stream is the block's output itself and the norm is written over it, the stream returned is
    what the block held before, not the norm."""
    b, w = rand((5, 3, cols), dtype, 1), rand((cols,), dtype, 2, 0.2, 1.0)
    s, want = ns.residual_norm(b, weight=w)
    assert s is b
    a = b.clone()
    s, y = ns.residual_norm(a, weight=w, out=a)
    assert y is a and torch.equal(y, want) and torch.equal(s, b)
    # through another view of the same rows
    a = b.clone()
    s, y = ns.residual_norm(a, weight=w, out=a.view(5, 3, cols))
    assert torch.equal(a, want) and torch.equal(s, b)
    # a block that is copied, since its rows are not evenly spaced, in the memory that the norm is written to
    a = b.clone()
    s, y = ns.residual_norm(a.transpose(0, 1), weight=w, out=a.view(3, 5, cols))
    assert torch.equal(y, want.transpose(0, 1)) and torch.equal(s, b.transpose(0, 1))
    # other columns of one buffer are not the block's: the stream is the block's output itself
    both = torch.cat([b.view(15, cols), b.view(15, cols)], 1)
    block = both[:, :cols]
    s, y = ns.residual_norm(block, weight=w, out=both[:, cols:])
    assert s is block and torch.equal(s, b.view(15, cols)) and torch.equal(y, want.view(15, cols))


def test_a_single_extra_gradient_is_clipped_as_a_whole(ns):
    """One launch's list of tensors, and the bits of the call with a list of one tensor."""
    ps = [torch.nn.Parameter(rand((64, 96), F32, 20))]
    ps[0].grad = rand((64, 96), F32, 21)
    table = rand((1000, 40), BF, 22)
    opt = ns.MuonNS5(ps)
    keep, one, two = ps[0].grad.clone(), table.clone(), table.clone()
    norm = opt.clip_grad_norm(0.5, extra=[one])
    clipped = ps[0].grad.clone()
    ps[0].grad.copy_(keep)
    assert torch.equal(opt.clip_grad_norm(0.5, extra=two), norm)
    assert torch.equal(one, two) and torch.equal(ps[0].grad, clipped) and not torch.equal(one, table)
    # a transposed one, whose elements lie side by side but not its rows'
    flat = rand((33, 65), F32, 23)
    ps[0].grad.copy_(keep)
    exact = float((keep.double().square().sum() + flat.double().square().sum()).sqrt())
    got = float(opt.clip_grad_norm(0.5, extra=flat.t()))
    assert abs(got - exact) <= 2.0 ** -23 * exact  # one rounding of an fp64 sum, and a margin of as much
