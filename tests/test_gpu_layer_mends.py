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
from test_gpu_layer import ACTS, BF, F32, U, act64, close, rand

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
