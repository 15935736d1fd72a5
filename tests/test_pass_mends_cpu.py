"""Calls of the operators of a training pass that once did something else than
documented, as far as they show without a GPU."""
import pytest
import torch

import newton_schulz_ns5_amd as ns


@pytest.mark.parametrize("shape", [(500, 8), (7,), ()])
def test_a_single_extra_gradient_is_one_tensor(monkeypatch, shape):
    """A tensor in the place of a list of them is that tensor, as clip_grad_norm has it, not its rows."""
    from newton_schulz_ns5_amd import pass_ops
    seen = []
    monkeypatch.setattr(pass_ops, "clip_grad_norm", lambda grads, max_norm, **how: seen.append(list(grads)))
    p = torch.nn.Parameter(torch.zeros(16, 32))
    p.grad = torch.ones(16, 32)
    extra = torch.ones(shape)
    opt = ns.MuonNS5([p])
    opt.clip_grad_norm(1.0, extra=extra)
    assert len(seen[0]) == 2 and seen[0][0] is p.grad and seen[0][1] is extra
    for several in ([extra, None], (extra,), iter([extra])):
        opt.clip_grad_norm(1.0, extra=several)
        grads = [t for t in seen[-1] if t is not None]
        assert len(grads) == 2 and grads[1] is extra
