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


def test_sizes_whose_gradient_is_summed_by_the_longest_pieces():
    """What test_gpu_pass_paths.py takes for pieces of 64 tokens is, by the slots in their workspace."""
    import ctypes
    from newton_schulz_ns5_amd import _lib
    from test_gpu_pass_paths import LONG_PIECES
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    need = ctypes.c_size_t()
    for tokens, rows, dim, dtype in LONG_PIECES:
        p = _lib.EmbeddingProblem(tokens=tokens, rows=rows, dim=dim, ids=1 << 40, w=1 << 42, w_row_stride=dim, y=1 << 44, y_row_stride=dim,
                                  w_dtype=_lib.MUON_F32, y_dtype=_lib.MUON_F32 if dtype is torch.float32 else _lib.MUON_BF16, scale=1.0)
        assert _lib.lib().muon_embedding_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(need)) == 0
        sort = 4 * up(4 * tokens) + up((tokens + 2047) // 2048 * 512 * 4) + 2048
        assert need.value - sort == up((tokens + 63) // 64 * 2 * dim * 4), (tokens, dim)
