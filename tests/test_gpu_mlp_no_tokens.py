"""A training step of the gated MLP block with no tokens (a rank or an expert
that got none): empty activations, weight gradients of zero."""
import pytest
import torch

pytestmark = pytest.mark.gpu

fg = pytest.importorskip("fp8_fine_grained_gb300")
from fp8_fine_grained_gb300 import mlp  # noqa: E402


@pytest.mark.parametrize("residual", [False, True])
def test_no_tokens(residual):
    D, I, dev = 256, 384, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    w = mlp.quantize(r(D), r(2 * I, D), r(D, I))
    x = r(0, D)
    y, h, saved = mlp.forward(x, x if residual else None, w, save=True)
    assert y.shape == (0, D) and h.shape == (0, D)
    grads = mlp.backward(x, saved, w, dres=x if residual else None)
    for t, shape, dtype in zip(grads, ((0, D), (2 * I, D), (D, I), (D,)), (torch.bfloat16,) + (torch.float32,) * 3):
        assert tuple(t.shape) == shape and t.dtype == dtype and t.is_cuda and not torch.any(t)
    norm = mlp.clip(grads, 1.0)
    assert norm.tolist() == [0.0, 1.0] and fg.device_status() == 0
