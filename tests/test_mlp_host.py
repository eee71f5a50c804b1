"""Refusals of the gated MLP block that come before any kernel (CPU)."""
import pytest
import torch

import fp8_fine_grained_gb300 as fg
from fp8_fine_grained_gb300 import mlp


@pytest.mark.parametrize("T", [1, 127, 129, 8191])
def test_saving_for_a_backward_pass_that_cannot_run(monkeypatch, T):
    """The backward pass groups the tokens by 128: other counts are refused when
    the forward pass is asked to save for it, not after the whole network's."""
    def reached(*a, **kw):
        raise AssertionError("a kernel was called")
    monkeypatch.setattr(fg, "fp8_rmsnorm", reached)
    x = torch.zeros(T, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="multiples of 128; got %d" % T):
        mlp.forward(x, None, mlp.Weights(*[None] * 5, 1e-6), save=True)
    with pytest.raises(AssertionError, match="a kernel was called"):
        mlp.forward(x, None, mlp.Weights(*[None] * 5, 1e-6))


@pytest.mark.parametrize("T", [0, 128, 1024])
def test_token_counts_that_it_takes(monkeypatch, T):
    class Reached(Exception):
        pass

    def reached(*a, **kw):
        raise Reached
    monkeypatch.setattr(fg, "fp8_rmsnorm", reached)
    with pytest.raises(Reached):
        mlp.forward(torch.zeros(T, 128, dtype=torch.bfloat16), None, mlp.Weights(*[None] * 5, 1e-6), save=True)
