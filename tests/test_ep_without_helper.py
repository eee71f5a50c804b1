"""The expert-parallel dispatch where the compiled helper could not be built: none of
the other calls of that layer needs it, so the plan comes out of torch."""
import sys

import pytest
import torch

import fp8_fine_grained_gb300 as fg
from fp8_fine_grained_gb300 import build as libbuild
from fp8_fine_grained_gb300 import ep


@pytest.fixture
def no_helper(monkeypatch):
    monkeypatch.setattr(fg, "_helper", None)
    monkeypatch.setitem(sys.modules, "fp8_fine_grained_gb300._tensors", None)   # (an import error)
    monkeypatch.delattr(fg, "_tensors", raising=False)


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""
    is_cuda = True


def ids(T=33, k=6, E=32):
    g = torch.Generator().manual_seed(3)
    t = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    t[torch.rand(T, k, generator=g) < 0.1] = -1
    return t


def same(a, b):
    assert torch.equal(a.dest.cpu(), b.dest) and torch.equal(a.send_counts.cpu(), b.send_counts) and a.n_send == b.n_send
    assert a.dest.dtype == b.dest.dtype and a.send_counts.dtype == b.send_counts.dtype


def test_helper_built(no_helper):
    assert not fg.helper_built()


def test_the_helper_is_built_here():
    libbuild.build()
    assert fg.helper_built()


def test_dispatch_without_the_helper(no_helper):
    t = ids()
    got = ep.plan_dispatch(t.as_subclass(OnGpu), 32, 4)
    same(ep.Plan(*(v.as_subclass(torch.Tensor) if isinstance(v, torch.Tensor) else v for v in got)), ep.plan_dispatch(t, 32, 4))


@pytest.mark.gpu
def test_dispatch_on_the_gpu_without_the_helper(no_helper):
    t = ids(700)
    same(ep.plan_dispatch(t.cuda(), 32, 4), ep.plan_dispatch(t, 32, 4))
    with pytest.raises(RuntimeError, match="not built"):
        fg.moe_plan(t.cuda(), 32)
