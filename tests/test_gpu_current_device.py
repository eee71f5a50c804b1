"""The operators between a gated MLP's GEMMs refuse tensors that are not on the
current device before anything is launched. The tensors here have no memory at
all (fake tensors that say cuda:1), so a call that does not refuse them cannot
reach a kernel either."""
import pytest
import torch

pytestmark = pytest.mark.gpu

fg = pytest.importorskip("fp8_fine_grained_gb300")
BF16, U8, F32 = torch.bfloat16, torch.uint8, torch.float32
MATCH = r"current device \(cuda:0\), not on cuda:1"


@pytest.fixture
def far(monkeypatch):
    from torch._subclasses import fake_tensor
    # (a fake tensor sets its device up first, which a machine may not have)
    monkeypatch.setattr(fake_tensor, "init_gpu_context", lambda device: None, raising=False)
    mode = fake_tensor.FakeTensorMode()

    def make(shape, dtype):
        with mode:
            return torch.empty(shape, dtype=dtype, device="cuda:1")
    return make


@pytest.fixture(autouse=True)
def first_device():
    assert torch.cuda.current_device() == 0


def refused(fn, *a, **kw):
    with pytest.raises(ValueError, match=MATCH):
        fn(*a, **kw)


@pytest.mark.parametrize("stream", [False, True])
def test_calls(far, stream):
    s = torch.cuda.Stream() if stream else None
    T, D, I, K = 128, 256, 128, 256
    x, w, r = far((T, D), BF16), far((D,), BF16), far((T,), F32)
    refused(fg.fp8_rmsnorm, x, w, q=far((T, D), U8), scales=far((D // 128, T), F32), rstd=r, stream=s)
    refused(fg.fp8_rmsnorm_t, x, r, w, qT=far((D, T), U8), scalesT=far((T // 128, D), F32), stream=s)
    refused(fg.fp8_rmsnorm_bwd, x, x, r, w, dx=far((T, D), BF16), dgamma=far((D,), F32), stream=s)
    refused(fg.fp8_gated_gemm, far((T, K), U8), far((K // 128, T), F32), far((2 * I, K), U8),
            far((2 * I // 128, K // 128), F32), h=far((T, I), U8), scales=far((I // 128, T), F32), stream=s)
    refused(fg.fp8_gated_bwd, far((T, 2 * I), BF16), far((T, I), BF16), q=far((T, 2 * I), U8),
            scales=far((2 * I // 128, T), F32), qT=far((2 * I, T), U8), scalesT=far((T // 128, 2 * I), F32),
            hqT=far((I, T), U8), hscalesT=far((T // 128, I), F32), stream=s)


def test_the_check_that_every_call_makes(far):
    H = fg._checks()
    near = torch.zeros(4, device="cuda:0")
    H.on_gpu(near, "a", None, "b")
    refused(H.on_gpu, None, "a", far((4,), F32), "b")
    with pytest.raises(ValueError, match="b must be on the other tensors' device"):
        H.on_gpu(near, "a", far((4,), F32), "b")
