"""The norm's bounded waits: a row that never arrives is reported, the launch
ends with the CTA's other rows and its copies in flight behind it, and the next
call is right. Sizes give the CTA that waits one row, more rows than its ring
has slots, and each width of kernel."""
import pytest
import torch

from tests import test_gpu_norm as N

pytestmark = pytest.mark.gpu

fg = pytest.importorskip("fp8_fine_grained_gb300")
ETIMEOUT = 5
SIZES = [(1, 256), (20000, 256), (9000, 512), (3, 1024), (4000, 1024), (3000, 7168), (1000, 12288)]


@pytest.fixture
def short_waits():
    fg.set_wait_limit_ns(50_000_000)
    yield
    fg.set_wait_limit_ns(2_000_000_000)
    fg.device_status()


@pytest.mark.parametrize("T,D", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_forward(short_waits, T, D, residual):
    x, r, w = N._inputs(T, D, seed=D)
    r = r if residual else None
    fg.inject_skip_first_load()
    fg.fp8_rmsnorm(x, w, N.EPS, residual=r)
    assert fg.device_status() == ETIMEOUT
    out = fg.fp8_rmsnorm(x, w, N.EPS, residual=r)
    assert fg.device_status() == 0                 # (the request was used up)
    N._check_fwd(x, r, w, out)


@pytest.mark.parametrize("T,D", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_backward(short_waits, T, D, residual):
    x, r, w = N._inputs(T, D, seed=D)
    rstd = torch.rand(T, device=N.DEV) + 0.5
    dres = r if residual else None
    fg.inject_skip_first_load()
    fg.fp8_rmsnorm_bwd(r, x, rstd, w, dres=dres)
    assert fg.device_status() == ETIMEOUT
    dx, dgamma = fg.fp8_rmsnorm_bwd(r, x, rstd, w, dres=dres)
    assert fg.device_status() == 0
    N._check_bwd(r, x, rstd, w, dres, dx, dgamma)


def test_a_call_without_rows_leaves_the_request_alone(short_waits):
    """Nothing is launched, so the request waits for the next launch."""
    x, r, w = N._inputs(4, 256, seed=1)
    fg.inject_skip_first_load()
    fg.fp8_rmsnorm(x[:0], w, N.EPS)
    assert fg.device_status() == 0
    fg.fp8_rmsnorm(x, w, N.EPS)
    assert fg.device_status() == ETIMEOUT
