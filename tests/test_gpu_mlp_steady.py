"""The MLP operators where every CTA is well past its first rows or tiles:
slots refilled and barriers in their further phases, chunk after chunk of one
tensor, outputs written over inputs whose later rows are still being fetched.
Sizes are for 152 SMs; the bounds are those of the operators' own tests."""
import math

import numpy as np
import pytest
import torch

from tests import test_gpu_gated as G
from tests import test_gpu_norm as N

pytestmark = pytest.mark.gpu

fg = pytest.importorskip("fp8_fine_grained_gb300")
DEV = "cuda"
U = N.U

# 6 to 16 rows per CTA, in each width of kernel
ROWS = [(9000, 512), (9001, 1152), (3000, 7168), (1500, 12288)]


@pytest.mark.parametrize("T,D", ROWS)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_forward(T, D, residual):
    x, r, w = N._inputs(T, D, seed=T)
    r = r if residual else None
    out = fg.fp8_rmsnorm(x, w, N.EPS, residual=r)
    assert fg.device_status() == 0
    N._check_fwd(x, r, w, out)


@pytest.mark.parametrize("T,D", ROWS)
@pytest.mark.parametrize("over", ["x", "residual"])
def test_norm_forward_in_place(T, D, over):
    x, r, w = N._inputs(T, D, seed=T + 1)
    want = fg.fp8_rmsnorm(x, w, N.EPS, residual=r)
    got = fg.fp8_rmsnorm(x, w, N.EPS, residual=r, h=x if over == "x" else r)
    assert fg.device_status() == 0
    assert got[2].data_ptr() == (x if over == "x" else r).data_ptr()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1][:, :T], got[1][:, :T])
    assert torch.equal(want[2], got[2]) and torch.equal(want[3], got[3])


def _bwd_inputs(T, D, seed):
    x, r, w = N._inputs(T, D, seed)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 1)
    dy = (torch.randn(T, D, generator=g, device=DEV) * 1e-3).to(torch.bfloat16)
    return x, torch.rand(T, generator=g, device=DEV) + 0.5, w, dy, (r * 1e-3).to(torch.bfloat16)


@pytest.mark.parametrize("T,D", ROWS)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_backward(T, D, residual):
    h, rstd, w, dy, dres = _bwd_inputs(T, D, seed=T)
    dres = dres if residual else None
    dx, dgamma = fg.fp8_rmsnorm_bwd(dy, h, rstd, w, dres=dres)
    assert fg.device_status() == 0
    N._check_bwd(dy, h, rstd, w, dres, dx, dgamma)


@pytest.mark.parametrize("T,D", ROWS + [(21, 640), (1, 256)])
@pytest.mark.parametrize("residual,over", [(False, "dy"), (True, "dy"), (True, "dres")])
def test_norm_backward_in_place(T, D, residual, over):
    h, rstd, w, dy, dres = _bwd_inputs(T, D, seed=T + 2)
    dres = dres if residual else None
    want = fg.fp8_rmsnorm_bwd(dy, h, rstd, w, dres=dres)
    buf = dy if over == "dy" else dres
    got = fg.fp8_rmsnorm_bwd(dy, h, rstd, w, dres=dres, dx=buf)
    assert fg.device_status() == 0 and got[0].data_ptr() == buf.data_ptr()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("M,K,I", [(4096, 256, 3328), (4000, 384, 3200), (1300, 128, 18432)])
@pytest.mark.parametrize("save", [False, True])
def test_gated_forward(M, K, I, save):
    """Five to ten persistent tiles per CTA; rows of every m-tile, every column."""
    ops = G._operands(M, K, I, seed=M + K)
    out = fg.fp8_gated_gemm(*ops, save=save)
    assert fg.device_status() == 0
    rng = np.random.default_rng(0)
    first = np.arange(0, M, 128)
    rows = np.unique(np.concatenate([first, np.minimum(first + rng.integers(0, 128, len(first)), M - 1), [M - 1]]))
    G._check_fwd(ops, out, rows=rows)
    again = fg.fp8_gated_gemm(*ops, save=save)
    assert torch.equal(out[0], again[0]) and torch.equal(out[1][:, :M], again[1][:, :M])


def _check_clip(grads, before, max_norm, norm, out):
    """The bounds of the clipping's own tests, in 64 bits on the device."""
    ref = math.sqrt(sum(float(b.double().pow(2).sum()) for b in before))
    got, coef = (float(v) for v in norm.cpu())
    assert abs(got - ref) <= 12 * U * ref
    c = min(1.0, max_norm / (ref + 1e-6))
    assert abs(coef - c) <= 14 * U * c
    for b, o in zip(before, out):
        for p in range(0, b.numel(), 1 << 26):
            want, have = b[p:p + (1 << 26)].double() * c, o[p:p + (1 << 26)].double()
            tol = 15 * U * want.abs()
            if b.dtype == torch.bfloat16:
                # half a spacing of bf16 values at the larger magnitude
                _, e = torch.frexp(torch.maximum(want.abs(), have.abs()).clamp(min=2.0 ** -126))
                tol += torch.ldexp(torch.ones_like(want), e - 9)
            assert bool(((have - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype,n,offset", [(torch.float32, 70000003, 0), (torch.float32, 70000003, 3),
                                            (torch.bfloat16, 150000007, 1), (torch.float32, 33000001, 2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_one_large_tensor(dtype, n, offset, in_place):
    """Many chunks of one tensor per CTA, on both sides of the size where the
    scaling changes its CTAs; starts off the 16-byte grid."""
    g = torch.Generator(device=DEV)
    g.manual_seed(n + offset)
    grad = (torch.randn(n + offset, generator=g, device=DEV) * 1e-3).to(dtype)[offset:]
    before = grad.clone()
    out = None if in_place else [torch.full((n,), 9.0, dtype=dtype, device=DEV)]
    max_norm = 0.3e-3 * math.sqrt(n)
    norm, got = fg.grad_clip([grad], max_norm, 1e-6, out=out)
    assert fg.device_status() == 0
    _check_clip([grad], [before], max_norm, norm, got)
    if not in_place:
        assert torch.equal(grad, before)


@pytest.mark.parametrize("scale", [1e14, 1e15, 1e17, 2e17])
def test_norms_beyond_the_square_root_of_a_float(scale):
    """Sums of squares on both sides of 1e30, where the root takes a rescaled
    sum, and past the largest float."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    grads = [(torch.randn(n, generator=g, device=DEV) * scale).to(t)
             for n, t in ((4001, torch.float32), (100003, torch.bfloat16), (7, torch.float32))]
    before = [t.clone() for t in grads]
    norm, out = fg.grad_clip(grads, 1.0, 1e-6, out=[torch.empty_like(t) for t in grads])
    _check_clip(grads, before, 1.0, norm, out)
