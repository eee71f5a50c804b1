"""The gated MLP block (mlp.py) as a whole: forward, backward and clipping
against the same block in 64 bits.

The kernels are checked element by element elsewhere; here the bound is that of
the quantisation. E4M3 rounds a value to 2^-4 relative at most, 2.6 % rms (an
even spread of the mantissa), so a product of two quantised matrices is off by
sqrt(2) * 2.6 % = 3.7 % rms and n such steps in a row by about sqrt(n) * 3.7 %:
forward two steps with a product of two projections in between, 3.7 * sqrt(3)
= 6.4 %; gradients up to five, 8.3 %. The bounds are 10 % and 14 % of the
result's 2-norm."""
import numpy as np
import pytest
import torch

from tests import mlp_ref as R

pytestmark = pytest.mark.gpu

fg = pytest.importorskip("fp8_fine_grained_gb300")
from fp8_fine_grained_gb300 import mlp  # noqa: E402

DEV = "cuda"
EPS = 1e-6


def f64(t):
    return t.double().cpu().numpy()


def _block(T, D, I, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    gamma = 1 + 0.2 * r(D)
    w13 = (r(2 * I, D) * D ** -0.5).to(torch.bfloat16)
    w2 = (r(D, I) * I ** -0.5).to(torch.bfloat16)
    x, res, dy, dres = (r(T, D).to(torch.bfloat16) for _ in range(4))
    return gamma, w13, w2, x, res, dy, dres


def _reference(gamma, w13, w2, x, res, dy, dres):
    I = w2.shape[1]
    h = f64((x.float() + res.float()).to(torch.bfloat16))
    gm, W13, W2, dY = f64(gamma), f64(w13), f64(w2), f64(dy)
    rstd = R.rms(h, EPS)
    n = h * rstd[:, None] * gm
    gu = n @ W13.T
    G, U = gu[:, :I], gu[:, I:]
    a = R.gate(G, U)
    y = a @ W2.T
    da = dY @ W2
    dG, dU, _ = R.gate_bwd(G, U, da)
    dgu = np.concatenate([dG, dU], 1)
    dn = dgu @ W13
    dx, dgamma, _, _ = R.norm_bwd(dn, h, rstd, gm)
    return y, h, dx + f64(dres), dgu.T @ n, dY.T @ a, dgamma


def _off(got, ref):
    return np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("T,D,I", [(128, 256, 384), (384, 512, 256)])
def test_training_step(T, D, I):
    args = _block(T, D, I, seed=T)
    gamma, w13, w2, x, res, dy, dres = args
    w = mlp.quantize(gamma, w13, w2, EPS)
    y, h, saved = mlp.forward(x, res, w, save=True)
    g = mlp.backward(dy, saved, w, dres=dres)
    assert fg.device_status() == 0
    ry, rh, rdx, rdw13, rdw2, rdgamma = _reference(*args)
    assert np.array_equal(f64(h), rh)
    assert _off(y, ry) < 0.10
    for got, ref in ((g.dx, rdx), (g.dw13, rdw13), (g.dw2, rdw2), (g.dgamma, rdgamma)):
        assert tuple(got.shape) == ref.shape
        assert _off(got, ref) < 0.14
    before = [f64(t) for t in (g.dw13, g.dw2, g.dgamma)]
    norm = np.sqrt(sum((b * b).sum() for b in before))
    got = mlp.clip(g, 0.5 * norm)
    assert abs(float(got[0]) - norm) < 1e-6 * norm and abs(float(got[1]) - 0.5) < 1e-5
    for t, b in zip((g.dw13, g.dw2, g.dgamma), before):
        assert np.allclose(f64(t), b * float(got[1]), rtol=1e-6, atol=0)


@pytest.mark.parametrize("T", [1, 3, 37, 200])
def test_serving_step(T):
    gamma, w13, w2, x, res, _, _ = _block(T, 512, 384, seed=T)
    w = mlp.quantize(gamma, w13, w2, EPS)
    y, h, saved = mlp.forward(x, res, w)
    assert saved is None and fg.device_status() == 0
    ref = _reference(gamma, w13, w2, x, res, x, x)
    assert _off(y, ref[0]) < 0.10


def test_a_chain_of_blocks_in_a_cuda_graph():
    """Decoding through three blocks, captured once and replayed on new input:
    equal to the same calls made directly."""
    T, D, I = 4, 512, 384
    ws = []
    for i in range(3):
        gamma, w13, w2, x, res, _, _ = _block(T, D, I, seed=40 + i)
        ws.append(mlp.quantize(gamma, w13, w2, EPS))

    def run(x, res):
        for w in ws:
            x, res, _ = mlp.forward(x, res, w)
        return x, res
    xs, rs = x.clone(), res.clone()
    run(xs, rs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(xs, rs)
    for k in range(3):
        xs.copy_(x * (k + 1))
        rs.copy_(res)
        graph.replay()
        want = run(xs, rs)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert fg.device_status() == 0


def test_mismatched_weights_are_refused():
    gamma, w13, w2, *_ = _block(8, 256, 128, seed=1)
    with pytest.raises(ValueError, match="w13 must be"):
        mlp.quantize(gamma, w13, w2.t().contiguous(), EPS)
    with pytest.raises(ValueError, match="w13 must be"):
        mlp.quantize(gamma[:128], w13, w2, EPS)
