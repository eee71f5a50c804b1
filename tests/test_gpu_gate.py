"""Precision of the gate's arithmetic where it is largest against the rounding
of its outputs: gates far out on the negative side, where an exponential whose
argument is rounded first is off by |g| 2^-24, and sigmoids below 2^-126.

Error bounds (u = 2^-24, no term that grows with |g|). The exponential e of -g
is good to 2 ulp and a correction's rounding (5 u), the sum 1 + e to u, the
reciprocal to 1 ulp (2 u): sigmoid(g) = 1 / (1 + e) is within 8 u relative, and
so is sigmoid(-g) = e / (1 + e), with one product more, except below 0.2, where
it is 9 u and enters beside a sigmoid(g) that is then within 4 u. Where the
result is subnormal, 2^-148 absolute. Every further product and sum adds u of
its own result.

The forward cases take their projections from one contraction block of few,
short products, so that the block's sum P is exact in FP32 and the projections
are round(P * round(sX * sW)) with FP32 roundings: known to the last bit."""
import numpy as np
import pytest
import torch

from tests import mlp_ref as R
from tests.gpu_util import rows_scales, to_np

pytestmark = pytest.mark.gpu

fg = pytest.importorskip("fp8_fine_grained_gb300")
DEV = "cuda"
U = R.U24
TINY = 2.0 ** -148


def f64(t):
    return t.double().cpu().numpy()


def sigmoid_bound(g):
    return 8 * U * R.sigmoid(g) + TINY


def encode(v):
    """E4M3 codes of values that E4M3 holds exactly."""
    table = {x: c for c, x in enumerate(R.DECODE) if c < 0x7F}
    return np.array([table[abs(x)] | (0x80 if x < 0 else 0) for x in v.reshape(-1)], np.uint8).reshape(v.shape)


def _exact_projections(M, I, base, up_scale, seed):
    """Operands (as the kernels take them) and the projections in FP32."""
    rng = np.random.default_rng(seed)
    K = 128
    x, w = np.zeros((M, K)), np.zeros((2 * I, K))
    x[:, 0] = 1.0
    x[:, 1:3] = rng.choice([1.0, 1.5], (M, 2))
    w[:I, 0] = base
    w[I:, 0] = rng.choice([-1.0, 1.0], I) * 4
    w[:, 1:3] = rng.integers(8, 16, (2 * I, 2)) / 32.0
    sx = (1 + 0.03 * rng.random(M)).astype(np.float32)
    sw = np.ones((2 * I // 128, 1), np.float32)
    sw[I // 128:] = up_scale
    P = (x @ w.T).astype(np.float32)                       # at most 13 bits
    assert np.array_equal(P, x @ w.T)
    s2 = sx[:, None] * np.repeat(sw[:, 0], 128)[None, :]   # one FP32 rounding
    gu = P * s2                                            # and another
    ld = (M + 3) // 4 * 4
    sxd = torch.zeros(1, ld, device=DEV)
    sxd[0, :M] = torch.from_numpy(sx).to(DEV)
    ops = (torch.from_numpy(encode(x)).to(DEV), sxd, torch.from_numpy(encode(w)).to(DEV),
           torch.from_numpy(sw).to(DEV))
    return ops, gu[:, :I].astype(np.float64), gu[:, I:].astype(np.float64)


# up to 32 tokens; 128-token tiles in clusters; persistent tiles
@pytest.mark.parametrize("M,I", [(32, 18432), (160, 4096), (1300, 2048)])
@pytest.mark.parametrize("base,up_scale", [(-48.0, 2.0 ** 20), (-88.0, 2.0 ** 30), (-16.0, 1.0), (3.0, 1.0)])
def test_forward(M, I, base, up_scale):
    ops, G, Up = _exact_projections(M, I, base, up_scale, seed=M)
    h, s, _ = fg.fp8_gated_gemm(*ops)
    assert fg.device_status() == 0
    sil = G * R.sigmoid(G)
    ref = sil * Up
    err = np.abs(G * Up) * sigmoid_bound(G) + 2 * U * np.abs(ref) + TINY * np.abs(Up)
    assert np.abs(ref).max(1).min() > 2.0 ** -119          # every row has codes of its own
    R.check_codes(to_np(h), rows_scales(s, M), ref, err, what="gate at %g" % base)


@pytest.mark.parametrize("base,spread", [(-88.0, 1.0), (-70.0, 3.0), (-48.0, 3.0), (-20.0, 3.0), (0.0, 2.0), (40.0, 5.0)])
def test_backward(base, spread):
    M, I = 512, 2048
    g = torch.Generator(device=DEV)
    g.manual_seed(int(base) + 100)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    gate = base + spread * (2 * torch.rand(M, I, generator=g, device=DEV) - 1)
    gu = torch.cat([gate, r(M, I) * 2.0 ** 15], 1).to(torch.bfloat16)
    dh = (r(M, I) * 2.0 ** 15).to(torch.bfloat16)
    q, s, qT, sT, hqT, hsT = fg.fp8_gated_bwd(gu, dh)
    assert fg.device_status() == 0
    G, Up, d = f64(gu[:, :I]), f64(gu[:, I:]), f64(dh)
    dG, dU, h = R.gate_bwd(G, Up, d)
    sg, es, ec = R.sigmoid(G), sigmoid_bound(G), sigmoid_bound(-G)
    a, c = np.abs(G) * sg, R.sigmoid(-G)
    ea = np.abs(G) * es + U * a + TINY
    slope = sg + G * sg * c
    eslope = es + ea * c + a * ec + ea * ec + U * np.abs(slope) + TINY
    eG = np.abs(d * Up) * (1 + U) * eslope + 3 * U * np.abs(dG)
    eU = np.abs(d) * ea + 2 * U * np.abs(dU)
    eh = np.abs(Up) * ea + 2 * U * np.abs(h)
    ref, err = np.concatenate([dG, dU], 1), np.concatenate([eG, eU], 1)
    R.check_codes(to_np(q), rows_scales(s, M), ref, err, what="gate gradient")
    R.check_codes(to_np(qT), rows_scales(sT, 2 * I), ref.T, err.T, what="gate gradient, transposed")
    R.check_codes(to_np(hqT), rows_scales(hsT, I), h.T, eh.T, what="activation, transposed")
