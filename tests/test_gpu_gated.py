"""GPU parity of the gated feed-forward (fp8_gated_gemm) and of its backward
pass (fp8_gated_bwd) against 64-bit forms.

Error bounds. The two projections obey the GEMM's bound 1e-5 * T (T the sum of
absolute scaled products, from the oracle). With eG and eU those bounds,
h = silu(G) U is off by at most 1.1 |U| eG + |silu(G)| eU + 1.1 eG eU (the
slope of silu stays below 1.1), plus the gate's own FP32 error |G U| err(sigmoid)
+ 3 u |h| (u = 2^-24). Backward, from bf16 G, U, dh: with d = err(sigmoid),
sg + a (1 - sg) is off by d (1 + |a|) + |G| d (1 - sg) + 4 u (sg + |a|), the
products add 3 u."""
import numpy as np
import pytest
import torch

import oracle
from tests import mlp_ref as R
from tests.gpu_util import check_gemm, rows_scales, to_np

pytestmark = pytest.mark.gpu

fg = pytest.importorskip("fp8_fine_grained_gb300")
DEV = "cuda"
U = R.U24


def f64(t):
    return t.double().cpu().numpy()


def _operands(M, K, I, seed, wscale=0.05):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = (torch.randn(M, K, generator=g, device=DEV) * torch.exp(torch.randn(K, generator=g, device=DEV))
         ).to(torch.bfloat16)
    w = (torch.randn(2 * I, K, generator=g, device=DEV) * wscale).to(torch.bfloat16)
    # the two projections' blocks have scales of their own
    w[:I] *= 0.5
    return fg.fp8_quant_1x128(x) + fg.fp8_quant_128x128(w)


def _check_fwd(ops, out, rows=None, pow2=False):
    xq, sx, wq, sw = ops
    h, s, gu = out
    M, I = xq.shape[0], wq.shape[0] // 2
    rows = np.arange(M) if rows is None else rows
    c, _, t = oracle.fprop(np.ascontiguousarray(to_np(xq)[rows]), np.ascontiguousarray(rows_scales(sx, M)[rows]),
                           to_np(wq), to_np(sw))
    c, t = np.asarray(c, np.float64), np.asarray(t, np.float64)
    if gu is not None:
        check_gemm(to_np(gu)[rows], c, t, True, "projections")
    G, Up, eG, eU = c[:, :I], c[:, I:], 1e-5 * t[:, :I], 1e-5 * t[:, I:]
    sil = G * R.sigmoid(G)
    ref = sil * Up
    err = (1.1 * np.abs(Up) * eG + np.abs(sil) * eU + 1.1 * eG * eU + np.abs(G * Up) * R.sigmoid_err(G)
           + 3 * U * np.abs(ref))
    R.check_codes(to_np(h)[rows], rows_scales(s, M)[rows], ref, err, pow2, "gated")


@pytest.mark.parametrize("M,K,I", [(1, 128, 128), (1, 1024, 384), (3, 384, 128), (17, 7168, 256), (32, 512, 2048),
                                   (33, 256, 640), (64, 2048, 256), (65, 1152, 384), (128, 512, 512), (129, 256, 256),
                                   (200, 640, 1152), (333, 1280, 384), (500, 384, 640),
                                   (2600, 256, 1024), (1537, 128, 1664)])
@pytest.mark.parametrize("save", [False, True])
def test_forward(M, K, I, save):
    ops = _operands(M, K, I, seed=M + K + I)
    out = fg.fp8_gated_gemm(*ops, save=save)
    assert fg.device_status() == 0
    assert (out[2] is not None) == save
    _check_fwd(ops, out)


@pytest.mark.parametrize("M,I", [(2, 384), (40, 384), (300, 384), (1300, 2048)])
def test_forward_pow2(M, I):
    ops = _operands(M, 512, I, seed=3)
    _check_fwd(ops, fg.fp8_gated_gemm(*ops, pow2=True), pow2=True)


@pytest.mark.parametrize("M,K,I", [(1, 7168, 18432), (24, 7168, 2048), (1300, 1024, 2048)])
def test_forward_workload_widths(M, K, I):
    """The framework's widths; rows sampled, every column checked."""
    ops = _operands(M, K, I, seed=5, wscale=0.02)
    rows = np.unique(np.concatenate([[0, M - 1], np.random.default_rng(0).integers(0, M, 6)]))
    _check_fwd(ops, fg.fp8_gated_gemm(*ops, save=True), rows=rows)
    assert fg.device_status() == 0


@pytest.mark.parametrize("M,I", [(5, 256), (40, 256), (150, 256), (1500, 1792)])
def test_saturated_gates_and_zero_rows(M, I):
    """Gates far out on both sides, and rows of zeros (scale 1, zero codes)."""
    xq, sx, wq, sw = _operands(M, 256, I, seed=8, wscale=1.0)
    sx = sx.clone()
    sx[:, 1] *= 2.0 ** 12
    sx[:, 2] *= 2.0 ** -40
    xq = xq.clone()
    xq[0] = 0
    out = fg.fp8_gated_gemm(xq, sx, wq, sw, save=True)
    assert fg.device_status() == 0
    assert torch.all(out[1][:, 0] == 1.0) and torch.all(out[0][0] & 0x7F == 0)
    _check_fwd((xq, sx, wq, sw), out)


@pytest.mark.parametrize("M,I", [(7, 256), (50, 256), (139, 256), (1411, 1792)])
def test_strides_and_untouched_padding(M, I):
    K = 384
    xq, sx, wq, sw = _operands(M, K, I, seed=11)
    xp = torch.zeros(M, K + 64, dtype=torch.uint8, device=DEV)
    xp[:, 32:32 + K] = xq
    wp = torch.zeros(2 * I, K + 128, dtype=torch.uint8, device=DEV)
    wp[:, 16:16 + K] = wq
    sp = torch.zeros(K // 128, M // 4 * 4 + 40, device=DEV)
    sp[:, :M] = sx[:, :M]
    h = torch.full((M + 2, I + 48), 0x33, dtype=torch.uint8, device=DEV)
    s = torch.full((I // 128, M // 4 * 4 + 12), -2.0, device=DEV)
    gu = torch.full((M + 1, 2 * I + 24), 9.0, dtype=torch.bfloat16, device=DEV)
    hv, guv = h[:M, :I], gu[:M, :2 * I]
    out = fg.fp8_gated_gemm(xp[:, 32:32 + K], sp, wp[:, 16:16 + K], sw, h=hv, scales=s, gu=guv)
    assert fg.device_status() == 0
    assert torch.all(h[:, I:] == 0x33) and torch.all(h[M:] == 0x33)
    assert torch.all(s[:, M:] == -2.0)
    assert torch.all(gu[:, 2 * I:] == 9.0) and torch.all(gu[M:] == 9.0)
    _check_fwd((xq, sx, wq, sw), out)
    plain = fg.fp8_gated_gemm(xq, sx, wq, sw, save=True)
    assert torch.equal(plain[0], hv) and torch.equal(plain[2], guv) and torch.equal(plain[1][:, :M], s[:, :M])


@pytest.mark.parametrize("M,I", [(1, 512), (40, 512), (200, 512), (1300, 2048)])
def test_forward_is_repeatable(M, I):
    ops = _operands(M, 2048, I, seed=12)
    a, b = fg.fp8_gated_gemm(*ops, save=True), fg.fp8_gated_gemm(*ops, save=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1][:, :M], b[1][:, :M]) and torch.equal(a[2], b[2])


def test_no_rows():
    xq, sx, wq, sw = _operands(4, 256, 256, seed=13)
    h, s, gu = fg.fp8_gated_gemm(xq[:0], sx, wq, sw, save=True)
    assert h.shape == (0, 256) and gu.shape == (0, 512)
    assert fg.device_status() == 0


@pytest.mark.parametrize("M,I", [(8, 256), (300, 256), (1300, 2048)])
def test_forward_reports_a_withheld_load(M, I):
    """A load that never lands: the bounded waits run out, the status word
    says so and the next launch is clean."""
    ops = _operands(M, 1024, I, seed=14)
    fg.set_wait_limit_ns(50_000_000)
    try:
        fg.inject_skip_first_load()
        fg.fp8_gated_gemm(*ops)
        assert fg.device_status() == 5  # FP8FG_ETIMEOUT
    finally:
        fg.set_wait_limit_ns(2_000_000_000)
    out = fg.fp8_gated_gemm(*ops)
    assert fg.device_status() == 0
    _check_fwd(ops, out)


def test_on_another_stream():
    """A side stream's outputs come from its own memory: nothing that is queued
    on the current stream can still be using it."""
    ops = _operands(100, 1024, 512, seed=15)
    gu, dh = _bwd_inputs(128, 256, seed=15)
    want, wantb = fg.fp8_gated_gemm(*ops), fg.fp8_gated_bwd(gu, dh)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    junk = [torch.full((100, 512), 7, dtype=torch.uint8, device=DEV) for _ in range(20)]
    del junk
    got, gotb = fg.fp8_gated_gemm(*ops, stream=side), fg.fp8_gated_bwd(gu, dh, stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1][:, :100], got[1][:, :100])
    assert all(torch.equal(a, b) for a, b in zip(wantb, gotb))
    assert torch.cuda.current_stream() != side


# ---------------------------------------------------------------- backward ----

def _bwd_inputs(M, I, seed, scale=1.5):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    gu = (torch.randn(M, 2 * I, generator=g, device=DEV) * scale).to(torch.bfloat16)
    dh = (torch.randn(M, I, generator=g, device=DEV) * 1e-3).to(torch.bfloat16)
    return gu, dh


def _check_bwd(gu, dh, out, pow2=False):
    q, s, qT, sT, hqT, hsT = out
    M, I = dh.shape
    G, Up, d = f64(gu[:, :I]), f64(gu[:, I:]), f64(dh)
    dG, dU, h = R.gate_bwd(G, Up, d)
    sg, es = R.sigmoid(G), R.sigmoid_err(G)
    a = np.abs(G) * sg
    ea = np.abs(G) * es + 2 * U * a
    eG = np.abs(d * Up) * (es * (1 + a) + ea * (1 - sg) + 4 * U * (sg + a)) + 3 * U * np.abs(dG)
    eU = np.abs(d) * ea + 2 * U * np.abs(dU)
    eh = np.abs(Up) * ea + 2 * U * np.abs(h)
    ref, err = np.concatenate([dG, dU], 1), np.concatenate([eG, eU], 1)
    R.check_codes(to_np(q), rows_scales(s, M), ref, err, pow2, "gate gradient")
    R.check_codes(to_np(qT), rows_scales(sT, 2 * I), ref.T, err.T, pow2, "gate gradient, transposed")
    R.check_codes(to_np(hqT), rows_scales(hsT, I), h.T, eh.T, pow2, "activation, transposed")


@pytest.mark.parametrize("M,I", [(128, 128), (128, 384), (256, 256), (640, 128), (384, 2048), (1280, 2048)])
@pytest.mark.parametrize("pow2", [False, True])
def test_backward(M, I, pow2):
    gu, dh = _bwd_inputs(M, I, seed=M + I)
    out = fg.fp8_gated_bwd(gu, dh, pow2=pow2)
    assert fg.device_status() == 0
    _check_bwd(gu, dh, out, pow2)


def test_backward_more_tiles_than_sms():
    gu, dh = _bwd_inputs(2048, 2560, seed=1)       # 320 tiles
    _check_bwd(gu, dh, fg.fp8_gated_bwd(gu, dh))


def test_backward_saturated_gates_and_zeros():
    gu, dh = _bwd_inputs(256, 256, seed=2, scale=40.0)
    dh[5] = 0
    dh[:128, 7] = 0
    gu[3] = 0
    gu[:, 9] = 0
    _check_bwd(gu, dh, fg.fp8_gated_bwd(gu, dh))
    assert fg.device_status() == 0


def test_backward_strides():
    M, I = 256, 384
    gu, dh = _bwd_inputs(M, I, seed=4)
    want = fg.fp8_gated_bwd(gu, dh)
    gup = torch.zeros(M, 2 * I + 40, dtype=torch.bfloat16, device=DEV)
    gup[:, 8:8 + 2 * I] = gu
    dhp = torch.zeros(M, I + 16, dtype=torch.bfloat16, device=DEV)
    dhp[:, :I] = dh
    u8 = lambda r, c: torch.full((r, c), 0x11, dtype=torch.uint8, device=DEV)  # noqa: E731
    f = lambda r, c: torch.full((r, c), -1.0, device=DEV)  # noqa: E731
    q, qT, hq = u8(M, 2 * I + 32), u8(2 * I, M + 16), u8(I, M + 48)
    s, sT, hs = f(2 * I // 128, M + 4), f(M // 128, 2 * I + 8), f(M // 128, I + 12)
    got = fg.fp8_gated_bwd(gup[:, 8:8 + 2 * I], dhp[:, :I], q=q[:, :2 * I], scales=s, qT=qT[:, :M], scalesT=sT,
                           hqT=hq[:, :M], hscalesT=hs)
    assert fg.device_status() == 0
    for a, b in zip(want, got):
        assert torch.equal(a, b[:, :a.shape[1]])
    assert torch.all(q[:, 2 * I:] == 0x11) and torch.all(qT[:, M:] == 0x11) and torch.all(hq[:, M:] == 0x11)
    assert torch.all(s[:, M:] == -1) and torch.all(sT[:, 2 * I:] == -1) and torch.all(hs[:, I:] == -1)


def test_backward_no_rows():
    gu, dh = _bwd_inputs(128, 256, seed=5)
    out = fg.fp8_gated_bwd(gu[:0], dh[:0])
    assert out[0].shape == (0, 512) and out[4].shape == (256, 0)
    assert fg.device_status() == 0


def test_backward_reports_a_withheld_load():
    gu, dh = _bwd_inputs(256, 256, seed=6)
    fg.set_wait_limit_ns(50_000_000)
    try:
        fg.inject_skip_first_load()
        fg.fp8_gated_bwd(gu, dh)
        assert fg.device_status() == 5  # FP8FG_ETIMEOUT
    finally:
        fg.set_wait_limit_ns(2_000_000_000)
    out = fg.fp8_gated_bwd(gu, dh)
    assert fg.device_status() == 0
    _check_bwd(gu, dh, out)


def test_backward_against_differences():
    """Central differences of the 64-bit gate against the dequantised
    gradients: a code is off by at most half an E4M3 step, 1/16 of its value
    or 2^-10 of its scale."""
    M, I = 128, 256
    gu, dh = _bwd_inputs(M, I, seed=7)
    q, s, *_ = fg.fp8_gated_bwd(gu, dh)
    sv = np.repeat(rows_scales(s, M).astype(np.float64), 128, 1)
    got = R.DECODE[to_np(q)] * sv
    G, Up, d = f64(gu[:, :I]), f64(gu[:, I:]), f64(dh)
    t = 1e-5
    num = np.concatenate([d * (R.gate(G + t, Up) - R.gate(G - t, Up)) / (2 * t),
                          d * (R.gate(G, Up + t) - R.gate(G, Up - t)) / (2 * t)], 1)
    assert np.all(np.abs(got - num) <= (1 / 16 + 1e-4) * np.abs(num) + 2.0 ** -10 * sv + 1e-8)
