"""GPU parity of the RMS norm with residual and E4M3 output (fp8_rmsnorm), of
its transposed form and of its backward pass, against 64-bit forms.

Error bounds (FP32 arithmetic, u = 2^-24). rstd: a thread adds at most 24
squares in sequence and two shuffle trees of 5 follow, 34 u relative on the sum
of squares, 17 u after the root, plus 4 u for the division, the addition and
rsqrtf: at most 24 u. y = h * rstd * gamma adds two products: 26 u |y|.
dx: the row's dot product carries 36 u of its absolute terms, the remaining
steps 8 u: 50 u of the bound tx, then half a bf16 ulp. dgamma: a CTA adds
ceil(T / grid) rows, the CTAs' sums are added at most 97 deep (T / 152 + 97) u
of the absolute terms."""
import numpy as np
import pytest
import torch

from tests import mlp_ref as R
from tests.gpu_util import bf16_ulp, rows_scales, to_np

pytestmark = pytest.mark.gpu

fg = pytest.importorskip("fp8_fine_grained_gb300")
DEV = "cuda"
U = R.U24
EPS = 1e-6


def f64(t):
    return t.double().cpu().numpy()


def _inputs(T, D, seed, gamma="bf16"):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    chan = torch.exp(torch.randn(D, generator=g, device=DEV))
    x = (torch.randn(T, D, generator=g, device=DEV) * chan).to(torch.bfloat16)
    r = (torch.randn(T, D, generator=g, device=DEV) * chan).to(torch.bfloat16)
    w = 1 + 0.3 * torch.randn(D, generator=g, device=DEV)
    return x, r, w.to(torch.bfloat16) if gamma == "bf16" else w


def _check_fwd(x, r, w, out, eps=EPS, pow2=False):
    q, s, h, rstd = out
    T, D = x.shape
    href = x if r is None else (x.float() + r.float()).to(torch.bfloat16)
    assert torch.equal(h.contiguous().view(torch.int16), href.contiguous().view(torch.int16))
    hd = f64(href)
    ref = R.rms(hd, eps)
    assert np.all(np.abs(f64(rstd)[:T] - ref) <= 24 * U * ref)
    y = hd * ref[:, None] * f64(w)
    R.check_codes(to_np(q), rows_scales(s, T), y, 26 * U * np.abs(y), pow2, "norm")


@pytest.mark.parametrize("T,D", [(1, 128), (1, 7168), (3, 256), (37, 384), (130, 2048), (129, 2176), (300, 7168),
                                 (1000, 128), (7, 8192), (5, 8320), (2, 18432), (700, 8064)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("gamma", ["bf16", "f32"])
def test_forward(T, D, residual, gamma):
    x, r, w = _inputs(T, D, seed=T + D, gamma=gamma)
    r = r if residual else None
    _check_fwd(x, r, w, fg.fp8_rmsnorm(x, w, EPS, residual=r))
    assert fg.device_status() == 0


@pytest.mark.parametrize("T,D", [(5, 512), (260, 7168)])
def test_forward_pow2(T, D):
    x, r, w = _inputs(T, D, seed=9)
    _check_fwd(x, r, w, fg.fp8_rmsnorm(x, w, EPS, residual=r, pow2=True), pow2=True)


def test_more_rows_than_the_grid_holds():
    """Every CTA strides over several rows (and alternates its scratch)."""
    x, r, w = _inputs(9001, 256, seed=4)
    _check_fwd(x, r, w, fg.fp8_rmsnorm(x, w, EPS, residual=r))


def test_strided_rows_and_untouched_padding():
    T, D = 33, 640
    x, r, w = _inputs(T, 1024, seed=2)
    xs, rs, ws = x[:, 128:128 + D], r[:, 256:256 + D], w[:D].contiguous()
    h = torch.full((T, D + 64), 7.0, dtype=torch.bfloat16, device=DEV)
    q = torch.full((T, D + 32), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((D // 128, T + 11), -3.0, device=DEV)
    rstd = torch.full((T + 5,), -1.0, device=DEV)
    out = fg.fp8_rmsnorm(xs, ws, EPS, residual=rs, h=h[:, :D], q=q[:, :D], scales=s, rstd=rstd)
    assert torch.all(h[:, D:] == 7.0) and torch.all(q[:, D:] == 0x55)
    assert torch.all(s[:, T:] == -3.0) and torch.all(rstd[T:] == -1.0)
    _check_fwd(xs, rs, ws, (out[0], out[1], out[2], out[3]))


def test_residual_stream_in_place():
    x, r, w = _inputs(65, 7168, seed=5)
    x0 = x.clone()
    ref = fg.fp8_rmsnorm(x, w, EPS, residual=r)
    out = fg.fp8_rmsnorm(x, w, EPS, residual=r, h=x)
    assert out[2].data_ptr() == x.data_ptr()
    T = x.shape[0]
    for i, (a, b) in enumerate(zip(ref, out)):
        assert torch.equal(a[:, :T] if i == 1 else a, b[:, :T] if i == 1 else b)
    _check_fwd(x0, r, w, out)


def test_rows_of_zeros_and_tiny_and_large_values():
    """A zero row: rstd = eps^-1/2 and all codes zero with scale 1."""
    x, r, w = _inputs(6, 512, seed=6)
    x[0] = 0
    x[1] *= 2.0 ** -60
    x[2] *= 2.0 ** 40
    x[3, :128] = 0
    x[4] = -x[4].abs()
    out = fg.fp8_rmsnorm(x, w, EPS)
    _check_fwd(x, None, w, out)
    assert torch.all(out[1][:, 0] == 1.0) and torch.all(out[0][0] & 0x7F == 0)


def test_eps_enters():
    x, r, w = _inputs(4, 256, seed=7)
    x *= 1e-3
    for eps in (1e-8, 1e-5, 0.5):
        _check_fwd(x, None, w, fg.fp8_rmsnorm(x, w, eps), eps=eps)


def test_no_rows():
    x, r, w = _inputs(4, 256, seed=8)
    q, s, h, rstd = fg.fp8_rmsnorm(x[:0], w, EPS, residual=r[:0])
    assert q.shape == (0, 256) and h.shape == (0, 256) and rstd.numel() == 0
    assert fg.device_status() == 0


@pytest.mark.parametrize("T,D", [(128, 128), (256, 2176), (384, 7168)])
@pytest.mark.parametrize("pow2", [False, True])
def test_transposed(T, D, pow2):
    x, r, w = _inputs(T, D, seed=T, gamma="f32" if pow2 else "bf16")
    q, s, h, rstd = fg.fp8_rmsnorm(x, w, EPS, residual=r)
    qT, sT = fg.fp8_rmsnorm_t(h, rstd, w, pow2=pow2)
    assert fg.device_status() == 0
    y = R.norm_y(f64(h), f64(w), EPS).T
    R.check_codes(to_np(qT), rows_scales(sT, D), y, 26 * U * np.abs(y), pow2, "transposed norm")


def _check_bwd(dy, h, rstd, w, dres, dx, dgamma):
    T, D = dy.shape
    ref, dg, tx, tg = R.norm_bwd(f64(dy), f64(h), f64(rstd)[:T], f64(w))
    if dres is not None:
        ref, tx = ref + f64(dres), tx + np.abs(f64(dres))
    got = f64(dx)
    tol = 50 * U * tx + 0.5 * bf16_ulp(np.maximum(np.abs(got), np.abs(ref)))
    assert np.all(np.abs(got - ref) <= tol)
    assert np.all(np.abs(f64(dgamma) - dg) <= (T / 152 + 97) * U * tg)


@pytest.mark.parametrize("T,D", [(1, 128), (1, 7168), (3, 256), (37, 384), (129, 2176), (300, 7168), (5, 8320),
                                 (2, 18432), (2000, 256), (700, 8192)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("gamma", ["bf16", "f32"])
def test_backward(T, D, residual, gamma):
    x, r, w = _inputs(T, D, seed=2 * T + D, gamma=gamma)
    q, s, h, rstd = fg.fp8_rmsnorm(x, w, EPS)
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    dy = (torch.randn(T, D, generator=g, device=DEV) * 1e-3).to(torch.bfloat16)
    dres = (torch.randn(T, D, generator=g, device=DEV) * 1e-3).to(torch.bfloat16) if residual else None
    dx, dgamma = fg.fp8_rmsnorm_bwd(dy, h, rstd, w, dres=dres)
    assert fg.device_status() == 0
    _check_bwd(dy, h, rstd, w, dres, dx, dgamma)
    again = fg.fp8_rmsnorm_bwd(dy, h, rstd, w, dres=dres)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dgamma)   # a fixed order of summation


@pytest.mark.parametrize("T", [2500, 4900, 7300])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("gamma", ["bf16", "f32"])
def test_backward_grids(T, residual, gamma):
    """Lengths where the variants take different numbers of CTAs: the
    workspace of (T, D) has to cover the largest."""
    x, r, w = _inputs(T, 1024, seed=T, gamma=gamma)
    dres = r if residual else None
    rstd = torch.rand(T, device=DEV) + 0.5
    dx, dgamma = fg.fp8_rmsnorm_bwd(r, x, rstd, w, dres=dres)
    assert fg.device_status() == 0
    _check_bwd(r, x, rstd, w, dres, dx, dgamma)


def test_backward_strided_and_in_place():
    T, D = 21, 640
    x, r, w = _inputs(T, 1024, seed=12)
    ws = w[:D].contiguous()
    hs = x[:, 128:128 + D]
    q, s, h, rstd = fg.fp8_rmsnorm(hs, ws, EPS)
    dy, dres = r[:, :D], r[:, 384:384 + D]
    dx, dgamma = fg.fp8_rmsnorm_bwd(dy, hs, rstd, ws, dres=dres)
    _check_bwd(dy, hs, rstd, ws, dres, dx, dgamma)
    buf = dres.clone()
    dx2, dgamma2 = fg.fp8_rmsnorm_bwd(dy, hs, rstd, ws, dres=buf, dx=buf)
    assert torch.equal(dx2, dx) and torch.equal(dgamma2, dgamma)


def test_backward_no_rows_gives_a_zero_dgamma():
    x, r, w = _inputs(4, 256, seed=8)
    dgamma = torch.full((256,), 5.0, device=DEV)
    fg.fp8_rmsnorm_bwd(x[:0], r[:0], torch.empty(0, device=DEV), w, dgamma=dgamma)
    assert fg.device_status() == 0
    assert torch.all(dgamma == 0)


def test_backward_against_differences():
    """The directional derivative of sum(dy * y) along v, by central
    differences of the 64-bit norm, is <dx, v>; dx carries a bf16 rounding of
    at most 2^-9 of each element and 50 u of its terms."""
    T, D = 6, 384
    x, r, w = _inputs(T, D, seed=20, gamma="f32")
    q, s, h, rstd = fg.fp8_rmsnorm(x, w, EPS)
    dy = r
    dx, dgamma = fg.fp8_rmsnorm_bwd(dy, h, rstd, w)
    hd, wd, dyd = f64(h), f64(w), f64(dy)
    rng = np.random.default_rng(0)
    _, _, tx, tg = R.norm_bwd(dyd, hd, f64(rstd), wd)
    for _ in range(5):
        v, t = rng.standard_normal((T, D)), 1e-4
        num = (dyd * (R.norm_y(hd + t * v, wd, EPS) - R.norm_y(hd - t * v, wd, EPS))).sum() / (2 * t)
        tol = (np.abs(v) * (2.0 ** -9 * np.abs(f64(dx)) + 50 * U * tx)).sum() + 1e-6 * np.abs(tx * v).sum()
        assert abs((f64(dx) * v).sum() - num) <= tol
        v = rng.standard_normal(D)
        num = (dyd * (R.norm_y(hd, wd + t * v, EPS) - R.norm_y(hd, wd - t * v, EPS))).sum() / (2 * t)
        assert abs((f64(dgamma) * v).sum() - num) <= (1e-6 * tg * np.abs(v)).sum() + 1e-5 * np.abs(tg * v).max()


def test_on_another_stream():
    """Launched on a side stream that first waits for its inputs; the
    backward's workspace may be reused by the current stream at once."""
    x, r, w = _inputs(2000, 2048, seed=30)
    want = fg.fp8_rmsnorm(x, w, EPS, residual=r)
    wantb = fg.fp8_rmsnorm_bwd(x, want[2], want[3], w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fg.fp8_rmsnorm(x, w, EPS, residual=r, stream=side)
    gotb = fg.fp8_rmsnorm_bwd(x, got[2], got[3], w, stream=side)
    junk = [torch.full((1 << 22,), float("nan"), device=DEV) for _ in range(8)]
    side.synchronize()
    for a, b in zip(want + wantb, got + gotb):
        assert torch.equal(a[:, :2000] if a.dim() == 2 and a.shape[0] == 16 else a,
                           b[:, :2000] if b.dim() == 2 and b.shape[0] == 16 else b)
    assert len(junk) == 8


def test_consecutive_calls_on_one_stream_see_each_other():
    """Each call's grid may start under the previous one's tail: a chain that
    feeds h forward must equal the same chain with waits in between."""
    x, r, w = _inputs(512, 7168, seed=31)
    a = b = x
    for _ in range(6):
        a = fg.fp8_rmsnorm(a, w, EPS, residual=r)[2]
    for _ in range(6):
        b = fg.fp8_rmsnorm(b, w, EPS, residual=r)[2]
        torch.cuda.synchronize()
    assert torch.equal(a, b)
