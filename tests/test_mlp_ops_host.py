"""Refusals of the operators between a gated MLP's GEMMs, without a GPU: the
C ABI's argument checks (they come before anything touches the device) and the
binding's checks of dtypes, layouts and extents. Also the 64-bit reference
forms themselves: their gradients against differences, and the code check
against codes made wrong on purpose."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_fine_grained_gb300 as fg
from fp8_fine_grained_gb300 import build as libbuild
from tests import mlp_ref as R

OK, EINVAL, EALIGN, EUNSUPPORTED = 0, 1, 2, 3
A, ODD = 0x10000, 0x10008          # never dereferenced
BF16, U8, F32 = torch.bfloat16, torch.uint8, torch.float32


@pytest.fixture(scope="module", autouse=True)
def L():
    libbuild.build()
    return fg.lib()


def _call(fn, names, base, **kw):
    unknown = set(kw) - set(names)
    assert not unknown, unknown
    a = dict(base, **kw)
    return fn(*[a[n] for n in names])


NORM = "x ldx r ldr gamma kind T D eps h ldh q ldq s ld_s rstd pow2 stream".split()
NORM_BASE = dict(x=A, ldx=256, r=A, ldr=256, gamma=A, kind=1, T=5, D=256, eps=1e-6, h=A, ldh=256, q=A, ldq=256, s=A,
                 ld_s=8, rstd=A, pow2=0, stream=None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(D=200), dict(D=18560), dict(eps=0.0), dict(eps=-1.0),
                                dict(eps=float("nan")), dict(eps=float("inf")), dict(pow2=2), dict(kind=7),
                                dict(ldx=248), dict(ldr=128), dict(ldh=128), dict(ldq=128), dict(ld_s=4),
                                dict(x=None), dict(gamma=None), dict(q=None), dict(s=None), dict(rstd=None),
                                dict(h=None), dict(T=1 << 31, ld_s=1 << 31)])
def test_norm_einval(L, kw):
    assert _call(L.fp8_rmsnorm, NORM, NORM_BASE, **kw) == EINVAL


@pytest.mark.parametrize("kw", [dict(x=ODD), dict(r=ODD), dict(gamma=ODD), dict(h=ODD), dict(q=ODD), dict(s=ODD),
                                dict(rstd=A + 2), dict(ldx=260), dict(ldr=257), dict(ldh=258), dict(ldq=264),
                                dict(ld_s=9)])
def test_norm_ealign(L, kw):
    assert _call(L.fp8_rmsnorm, NORM, NORM_BASE, **kw) == EALIGN


def test_norm_nothing_to_do(L):
    assert _call(L.fp8_rmsnorm, NORM, NORM_BASE, T=0, x=None, q=None) == OK
    assert _call(L.fp8_rmsnorm, NORM, NORM_BASE, D=0) == OK


NT = "h ldh rstd gamma kind T D q ldq s ld_s pow2 stream".split()
NT_BASE = dict(h=A, ldh=256, rstd=A, gamma=A, kind=0, T=128, D=256, q=A, ldq=128, s=A, ld_s=256, pow2=0, stream=None)


@pytest.mark.parametrize("kw,rc", [(dict(T=100), EINVAL), (dict(D=130), EINVAL), (dict(ldq=112), EINVAL),
                                   (dict(ld_s=128), EINVAL), (dict(ldh=128), EINVAL), (dict(kind=2), EINVAL),
                                   (dict(h=None), EINVAL), (dict(s=None), EINVAL), (dict(q=ODD), EALIGN),
                                   (dict(ldq=136), EALIGN), (dict(ld_s=258), EALIGN), (dict(T=0), OK)])
def test_norm_transposed_refusals(L, kw, rc):
    assert _call(L.fp8_rmsnorm_t, NT, NT_BASE, **kw) == rc


NB = "dy lddy h ldh rstd gamma kind dres lddres T D dx lddx dgamma ws bytes stream".split()
NB_BASE = dict(dy=A, lddy=256, h=A, ldh=256, rstd=A, gamma=A, kind=0, dres=A, lddres=256, T=4, D=256, dx=A, lddx=256,
               dgamma=A, ws=A, bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,rc", [(dict(T=-1), EINVAL), (dict(D=64), EINVAL), (dict(lddy=128), EINVAL),
                                   (dict(ldh=128), EINVAL), (dict(lddx=128), EINVAL), (dict(lddres=128), EINVAL),
                                   (dict(dgamma=None), EINVAL), (dict(ws=None), EINVAL), (dict(dy=None), EINVAL),
                                   (dict(kind=5), EINVAL), (dict(dy=ODD), EALIGN), (dict(dgamma=ODD), EALIGN),
                                   (dict(ws=ODD), EALIGN), (dict(lddy=260), EALIGN), (dict(lddres=260), EALIGN),
                                   (dict(D=0), OK)])
def test_norm_backward_refusals(L, kw, rc):
    assert _call(L.fp8_rmsnorm_bwd, NB, NB_BASE, **kw) == rc


GF = "xq sx ldx ld_sx wq sw ldw M I K h ldh s ld_s gu ldgu pow2 stream".split()
GF_BASE = dict(xq=A, sx=A, ldx=256, ld_sx=8, wq=A, sw=A, ldw=256, M=5, I=128, K=256, h=A, ldh=128, s=A, ld_s=8, gu=A,
               ldgu=256, pow2=0, stream=None)


@pytest.mark.parametrize("kw,rc", [(dict(M=-1), EINVAL), (dict(I=100), EINVAL), (dict(K=0), EINVAL), (dict(K=200), EINVAL),
                                   (dict(ldx=240), EINVAL), (dict(ldw=128), EINVAL), (dict(ld_sx=4), EINVAL),
                                   (dict(ldh=64), EINVAL), (dict(ld_s=4), EINVAL), (dict(ldgu=248), EINVAL),
                                   (dict(pow2=3), EINVAL), (dict(xq=None), EINVAL), (dict(sw=None), EINVAL),
                                   (dict(h=None), EINVAL), (dict(I=1 << 30, ldh=1 << 30), EINVAL), (dict(xq=ODD), EALIGN),
                                   (dict(wq=ODD), EALIGN), (dict(h=ODD), EALIGN), (dict(gu=ODD), EALIGN),
                                   (dict(ldx=264), EALIGN), (dict(ldgu=260), EALIGN), (dict(ld_sx=9), EALIGN),
                                   (dict(sw=A + 2), EALIGN), (dict(M=0), OK), (dict(I=0), OK)])
def test_gated_refusals(L, kw, rc):
    assert _call(L.fp8_gated_gemm, GF, GF_BASE, **kw) == rc


GB = "gu ldgu dh lddh M I q ldq s ld_s qT ldqT sT ld_sT hT ldhT hs ld_hs pow2 stream".split()
GB_BASE = dict(gu=A, ldgu=256, dh=A, lddh=128, M=128, I=128, q=A, ldq=256, s=A, ld_s=128, qT=A, ldqT=128, sT=A,
               ld_sT=256, hT=A, ldhT=128, hs=A, ld_hs=128, pow2=0, stream=None)


@pytest.mark.parametrize("kw,rc", [(dict(M=64), EINVAL), (dict(I=64), EINVAL), (dict(ldgu=128), EINVAL),
                                   (dict(lddh=64), EINVAL), (dict(ldq=128), EINVAL), (dict(ld_s=64), EINVAL),
                                   (dict(ldqT=64), EINVAL), (dict(ld_sT=128), EINVAL), (dict(ldhT=64), EINVAL),
                                   (dict(ld_hs=64), EINVAL), (dict(hT=None), EINVAL), (dict(gu=ODD), EALIGN),
                                   (dict(hs=ODD), EALIGN), (dict(ldgu=260), EALIGN), (dict(ldhT=136), EALIGN),
                                   (dict(pow2=-1), EINVAL), (dict(M=0), OK)])
def test_gated_backward_refusals(L, kw, rc):
    assert _call(L.fp8_gated_bwd, GB, GB_BASE, **kw) == rc


def _clip(L, rows, max_norm=1.0, eps=1e-6, norm=A, ws=A, nbytes=1 << 30, count=None):
    flat = [v for r in rows for v in r]
    table = (ctypes.c_int64 * max(1, len(flat)))(*flat)
    return L.fp8fg_grad_clip(table, len(rows) if count is None else count, max_norm, eps, norm, ws, nbytes, None)


def test_clip_refusals(L):
    ok = (A, A, 10, 0)
    for rows, rc in (([(A, A, 10, 2)], EINVAL), ([(A, A, -1, 0)], EINVAL), ([(0, A, 10, 0)], EINVAL),
                     ([ok, (A, 0, 10, 0)], EINVAL), ([(A + 2, A, 10, 0)], EALIGN), ([ok, (A, A + 1, 10, 1)], EALIGN)):
        assert _clip(L, rows) == rc
    for kw in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(eps=-1.0), dict(eps=float("nan")), dict(norm=None),
               dict(ws=None), dict(count=-1), dict(count=1 << 20)):
        assert _clip(L, [ok], **kw) == EINVAL
    assert _clip(L, [ok], norm=A + 1) == EALIGN and _clip(L, [ok], ws=A + 4) == EALIGN


# ------------------------------------------------------------- the binding ----

def z(shape, dtype):
    return torch.zeros(shape, dtype=dtype)


def expect(msg, fn, *a, **kw):
    with pytest.raises(ValueError, match=msg):
        fn(*a, **kw)


def test_binding_norm():
    x, w = z((4, 256), BF16), z((256,), BF16)
    expect("CUDA tensor", fg.fp8_rmsnorm, x, w)
    expect("x must be", fg.fp8_rmsnorm, x.float(), w)
    expect("row-major", fg.fp8_rmsnorm, z((256, 4), BF16).t(), w)
    expect("gamma", fg.fp8_rmsnorm, x, w[:128])
    expect("gamma", fg.fp8_rmsnorm, x, z((512,), BF16)[::2])
    expect("float32 or bfloat16", fg.fp8_rmsnorm, x, w.double())
    expect("residual", fg.fp8_rmsnorm, x, w, residual=x[:3])
    expect("residual", fg.fp8_rmsnorm, x, w, residual=x.float())
    expect("h must cover", fg.fp8_rmsnorm, x, w, residual=x, h=z((3, 256), BF16))
    expect("only with a residual", fg.fp8_rmsnorm, x, w, h=x)
    expect("q must cover", fg.fp8_rmsnorm, x, w, q=z((4, 128), U8))
    expect("scales must cover", fg.fp8_rmsnorm, x, w, scales=z((2, 3), F32))
    expect("rstd", fg.fp8_rmsnorm, x, w, rstd=z((3,), F32))
    expect("rstd", fg.fp8_rmsnorm, x, w, rstd=z((8,), F32)[::2])
    expect("x must be a tensor", fg.fp8_rmsnorm, [1.0], w)
    expect("rstd must be a tensor", fg.fp8_rmsnorm, x, w, rstd=3)
    expect("row-major", fg.fp8_rmsnorm, x.to_sparse(), w)
    expect("row-major", fg.fp8_rmsnorm, z((4, 2, 128), BF16), w)


def test_binding_norm_transposed_and_backward():
    h, w, r = z((128, 256), BF16), z((256,), F32), z((128,), F32)
    expect("CUDA tensor", fg.fp8_rmsnorm_t, h, r, w)
    expect("rstd", fg.fp8_rmsnorm_t, h, r[:100], w)
    expect("qT must cover", fg.fp8_rmsnorm_t, h, r, w, qT=z((256, 64), U8))
    expect("scalesT must cover", fg.fp8_rmsnorm_t, h, r, w, scalesT=z((1, 128), F32))
    expect("CUDA tensor", fg.fp8_rmsnorm_bwd, h, h, r, w)
    expect("dy must be", fg.fp8_rmsnorm_bwd, h.float(), h, r, w)
    expect("h must cover", fg.fp8_rmsnorm_bwd, h, h[:100], r, w)
    expect("rstd", fg.fp8_rmsnorm_bwd, h, h, r.double(), w)
    expect("dres must cover", fg.fp8_rmsnorm_bwd, h, h, r, w, dres=h[:, :128])
    expect("dx must be", fg.fp8_rmsnorm_bwd, h, h, r, w, dx=h.float())
    expect("dgamma", fg.fp8_rmsnorm_bwd, h, h, r, w, dgamma=z((255,), F32))


def test_binding_gated():
    M, K, I = 5, 256, 128
    xq, sx, wq, sw = z((M, K), U8), z((2, 8), F32), z((2 * I, K), U8), z((2, 2), F32)
    expect("CUDA tensor", fg.fp8_gated_gemm, xq, sx, wq, sw)
    expect("K = 256", fg.fp8_gated_gemm, xq, sx, wq[:, :128], sw)
    expect("up rows", fg.fp8_gated_gemm, xq, sx, z((129, K), U8), sw)
    expect("sw must be", fg.fp8_gated_gemm, xq, sx, wq, z((2, 4), F32)[:, :2])
    expect("sw must be", fg.fp8_gated_gemm, xq, sx, wq, z((3, 2), F32))
    expect("sx must cover", fg.fp8_gated_gemm, xq, sx[:, :4], wq, sw)
    expect("h must cover", fg.fp8_gated_gemm, xq, sx, wq, sw, h=z((M, 64), U8))
    expect("scales must cover", fg.fp8_gated_gemm, xq, sx, wq, sw, scales=z((1, 4), F32))
    expect("gu must cover", fg.fp8_gated_gemm, xq, sx, wq, sw, gu=z((M, I), BF16))
    expect("gu must be", fg.fp8_gated_gemm, xq, sx, wq, sw, gu=z((M, 2 * I), F32))
    gu, dh = z((128, 2 * I), BF16), z((128, I), BF16)
    expect("CUDA tensor", fg.fp8_gated_bwd, gu, dh)
    expect("gu must be", fg.fp8_gated_bwd, gu[:, :I], dh)
    expect("dh must be", fg.fp8_gated_bwd, gu, dh.float())
    expect("q must cover", fg.fp8_gated_bwd, gu, dh, q=z((128, I), U8))
    expect("qT must cover", fg.fp8_gated_bwd, gu, dh, qT=z((I, 128), U8))
    expect("hscalesT must cover", fg.fp8_gated_bwd, gu, dh, hscalesT=z((1, 64), F32))


def test_binding_clip():
    g = [z((4, 5), F32), z((7,), BF16)]
    expect("CUDA tensor", fg.grad_clip, g, 1.0)
    expect("at least one", fg.grad_clip, [], 1.0)
    expect("float32 or bfloat16", fg.grad_clip, [z((3,), torch.float16)], 1.0)
    expect("contiguous", fg.grad_clip, [z((4, 6), F32).t()], 1.0)
    expect("one tensor per", fg.grad_clip, g, 1.0, out=g[:1])
    expect("match", fg.grad_clip, g, 1.0, out=[g[0], z((8,), BF16)])
    expect("match", fg.grad_clip, g, 1.0, out=[g[0], z((7,), F32)])
    expect("contiguous", fg.grad_clip, g, 1.0, out=[g[0], z((14,), BF16)[::2]])


# ------------------------------------------------------ the reference forms ----

def test_reference_gradients_against_differences():
    rng = np.random.default_rng(1)
    h, w, dy = rng.standard_normal((3, 128)), 1 + rng.standard_normal(128), rng.standard_normal((3, 128))
    eps, t = 1e-3, 1e-6
    dx, dg, _, _ = R.norm_bwd(dy, h, R.rms(h, eps), w)
    for _ in range(4):
        v = rng.standard_normal(h.shape)
        num = (dy * (R.norm_y(h + t * v, w, eps) - R.norm_y(h - t * v, w, eps))).sum() / (2 * t)
        assert abs(num - (dx * v).sum()) < 1e-7 * np.abs(dx * v).sum()
        v = rng.standard_normal(w.shape)
        num = (dy * (R.norm_y(h, w + t * v, eps) - R.norm_y(h, w - t * v, eps))).sum() / (2 * t)
        assert abs(num - (dg * v).sum()) < 1e-7 * np.abs(dg * v).sum()
    g, u = 3 * rng.standard_normal(500), rng.standard_normal(500)
    dG, dU, a = R.gate_bwd(g, u, np.ones(500))
    assert np.allclose(dG, (R.gate(g + t, u) - R.gate(g - t, u)) / (2 * t), rtol=1e-6, atol=1e-8)
    assert np.allclose(dU, (R.gate(g, u + t) - R.gate(g, u - t)) / (2 * t), rtol=1e-6, atol=1e-8)
    assert np.allclose(a, R.gate(g, u))


def test_code_check_finds_wrong_codes_and_scales():
    rng = np.random.default_rng(2)
    ref = rng.standard_normal((4, 256))
    s = np.abs(ref).reshape(4, 2, 128).max(2) / 448
    v = ref / np.repeat(s, 128, 1)
    grid = np.sort(R.DECODE[np.isfinite(R.DECODE)])
    order = np.argsort(np.where(np.isfinite(R.DECODE), R.DECODE, 1e9), kind="stable")
    codes = order[np.abs(grid[:, None, None] - v).argmin(0)].astype(np.uint8)
    R.check_codes(codes, s, ref, 0.0)
    wrong = codes.copy()
    wrong[2, 100] ^= 1                                   # the neighbouring code
    with pytest.raises(AssertionError, match="nearest"):
        R.check_codes(wrong, s, ref, 0.0)
    off = s.copy()
    off[1, 1] *= 1.001
    with pytest.raises(AssertionError, match="scale"):
        R.check_codes(codes, off, ref, 0.0)


def test_checks_of_the_helper():
    from fp8_fine_grained_gb300 import _tensors as H
    m = z((6, 10), BF16)[:, 2:8]
    assert H.matrix(m, BF16, 6, 6, "m") == 10
    assert H.matrix(z((0, 5), U8), U8, 0, 5, "m") == 5
    assert H.vector(z((4,), F32), F32, 3, "v") is None
    assert H.on_gpu(None, "a", None, "b") is None
    assert H.norm_weight(z((5,), F32), 5) == fg.OUT_F32 and H.norm_weight(z((5,), BF16), 5) == fg.OUT_BF16
    expect("gamma must be a contiguous vector of 4", H.norm_weight, z((5,), F32), 4)
    expect("gamma must be a contiguous vector of 5", H.norm_weight, z((10,), F32)[::2], 5)
    expect("gamma must be a tensor", H.norm_weight, [1.0], 1)
    expect("m must cover", H.matrix, m, BF16, 7, 6, "m")
    expect("m must be torch.uint8", H.matrix, m, U8, 1, 1, "m")
    expect("v must be a contiguous vector of at least 5", H.vector, z((4,), F32), F32, 5, "v")
    expect("b must be a CUDA tensor", H.on_gpu, None, "a", m, "b")
    for args in ((), (m, BF16, 1, 1), (m, 3, 1, 1, "m"), (m, BF16, 1, 1, 7)):
        expect("bad call", H.matrix, *args)
    with pytest.raises(TypeError):
        H.matrix(m, BF16, 1.5, 1, "m")


def test_tensor_table():
    """The refusals of the helper that writes the clipping's table (the device
    is looked at last)."""
    from fp8_fine_grained_gb300 import _tensors
    flat = torch.arange(20, dtype=F32)
    with pytest.raises(ValueError, match="CUDA"):
        _tensors.describe([flat], [flat])
    for args in ((), ([],), ([flat], (flat,)), ([flat], [])):
        with pytest.raises(ValueError, match="two lists"):
            _tensors.describe(*args)
    with pytest.raises(ValueError, match="hold tensors"):
        _tensors.describe([flat, 3], [flat, flat])
    with pytest.raises(ValueError, match="contiguous"):
        _tensors.describe([flat.to_sparse()], [flat])
    with pytest.raises(ValueError, match="contiguous"):
        _tensors.describe([flat[::2]], [flat[:10]])
    assert _tensors.describe([], []) == b""


def test_library_calls_of_the_helper():
    """The helper's calls: a tensor is its data pointer, None is NULL, and the
    library's own refusals come back as its status codes."""
    H = fg._checks()
    x = torch.zeros(2, 128, dtype=BF16)
    with pytest.raises(ValueError, match="bad call of the library"):
        H.fp8_rmsnorm(x, 128)
    with pytest.raises(TypeError):
        H.fp8_rmsnorm_t(x, 128, x, x, "1", 2, 128, x, 2, x, 128, 0, 0)
    with pytest.raises(TypeError):
        H.fp8_rmsnorm_t(object(), 128, x, x, 1, 2, 128, x, 2, x, 128, 0, 0)
    ok, einval = 0, fg.lib().fp8_rmsnorm_t(0, 128, 0, 0, 1, 3, 128, 0, 128, 0, 128, 0, 0)    # 3 rows
    assert einval != ok
    assert H.fp8_rmsnorm_t(x, 128, x, x, 1, 3, 128, x, 128, x, 128, 0, 0) == einval
    assert H.fp8_rmsnorm_t(None, 128, None, None, 1, 128, 128, None, 128, None, 128, 0, 0) == einval   # NULL
    assert H.fp8_rmsnorm_t(None, 128, None, None, 1, 0, 128, None, 0, None, 128, 0, 0) == ok            # no rows


def test_allocation_of_the_helper():
    H = fg._checks()
    x = torch.zeros(3)
    a, b = H.empty(x, U8, 5), H.empty(x, BF16, 5, 6)
    assert a.shape == (5,) and a.dtype is U8 and b.shape == (5, 6) and b.dtype is BF16 and b.is_contiguous()
    assert H.empty(x, F32, 0, 4).shape == (0, 4)
    for args in ((x, U8), (x, 3, 1), (3, U8, 1), (x, U8, 1, 1, 1)):
        with pytest.raises(ValueError, match="bad call"):
            H.empty(*args)
    with pytest.raises(RuntimeError, match="negative"):
        H.empty(x, U8, -1)
