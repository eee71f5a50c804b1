"""Tensors of one row: torch gives the stride of a dimension of size one no
meaning and keeps whatever a transposition or a view left there, so a decoding
step's single token may come with any."""
import pytest
import torch

import fp8_fine_grained_gb300 as fg

BF16, U8, F32 = torch.bfloat16, torch.uint8, torch.float32


def odd(t):
    """The same row, contiguous, with a row stride of 1."""
    v = t.reshape(-1, 1).t()
    assert v.shape == t.shape and v.stride() == (1, 1) and v.is_contiguous()
    return v


def test_row_pitch():
    H = fg._checks()
    for dtype in (BF16, U8, F32):
        assert H.matrix(odd(torch.zeros(1, 256, dtype=dtype)), dtype, 1, 256, "m") == 256
    assert H.matrix(odd(torch.zeros(1, 250)), F32, 1, 250, "m") == 256
    assert H.matrix(torch.zeros(3, 300)[1:2, :257], F32, 1, 257, "m") == 272
    assert H.matrix(torch.zeros(3, 300)[:, :257], F32, 1, 257, "m") == 300
    with pytest.raises(ValueError, match="m must cover"):
        H.matrix(odd(torch.zeros(1, 256)), F32, 2, 256, "m")


@pytest.mark.gpu
def test_one_token():
    D, I = 512, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    x, res, w, dy = r(1, D), r(1, D), r(D), r(1, D)
    want = fg.fp8_rmsnorm(x, w, residual=res)
    got = fg.fp8_rmsnorm(odd(x), w, residual=odd(res), h=odd(torch.empty_like(x)), q=odd(torch.empty_like(want[0])))
    assert torch.equal(want[0], got[0]) and torch.equal(want[1][:, :1], got[1][:, :1])
    assert torch.equal(want[2], got[2]) and torch.equal(want[3], got[3])
    wantb = fg.fp8_rmsnorm_bwd(dy, want[2], want[3], w, dres=res)
    gotb = fg.fp8_rmsnorm_bwd(odd(dy), odd(want[2]), want[3], w, dres=odd(res), dx=odd(torch.empty_like(dy)))
    assert all(torch.equal(a, b) for a, b in zip(wantb, gotb))
    wq, sw = fg.fp8_quant_128x128(r(2 * I, D))
    wantg = fg.fp8_gated_gemm(want[0], want[1], wq, sw, save=True)
    gotg = fg.fp8_gated_gemm(odd(want[0]), want[1], wq, sw, h=odd(torch.empty_like(wantg[0])),
                             gu=odd(torch.empty_like(wantg[2])))
    assert torch.equal(wantg[0], gotg[0]) and torch.equal(wantg[1][:, :1], gotg[1][:, :1])
    assert torch.equal(wantg[2], gotg[2])
    assert fg.device_status() == 0


@pytest.mark.gpu
def test_one_group_of_rows_or_columns():
    """Scales of one group: rows of their own pitch, one of them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn(128, 128, generator=g, device="cuda").to(BF16)
    w = torch.ones(128, device="cuda")
    q, s, h, rstd = fg.fp8_rmsnorm(x, w)
    qo, so, _, _ = fg.fp8_rmsnorm(x, w, scales=odd(torch.empty_like(s)))
    t, to = fg.fp8_rmsnorm_t(h, rstd, w), fg.fp8_rmsnorm_t(h, rstd, w, scalesT=odd(torch.empty(1, 128, device="cuda")))
    assert torch.equal(q, qo) and torch.equal(s, so)
    assert all(torch.equal(a, b) for a, b in zip(t, to))
    assert fg.device_status() == 0
