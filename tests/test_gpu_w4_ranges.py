"""4-bit products where x and the weight's scales stand at opposite ends of FP32's
range: the products are in it, the sums of x times the codes alone are not."""
import pytest
import torch

from tests.test_gpu_w4 import check, rows, want, weights

pytestmark = pytest.mark.gpu
fg = pytest.importorskip("fp8_fine_grained_gb300")
F32 = torch.float32


def tolerance(x, s, tol):
    """Beside the bound of the sums: of an entry of x that is 2^-31 of its block's largest or less, up to 2^-39 of
    the largest may be lost (half a step of FP16's 2^-24, the largest at 2^14 or more), times codes of at most 8 in
    128 columns; and 2^-125 a group."""
    most = x.double().abs().view(x.shape[0], -1, 128).amax(2)
    scale = s.double().view(s.shape[0], x.shape[1] // 128, -1).amax(2)
    return tol + 2.0 ** -39 * 8 * 128 * most @ scale.t() + 2.0 ** -125 * s.shape[1]


@pytest.mark.parametrize("kind,group", [("e2m1", 128), ("e2m1", 32), ("int4", 64)])
@pytest.mark.parametrize("px,ps", [(124, -30), (124, -60), (110, -100), (124, -126), (100, 0), (-100, 100), (-122, 120), (-122, 20),
                                   (0, -120), (0, 115)])
def test_opposite_ends(kind, group, px, ps):
    q, s = weights(21, kind, group, 40, 1024)
    s = (s * 2.0 ** ps).contiguous()
    x = rows(22, 6, 1024, 0.0)
    x = (x.double() * 2.0 ** px).to(torch.bfloat16)
    v, tol = want(x, q, s, kind, False)
    tol = tolerance(x, s, tol)
    assert float(v.abs().max()) < 2.0 ** 127 and torch.isfinite(x).all()
    for n in (1, 6):
        check(fg.w4_matvec(x[:n], q, s, kind=kind, out_dtype=F32), v[:n], tol[:n])


def test_both_ends_in_one_row():
    """Columns of large x under small scales beside columns of small x under large ones."""
    q, s = weights(23, "e2m1", 128, 40, 1024)
    x = rows(24, 5, 1024, 0.0).double()
    for b in range(8):
        p = 120 if b % 2 else -110
        x[:, 128 * b:128 * b + 128] *= 2.0 ** p
        s[:, b] *= 2.0 ** -p
    x = x.to(torch.bfloat16)
    v, tol = want(x, q, s.contiguous(), "e2m1", False)
    check(fg.w4_matvec(x, q, s.contiguous(), out_dtype=F32), v, tolerance(x, s, tol))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
def test_an_infinity_among_zeros(bad):
    """Its block has no finite entry to take a scale from."""
    q, s = weights(25, "e2m1", 128, 48, 512)
    s = s * 2.0 ** -40
    q |= 0x22                                # (no code is zero)
    x = torch.zeros(3, 512, device="cuda", dtype=torch.bfloat16)
    x[1, 200] = bad
    y = fg.w4_matvec(x, q, s, out_dtype=F32)
    assert (y[[0, 2]] == 0).all() and torch.isinf(y[1]).all()
    sign = torch.where((q[:, 100] & 8) > 0, -1.0, 1.0)   # (column 200: the low half of byte 100)
    assert torch.equal(torch.sign(y[1]), sign * (1.0 if bad > 0 else -1.0))
