"""GPU parity of grad_clip against 64-bit forms.

Error bounds (u = 2^-24): a thread adds 16 squares in sequence and three
levels of such sums in FP32, plus two single elements: at most 21 u on the sum
of squares, 10.5 u on the norm after the root, 1.5 u for the root; the
factor adds an addition and a quotient: 14 u; the product one more: 15 u, and
half a bf16 ulp for bf16 tensors."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_util import bf16_ulp

pytestmark = pytest.mark.gpu

fg = pytest.importorskip("fp8_fine_grained_gb300")
DEV = "cuda"
U = 2.0 ** -24
EPS = 1e-6


def f64(t):
    return t.double().cpu().numpy().reshape(-1)


def _grads(sizes, types, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return [(torch.randn(n, generator=g, device=DEV) * scale).to(t) for n, t in zip(sizes, types)]


def _check(grads, before, max_norm, norm, out, eps=EPS):
    ref = math.sqrt(sum(float((b * b).sum()) for b in before))
    got, coef = (float(v) for v in norm.cpu())
    assert abs(got - ref) <= 12 * U * ref
    c = min(1.0, max_norm / (ref + eps))
    assert abs(coef - c) <= 14 * U * c
    for g, b, o in zip(grads, before, out):
        want, have = b * c, f64(o)
        tol = 15 * U * np.abs(want)
        if g.dtype == torch.bfloat16:
            tol = tol + 0.5 * bf16_ulp(np.maximum(np.abs(want), np.abs(have)))
        assert np.all(np.abs(have - want) <= tol)


F, B = torch.float32, torch.bfloat16


@pytest.mark.parametrize("sizes", [[1], [3, 5], [7, 0, 130, 1], [8192], [8193, 4096], [100003, 17, 65536, 40000],
                                   [3000017]])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("in_place", [False, True])
def test_clip(sizes, kind, in_place):
    types = [{"f32": F, "bf16": B, "mixed": (F, B)[i % 2]}[kind] for i in range(len(sizes))]
    grads = _grads(sizes, types, seed=sum(sizes))
    before = [f64(g) for g in grads]
    out = None if in_place else [torch.full_like(g, 9.0) for g in grads]
    max_norm = 0.3 * math.sqrt(sum(sizes))
    norm, got = fg.grad_clip(grads, max_norm, EPS, out=out)
    assert fg.device_status() == 0
    _check(grads, before, max_norm, norm, got)
    if in_place:
        assert all(a.data_ptr() == b.data_ptr() for a, b in zip(grads, got))
    else:
        assert all(np.array_equal(f64(g), b) for g, b in zip(grads, before))


@pytest.mark.parametrize("dtype", [F, B])
def test_every_alignment_of_views_into_a_bucket(dtype):
    """Tensors one behind the other with no padding, inputs and outputs at
    offsets of their own: heads, tails and, where the two differ modulo 16
    bytes, the scalar path. The bytes between the outputs stay."""
    sizes = [1, 2, 3, 4, 5, 6, 7, 8, 9, 15, 31, 33, 257, 1027, 8200, 20001]
    flat = _grads([sum(sizes)], [dtype], seed=3)[0]
    grads = list(flat.split(sizes))
    before = [f64(g) for g in grads]
    buf = torch.full((sum(sizes) + 3 * len(sizes) + 5,), 4.0, dtype=dtype, device=DEV)
    out, at, gaps = [], 1, [0]
    for i, n in enumerate(sizes):
        out.append(buf[at:at + n])
        at += n
        gap = i % 4
        gaps += list(range(at, at + gap))
        at += gap
    norm, _ = fg.grad_clip(grads, 10.0, EPS, out=out)
    _check(grads, before, 10.0, norm, out)
    assert torch.all(buf[torch.tensor(gaps, device=DEV)] == 4.0) and torch.all(buf[at:] == 4.0)


def test_norm_below_the_limit_leaves_gradients_alone():
    grads = _grads([5000, 77], [F, B], seed=4)
    keep = [g.clone() for g in grads]
    norm, out = fg.grad_clip(grads, 1e6, EPS)
    assert float(norm[1]) == 1.0
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    other = [torch.empty_like(g) for g in grads]
    fg.grad_clip(grads, 1e6, EPS, out=other)
    assert all(torch.equal(a, b) for a, b in zip(other, keep))


def test_shapes_and_many_tensors():
    """More tensors than one launch takes, of several dimensions, some empty."""
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    shapes = [((i * 37) % 23, (i * 11) % 9 + 1) if i % 3 else ((i * 53) % 211,) for i in range(2500)]
    grads = [torch.randn(*s, generator=g, device=DEV).to((F, B)[i % 2]) for i, s in enumerate(shapes)]
    before = [f64(t) for t in grads]
    norm, out = fg.grad_clip(grads, 1.0, EPS)
    assert fg.device_status() == 0
    _check(grads, before, 1.0, norm, out)


def test_scales_of_the_values():
    """Tiny and large gradients in one list, and a max_norm of zero."""
    grads = _grads([4000], [F], seed=6, scale=1e-8) + _grads([4000], [F], seed=7, scale=1e12)
    before = [f64(g) for g in grads]
    norm, out = fg.grad_clip(grads, 1.0, EPS, out=[torch.empty_like(g) for g in grads])
    _check(grads, before, 1.0, norm, out)
    norm, out = fg.grad_clip(grads, 0.0, EPS)
    assert float(norm[1]) == 0.0 and all(torch.all(o == 0) for o in out)


def test_zeros_infinities_and_nan():
    z = [torch.zeros(1000, device=DEV)]
    norm, out = fg.grad_clip(z, 1.0, EPS)
    assert float(norm[0]) == 0.0 and float(norm[1]) == 1.0 and torch.all(out[0] == 0)
    g = _grads([1000, 500], [F, B], seed=8)
    g[0][17] = float("inf")
    norm, out = fg.grad_clip(g, 1.0, EPS)
    assert math.isinf(float(norm[0])) and float(norm[1]) == 0.0
    assert torch.isnan(out[0][17]) and torch.all(out[1] == 0) and int(torch.isnan(out[0]).sum()) == 1
    g = _grads([1000, 500], [F, B], seed=9)
    g[1][3] = float("nan")
    norm, out = fg.grad_clip(g, 1e9, EPS)
    assert all(torch.all(torch.isnan(o)) for o in out) and torch.isnan(norm).all()


def test_repeatable_and_on_another_stream():
    grads = _grads([1000003, 70001], [F, B], seed=10)
    want = fg.grad_clip(grads, 1.0, EPS, out=[torch.empty_like(g) for g in grads])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fg.grad_clip(grads, 1.0, EPS, out=[torch.empty_like(g) for g in grads], stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and all(torch.equal(a, b) for a, b in zip(want[1], got[1]))


def test_table_rows_of_views():
    """What the helper reads from views, several types and empty tensors."""
    import struct
    from fp8_fine_grained_gb300 import _tensors
    flat, out = _grads([100], [F], seed=1)[0], torch.empty(100, device=DEV)
    b = torch.zeros(3, 0, dtype=B, device=DEV)
    rows = struct.unpack("<" + "qqqii" * 3, _tensors.describe([flat[3:10], b, flat[10:].view(9, 10)],
                                                         [out[5:12], b, out[10:].view(90)]))
    assert rows[0:5] == (flat.data_ptr() + 12, out.data_ptr() + 20, 7, 0, 0)
    assert rows[7:10] == (0, 1, 0)
    assert rows[10:15] == (flat.data_ptr() + 40, out.data_ptr() + 40, 90, 0, 0)
