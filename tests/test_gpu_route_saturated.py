"""The router's order where scores are rounded to 0 or 1: against decimal arithmetic
that neither saturates nor underflows. Without a bias the order is that of the scores
as real numbers."""
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

from tests.test_gpu_route import rnd

pytestmark = pytest.mark.gpu
fg = pytest.importorskip("fp8_fine_grained_gb300")
NINF, INF = float("-inf"), float("inf")


def scores(row, score):
    """Scores of finite or masked logits, in decimal (a score that is masked: None)."""
    l = [None if v == NINF or v != v else Decimal(float(v)) for v in row]
    if score == "sigmoid":
        return [None if v is None else 1 / (1 + (-v).exp()) for v in l]
    top = max(v for v in l if v is not None)     # (the row's sum divides all of them)
    return [None if v is None else (v - top).exp() for v in l]


def choice(row, k, score, groups, top_groups, group_top):
    with localcontext() as c:
        # (1 - exp(-l) has l / ln 10 nines; scores near 0 need no more digits)
        c.prec, c.Emin, c.Emax = 40 + int(max(0.0, *(v for v in row if v < INF)) / 2.3), -10 ** 17, 10 ** 17
        s = scores(row, score)
        n = len(row) // groups
        best = [sorted((v for v in s[g * n:(g + 1) * n] if v is not None), reverse=True)[:group_top] for g in range(groups)]
        value = [sum(b) if b else Decimal(-1) for b in best]
        c.prec -= 15                             # (equal sums come out equal: their rounding is far below this)
        value = [+v for v in value]
        kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
        order = sorted((e for e in range(len(row)) if e // n in kept and s[e] is not None), key=lambda e: (-s[e], e))[:k]
        return order + [-1] * (k - len(order))


def check(logits, k, **kw):
    ids, gates = fg.moe_route(logits, k, **kw)
    want = [choice(r, k, kw["score"], kw["groups"], kw["top_groups"], kw["group_top"]) for r in logits.double().cpu().numpy()]
    assert np.array_equal(ids.cpu().numpy(), np.array(want))
    assert torch.isfinite(gates).all() and fg.device_status() == 0
    return ids


KINDS = [dict(score=s, groups=g, top_groups=t, group_top=p)
         for s in ("sigmoid", "softmax") for g, t in ((1, 1), (4, 1), (4, 3)) for p in (1, 2)]


@pytest.mark.parametrize("kw", KINDS)
@pytest.mark.parametrize("shift,spread", [(40.0, 1.0), (36.0, 3.0), (70.0, 20.0), (15.0, 0.5), (500.0, 30.0), (692.0, 6.0)])
def test_close_to_one(kw, shift, spread):
    check(shift + spread * rnd(41, 20, 16), 3, **kw)
    check((shift + spread * rnd(42, 20, 16)).to(torch.bfloat16), 3, **kw)


@pytest.mark.parametrize("kw", KINDS)
@pytest.mark.parametrize("shift,spread", [(-100.0, 5.0), (-300.0, 100.0), (-1000.0, 60.0), (-692.0, 6.0)])
def test_close_to_zero(kw, shift, spread):
    check(shift + spread * rnd(43, 12, 16), 3, **kw)


@pytest.mark.parametrize("kw", KINDS)
def test_one_far_above_the_others(kw):
    """The others' softmax underflows; a sigmoid of 1 stands beside smaller ones in every group."""
    logits = rnd(44, 12, 16)
    logits[:, 5] = 900.0
    check(logits, 3, **kw)
    logits[:, 1::4] = 60.0                  # the same best in every group: the second decides
    logits[::2, 2::4] -= 40.0
    check(logits, 3, **kw)


@pytest.mark.parametrize("kw", KINDS)
def test_equal_sums_and_masks(kw):
    """x and -x have the same sum of sigmoids for every x; groups without experts, and of one."""
    logits = torch.full((3, 16), -50.0, device="cuda")
    for g, x in enumerate((0.5, 3.0, 0.0, 20.0)):
        logits[0, 4 * g], logits[0, 4 * g + 2] = x, -x
    logits[1:, ::4] = 45.0
    logits[1, 8:12] = NINF
    logits[2, 5:8] = NINF
    logits[2, 9] = 46.0
    check(logits, 3, **kw)


def test_no_groups_and_groups_that_are_all_kept():
    """The same order either way."""
    logits = 45 + 5 * rnd(45, 50, 64)
    want, _ = fg.moe_route(logits, 8, score="sigmoid")
    for groups in (2, 4, 16):
        got, _ = fg.moe_route(logits, 8, score="sigmoid", groups=groups, top_groups=groups)
        assert torch.equal(got, want)


@pytest.mark.parametrize("group_top", [1, 2])
def test_with_a_bias_the_scores_are_those_of_64_bits(group_top):
    """As the header says: above 37 a sigmoid is 1 there."""
    logits = torch.tensor([[38.0, 60.0, 39.0, 45.0, 1.0, 50.0, 40.0, 41.0]], device="cuda")
    ids, _ = fg.moe_route(logits, 4, bias=torch.zeros(8, device="cuda"))
    assert ids.tolist() == [[0, 1, 2, 3]]
    ids, _ = fg.moe_route(logits, 4, bias=torch.zeros(8, device="cuda"), groups=2, top_groups=1, group_top=group_top)
    assert ids.tolist() == [[0, 1, 2, 3]]
