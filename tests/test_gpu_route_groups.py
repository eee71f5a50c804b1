"""The router's comparison of groups where a group's two best choices are far larger
than their sum: their rounding is that of the choices."""
import pytest
import torch

from tests.test_gpu_route import check_route, rnd

pytestmark = pytest.mark.gpu


def test_two_choices_of_opposite_signs():
    """1.0200885 and 1.0200887 in 64 bits, 1.0200920 and 1.0200888 where each choice is rounded to FP32."""
    logits = torch.tensor([[1.0056078, -0.9054694, 0.6697878, -0.5813015]], device="cuda")
    bias = torch.tensor([64.0, -64.0, 0.0, 0.0], device="cuda")
    ids, _ = check_route(logits, bias, 2, groups=2, top_groups=1)
    assert ids.tolist() == [[2, 3]]


@pytest.mark.parametrize("size", [8.0, 64.0, 1e3, 1e4])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_large_biases_of_both_signs(size, score, group_top):
    """Groups of two whose biases cancel; then groups of eight of which two members' do."""
    logits = 1.5 * rnd(int(size), 600, 8)
    bias = size * torch.tensor([1.0, -1.0, 0.0, 0.0, -0.5, 0.5, 1.0, -1.0], device="cuda")
    for top_groups in (1, 2, 3):
        check_route(logits, bias, 2, score=score, groups=4, top_groups=top_groups, group_top=group_top)
    logits = 1.5 * rnd(int(size) + 1, 200, 64)
    bias = torch.full((8, 8), -2 * size, device="cuda")
    bias[:, 3], bias[:, 5] = size, -size
    check_route(logits, bias.view(-1), 4, score=score, groups=8, top_groups=4, group_top=group_top)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_lowest_and_largest_biases(score, group_top):
    """A group of experts with the lowest finite bias is worth more than one with none left, whatever its index;
    sums of two such biases are compared, not lost."""
    kw = dict(score=score, groups=4, group_top=group_top)
    lowest = torch.finfo(torch.float32).min
    logits = rnd(31, 5, 8)
    masked = logits.clone()
    masked[:, [0, 1, 4, 5, 6, 7]] = float("-inf")
    for top_groups in (1, 2, 3):
        ids, _ = check_route(masked, torch.full((8,), lowest, device="cuda"), 2, top_groups=top_groups, **kw)
        assert (ids >= 2).all() and (ids < 4).all()
        for bias in ([lowest] * 8, [-lowest] * 8, [lowest, lowest, lowest, 0, 0, 0, 1, 1],
                     [lowest, -lowest, 0, 0, -lowest, lowest, -lowest, -lowest], [lowest / 2] * 4 + [lowest] * 4):
            bias = torch.tensor(bias, device="cuda")
            check_route(logits, bias, 2, top_groups=top_groups, **kw)
            check_route(masked, bias, 2, top_groups=top_groups, **kw)
    bias = torch.full((64,), lowest, device="cuda")
    bias[5::9] = 0.25
    for top_groups in (2, 5):
        check_route(rnd(32, 40, 64), bias, 6, score=score, groups=8, top_groups=top_groups, group_top=group_top)
