"""The router over scores at the ends of the numbers and where sums cancel: the choice is the 64-bit one all the same."""
import pytest
import torch

import test_gpu_ops_scores as scores
from combine_persistent_warp_gb300 import ops

pytestmark = pytest.mark.gpu
LOWEST = {torch.float32: torch.finfo(torch.float32).min, torch.bfloat16: torch.finfo(torch.bfloat16).min, torch.float16: torch.finfo(torch.float16).min}


def _agree(l, k, score, bias, groups, kept, mask=None):
    idx, _ = ops.route_scores(l, k, score=score, bias=bias, groups=groups, topk_groups=kept, token_mask=mask)
    want = scores._choice(l, k, score, bias, groups, kept, 2)
    if mask is not None:
        want = torch.where(mask[:, None], want, -1)
    assert torch.equal(idx, want)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [40, 5000, 9000])
def test_logits_of_the_lowest_value_have_a_score_of_zero(T, dtype, score):
    """Experts masked with their type's lowest value, or others near it: a score of 0, not one far below."""
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")
    l = (1.5 * torch.randn(T, 64, generator=g, device="cuda")).to(dtype)
    l[rand(T, 64) < 0.5] = LOWEST[dtype]
    l[rand(T, 64) < 0.2] = 0.9 * LOWEST[dtype]
    l[7] = LOWEST[dtype]
    l[8, 8:] = LOWEST[dtype]
    l[9] = -LOWEST[dtype]
    l[10, 5:] = -float("inf")
    for b in (None, torch.zeros(64, device="cuda"), scores._bias(64), 10 * scores._bias(64)):
        for groups, kept in ((1, 1), (8, 3), (16, 5)):
            if b is None and groups == 1:   # (the logits themselves decide)
                continue
            _agree(l, 8, score, b, groups, kept)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [40, 9000])
def test_huge_biases_beside_huge_logits(T, score):
    g = torch.Generator(device="cuda").manual_seed(T)
    pick = lambda values, *s: torch.tensor(values, device="cuda")[torch.randint(0, len(values), s, generator=g, device="cuda")]
    l = pick([0.0, 1e38, -1e38, 3e38, -3e38, 1.0, -1.0], T, 64)
    for values in ([3.3e38, 2.5e38, 1e38], [3.3e38, -3.3e38, 0.1], [-3e38, -1e38, 1.0, 3.4e38], [float("inf"), 1e38, -float("inf"), 0.2]):
        b = pick(values, 64)
        for groups, kept in ((1, 1), (8, 3)):
            _agree(l, 4, score, b, groups, kept)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [300, 5000, 20000])
def test_sums_past_the_largest_number(T, score):
    g = torch.Generator(device="cuda").manual_seed(T)
    l = 1.5 * torch.randn(T, 64, generator=g, device="cuda")
    for at in ({8: -3.4e38, 9: -3.4e38}, {8: 3.4e38, 9: 3.3e38, 10: -3.4e38}, {8: -3.4e38, 9: -3.4e38, 10: -3.3e38, 11: 3.4e38, 12: 3.3e38, 13: 3.2e38}):
        b = scores._bias(64)
        for e, v in at.items():
            b[e] = v
        for groups, kept in ((8, 3), (32, 9)):
            _agree(l, 4, score, b, groups, kept)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("B", [0.9, 1.0, 4.0, 16.0, 32.0, 100.0, 1e4, 1e9])
@pytest.mark.parametrize("T,groups,per,k", [(300, 8, 2, 4), (5000, 16, 2, 6), (20000, 8, 2, 8), (20000, 4, 3, 3), (9000, 8, 16, 8), (500, 32, 2, 8),
                                            (700, 32, 32, 4)])
def test_biases_that_cancel_in_a_group(T, groups, per, k, B, score):
    """32 bits hold c = score + bias to half a step of its size, which stays when a group's sum cancels: with B and -B the sums
    are near 1 and each c is up to B 2^-24 off.  One expert of each group is favoured by B and the others are held back by as much: the sums of a group's two best are
    close together, in another order than the first or the second of them.  (No two are equal: 64-bit sums of equal parts in
    another order need not be.)"""
    g = torch.Generator(device="cuda").manual_seed(T + groups)
    E = groups * per
    rows = torch.arange(groups, device="cuda")
    best = torch.randint(0, per, (groups,), generator=g, device="cuda")
    bias = torch.full((groups, per), -B, device="cuda")
    bias[rows, best] = B
    mask = torch.rand(T, generator=g, device="cuda") > 0.1
    rank = torch.rand(T, groups, generator=g, device="cuda").argsort(1)
    for dtype, at, step, far, apart in ((torch.float32, 0.0, 2.0 ** -22, 128, 4), (torch.float32, 0.3, 2.0 ** -20, 128, 4),
                                        (torch.bfloat16, 2.0, 2.0 ** -6, 8, 1)):
        x = torch.randint(-far, far + 1, (T, groups), generator=g, device="cuda")
        n = (apart * rank - x)[:, :, None].repeat(1, 1, per)
        n[:, rows, best] = x
        l = (at + n * step).view(T, E).to(dtype)
        _agree(l, k, score, bias.view(-1), groups, groups // 2)
        _agree(l, k, score, bias.view(-1), groups, 1 if k <= per else groups - 1, mask)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [300, 5000, 20000])
def test_a_group_held_back_by_much_leaves_the_others_as_they_are(T, score):
    """Biases of very different size side by side, the largest in groups that stay or do not."""
    g = torch.Generator(device="cuda").manual_seed(T)
    l = 1.5 * torch.randn(T, 64, generator=g, device="cuda")
    plain = scores._bias(64)
    for at in ({3: -1e9, 4: 1e9}, {8: -1e9, 9: -1e9}, {8: 1e9, 9: -1e9, 16: 1e9, 17: -1e9}, {0: 1e30, 1: -1e30, 63: -100.0}):
        b = plain.clone()
        for e, v in at.items():
            b[e] = v
        for groups, kept in ((8, 3), (32, 9)):
            _agree(l, 4, score, b, groups, kept)
        far = b.view(32, 2).clone()
        far[5] = torch.tensor([1e9, -1e9], device="cuda")
        _agree(l, 4, score, far.view(-1), 32, 8)
