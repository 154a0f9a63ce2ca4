"""The router over scores and its gradient against 64-bit formulas.

The choice has to be the 64-bit one exactly.  Bounds of the weights, with e = 2^-24 and L the largest |logit|: a
score is (L + 8) e relative off (the exponent's rounding, 2 of the exponential, a sum and a quotient), so quotients of scores
2 (L + 8) e and 16 e for their sum and the roundings after it; the gradient twice that of its parts and k e of their sum,
and half a step of its type.
"""
import pytest
import torch

from combine_persistent_warp_gb300 import ops

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}


def _scores(l, score):
    l = l.double()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    p = torch.exp(l - l.amax(1, keepdim=True))
    return p / p.sum(1, keepdim=True)


def _ordered(c):
    """NaN as one value, the largest: a sort goes by its bits, the sign among them."""
    return torch.sort(c.masked_fill(c.isnan(), float("nan")), dim=-1, descending=True, stable=True)


def _choice(l, k, score, bias, groups, kept, top):
    T, E = l.shape
    c = _scores(l, score)
    if bias is not None:
        c = c + bias.double()
    c = torch.where(l == -float("inf"), -float("inf"), c)
    if kept < groups:
        v = _ordered(c.view(T, groups, -1)).values[:, :, :top]
        # fewer than `top` candidates: the sum of those there are
        g = torch.where(v[:, :, :1].isneginf().squeeze(2), -float("inf"), v.masked_fill(v.isneginf(), 0.0).sum(2))
        order = _ordered(g).indices[:, :kept]
        stays = torch.zeros_like(g, dtype=torch.bool).scatter_(1, order, True) & ~g.isneginf()
        c = torch.where(stays[:, :, None], c.view(T, groups, -1), -float("inf")).view(T, E)
    v, idx = _ordered(c)
    return torch.where(v[:, :k].isneginf(), -1, idx[:, :k])


def _log_scores(l, score):
    return torch.nn.functional.logsigmoid(l) if score == "sigmoid" else torch.log_softmax(l, 1)


def _weights(l, idx, score, renorm, scale):
    s = _log_scores(l.double(), score).gather(1, idx.clamp_min(0)).masked_fill(idx < 0, -float("inf"))
    w = torch.softmax(s, 1).nan_to_num(0.0) if renorm else s.exp()
    return scale * w


def _check(l, k, score="sigmoid", bias=None, groups=1, kept=None, top=2, renorm=True, scale=1.0, mask=None):
    kept = groups if kept is None else kept
    idx, w = ops.route_scores(l, k, score=score, bias=bias, groups=groups, topk_groups=kept, group_top=top, renormalize=renorm,
                              scale=scale, token_mask=mask)
    want = _choice(l, k, score, bias, groups, kept, top)
    if mask is not None:
        want = torch.where(mask[:, None], want, -1)
    assert torch.equal(idx, want)
    L = l.masked_fill(l.isinf(), 0).abs().max().item() if l.numel() else 0.0
    ref = _weights(l, idx, score, renorm, scale)
    rel = (2 * (L + 8) + 16 + l.shape[1] / 2) * E24
    assert ((w.double() - ref).abs() <= rel * ref + 2.0 ** -126).all()
    dw = torch.randn(w.shape, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    got = ops.route_scores_backward(dw, idx, w, l, score=score, renormalize=renorm, scale=scale)
    d = dw.double().masked_fill(idx < 0, 0.0)
    leaf = l.double().clone().requires_grad_()
    ls = torch.where(idx < 0, -float("inf"), _log_scores(leaf.masked_fill(leaf.isneginf(), -1e4), score).gather(1, idx.clamp_min(0)))
    some = (idx >= 0).any(1)
    out = (torch.softmax(ls[some], 1) if renorm else ls[some].exp()) * scale
    (out * d[some]).sum().backward()
    grad = torch.where(l.isneginf(), 0.0, leaf.grad)
    parts = (ref * d.abs()).sum(1, keepdim=True)
    hot = torch.zeros_like(grad).scatter_add_(1, idx.clamp_min(0), torch.where(idx < 0, 0.0, ref * d.abs() + ref / scale * parts))
    if score == "softmax" and not renorm:
        hot = hot + _scores(l.masked_fill(l.isneginf(), -1e4), score) * parts
    # (the reference's zeros are sums that cancel in 64 bits: some 30 roundings, 2^-48 in all, of parts no larger than these)
    bound = 2 * (rel + k * E24) * hot + 2.0 ** -48 * parts + U[l.dtype] * grad.abs() + TINY[l.dtype]
    assert got.dtype == l.dtype and ((got.double() - grad).abs() <= bound).all()
    return idx, w


def _logits(T, E, dtype, seed=0, std=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (std * torch.randn(T, E, generator=g, device="cuda")).to(dtype)


def _bias(E, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 99)
    return torch.randint(-200, 201, (E,), generator=g, device="cuda").float() * 0.001


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score,renorm,scale", [("sigmoid", True, 2.5), ("sigmoid", False, 1.0), ("softmax", True, 1.0), ("softmax", False, 0.5)])
@pytest.mark.parametrize("T,E,k,groups,kept,top", [(1, 1, 1, 1, 1, 1), (1, 32, 8, 4, 2, 2), (33, 60, 7, 4, 2, 1), (257, 128, 8, 8, 4, 2), (3, 256, 8, 8, 4, 2),
                                                   (40, 256, 32, 32, 5, 2), (5, 1024, 32, 16, 3, 2), (17, 160, 6, 8, 3, 1), (9, 31, 31, 1, 1, 2),
                                                   (130, 72, 5, 3, 1, 2), (8, 1023, 9, 11, 2, 2), (1000, 64, 6, 1, 1, 2)])
def test_choice_weights_and_gradient(T, E, k, groups, kept, top, score, renorm, scale, dtype):
    l = _logits(T, E, dtype)
    for bias in (None, _bias(E)):
        _check(l, k, score, bias, groups, kept, top, renorm, scale)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 3)])
def test_values_that_32_bits_cannot_tell_apart(score, groups, kept):
    """Scores next to 1, or next to each other: the choice is the 64-bit one all the same."""
    E = 64
    g = torch.Generator(device="cuda").manual_seed(3)
    l = torch.rand(300, E, generator=g, device="cuda") * 12 + 16          # 1 - s between 1e-7 and 1e-12
    bias = torch.randint(0, 2, (E,), generator=g, device="cuda").float() * 0.25
    _check(l, 8, score, bias, groups, kept)
    near = 1.0 + torch.randint(0, 4, (300, E), generator=g, device="cuda") * 2.0 ** -23
    _check(near, 8, score, bias, groups, kept)
    _check(-near - 20, 6, score, bias, groups, kept)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_ties_go_to_the_lowest(score):
    zero = torch.zeros(5, 128, device="cuda", dtype=torch.bfloat16)
    for bias in (None, torch.zeros(128, device="cuda")):
        idx, _ = _check(zero, 8, score, bias, 8, 3)
        assert torch.equal(idx, torch.arange(8, device="cuda").expand(5, 8))
    few = (torch.randint(0, 3, (400, 96), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 0.5).bfloat16()
    _check(few, 7, score, torch.zeros(96, device="cuda"), 6, 2)
    _check(few, 7, score, None, 6, 2, 1)
    _check(torch.where(few == 0, -0.0, few.float()), 7, score, None)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
def test_absent_experts_masked_tokens_and_empty_groups(score, bias):
    l = _logits(64, 48, torch.float32)
    l[:, 5] = -float("inf")
    l[3] = -float("inf")                       # nothing to choose
    l[4, 1:] = -float("inf")                   # one expert
    l[5, 8:] = -float("inf")                   # one group
    l[6, 10:] = -float("inf")                  # two candidates in the second group
    l[7, 9:] = -float("inf")                   # one in the second
    b = _bias(48) if bias else None
    mask = torch.ones(64, dtype=torch.bool, device="cuda")
    mask[10:20] = False
    for renorm in (True, False):
        idx, w = _check(l, 8, score, b, 6, 2, 2, renorm, 2.5, mask)
        assert (idx[3] == -1).all() and (w[3] == 0).all() and (idx[10:20] == -1).all() and (w[idx < 0] == 0).all()
    if bias:
        b2 = b.clone()
        b2[7] = -float("inf")                  # an expert that the bias excludes
        idx, _ = ops.route_scores(_logits(64, 48, torch.float32), 30, score=score, bias=b2)
        assert not (idx == 7).any()


def test_nan_counts_as_the_largest_and_padding_is_not_read():
    l = _logits(8, 40, torch.float32)
    l[2, 17] = float("nan")
    mask = torch.ones(8, dtype=torch.bool, device="cuda")
    mask[5] = False
    l[5] = float("nan")
    idx, w = ops.route_scores(l, 4, bias=_bias(40), token_mask=mask)
    assert idx[2, 0] == 17 and w[2].isnan().all() and (idx[5] == -1).all() and (w[5] == 0).all() and not w[[0, 1, 3, 4, 6, 7]].isnan().any()
    d = ops.route_scores_backward(torch.ones_like(w), idx, w, l)
    assert (d[5] == 0).all() and not d[[0, 1, 3, 4, 6, 7]].isnan().any()


def test_tiny_scores_have_their_quotients():
    l = -_logits(20, 16, torch.float32).abs() - 150
    idx, w = _check(l, 4, "sigmoid", None)
    assert ((w.sum(1) - 1).abs() < 1e-5).all()
    idx, w = ops.route_scores(l + 20000, 4, score="sigmoid")
    assert ((w - 0.25).abs() < 1e-6).all()


def test_an_expert_in_two_slots_gets_both_gradients():
    l = _logits(6, 40, torch.float32)
    idx = torch.randint(0, 3, (6, 5), device="cuda")
    w, dw = torch.rand(6, 5, device="cuda"), torch.randn(6, 5, device="cuda")
    for score in ("sigmoid", "softmax"):
        got = ops.route_scores_backward(dw, idx, w, l, score=score, renormalize=False)
        if score == "sigmoid":
            part = (w * dw).double() * (1 - _scores(l, score).gather(1, idx))
            want = torch.zeros(6, 40, dtype=torch.float64, device="cuda").scatter_add_(1, idx, part)
        else:
            p = _scores(l, score)
            want = p * (torch.zeros_like(p).scatter_add_(1, idx, dw.double()) - (w * dw).double().sum(1, keepdim=True))
        # five terms of at most 4, 32 roundings of each
        assert ((got.double() - want).abs() <= 5 * 4 * 32 * E24).all()


def test_strided_logits_streams_graphs_and_equal_bits():
    big = _logits(500, 131, torch.bfloat16)
    l, bias = big[:, 1:129], _bias(128)
    args = dict(bias=bias, groups=8, topk_groups=4, scale=2.5)
    idx, w = _check(l, 8, "sigmoid", bias, 8, 4, scale=2.5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    i2, w2 = ops.route_scores(l, 8, stream=s, **args)
    d2 = ops.route_scores_backward(w2, i2, w2, l, scale=2.5, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(idx, i2) and torch.equal(w, w2)
    live = l.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        i3, w3 = ops.route_scores(live, 8, **args)
        d3 = ops.route_scores_backward(w3, i3, w3, live, scale=2.5)
    g.replay()
    assert torch.equal(i3, idx) and torch.equal(w3, w) and torch.equal(d3, d2)
    live.copy_(l.flip(0))
    g.replay()
    assert torch.equal(i3, idx.flip(0)) and torch.equal(w3, w.flip(0))
    e = l[:0]
    assert ops.route_scores(e, 8, **args)[0].shape == (0, 8)
    assert ops.route_scores_backward(w[:0], idx[:0], w[:0], e).shape == (0, 128)


def test_choice_feeds_the_expert_order():
    l = _logits(300, 32, torch.bfloat16)
    idx, w = ops.route_scores(l, 4, bias=_bias(32), groups=4, topk_groups=2)
    order = ops.expert_order(idx, 32)
    assert order.status.item() == 0 and order.offsets[-1].item() == 1200


def test_gradient_against_differences():
    l = _logits(4, 12, torch.float32)
    dw = torch.randn(4, 3, device="cuda")
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            idx, w = ops.route_scores(l, 3, score=score, renormalize=renorm, scale=1.5)
            got = ops.route_scores_backward(dw, idx, w, l, score=score, renormalize=renorm, scale=1.5)
            f = lambda v: (_weights(v, idx, score, renorm, 1.5) * dw).sum()
            for e in range(12):
                d = torch.zeros(4, 12, dtype=torch.float64, device="cuda")
                d[2, e] = 1e-5
                # the differences are 1e-9 off, the gradient some hundred roundings of terms of at most 4
                assert abs((f(l.double() + d) - f(l.double() - d)) / 2e-5 - got[2, e].double()) <= 1e-4


@pytest.mark.parametrize("T,k", [(6143, 8), (6145, 8), (6147, 16), (16384, 8), (16387, 7), (16385, 16), (16386, 20)])
@pytest.mark.parametrize("score,bias,groups,kept", [("sigmoid", True, 8, 4), ("sigmoid", True, 1, 1), ("softmax", False, 1, 1), ("sigmoid", False, 8, 3)])
def test_long_batches(T, k, score, bias, groups, kept):
    """Several tokens a warp, the last warp's not all there, some of them masked; a bias past what the words hold in fixed point."""
    for dtype in (torch.bfloat16, torch.float32):
        l = _logits(T, 96, dtype, seed=T)
        mask = torch.rand(T, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") > 0.1
        b = _bias(96) if bias else None
        _check(l, k, score, b, groups, kept, mask=mask)
        if bias:
            b = 5 * b
            b[3] = -float("inf")
            _check(l, k, score, b, groups, kept, scale=0.5)


@pytest.mark.parametrize("k", [5, 31, 32])
def test_large_logits_without_a_bias_are_in_their_own_order(k):
    """Sigmoids that are 1 in 64 bits too: what the choice goes by without a bias are the logits."""
    g = torch.Generator(device="cuda").manual_seed(9)
    l = 40.0 + 100 * torch.rand(30, 70, generator=g, device="cuda")
    for v in (l, l.bfloat16()):
        idx, w = ops.route_scores(v, k)
        assert torch.equal(idx, torch.sort(v, dim=1, descending=True, stable=True).indices[:, :k])
        assert ((w - 1.0 / k).abs() <= 8 * E24).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,groups,kept", [(64, 1, 1, 1), (64, 6, 1, 1), (64, 6, 8, 3), (72, 9, 3, 1), (512, 32, 16, 5)])
def test_biases_and_logits_that_are_no_ordinary_numbers(score, E, k, groups, kept):
    """A NaN is the largest and an infinite or huge bias takes its place in the order, as in 64 bits; the tail of a batch whose
    groups are all equal, and tokens that are masked, are left alone."""
    inf, nan = float("inf"), float("nan")
    l = _logits(6145, E, torch.float32)
    l[1, 3] = nan
    l[2, 40] = inf
    l[3, 5:9] = -nan
    l[4, ::2] = -inf
    l[4, 1] = nan
    l[5, 60], l[5, 61] = inf, nan
    l[6] = nan
    l[7] = inf
    plain = _bias(E)
    for at in ({}, {7: nan}, {9: inf}, {9: inf, 40: inf, 50: nan}, {9: 3.4e38, 10: 3.2e38, 30: inf, 63: 3.3e38}, {3: -inf, 5: nan, 40: -3.4e38}):
        b = plain.clone()
        for e, v in at.items():
            b[e] = v
        for rows in (l[:40], l):
            idx, _ = ops.route_scores(rows, k, score=score, bias=b, groups=groups, topk_groups=kept)
            assert torch.equal(idx, _choice(rows, k, score, b, groups, kept, 2))
    mask = torch.arange(6145, device="cuda") % 3 != 0
    same = torch.zeros(6145, E, device="cuda")
    for b in (None, torch.zeros(E, device="cuda")):
        _check(same, k, score, b, groups, kept, mask=mask)


@pytest.mark.parametrize("T,k", [(40, 8), (40, 1), (40, 32), (6145, 8), (16385, 8), (16385, 1)])
def test_chains_of_ties_and_of_near_values(T, k):
    """Around the last slot: equal values with and without nearly equal ones among them, in and out of order."""
    g = torch.Generator(device="cuda").manual_seed(T + k)
    ints = lambda n, *size: torch.randint(0, n, size, generator=g, device="cuda").float()
    zero = torch.zeros(64, device="cuda")
    step = ints(3, 64) * 0.25
    for l in (ints(2, T, 64), ints(12, T, 64) * 0.25, 1 + ints(3, T, 64) * 2.0 ** -23, ints(2, T, 64) + ints(2, T, 64) * 2.0 ** -22,
              (ints(2, T, 64) + 16) * (1 + ints(2, T, 64) * 2.0 ** -23), torch.zeros(T, 64, device="cuda")):
        for b in (zero, step, step + ints(2, 64) * 2.0 ** -24, 3 * step):
            for groups, kept in ((1, 1), (4, 2)):
                if k <= kept * 64 // groups:
                    idx, _ = ops.route_scores(l, k, bias=b, groups=groups, topk_groups=kept)
                    assert torch.equal(idx, _choice(l, k, "sigmoid", b, groups, kept, 2))


@pytest.mark.parametrize("T,k", [(2051, 5), (2050, 16), (32771, 8)])
@pytest.mark.parametrize("E", [40, 37])
def test_gradient_of_several_tokens_a_warp(T, k, E):
    """Experts in several slots, empty slots, and a last warp whose tokens are not all there."""
    g = torch.Generator(device="cuda").manual_seed(T + E)
    l = _logits(T, E, torch.float32)
    idx = torch.randint(-1, 6, (T, k), generator=g, device="cuda")
    w, dw = torch.rand(T, k, generator=g, device="cuda"), torch.randn(T, k, generator=g, device="cuda").clamp(-4, 4)
    got = ops.route_scores_backward(dw, idx, w, l, renormalize=False)
    at = idx.clamp_min(0)
    part = (w * dw).double() * (1 - _scores(l, "sigmoid").gather(1, at))
    want = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_add_(1, at, part.masked_fill(idx < 0, 0.0))
    # at most 16 terms of at most 4, 32 roundings of each
    assert ((got.double() - want).abs() <= k * 4 * 32 * E24).all()
    half = ops.route_scores_backward(dw, idx, w, l.bfloat16(), renormalize=False)
    part = (w * dw).double() * (1 - _scores(l.bfloat16(), "sigmoid").gather(1, at))
    want = torch.zeros_like(want).scatter_add_(1, at, part.masked_fill(idx < 0, 0.0))
    assert ((half.double() - want).abs() <= k * 4 * 32 * E24 + U[torch.bfloat16] * want.abs() + 2.0 ** -126).all()
