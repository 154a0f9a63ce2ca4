"""The router, its gradient and the expert-major order against plain forms: indices and orders
equal, weights within fp32 rounding of 64-bit softmaxes.

Weights: expf is at most 2 ulp off and its argument carries one rounding of a difference of at most
|l| magnitudes, so p is off by (4 + |d|)*2^-24 relative, d the difference of two logits; sums of at most 1024
positive terms add 64*2^-24.  The bound below is (80 + 2*max|d|) * 2^-24 relative.
"""
import math

import pytest
import torch

from combine_persistent_warp_gb300 import ops

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -10}


def _logits(T, E, dtype, seed=0, std=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, E, generator=g, device="cuda") * std).to(dtype)


def _plain(logits, k, renorm, mask=None):
    l = logits.double()
    key = torch.where(l.isnan(), math.inf, l)       # NaN above everything that these tests hold
    val, idx = torch.sort(key, dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    dead = val == -math.inf
    real = torch.gather(l, 1, idx)
    p = torch.exp(real - real[:, :1])
    p = torch.where(dead, 0.0, p)
    den = p.sum(1, keepdim=True) if renorm else torch.exp(l - real[:, :1]).sum(1, keepdim=True)
    w = torch.where(dead, 0.0, p / den)
    idx = torch.where(dead, -1, idx)
    if mask is not None:
        idx = torch.where(mask[:, None], idx, -1)
        w = torch.where(mask[:, None], w, 0.0)
    return idx, w


def _close(w, rw, logits):
    l = logits.double()
    l = l[l.isfinite()]
    spread = float(l.max() - l.min()) if l.numel() else 0.0
    assert torch.equal(w.isnan(), rw.isnan())
    ok = ~rw.isnan()
    assert ((w.double() - rw).abs()[ok] <= (80 + 2 * spread) * E24 * rw.abs()[ok] + 1e-37).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (5, 8, 8), (128, 32, 8), (33, 33, 4), (1000, 64, 6), (17, 100, 32),
                                   (300, 128, 8), (9, 256, 8), (7, 257, 3), (4, 1000, 32), (3, 1024, 1)])
def test_forward(T, E, k, dtype, renorm):
    l = _logits(T, E, dtype)
    idx, w = ops.route_topk(l, k, renormalize=renorm)
    ridx, rw = _plain(l, k, renorm)
    assert torch.equal(idx, ridx)
    _close(w, rw, l)


def test_ties_go_to_the_lowest_expert():
    l = torch.zeros(4, 100, device="cuda")
    l[1] = -0.0
    l[1, 50] = 0.0
    l[2, 7:] = 1.0
    l[3] = torch.finfo(torch.float32).min
    idx, w = ops.route_topk(l, 5)
    assert idx.tolist() == [[0, 1, 2, 3, 4]] * 2 + [[7, 8, 9, 10, 11]] + [[0, 1, 2, 3, 4]]
    assert (w - 0.2).abs().max() <= 4 * E24


@pytest.mark.parametrize("renorm", [True, False])
def test_masked_experts_and_tokens(renorm):
    T, E, k = 64, 40, 6
    l = _logits(T, E, torch.float32, 3)
    g = torch.Generator(device="cuda").manual_seed(1)
    l[torch.rand(T, E, generator=g, device="cuda") < 0.9] = -math.inf      # rows with fewer than k left
    l[5] = -math.inf                                                       # and none
    mask = torch.rand(T, generator=g, device="cuda") < 0.7
    mask[7], mask[8] = False, False
    l[7], l[8, ::2] = math.nan, math.inf                                   # in a masked token: nothing leaks
    idx, w = ops.route_topk(l, k, token_mask=mask, renormalize=renorm)
    ridx, rw = _plain(l, k, renorm, mask)
    rw = torch.where(ridx < 0, 0.0, rw)
    assert torch.equal(idx, ridx)
    _close(w, rw, l)
    assert (idx[5] == -1).all() and (w[5] == 0).all()
    dw = torch.randn(T, k, generator=g, device="cuda")
    dw[7] = math.nan
    d = ops.route_topk_backward(dw, idx, w, l, renormalize=renorm)
    assert (d[~mask] == 0).all() and (d[5] == 0).all() and d[mask].isfinite().all()


def test_nan_and_infinite_logits_show():
    l = _logits(3, 16, torch.float32)
    l[0, 9] = math.nan
    l[1, 4] = math.inf
    idx, w = ops.route_topk(l, 4)
    assert idx[0, 0] == 9 and w[0].isnan().all() and ((idx[0] >= 0) & (idx[0] < 16)).all()
    assert idx[1, 0] == 4 and w[1, 0].isnan()
    assert w[2].isfinite().all()


def test_strided_logits():
    big = _logits(50, 96, torch.bfloat16)
    l = big[:, 3:67]
    idx, w = ops.route_topk(l, 4)
    ridx, rw = _plain(l, 4, True)
    assert torch.equal(idx, ridx)
    _close(w, rw, l)


def _grad(l, idx, dw, renorm):
    """Gradient of sum(dw * w) through 64-bit autograd of the softmax, the choice held."""
    x = l.double().requires_grad_()
    p = torch.softmax(x, 1)
    w = torch.gather(p, 1, idx.clamp_min(0)) * (idx >= 0)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    (w * dw.double()).sum().backward()
    return x.grad, w.detach()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 8), (128, 32, 8), (33, 33, 4), (300, 128, 8), (7, 257, 3), (4, 1000, 32)])
def test_backward(T, E, k, dtype, renorm):
    l = _logits(T, E, dtype, 5)
    idx, w = ops.route_topk(l, k, renormalize=renorm)
    g = torch.Generator(device="cuda").manual_seed(2)
    dw = torch.randn(T, k, generator=g, device="cuda")
    d = ops.route_topk_backward(dw, idx, w, l, renormalize=renorm)
    rd, rw = _grad(l, idx, dw, renorm)
    scale = (rw * dw.double().abs()).sum(1, keepdim=True) + (rw.max(1).values * dw.double().abs().max(1).values)[:, None]
    tiny = 2.0 ** -24 if dtype == torch.float16 else 0.0
    assert ((d.double() - rd).abs() <= 200 * E24 * scale + U[dtype] * rd.abs() + tiny).all()
    assert d.dtype == dtype
    if renorm:
        rest = torch.ones(T, E, dtype=torch.bool, device="cuda").scatter_(1, idx, False)
        assert (d[rest] == 0).all()


@pytest.mark.parametrize("renorm", [True, False])
def test_backward_against_differences(renorm):
    T, E, k, h = 8, 24, 5, 1e-5
    l = _logits(T, E, torch.float32, 6)
    idx, w = ops.route_topk(l, k, renormalize=renorm)
    g = torch.Generator(device="cuda").manual_seed(2)
    dw = torch.randn(T, k, generator=g, device="cuda")
    d = ops.route_topk_backward(dw, idx, w, l, renormalize=renorm)
    v = torch.randn(T, E, generator=g, device="cuda", dtype=torch.double)

    def f(x):
        e = torch.exp(x)
        c = torch.gather(e, 1, idx)
        return (c / (c if renorm else e).sum(1, keepdim=True) * dw.double()).sum()

    diff = (f(l.double() + h * v) - f(l.double() - h * v)) / (2 * h)
    assert abs((d.double() * v).sum() - diff) <= 1e-5 * (1 + d.double().norm() * v.norm())


# ------------------------------------------------------------------ expert-major order ----
def _plain_order(idx, E):
    flat = idx.reshape(-1)
    key = torch.where((flat < 0) | (flat >= E), E, flat)
    at = torch.argsort(key, stable=True)
    rows = torch.empty_like(at)
    rows[at] = torch.arange(at.numel(), device=at.device)
    rows = torch.where(key == E, -1, rows).view_as(idx).int()
    counts = torch.bincount(key, minlength=E + 1)[:E]
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int(), rows


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 32), (3, 2, 1000), (128, 8, 32), (512, 8, 128), (513, 8, 128), (4096, 8, 32),
                                   (4097, 7, 1024), (16384, 8, 128), (20001, 5, 257), (150000, 8, 64), (300000, 4, 1024),
                                   (700, 8, 680), (5000, 8, 681), (5000, 8, 682), (5000, 8, 683), (700, 8, 682)])
@pytest.mark.parametrize("kind", ["uniform", "skewed", "one"])
def test_order(T, k, E, kind):
    g = torch.Generator(device="cuda").manual_seed(T + k)
    if kind == "one":
        idx = torch.full((T, k), E - 1, dtype=torch.int64, device="cuda")
    else:
        u = torch.rand(T, k, generator=g, device="cuda")
        idx = ((u if kind == "uniform" else u ** 4) * E).long().clamp_max(E - 1)
        idx[torch.rand(T, k, generator=g, device="cuda") < 0.05] = -1
    order = ops.expert_order(idx, E)
    off, rows = _plain_order(idx, E)
    assert torch.equal(order.offsets, off) and torch.equal(order.rows, rows) and order.status.item() == 0


def test_order_of_skipped_and_bad_ids():
    idx = torch.full((40, 4), -1, dtype=torch.int64, device="cuda")
    o = ops.expert_order(idx, 6)
    assert (o.offsets == 0).all() and (o.rows == -1).all() and o.status.item() == 0
    for bad in (6, -2, 1 << 40):
        idx[3, 1], idx[9, 0] = bad, 5
        o = ops.expert_order(idx, 6)
        assert o.status.item() == 6                      # MOE_ERR_BAD_INDEX
        assert o.rows[9, 0] == 0 and o.offsets.tolist() == [0] * 6 + [1] and (o.rows >= 0).sum() == 1
    e = ops.expert_order(torch.zeros(0, 4, dtype=torch.int64, device="cuda"), 3)
    assert e.offsets.tolist() == [0, 0, 0, 0] and e.rows.shape == (0, 4)


def test_refusals_of_tensors():
    l = _logits(4, 8, torch.float32)
    idx, w = ops.route_topk(l, 2)
    with pytest.raises(ops.MoeError):
        ops.route_topk(l, 9)
    with pytest.raises(TypeError):
        ops.route_topk(l.long(), 2)
    with pytest.raises(TypeError):
        ops.route_topk(l, 2, token_mask=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        ops.route_topk(l, 2, token_mask=torch.ones(3, device="cuda", dtype=torch.bool))
    with pytest.raises(TypeError):
        ops.route_topk_backward(w.half(), idx, w, l)
    with pytest.raises(TypeError):
        ops.expert_order(idx.int(), 8)
    with pytest.raises(ops.MoeError):
        ops.expert_order(idx, 2000)
