"""16-bit types in their own right: the router over every value that they have, and fp16 results within
fp16's own unit roundoff, 2^-11 (the other files' bounds take 2^-10), of the same 64-bit forms.

Gate weights: as in test_gpu_ops_router.py, (80 + 2 |d|) * 2^-24 relative, d the difference from the token's
largest logit; from |d| = 88 on a weight is below 2^-126 and need not be more than tiny.
"""
import math

import pytest
import test_gpu_ops_grouped as grouped
import test_gpu_ops_norm as norm
import test_gpu_ops_router as router
import test_gpu_ops_rows as rows
import torch

from combine_persistent_warp_gb300 import ops

pytestmark = pytest.mark.gpu
HALF = [torch.bfloat16, torch.float16]
E24 = 2.0 ** -24


def _plain(l, k, mask=None):
    """Indices by value, then lowest index, NaN above +inf, -inf never."""
    key = l.double()
    key = torch.where(key == math.inf, 1e300, key)
    key = torch.where(l.isnan(), 1e301, key)
    val, idx = torch.sort(key, dim=1, descending=True, stable=True)
    idx = torch.where(val[:, :k] == -math.inf, -1, idx[:, :k])
    return idx if mask is None else torch.where(mask[:, None], idx, -1)


def _check(l, k, renorm, mask=None):
    idx, w = ops.route_topk(l, k, token_mask=mask, renormalize=renorm)
    assert torch.equal(idx, _plain(l, k, mask))
    assert (w[idx < 0] == 0).all()
    v = torch.where(idx < 0, -math.inf, l.double().gather(1, idx.clamp_min(0)))
    top = v[:, :1]
    finite = top[:, 0].isfinite()                         # (no NaN or +inf on top, and something chosen)
    p = torch.exp(v - top)
    den = p.sum(1, keepdim=True) if renorm else torch.exp(l.double() - top).sum(1, keepdim=True)
    ref = (p / den)[finite]
    bound = (80 + 2 * (v - top)[finite].abs().clamp_max(88)) * E24 * ref + 2.0 ** -126
    assert ((w.double()[finite] - ref).abs() <= bound).all()
    return idx, w


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(8, 3), (32, 8), (33, 8), (128, 8), (256, 6), (1000, 32)])
def test_router_over_all_bit_patterns(E, k, renorm, dtype):
    """Subnormals, both zeros, the largest and lowest finite values, infinities and NaNs among the others,
    and rows of few values, so that most of their logits are ties."""
    g = torch.Generator(device="cuda").manual_seed(E)
    T = max(65536 // E, 64)
    every = torch.randint(-32768, 32768, (T, E), generator=g, device="cuda").to(torch.int16).view(dtype)
    finite = torch.where(every.isfinite(), every, torch.tensor(0.0, dtype=dtype, device="cuda"))
    tiny, low = torch.tensor([1, 2, -32767, -32766], dtype=torch.int16).view(dtype), torch.finfo(dtype).min
    few = torch.cat([tiny, torch.tensor([0.0, -0.0, low, -low, -math.inf, 1.0, -1.0], dtype=dtype)]).cuda()
    ties = few[torch.randint(0, few.numel(), (T, E), generator=g, device="cuda")]
    mask = torch.rand(T, generator=g, device="cuda") < 0.8
    for l in (every, finite, ties):
        _check(l, k, renorm)
        _check(l, k, renorm, mask)


@pytest.mark.parametrize("dtype", HALF)
def test_router_ties_and_the_lowest_value(dtype):
    l = torch.zeros(5, 100, device="cuda", dtype=dtype)
    l[1] = -0.0
    l[1, 50] = 0.0
    l[2, 7:] = 1.0
    l[3] = torch.finfo(dtype).min
    l[4] = -math.inf
    l[4, 60], l[4, 61] = torch.finfo(dtype).min, -torch.finfo(dtype).smallest_normal
    idx, w = ops.route_topk(l, 5)
    assert idx.tolist() == [[0, 1, 2, 3, 4]] * 2 + [[7, 8, 9, 10, 11], [0, 1, 2, 3, 4], [61, 60, -1, -1, -1]]
    assert (w[:4] - 0.2).abs().max() <= 4 * E24 and w[4].tolist() == [1.0, 0.0, 0.0, 0.0, 0.0]


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("renorm", [True, False])
def test_router_masked_experts_and_tokens(renorm, dtype):
    T, E, k = 64, 40, 6
    l = router._logits(T, E, dtype, 3)
    g = torch.Generator(device="cuda").manual_seed(1)
    l[torch.rand(T, E, generator=g, device="cuda") < 0.9] = -math.inf
    l[5] = -math.inf
    mask = torch.rand(T, generator=g, device="cuda") < 0.7
    mask[7], mask[8] = False, False
    l[7], l[8, ::2] = math.nan, math.inf
    idx, w = _check(l, k, renorm, mask)
    dw = torch.randn(T, k, generator=g, device="cuda")
    dw[7] = math.nan
    d = ops.route_topk_backward(dw, idx, w, l, renormalize=renorm)
    assert (d[~mask] == 0).all() and (d[5] == 0).all() and d[mask].isfinite().all()


@pytest.mark.parametrize("dtype", HALF)
def test_router_nan_and_infinity_show(dtype):
    l = router._logits(4, 16, dtype)
    l[0, 9] = math.nan
    l[1, 4] = math.inf
    l[3, 2], l[3, 11] = math.inf, -math.nan
    idx, w = ops.route_topk(l, 4)
    assert idx[0, 0] == 9 and idx[1, 0] == 4 and idx[3, :2].tolist() == [11, 2]
    assert w[0].isnan().all() and w[1, 0].isnan() and w[3].isnan().all() and w[2].isfinite().all()


@pytest.fixture
def fp16_roundoff(monkeypatch):
    for m in (grouped, norm, router, rows):
        monkeypatch.setitem(m.U, torch.float16, 2.0 ** -11)


@pytest.mark.parametrize("T,H", [(1, 8), (9, 1001), (130, 4096), (700, 1024), (2, 16384), (1300, 264)])
def test_norm_within_fp16_roundoff(T, H, fp16_roundoff):
    x, g, b, dy = norm._inputs(T, H, torch.float16, torch.float16)
    norm._check_forward(x, g, b, ops.layer_norm(x, g, b))
    norm._check_backward(x, g, dy)


@pytest.mark.parametrize("T,k,H,E", rows.SIZES)
def test_rows_within_fp16_roundoff(T, k, H, E, fp16_roundoff):
    rows.test_combine_and_its_gradients(T, k, H, E, torch.float16, True)


@pytest.mark.parametrize("T,E,k", [(5, 8, 8), (33, 33, 4), (300, 128, 8)])
@pytest.mark.parametrize("renorm", [True, False])
def test_router_gradient_within_fp16_roundoff(T, E, k, renorm, fp16_roundoff):
    router.test_backward(T, E, k, torch.float16, renorm)


@pytest.mark.parametrize("sizes,N,K", [([5, 0, 1], 264, 200), ([257, 255], 512, 136), ([300, 1, 0, 700, 513], 320, 448), ([1], 256, 4096)])
def test_products_within_fp16_roundoff(sizes, N, K, fp16_roundoff):
    grouped._check(*grouped._case(sizes, N, K, torch.float16))
