"""The autograd functions on the GPU in the forms that the operators document: parameters that are absent."""
import pytest
import torch

from combine_persistent_warp_gb300 import ops, training

pytestmark = pytest.mark.gpu


def _order(T, k, E, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ops.expert_order(torch.randint(-1, E, (T, k), generator=g, device="cuda"), E)


@pytest.mark.parametrize("with_weight", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
def test_layer_norm_without_weight_or_bias(with_weight, with_bias):
    # fp32 sums of 64 and 33 terms: a few dozen roundings of 2^-24 on values of up to about 30
    torch.manual_seed(0)
    x = torch.randn(33, 64, device="cuda", requires_grad=True)
    g = torch.randn(64, device="cuda", requires_grad=True) if with_weight else None
    b = torch.randn(64, device="cuda", requires_grad=True) if with_bias else None
    dy = torch.randn(33, 64, device="cuda")
    training.layer_norm(x, g, b).backward(dy)
    want = [t.detach().double().requires_grad_() if t is not None else None for t in (x, g, b)]
    torch.nn.functional.layer_norm(want[0], (64,), want[1], want[2]).backward(dy.double())
    for got, ref in zip((x, g, b), want):
        if got is not None:
            assert (got.grad - ref.grad).abs().max() <= 1e-4


def test_combine_without_gate_weights():
    o = _order(20, 3, 4)
    y = torch.randn(60, 24, device="cuda", requires_grad=True)
    dout = torch.randn(20, 24, device="cuda")
    training.combine_rows(y, o, None).backward(dout)
    want = torch.zeros(60, 24, device="cuda")
    named = o.rows >= 0
    want[o.rows[named].long()] = dout[named.nonzero()[:, 0]]
    assert torch.equal(y.grad, want)


def test_a_bias_in_fp32_without_a_weight():
    torch.manual_seed(3)
    x = torch.randn(40, 64, device="cuda").bfloat16()
    b = torch.randn(64, device="cuda", requires_grad=True)
    dy = torch.randn(40, 64, device="cuda").bfloat16()
    training.layer_norm(x, None, b).backward(dy)
    assert b.grad.dtype == torch.float32
    # a 40-term sum in fp32, not a bf16 of it
    assert ((b.grad - dy.double().sum(0)).abs() <= 40 * 2.0 ** -24 * dy.double().abs().sum(0)).all()


@pytest.mark.parametrize("rows", [1, 5])
def test_gradients_that_start_anywhere(rows):
    """The gradient of y in torch.cat([s, y.view(-1)]) is contiguous and starts behind s."""
    torch.manual_seed(4)
    off = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device="cuda")
    x = torch.randn(rows, 64, device="cuda").bfloat16().requires_grad_()
    w = torch.randn(2, 72, 64, device="cuda").bfloat16().requires_grad_()
    y = training.grouped_mm(x, w, off)
    d = torch.randn(rows * 72 + 3, device="cuda").bfloat16()
    torch.cat([torch.zeros(3, device="cuda", dtype=torch.bfloat16), y.view(-1)]).backward(d)
    dy = d[3:].clone().view(rows, 72)
    assert torch.equal(x.grad, ops.grouped_mm_dx(dy, w.detach(), off))
    assert torch.equal(w.grad, ops.grouped_mm_dw(dy, x.detach(), off))
    # a part of a wider gradient
    x.grad = None
    wide = torch.randn(rows, 77, device="cuda").bfloat16()
    training.grouped_mm(x, w, off).backward(wide[:, 5:])
    assert torch.equal(x.grad, ops.grouped_mm_dx(wide[:, 5:].clone(), w.detach(), off))


@pytest.mark.parametrize("T,H", [(0, 64), (1, 64), (300, 512), (40, 1001), (3000, 2048), (3000, 2049), (5, 12000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients_that_are_not_asked_for(T, H, dtype):
    torch.manual_seed(5)
    x, dy = torch.randn(T, H, device="cuda").to(dtype), torch.randn(T, H, device="cuda").to(dtype)
    g = torch.randn(H, device="cuda").to(dtype)
    _, mean, rstd = ops.layer_norm(x, g)
    full = ops.layer_norm_backward(dy, x, g, mean, rstd)
    for weight_grad, bias_grad in ((False, False), (True, False), (False, True)):
        part = ops.layer_norm_backward(dy, x, g, mean, rstd, weight_grad=weight_grad, bias_grad=bias_grad)
        for a, b, asked in zip(part, full, (True, weight_grad, bias_grad)):
            assert torch.equal(a, b) if asked else a is None
    o = _order(T, 2, 4)
    y, w = torch.randn(2 * T, H, device="cuda").to(dtype), torch.rand(T, 2, device="cuda")
    dout = torch.randn(T, H, device="cuda").to(dtype)
    dy, dw = ops.combine_rows_backward(dout, y, o.rows, w, o.offsets, gate_grad=False)
    assert dw is None and torch.equal(dy, ops.combine_rows_backward(dout, y, o.rows, w, o.offsets)[0])


@pytest.mark.parametrize("held", [float("nan"), float("inf"), 1e30, 0.0])
def test_what_unrouted_tokens_hold_reaches_no_gradient(held):
    torch.manual_seed(6)
    block = training.MoEBlock(4, 64, 64, 2, std=0.1).cuda()
    x = torch.randn(50, 64, device="cuda").bfloat16()
    mask = torch.arange(50, device="cuda") % 3 != 0
    want = {}
    for fill in (1.0, held):
        v = torch.where(mask[:, None], x, fill).requires_grad_()
        block.zero_grad()
        out = block(v, mask)
        out[mask].float().square().mean().backward()
        got = dict({n: p.grad.clone() for n, p in block.named_parameters()}, x=v.grad, out=out[mask].detach())
        assert all(t.isfinite().all() for t in got.values()) and not v.grad[~mask].any()
        want = want or got
    for n, t in want.items():
        assert torch.equal(t, got[n]), n
