"""The autograd functions of `training` around stand-ins of the operators on the CPU: which gradients they
return, of which type, and what they hand to the operators."""
import pytest
import torch

from combine_persistent_warp_gb300 import ops, training


def _layer_norm(x, weight=None, bias=None, eps=1e-5):
    f = x.float()
    mean = f.mean(1)
    rstd = (f.var(1, unbiased=False) + eps).rsqrt()
    y = (f - mean[:, None]) * rstd[:, None]
    y = y * weight.float() if weight is not None else y
    return (y + bias.float() if bias is not None else y).to(x.dtype), mean, rstd


def _layer_norm_backward(dy, x, weight, mean, rstd, *, param_dtype=None, weight_grad=True, bias_grad=True):
    xh = (x.float() - mean[:, None]) * rstd[:, None]
    d = dy.float()
    g = d * weight.float() if weight is not None else d
    dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * rstd[:, None]
    to = weight.dtype if weight is not None else param_dtype or x.dtype
    return dx.to(x.dtype), (d * xh).sum(0).to(to) if weight_grad else None, d.sum(0).to(to) if bias_grad else None


def _combine_rows(y, rows, w=None):
    v = y[rows.clamp_min(0).long()].float() * (w if w is not None else torch.ones(rows.shape))[:, :, None]
    return torch.where((rows < 0)[:, :, None], 0.0, v).sum(1).to(y.dtype)


def _combine_rows_backward(dout, y, rows, w, offsets, *, gate_grad=True):
    named = rows >= 0
    at = rows[named].long()
    weights = w if w is not None else torch.ones(rows.shape)
    dy = torch.zeros_like(y, dtype=torch.float32)
    dy[at] = (weights[:, :, None] * dout.float()[:, None])[named]
    dw = torch.zeros(rows.shape)
    dw[named] = (y[at].float() * dout.float()[named.nonzero()[:, 0]]).sum(1)
    return dy.to(y.dtype), dw if gate_grad else None


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    for f in (_layer_norm, _layer_norm_backward, _combine_rows, _combine_rows_backward):
        monkeypatch.setattr(ops, f.__name__[1:], f)


ORDER = ops.ExpertOrder(torch.tensor([0, 2, 5], dtype=torch.int32), torch.tensor([[0, 2], [1, -1], [3, 4]], dtype=torch.int32),
                        torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("with_weight", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
def test_layer_norm_without_weight_or_bias(with_weight, with_bias):
    torch.manual_seed(0)
    x = torch.randn(5, 16, requires_grad=True)
    g = torch.randn(16, requires_grad=True) if with_weight else None
    b = torch.randn(16, requires_grad=True) if with_bias else None
    dy = torch.randn(5, 16)
    training.layer_norm(x, g, b).backward(dy)
    want = [t.detach().clone().requires_grad_() if t is not None else None for t in (x, g, b)]
    torch.nn.functional.layer_norm(want[0], (16,), want[1], want[2]).backward(dy)
    for got, ref in zip((x, g, b), want):
        if got is not None:
            assert (got.grad - ref.grad).abs().max() <= 1e-5


def test_combine_without_gate_weights():
    y = torch.randn(6, 8, requires_grad=True)
    dout = torch.randn(3, 8)
    training.combine_rows(y, ORDER, None).backward(dout)
    want = torch.zeros(6, 8)
    for t, j in ORDER.rows.ge(0).nonzero().tolist():
        want[ORDER.rows[t, j]] = dout[t]
    assert torch.equal(y.grad, want)


def test_a_bias_in_fp32_without_a_weight_keeps_its_gradients_bits():
    torch.manual_seed(3)
    x = torch.randn(7, 16).bfloat16()
    b = torch.zeros(16, requires_grad=True)
    dy = torch.randn(7, 16).bfloat16()
    training.layer_norm(x, None, b).backward(dy)
    assert torch.equal(b.grad, dy.float().sum(0))       # not rounded to x's type on its way


def _views():
    flat = torch.arange(3 + 4 * 64, dtype=torch.float32).bfloat16()
    wide = torch.randn(5, 67).bfloat16()
    return {"contiguous off a 16-byte boundary": flat[3:].view(4, 64), "one row of an odd stride": wide[:1, :64],
            "one row inside a row": wide[2:3, 3:67], "expanded": flat[:1].expand(4, 64), "transposed": torch.randn(64, 4).bfloat16().t(),
            "odd stride": wide[:, :64]}


@pytest.mark.parametrize("kind", _views())
def test_gradients_reach_the_operators_on_16_byte_boundaries(kind):
    t = _views()[kind]
    r = training._rows(t)
    assert torch.equal(r, t) or t.isnan().any()
    assert r.data_ptr() % 16 == 0 and r.stride(1) == 1 and r.stride(0) >= r.shape[1] and r.stride(0) * r.element_size() % 16 == 0


def test_gradients_that_fit_are_not_copied():
    t = torch.randn(4, 64).bfloat16()
    assert training._rows(t) is t


def test_rows_of_an_odd_width_are_not_copied():
    """No copy puts them on 16-byte boundaries, and what has such rows takes them as they are."""
    for t in (torch.randn(4, 33).bfloat16(), torch.arange(3 + 4 * 33).bfloat16()[3:].view(4, 33)):
        assert training._rows(t) is t


def test_gradients_of_frozen_parameters_are_not_asked_for(monkeypatch):
    seen = []
    for name in ("layer_norm_backward", "combine_rows_backward"):
        f = getattr(ops, name)
        monkeypatch.setattr(ops, name, lambda *a, _f=f, **k: (seen.append(k), _f(*a, **k))[1])
    x, g, b = torch.randn(3, 16, requires_grad=True), torch.randn(16), torch.randn(16, requires_grad=True)
    training.layer_norm(x, g, b).sum().backward()
    assert g.grad is None and b.grad is not None and not seen[0]["weight_grad"] and seen[0]["bias_grad"]
    y, w = torch.randn(6, 8, requires_grad=True), torch.rand(3, 2)
    training.combine_rows(y, ORDER, w).sum().backward()
    assert w.grad is None and not seen[1]["gate_grad"]
    training.combine_rows(y, ORDER, w.requires_grad_()).sum().backward()
    assert w.grad is not None and seen[2]["gate_grad"]
