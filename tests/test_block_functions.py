"""The autograd functions of a block with an RMS norm, scored routing and 8-bit checkpoints, around stand-ins of
the operators on the CPU: which gradients they return, and what they hand to the operators."""
import pytest
import torch

from combine_persistent_warp_gb300 import ops, training


def _rms_norm(x, weight=None, eps=1e-6, *, residual=None):
    h = x if residual is None else x + residual
    rstd = (h.square().mean(1) + eps).rsqrt()
    y = h * rstd[:, None]
    return (y if weight is None else y * weight), rstd, h


def _rms_norm_backward(dy, h, weight, rstd, *, dh=None, param_dtype=None, weight_grad=True):
    xh = h * rstd[:, None]
    a = dy if weight is None else dy * weight
    dx = (a - xh * (a * xh).mean(1, keepdim=True)) * rstd[:, None]
    return dx if dh is None else dx + dh, (dy * xh).sum(0) if weight_grad else None


def _swiglu(gu):
    g, u = gu.chunk(2, 1)
    return g * torch.sigmoid(g) * u


def _swiglu_backward(dact, gu):
    g, u = gu.chunk(2, 1)
    s = torch.sigmoid(g)
    return torch.cat([dact * u * (s + g * s * (1 - s)), dact * g * s], 1)


def _checkpoint_rows(x):
    return x.clone(), torch.zeros(len(x), 1)


def _grouped(x, w, offsets):
    return torch.cat([x[a:b] @ w[e].t() for e, (a, b) in enumerate(zip(offsets[:-1], offsets[1:]))])


STAND_INS = dict(
    rms_norm=_rms_norm, rms_norm_backward=_rms_norm_backward, swiglu=_swiglu, swiglu_backward=_swiglu_backward,
    swiglu_checkpoint=lambda gu: (_swiglu(gu), *_checkpoint_rows(gu)),
    swiglu_checkpoint_backward=lambda dact, codes, scales: (_swiglu_backward(dact, codes), _swiglu(codes)),
    checkpoint_rows=_checkpoint_rows, restore_rows=lambda codes, scales, dtype: codes.to(dtype),
    gather_rows=lambda x, rows, offsets: torch.zeros(rows.numel(), x.shape[1]).index_copy_(
        0, rows.reshape(-1).long(), x.repeat_interleave(rows.shape[1], 0)),
    combine_rows=lambda y, rows, w=None: (y[rows.long()] * (1.0 if w is None else w[:, :, None])).sum(1),
    grouped_mm=_grouped, grouped_mm_dx=lambda dy, w, offsets: _grouped(dy, w.transpose(1, 2), offsets),
    grouped_mm_dw=lambda dy, x, offsets: torch.stack([dy[a:b].t() @ x[a:b] for a, b in zip(offsets[:-1], offsets[1:])]))


def _combine_rows_backward(dout, y, rows, w, offsets, *, gate_grad=True):
    dy = torch.zeros_like(y)
    dy[rows.long()] = (torch.ones(rows.shape) if w is None else w)[:, :, None] * dout[:, None]
    return dy, (y[rows.long()] * dout[:, None]).sum(2) if gate_grad else None


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    for name, f in STAND_INS.items():
        monkeypatch.setattr(ops, name, f)
    monkeypatch.setattr(ops, "combine_rows_backward", _combine_rows_backward)


ORDER = ops.ExpertOrder(torch.tensor([0, 2, 6], dtype=torch.int32), torch.tensor([[0, 2], [1, 5], [3, 4]], dtype=torch.int32),
                        torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("use", ["both", "norm", "sum"])
def test_the_sum_and_the_norm_have_their_gradients(use):
    torch.manual_seed(0)
    x, r, g = (torch.randn(5, 16, requires_grad=True) for _ in range(3))
    w = torch.randn(16, requires_grad=True)
    d, e = torch.randn(5, 16), torch.randn(5, 16)

    def loss(y, h):
        return (0.0 if use == "sum" else (y * d).sum()) + (0.0 if use == "norm" else (h * e).sum())

    loss(*training.rms_norm(x, w, residual=r)).backward()
    got = [t.grad for t in (x, r, w)]
    for t in (x, r, w):
        t.grad = None
    h = x + r
    loss(h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w, h).backward()
    for a, t in zip(got, (x, r, w)):
        assert (a is None and use == "sum") or (a - t.grad).abs().max() <= 1e-5


def test_norm_without_a_residual_gives_its_input_back():
    x, w = torch.randn(3, 8, requires_grad=True), torch.ones(8)
    y, h = training.rms_norm(x, w)
    assert h is x
    (y + h).sum().backward()
    want = torch.autograd.grad((_rms_norm(x, w)[0] + x).sum(), x)[0]
    assert (x.grad - want).abs().max() <= 1e-6 and w.grad is None


@pytest.mark.parametrize("checkpoint", [False, True])
def test_swiglu_keeps_what_it_is_asked_to(checkpoint, monkeypatch):
    asked = []
    for name in ("swiglu", "swiglu_checkpoint"):
        monkeypatch.setattr(ops, name, lambda gu, _f=getattr(ops, name), _n=name: (asked.append(_n), _f(gu))[1])
    gu, d = torch.randn(4, 10, requires_grad=True), torch.randn(4, 5)
    training.swiglu(gu, checkpoint).backward(d)
    assert (gu.grad - torch.autograd.grad((_swiglu(gu) * d).sum(), gu)[0]).abs().max() <= 1e-6
    with torch.no_grad():
        training.swiglu(gu, checkpoint)
    assert asked == ["swiglu_checkpoint" if checkpoint else "swiglu", "swiglu"]


@pytest.mark.parametrize("frozen", [(), ("h",), ("w",), ("gu", "down"), ("h", "gu"), ("h", "gu", "down")])
def test_experts_gradients(frozen):
    torch.manual_seed(1)
    t = dict(h=torch.randn(3, 8), w=torch.rand(3, 2), gu=torch.randn(2, 12, 8), down=torch.randn(2, 8, 6))
    for n, v in t.items():
        v.requires_grad_(n not in frozen)
    d = torch.randn(3, 8)
    training.experts(t["h"], ORDER, t["w"], t["gu"], t["down"]).backward(d)
    rows = torch.zeros(6, 8).index_copy(0, ORDER.rows.reshape(-1).long(), t["h"].repeat_interleave(2, 0))
    y = _grouped(_swiglu(_grouped(rows, t["gu"], ORDER.offsets)), t["down"], ORDER.offsets)
    want = torch.autograd.grad(((y[ORDER.rows.long()] * t["w"][:, :, None]).sum(1) * d).sum(), [v for n, v in t.items() if n not in frozen])
    for (n, v), g in zip([(n, v) for n, v in t.items() if n not in frozen], want):
        assert (v.grad - g).abs().max() <= 1e-4, n
    assert all(t[n].grad is None for n in frozen)
    with torch.no_grad():
        assert torch.equal(training.experts(t["h"], ORDER, t["w"], t["gu"], t["down"]), (y[ORDER.rows.long()] * t["w"][:, :, None]).sum(1))


def test_block_arguments():
    with pytest.raises(ValueError, match="norm"):
        training.MoEBlock(2, 8, 8, 1, norm="batch")
    with pytest.raises(ValueError, match="score"):
        training.MoEBlock(2, 8, 8, 1, groups=2)
    with pytest.raises(ValueError, match="balance"):
        training.MoEBlock(2, 8, 8, 1).update_balance()
    with pytest.raises(ValueError, match="residual"):
        training.MoEBlock(2, 8, 8, 1)(torch.zeros(1, 8), residual=torch.zeros(1, 8))
    plain = training.MoEBlock(2, 8, 8, 1)
    assert set(plain.state_dict()) == {"norm_weight", "norm_bias", "router", "w_gate_up", "w_down"}
    block = training.MoEBlock(2, 8, 8, 1, norm="rms", score="sigmoid", balance=True)
    assert set(block.state_dict()) == {"norm_weight", "router", "w_gate_up", "w_down", "balance_bias"}


def test_balance_moves_against_the_loads():
    block = training.MoEBlock(4, 8, 8, 1, score="sigmoid", balance=True)
    block.load += torch.tensor([10, 0, 5, 5])
    block.update_balance(0.5)
    assert block.balance_bias.tolist() == [-0.5, 0.5, 0.0, 0.0] and not block.load.any()


def test_a_change_of_type_leaves_the_biases_as_they_are():
    block = training.MoEBlock(4, 32, 32, 2, score="sigmoid", balance=True)
    block.balance_bias += torch.tensor([1.001, -0.002, 0.0, 1e-9])
    kept = block.balance_bias.clone()
    for change in (lambda: block.half(), lambda: block.to(torch.bfloat16), lambda: block.float().bfloat16(), lambda: block.to("cpu")):
        change()
        assert block.balance_bias.dtype == torch.float32 and torch.equal(block.balance_bias, kept)
        assert block.load.dtype == torch.int64 and block.balance_bias is dict(block.named_buffers())["balance_bias"]
    assert block.router.dtype == torch.bfloat16
    assert torch.equal(block.state_dict()["balance_bias"], kept)
    training.MoEBlock(4, 32, 32, 2).half()


@pytest.mark.parametrize("options", [dict(topk_groups=1), dict(group_top=1), dict(groups=2), dict(renormalize=False), dict(scale=2.0), dict(balance=True)])
def test_options_of_the_scores_need_them(options):
    with pytest.raises(ValueError, match="need a score"):
        training.MoEBlock(4, 32, 32, 2, **options)
