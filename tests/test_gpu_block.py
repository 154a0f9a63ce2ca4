"""A block with an RMS norm, scored routing and 8-bit checkpoints: its output and gradients against a plain
64-bit block, and its pieces against the operators one by one.

Tolerances: the block rounds to bf16 (u = 2^-8) after the norm, each product, the SwiGLU and the combine; a relative error
of the sums of a few such roundings stays below 8u of the whole tensor's norm, forward and (through twice as many
steps) 16u backward.  The 8-bit checkpoints add to the gradients: a step is at most 2^-6 of the largest of 32
values, about 2.5 of their deviation, and uniform errors of half a step at most have a deviation of 2^-6 * 2.5 / sqrt(12), 1.1% of
the values'; gate, up and the down products' rows in quadrature 2%, inside the 16u (6%) with the roundings' 2%.
"""
import os
import sys
import threading

import pytest
import torch

from combine_persistent_warp_gb300 import ops, training

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U16 = 2.0 ** -8


def _plain(block, x, residual, idx):
    """The block in 64 bits with the experts chosen as given; returns output and leaves."""
    p = {n: v.detach().double().requires_grad_() for n, v in block.named_parameters()}
    x = x.detach().double().requires_grad_()
    r = residual.detach().double().requires_grad_() if residual is not None else None
    s = x if r is None else x + r
    if block.norm == "rms":
        h = s * (s.square().mean(1, keepdim=True) + block.eps).rsqrt() * p["norm_weight"]
    else:
        c = s - s.mean(1, keepdim=True)
        h = c * (c.square().mean(1, keepdim=True) + block.eps).rsqrt() * p["norm_weight"] + p["norm_bias"]
    logits = h @ p["router"].t()
    if block.routing is None:
        w = torch.softmax(logits.gather(1, idx.clamp_min(0)), 1)
    else:
        score = torch.sigmoid(logits) if block.routing["score"] == "sigmoid" else torch.softmax(logits, 1)
        w = score.gather(1, idx.clamp_min(0))
        w = block.routing["scale"] * (w / w.sum(1, keepdim=True) if block.routing["renormalize"] else w)
    out = s
    for e in range(block.E):
        gu = h @ p["w_gate_up"][e].t()
        y = (torch.nn.functional.silu(gu[:, :block.I]) * gu[:, block.I:]) @ p["w_down"][e].t()
        out = out + ((idx == e) * w).sum(1, keepdim=True) * y
    return out, x, r, p


FORMS = {"rms": dict(norm="rms"), "checkpoint": dict(checkpoint=True),
         "sigmoid groups": dict(score="sigmoid", groups=4, topk_groups=2, scale=2.5, balance=True),
         "softmax": dict(score="softmax", renormalize=False, norm="rms"),
         "all": dict(norm="rms", score="sigmoid", groups=4, topk_groups=3, balance=True, checkpoint=True)}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,E,H,I,topk,masked", [(1, 4, 64, 64, 2, False), (300, 8, 256, 128, 2, False), (257, 12, 136, 72, 3, True)])
def test_block_against_a_plain_one(T, E, H, I, topk, masked, form, monkeypatch):
    torch.manual_seed(1)
    block = training.MoEBlock(E, H, I, topk, std=0.1, **FORMS[form]).cuda()
    if block.balance_bias is not None:
        block.balance_bias += 0.01 * torch.randn(E, device="cuda")
    x = torch.randn(T, H, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    r = torch.randn(T, H, device="cuda", dtype=torch.bfloat16, requires_grad=True) if block.norm == "rms" else None
    mask = (torch.rand(T, device="cuda") < 0.7) if masked else None
    call = (lambda: block(x, mask)) if r is None else (lambda: block(x, mask, residual=r))
    seen = []
    keep = ops.expert_order
    monkeypatch.setattr(ops, "expert_order", lambda idx, E, **k: (seen.append(idx), keep(idx, E, **k))[1])
    out = call()
    assert torch.equal(call(), out)          # the same bits again
    with torch.no_grad():
        assert torch.equal(call(), out)
    idx = seen[0]
    if masked:
        assert (idx[~mask] == -1).all()
        assert torch.equal(out[~mask], x[~mask] if r is None else (x + r)[~mask])
    if block.load is not None:
        assert block.load.sum().item() == 3 * (idx >= 0).sum().item()
    ref, rx, rr, rp = _plain(block, x, r, idx)
    d = torch.randn_like(out)
    out.backward(d)
    ref.backward(d.double())
    rel = lambda a, b: ((a.double() - b).norm() / b.norm().clamp_min(1e-30)).item()
    assert rel(out, ref) <= 8 * U16
    assert rel(x.grad, rx.grad) <= 16 * U16
    if r is not None:
        assert torch.equal(r.grad, x.grad)
    for n, v in block.named_parameters():
        assert rel(v.grad, rp[n].grad) <= 16 * U16, n
    assert ops.get_error() == 0


def test_experts_are_the_operators_one_by_one():
    torch.manual_seed(2)
    T, E, H, I, k = 120, 5, 128, 72, 3
    h = torch.randn(T, H, device="cuda").bfloat16().requires_grad_()
    gu_w = (0.1 * torch.randn(E, 2 * I, H, device="cuda")).bfloat16().requires_grad_()
    down = (0.1 * torch.randn(E, H, I, device="cuda")).bfloat16().requires_grad_()
    idx, w = ops.route_scores(torch.randn(T, E, device="cuda"), k)
    idx[::7, 1] = -1
    order = ops.expert_order(idx, E)
    w.requires_grad_()
    d = torch.randn(T, H, device="cuda").bfloat16()
    out = training.experts(h, order, w, gu_w, down)
    out.backward(d)
    with torch.no_grad():
        rows = ops.gather_rows(h, order.rows, order.offsets)
        gu = ops.grouped_mm(rows, gu_w, order.offsets)
        act, codes, scales = ops.swiglu_checkpoint(gu)
        y = ops.grouped_mm(act, down, order.offsets)
        assert torch.equal(out, ops.combine_rows(y, order.rows, w))
        dy, dw = ops.combine_rows_backward(d, ops.restore_rows(*ops.checkpoint_rows(y), torch.bfloat16), order.rows, w, order.offsets)
        dgu, again = ops.swiglu_checkpoint_backward(ops.grouped_mm_dx(dy, down, order.offsets), codes, scales)
        assert torch.equal(w.grad, dw) and torch.equal(down.grad, ops.grouped_mm_dw(dy, again, order.offsets))
        assert torch.equal(gu_w.grad, ops.grouped_mm_dw(dgu, rows, order.offsets))
        assert torch.equal(h.grad, ops.combine_rows(ops.grouped_mm_dx(dgu, gu_w, order.offsets), order.rows))


def test_checkpoints_hold_less_memory():
    torch.manual_seed(3)
    sizes = {}
    for checkpoint in (False, True):
        block = training.MoEBlock(4, 1024, 1024, 2, score="sigmoid", checkpoint=checkpoint).cuda()
        x = torch.randn(4096, 1024, device="cuda", dtype=torch.bfloat16, requires_grad=True)
        block(x).sum().backward()
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        out = block(x)
        sizes[checkpoint] = torch.cuda.memory_allocated() - before
        del out
    rows, I, H = 8192, 1024, 1024
    # kept anyway: the output, h, x; of the rows, in bytes: 2 H gathered, 4 I gate and up, 2 I each of silu, the product and
    # the down products' 2 H, against 2 I + H codes and a byte for 32 of them
    saved = rows * (2 * H + 4 * I + 4 * I + 2 * H - (2 * I + H) * 33 / 32)
    assert sizes[False] - sizes[True] >= 0.95 * saved


@pytest.mark.parametrize("held", [float("nan"), float("inf"), 1e30])
def test_what_unrouted_tokens_hold_reaches_no_gradient(held):
    torch.manual_seed(6)
    block = training.MoEBlock(4, 64, 64, 2, std=0.1, **dict(FORMS["all"], groups=2, topk_groups=1)).cuda()
    x, r = torch.randn(50, 64, device="cuda").bfloat16(), torch.randn(50, 64, device="cuda").bfloat16()
    mask = torch.arange(50, device="cuda") % 3 != 0
    want = {}
    for fill in (1.0, held):
        v, u = (torch.where(mask[:, None], t, fill).requires_grad_() for t in (x, r))
        block.zero_grad()
        out = block(v, mask, residual=u)
        out[mask].float().square().mean().backward()
        got = dict({n: p.grad.clone() for n, p in block.named_parameters()}, x=v.grad, r=u.grad, out=out[mask].detach())
        assert all(t.isfinite().all() for t in got.values()) and not v.grad[~mask].any() and not u.grad[~mask].any()
        want = want or got
    for n, t in want.items():
        assert torch.equal(t, got[n]), n


def test_backward_in_a_graph():
    """A whole step, captured (its warm-up on the capture's own stream) and replayed on other inputs."""
    torch.manual_seed(7)
    block = training.MoEBlock(4, 64, 64, 2, std=0.1, **dict(FORMS["all"], groups=2, topk_groups=1)).cuda()
    x, d = torch.randn(80, 64, device="cuda").bfloat16(), torch.randn(80, 64, device="cuda").bfloat16()

    def step(v):
        block.zero_grad(set_to_none=True)
        out = block(v, residual=d)
        out.backward(d)
        return out.detach()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step(x)
    torch.cuda.current_stream().wait_stream(s)
    live = x.clone()
    block.zero_grad(set_to_none=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = step(live)
    grads = {n: p.grad for n, p in block.named_parameters()}
    live.copy_(x.flip(0))
    g.replay()
    torch.cuda.synchronize()
    got = dict({n: t.clone() for n, t in grads.items()}, out=out.clone())
    want = dict(out=step(x.flip(0)), **{n: p.grad for n, p in block.named_parameters()})
    for n, t in want.items():
        assert torch.equal(t, got[n]), n


def test_serving_through_the_fused_layer():
    torch.manual_seed(8)
    block = training.MoEBlock(8, 256, 128, 2, std=0.05, **FORMS["all"]).cuda()
    x, r = torch.randn(64, 256, device="cuda").bfloat16(), torch.randn(64, 256, device="cuda").bfloat16()
    layer = block.serving_layer(64)
    got = block.serve(layer, x, residual=r)
    with torch.no_grad():
        block.eval()
        full = block(x, residual=r)
    base = (x + r).float()
    # FP8 (e4m3) operands carry 2^-4 relative steps: about 3% a tensor, three tensors deep
    assert ((got.float() - full.float()).norm() / (full.float() - base).norm()).item() < 0.15
    assert layer.get_error() == 0 and ops.get_error() == 0
    layer.close()


def test_example_trains_and_serves():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_moe_block as ex
    block, first, last = ex.train(steps=10, tokens=512, **ex.SCORES)
    assert first == first and last == last
    assert all(p.grad is not None and p.grad.isfinite().all() for p in block.parameters())
    assert block.balance_bias.any()
    assert ex.serve(block, tokens=256) < 0.15     # (FP8 operands, as above)


def test_empty_batch():
    block = training.MoEBlock(4, 64, 64, 2, std=0.1, **dict(FORMS["all"], groups=2, topk_groups=1)).cuda()
    x, r = (torch.randn(0, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True) for _ in range(2))
    for mask in (None, torch.ones(0, dtype=torch.bool, device="cuda")):
        out = block(x, mask, residual=r)
        assert out.shape == (0, 64)
        out.sum().backward()
    assert x.grad.shape == r.grad.shape == (0, 64) and not block.load.any()
    assert all(p.grad is not None and not p.grad.any() for p in block.parameters())


def test_two_threads_on_their_own_streams():
    """Steps of two blocks side by side give the bits that each gives alone."""
    torch.manual_seed(10)
    blocks = [training.MoEBlock(8, 256, 136, 2, std=0.1, **dict(FORMS["all"], topk_groups=2)).cuda() for _ in range(2)]
    data = [(torch.randn(T, 256, device="cuda").bfloat16(), torch.randn(T, 256, device="cuda").bfloat16()) for T in (300, 1111)]

    def step(i):
        x, r = (t.clone().requires_grad_() for t in data[i])
        blocks[i].zero_grad(set_to_none=True)
        out = blocks[i](x, residual=r)
        out.backward(data[i][1])
        return [out.detach(), x.grad, *(p.grad for p in blocks[i].parameters())]

    alone = [step(i) for i in range(2)]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got = step(i)
                    torch.cuda.current_stream().synchronize()
                    wrong.extend((i, n) for n, (a, b) in enumerate(zip(got, alone[i])) if not torch.equal(a, b))
        except Exception as e:
            wrong.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
