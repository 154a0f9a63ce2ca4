"""Calls one after the other, each launched ahead of the one before and into memory that earlier ones had: the
same bits as with the GPU waited for after every call."""
import pytest
import torch

from combine_persistent_warp_gb300 import ops

pytestmark = pytest.mark.gpu


def _run(M, I, steps, wait, dtype):
    """A chain whose every buffer comes back from the allocator a call or two later, with other values."""
    sync = torch.cuda.synchronize if wait else (lambda: None)
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(M, 2 * I, generator=g, device="cuda").to(dtype)
    w = (1 + 0.1 * torch.randn(2 * I, generator=g, device="cuda")).to(dtype)
    E = 16
    seen = []

    def call(f, *a, **k):
        r = f(*a, **k)
        sync()
        return r

    for _ in range(steps):
        act, codes, scales = call(ops.swiglu_checkpoint, h)
        dgu, again = call(ops.swiglu_checkpoint_backward, act, codes, scales)
        y, rstd, s = call(ops.rms_norm, dgu, w, residual=h)
        dx, dw = call(ops.rms_norm_backward, dgu, s, w, rstd, dh=y)
        kept = call(ops.checkpoint_rows, dx)
        h = call(ops.restore_rows, *kept, dtype)
        idx, gate = call(ops.route_scores, h[:, :E], 4, groups=4, topk_groups=2)
        d = call(ops.route_scores_backward, gate, idx, gate, h[:, :E])
        h = call(ops.rms_norm, h, w)[0]
        seen += [again, dw, d, idx]
        del act, codes, scales, dgu, y, rstd, s, dx, kept, gate
    seen.append(h)
    torch.cuda.synchronize()
    return seen


@pytest.mark.parametrize("M,I,dtype", [(5, 64, torch.bfloat16), (700, 512, torch.bfloat16), (6000, 1024, torch.bfloat16), (3000, 333, torch.float32),
                                       (2000, 1003, torch.float16)])
def test_a_chain_of_calls_has_the_bits_of_calls_apart(M, I, dtype):
    apart = _run(M, I, 12, True, dtype)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(_run(M, I, 12, False, dtype), apart))


def test_a_captured_chain_has_the_bits_of_calls_apart():
    M, I, dtype = 900, 512, torch.bfloat16
    x, w = torch.randn(M, 2 * I, device="cuda").to(dtype), torch.ones(2 * I, device="cuda", dtype=dtype)

    def chain(v):
        for _ in range(6):
            act, codes, scales = ops.swiglu_checkpoint(v)
            dgu, _ = ops.swiglu_checkpoint_backward(act, codes, scales)
            v = ops.rms_norm(dgu, w, residual=v)[0]
            v = ops.restore_rows(*ops.checkpoint_rows(v), dtype)
        return v

    live = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(live)
    for i in range(5):
        live.copy_(x.roll(i, 0))
        graph.replay()
        assert torch.equal(out, chain(x.roll(i, 0)))


def test_two_streams_at_once():
    g = torch.Generator(device="cuda").manual_seed(3)
    x = [torch.randn(3000, 2048, generator=g, device="cuda").bfloat16() for _ in range(2)]
    w = torch.ones(2048, device="cuda").bfloat16()
    want = [ops.rms_norm(v, w, residual=v) for v in x]
    back = [ops.rms_norm_backward(v, o[2], w, o[1], dh=v) for v, o in zip(x, want)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    for _ in range(10):
        got = []
        for v, s in zip(x, streams):
            with torch.cuda.stream(s):
                o = ops.rms_norm(v, w, residual=v)
                got.append((o, ops.rms_norm_backward(v, o[2], w, o[1], dh=v)))
        torch.cuda.synchronize()
        for (o, b), p, q in zip(got, want, back):
            assert all(torch.equal(m, n) for m, n in zip(o, p)) and all(torch.equal(m, n) for m, n in zip(b, q))
