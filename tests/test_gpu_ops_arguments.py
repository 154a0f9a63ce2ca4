"""What the operators' Python entry points take and refuse on the GPU."""
import threading
import time

import pytest
import torch

from combine_persistent_warp_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [0, 1])
def test_the_stride_of_a_single_row_may_be_anything(rows):
    torch.manual_seed(0)
    base = torch.randn(3, 67 * 128 + 3, device="cuda").bfloat16()
    x, dy = base[:rows, :256], base[1:1 + rows, 5:5 + 128].clone().as_strided((rows, 128), (131, 1))
    assert rows == 0 or x.stride(0) % 8 and dy.stride(0) % 8
    w = torch.randn(2, 128, 256, device="cuda").bfloat16()
    off = torch.tensor([0, 0, rows], dtype=torch.int32, device="cuda")
    plain = lambda t: t.clone(memory_format=torch.contiguous_format)
    assert torch.equal(ops.grouped_mm(x, w, off), ops.grouped_mm(plain(x), w, off))
    assert torch.equal(ops.grouped_mm_dx(dy, w, off), ops.grouped_mm_dx(plain(dy), w, off))
    assert torch.equal(ops.grouped_mm_dw(dy, x, off), ops.grouped_mm_dw(plain(dy), plain(x), off))
    out = torch.zeros(3, 131, device="cuda").bfloat16()[:rows, :128]
    assert torch.equal(ops.grouped_mm(x, w, off, out=out), ops.grouped_mm(plain(x), w, off))
    for a, b in zip(ops.layer_norm_fp8(x), ops.layer_norm_fp8(plain(x))):
        assert torch.equal(a, b)


def _products():
    torch.manual_seed(1)
    x, dy = torch.randn(6, 64, device="cuda").bfloat16(), torch.randn(6, 72, device="cuda").bfloat16()
    w = torch.randn(2, 72, 64, device="cuda").bfloat16()
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    return [(lambda out: ops.grouped_mm(x, w, off, out=out), (6, 72)), (lambda out: ops.grouped_mm_dx(dy, w, off, out=out), (6, 64)),
            (lambda out: ops.grouped_mm_dw(dy, x, off, out=out), (2, 72, 64)),
            (lambda out: ops.grouped_mm_dw(dy, x, off, out=out, accumulate=True), (2, 72, 64))]


@pytest.mark.parametrize("which", range(4))
def test_an_output_that_autograd_saved_and_a_call_overwrote_raises(which):
    call, shape = _products()[which]
    out = torch.ones(shape, device="cuda", dtype=torch.bfloat16)
    p = torch.ones(shape, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    z = (p * out).sum()                      # saves out
    v = out._version
    assert call(out) is out and out._version == v + 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()
    with torch.inference_mode():
        fresh = torch.ones(shape, device="cuda", dtype=torch.bfloat16)
        assert call(fresh) is fresh


def test_an_output_that_overlaps_an_input_is_refused():
    torch.manual_seed(2)
    bf = dict(device="cuda", dtype=torch.bfloat16)
    w = torch.randn(2, 64, 64, **bf)
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    x = torch.randn(6, 64, **bf)
    for f, name in ((ops.grouped_mm, "x"), (ops.grouped_mm_dx, "dy")):
        for out, what in ((x, name), (w[0, :6], "w")):
            with pytest.raises(ValueError, match=f"out overlaps {what}"):
                f(x, w, off, out=out)
    # rows of one buffer: apart, and one column in common
    wide = torch.randn(6, 136, **bf)
    part = wide[:, :64]
    want = ops.grouped_mm(part.clone(), w, off)
    assert torch.equal(ops.grouped_mm(part, w, off, out=wide[:, 72:]), want)
    assert torch.equal(part, wide[:, :64])
    with pytest.raises(ValueError, match="overlaps"):
        ops.grouped_mm(part, w, off, out=wide[:, 56:120])
    # of the same buffer at different strides: rows 0, 2, ... of it and rows 1, 3, ..., and all rows
    rows = torch.randn(12, 64, **bf)
    assert torch.equal(ops.grouped_mm(rows[::2], w, off, out=rows[1::2]), ops.grouped_mm(rows[::2].clone(), w, off))
    with pytest.raises(ValueError, match="overlaps"):
        ops.grouped_mm(rows[::2], w, off, out=rows[:6])
    both = torch.randn(13, 64, **bf)
    assert ops.grouped_mm(both[:6], w, off, out=both[6:12]) is not None
    buf = torch.randn(64 * 64, **bf)
    inside, apart, one = buf[:6 * 64].view(6, 64), torch.randn(6, 64, **bf), torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    for dy, x, what in ((inside, apart, "dy"), (apart, inside, "x")):
        with pytest.raises(ValueError, match=f"out overlaps {what}"):
            ops.grouped_mm_dw(dy, x, one, out=buf.view(1, 64, 64))


def test_other_threads_run_while_get_error_waits():
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.wait(0.005):
            ticks.append(time.monotonic())

    t = threading.Thread(target=tick)
    t.start()
    torch.cuda.synchronize()
    torch.cuda._sleep(1_000_000_000)         # about half a second of the stream
    start = time.monotonic()
    assert ops.get_error() == 0
    end = time.monotonic()
    stop.set()
    t.join()
    assert end - start > 0.2
    assert sum(start < x < end for x in ticks) >= 5


def test_numbers_past_31_bits_are_refused():
    logits = torch.zeros(4, 8, device="cuda")
    idx = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    for far in (1 << 32, -(1 << 32), -(1 << 40)):
        with pytest.raises(ValueError, match="31 bits"):
            ops.route_topk(logits, 2 + far)
        with pytest.raises(ValueError, match="31 bits"):
            ops.expert_order(idx, 8 + far)
