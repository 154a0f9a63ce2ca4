"""Rows into and out of expert order, with gradients, against 64-bit plain forms.

Bounds: a combined value is a sum of k fp32 products, (k + 1)*2^-24 * sum|w*y| off before the rounding u
of its type; a gate weight's gradient is an fp32 sum of H products, at most (H/32 + 16)*2^-24 of the
sum of magnitudes (a thread's run, then a tree); a row's gradient is one product, rounded once.
"""
import pytest
import torch

from combine_persistent_warp_gb300 import native, ops

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -10}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -24}


def _case(T, k, H, E, dtype, skip=0.1, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda")
    idx[torch.rand(T, k, generator=g, device="cuda") < skip] = -1
    o = ops.expert_order(idx, E)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return o, r(T, H).to(dtype), r(T * k, H).to(dtype), r(T, k).abs(), r(T, H).to(dtype)


SIZES = [(1, 1, 8, 1), (1, 8, 7168, 32), (3, 2, 5, 4), (17, 3, 1001, 5), (128, 8, 256, 8), (40, 32, 72, 64), (9, 9, 4104, 3),
         (300, 6, 640, 16)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,k,H,E", SIZES)
def test_gather(T, k, H, E, dtype):
    o, x, _, _, _ = _case(T, k, H, E, dtype)
    out = ops.gather_rows(x, o.rows, o.offsets)
    ref = torch.zeros_like(out)
    named = o.rows >= 0
    ref[o.rows[named].long()] = x[named.nonzero()[:, 0]]
    assert torch.equal(out, ref)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,k,H,E", SIZES)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_and_its_gradients(T, k, H, E, dtype, weighted):
    o, _, y, w, dout = _case(T, k, H, E, dtype)
    named = o.rows >= 0
    y[int(o.offsets[-1]):] = float("nan")             # rows of no slot are not read
    w[~named] = float("nan")                          # nor are skipped slots' weights
    w = w if weighted else None
    out = ops.combine_rows(y, o.rows, w)
    yr = torch.where(named[:, :, None], y[o.rows.clamp_min(0).long()].double(), 0.0)
    wr = torch.where(named, w.double() if weighted else 1.0, 0.0)
    terms = wr[:, :, None] * yr
    ref = terms.sum(1)
    assert ((out.double() - ref).abs() <= (k + 1) * E24 * terms.abs().sum(1) + U[dtype] * ref.abs() + TINY[dtype]).all()
    dy, dw = ops.combine_rows_backward(dout, y, o.rows, w, o.offsets)
    rdy = torch.zeros(T * k, H, dtype=torch.double, device="cuda")
    rdy[o.rows[named].long()] = (wr[:, :, None] * dout.double()[:, None, :])[named]
    assert ((dy.double() - rdy).abs() <= (U[dtype] + E24) * rdy.abs() + TINY[dtype]).all()
    prod = yr * dout.double()[:, None, :]
    assert ((dw.double() - prod.sum(2)).abs() <= (H / 32 + 16) * E24 * prod.abs().sum(2)).all()
    assert (dw[~named] == 0).all() and (dy[int(o.offsets[-1]):] == 0).all()


def test_gradients_against_differences():
    T, k, H, E, h = 7, 3, 40, 4, 1e-4
    o, x, y, w, dout = _case(T, k, H, E, torch.float32)
    named = (o.rows >= 0)[:, :, None]
    g = torch.Generator(device="cuda").manual_seed(4)

    def f(y, w):
        v = torch.where(named, y[o.rows.clamp_min(0).long()], 0.0)
        return ((v * w[:, :, None]).sum(1) * dout.double()).sum()

    dy, dw = ops.combine_rows_backward(dout, y, o.rows, w, o.offsets)
    vy = torch.randn(y.shape, generator=g, device="cuda", dtype=torch.double)
    vw = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.double)
    yd, wd = y.double(), w.double()
    for got, diff in (((dy.double() * vy).sum(), (f(yd + h * vy, wd) - f(yd - h * vy, wd)) / (2 * h)),
                      ((dw.double() * vw).sum(), (f(yd, wd + h * vw) - f(yd, wd - h * vw)) / (2 * h))):
        assert abs(got - diff) <= 1e-5 * (1 + abs(diff)) * 10
    # the gradient of gather is combine with unit weights: <gather(x), v> = <x, combine(v)>
    v = torch.randn(T * k, H, generator=g, device="cuda")
    left = (ops.gather_rows(x, o.rows, o.offsets).double() * v.double()).sum()
    right = (x.double() * ops.combine_rows(v, o.rows).double()).sum()
    assert abs(left - right) <= 1e-5 * (1 + abs(left)) * 10


def test_all_slots_skipped_and_empty_batches():
    rows = torch.full((6, 2), -1, dtype=torch.int32, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x = torch.full((6, 64), float("nan"), device="cuda")
    y = torch.full((12, 64), float("inf"), device="cuda")
    w = torch.ones(6, 2, device="cuda")
    assert (ops.gather_rows(x, rows, off) == 0).all()
    assert (ops.combine_rows(y, rows, w) == 0).all()
    dy, dw = ops.combine_rows_backward(x, y, rows, w, off)
    assert (dy == 0).all() and (dw == 0).all()
    e = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    assert ops.gather_rows(x[:0], e, off).shape == (0, 64)
    assert ops.combine_rows(y[:0], e).shape == (0, 64)
    assert ops.combine_rows_backward(x[:0], y[:0], e, None, off)[0].shape == (0, 64)


def test_rows_outside_the_tensor_are_left_out():
    rows = torch.tensor([[0, 5], [7, -3]], dtype=torch.int32, device="cuda")
    y = torch.arange(4.0, device="cuda")[:, None].repeat(1, 16) + 1
    assert torch.equal(ops.combine_rows(y, rows), torch.tensor([[1.0], [0.0]], device="cuda").repeat(1, 16))


def test_strided_inputs_and_another_stream():
    o, x, y, w, dout = _case(50, 4, 256, 8, torch.bfloat16)
    wide = torch.randn(50, 700, device="cuda").bfloat16()
    for at in (0, 8, 3):
        v = wide[:, at:at + 256]
        assert torch.equal(ops.gather_rows(v, o.rows, o.offsets), ops.gather_rows(v.contiguous(), o.rows, o.offsets))
        a = ops.combine_rows_backward(v, y, o.rows, w, o.offsets)
        b = ops.combine_rows_backward(v.contiguous(), y, o.rows, w, o.offsets)
        assert torch.equal(a[0], b[0]) and (a[1] - b[1]).abs().max() <= 1e-4
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ops.combine_rows(y, o.rows, w, stream=s)
    s.synchronize()
    assert torch.equal(got, ops.combine_rows(y, o.rows, w))


CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _inside(t, at, fill):
    """A copy of t, `at` elements into a buffer that holds `fill` before and after it."""
    b = torch.full((at + t.numel() + 16,), fill, dtype=t.dtype, device="cuda")
    v = b[at:at + t.numel()].view(t.shape)
    v.copy_(t)
    return v, b


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (1, 2, 9), (2, 1, 64), (3, 4, 31), (5, 3, 97), (4, 9, 513), (40, 4, 333), (7, 8, 775),
                                   (3, 2, 3001), (2500, 5, 775), (2500, 2, 1543)])
@pytest.mark.parametrize("at", [(1, 1, 1, 1), (0, 3, 0, 2), (5, 0, 6, 0)])
def test_rows_of_any_alignment(T, k, H, dtype, at):
    # every matrix between values that no result may hold, and every result between values that stay
    o, x, y, w, dout = _case(T, k, H, 4, dtype, seed=H)
    M = T * k
    named = o.rows >= 0
    y[int(o.offsets[-1]):] = float("nan")
    x = torch.cat([x, torch.full((T, 3), float("nan"), dtype=dtype, device="cuda")], 1)   # a stride of H + 3
    x = _inside(x, at[0], float("nan"))[0]
    d = _inside(torch.cat([dout, torch.full_like(x[:, :2], float("nan"))], 1), at[0], float("nan"))[0]
    y = _inside(y, at[1], float("nan"))[0]
    results = [_inside(torch.zeros(r, H, dtype=dtype, device="cuda"), at[i], 7.0) for r, i in ((M, 2), (T, 3), (M, 3))]
    (rows, rows_b), (out, out_b), (dy, dy_b) = results
    dw = torch.empty(T, k, device="cuda")
    lib, s, c = native.load(), torch.cuda.current_stream().cuda_stream, CODE[dtype]
    q = lambda t: t.data_ptr()
    assert lib.moe_gather_rows(T, k, H, 4, M, q(x), H + 3, c, q(o.rows), q(o.offsets), q(rows), s) == 0
    assert lib.moe_combine_rows(T, k, H, M, q(y), c, q(o.rows), q(w), q(out), s) == 0
    assert lib.moe_combine_rows_backward(T, k, H, 4, M, q(d), H + 2, q(y), c, q(o.rows), q(w), q(o.offsets), q(dy), q(dw), s) == 0
    torch.cuda.synchronize()
    for (v, b), i in zip(results, (2, 3, 3)):
        assert (b[:at[i]] == 7).all() and (b[at[i] + v.numel():] == 7).all()
    ref = torch.zeros_like(rows)
    ref[o.rows[named].long()] = x[:, :H][named.nonzero()[:, 0]]
    assert torch.equal(rows, ref)
    yr = torch.where(named[:, :, None], y[o.rows.clamp_min(0).long()].double(), 0.0)
    wr = torch.where(named, w.double(), 0.0)
    terms = wr[:, :, None] * yr
    assert ((out.double() - terms.sum(1)).abs() <= (k + 1) * E24 * terms.abs().sum(1) + U[dtype] * terms.sum(1).abs() + TINY[dtype]).all()
    d = dout.double()[:, None, :]
    rdy = torch.zeros(M, H, dtype=torch.double, device="cuda")
    rdy[o.rows[named].long()] = (wr[:, :, None] * d)[named]
    assert ((dy.double() - rdy).abs() <= (U[dtype] + E24) * rdy.abs() + TINY[dtype]).all()
    assert ((dw.double() - (yr * d).sum(2)).abs() <= (H / 32 + 16) * E24 * (yr * d).abs().sum(2)).all()


def test_offsets_past_32_bits():
    T, k, H = 37501, 8, 7168            # 2.15e9 elements in expert order
    x = torch.randn(T, H, device="cuda", dtype=torch.bfloat16)
    idx = torch.arange(k, device="cuda").repeat(T, 1)
    o = ops.expert_order(idx, k)
    rows = ops.gather_rows(x, o.rows, o.offsets)
    assert torch.equal(rows[-100:], x[-100:]) and torch.equal(rows[T * 7:T * 7 + 50], x[:50])
    w = torch.full((T, k), 0.125, device="cuda")
    assert torch.equal(ops.combine_rows(rows, o.rows, w), x)


def test_refusals_of_tensors():
    o, x, y, w, dout = _case(4, 2, 64, 3, torch.bfloat16)
    with pytest.raises(ValueError):
        ops.gather_rows(x[:3], o.rows, o.offsets)
    with pytest.raises(TypeError):
        ops.gather_rows(x, o.rows.long(), o.offsets)
    with pytest.raises(TypeError):
        ops.combine_rows(y, o.rows, w.half())
    with pytest.raises(ValueError):
        ops.combine_rows(y.t(), o.rows, w)
    with pytest.raises(TypeError):
        ops.combine_rows_backward(dout.float(), y, o.rows, w, o.offsets)
    with pytest.raises(ValueError):
        ops.combine_rows_backward(dout, y, o.rows, w[:, :1], o.offsets)
