"""The experts' activation, its gradients, and rows in 8 bits, against 64-bit formulas.

Bounds, with u half a step of the output's type and e = 2^-24: the logistic function is (1.5 |g| + 8) e relative off (the
exponent's rounding and those of the instructions behind it), a product of it two or three roundings more, and
s + g s (1 - s) that of its two parts.  Below 2^-126 it may be zero.  The 8-bit form is exact: its codes, its scales and what they stand for.
"""
import pytest
import torch

from combine_persistent_warp_gb300 import ops

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _power(n):
    """2^n in 64 bits, from its exponent field (torch.ldexp multiplies by a 32-bit power)."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _kept(x):
    """(codes, scale bytes, values) of rows in the 8-bit format, in 64 bits."""
    M, H = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -H % 32)).view(M, -1, 32)
    big = v.abs().amax(2)
    bad = ~v.isfinite().all(2)
    _, exponent = torch.frexp(big.masked_fill(bad, 1.0))
    b = torch.where(big > 0, exponent.long() - 1 + 127, 0).clamp_min(7).masked_fill(bad, 255)
    step = _power((b - 133).masked_fill(bad, 0))
    n = (v / step[:, :, None]).round().clamp(-127, 127)
    value = torch.where(bad[:, :, None], float("nan"), n * step[:, :, None]).view(M, -1)[:, :H]
    return n.nan_to_num(0).to(torch.int8).view(M, -1)[:, :H], b.to(torch.uint8), value


def _same(a, b):
    return torch.equal(torch.nan_to_num(a, nan=12345.0), torch.nan_to_num(b, nan=12345.0)) and torch.equal(a.isnan(), b.isnan())


def _check_act(act, gu):
    g, u = gu.double().chunk(2, 1)
    ref = g * torch.sigmoid(g) * u
    bound = ((1.5 * g.abs() + 12) * E24 + U[act.dtype]) * ref.abs() + (1 + g.abs()) * (1 + u.abs()) * 2.0 ** -126 + TINY[act.dtype]
    assert ((act.double() - ref).abs() <= bound).all()


def _check_grad(dgu, da, gu):
    g, u = gu.double().chunk(2, 1)
    d, s = da.double(), torch.sigmoid(g)
    low = (1 + d.abs()) * (1 + g.abs()) * (1 + u.abs()) * 2.0 ** -125 + TINY[dgu.dtype]
    dg, du = dgu.double().chunk(2, 1)
    ref = d * u * s * (1 + g * (1 - s))
    assert ((dg - ref).abs() <= (d * u).abs() * s * (1 + g.abs()) * (1.5 * g.abs() + 20) * E24 + U[dgu.dtype] * ref.abs() + low).all()
    ref = d * g * s
    assert ((du - ref).abs() <= ((1.5 * g.abs() + 12) * E24 + U[dgu.dtype]) * ref.abs() + low).all()


def _inputs(M, I, dtype, seed=0, std=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (std * torch.randn(M, 2 * I, generator=g, device="cuda")).to(dtype), torch.randn(M, I, generator=g, device="cuda").to(dtype)


def _check_all(gu, da):
    I = da.shape[1]
    act = ops.swiglu(gu)
    _check_act(act, gu)
    _check_grad(ops.swiglu_backward(da, gu), da, gu)
    again, codes, scales = ops.swiglu_checkpoint(gu)
    assert torch.equal(act, again)
    cg, sg, vg = _kept(gu[:, :I])
    cu, su, vu = _kept(gu[:, I:])
    assert torch.equal(codes, torch.cat([cg, cu], 1)) and torch.equal(scales, torch.cat([sg, su], 1))
    dgu, act = ops.swiglu_checkpoint_backward(da, codes, scales)
    kept = torch.cat([vg, vu], 1)
    _check_act(act, kept)
    _check_grad(dgu, da, kept)


SIZES = [(1, 1), (1, 8), (3, 5), (2, 31), (2, 32), (5, 33), (4, 40), (7, 100), (300, 72), (9, 256), (9, 257), (5, 1000), (33, 1403), (130, 2048),
         (1024, 2048), (3, 4096), (2, 8200), (257, 136), (70, 1536)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,I", SIZES)
def test_activation_gradient_and_checkpoint(M, I, dtype):
    _check_all(*_inputs(M, I, dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_large_and_small_gates(dtype):
    gu, da = _inputs(40, 320, dtype, std=30.0)
    _check_all(gu, da)
    gu = gu * 2.0 ** -12
    _check_all(gu, da)
    gu = torch.zeros(6, 128, device="cuda", dtype=dtype)
    _check_all(gu, da[:6, :64])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("I,off,pitch", [(64, 0, 200), (64, 3, 131), (100, 1, 203), (256, 8, 528), (33, 0, 80)])
def test_strided_and_unaligned_rows(I, off, pitch, dtype):
    g0, d0 = _inputs(21, I, dtype)
    flat = torch.full((21 * pitch + off,), float("nan"), device="cuda", dtype=dtype)[off:]
    gu = flat.as_strided((21, 2 * I), (pitch, 1))
    gu.copy_(g0)
    flat = torch.full((21 * pitch + off,), float("nan"), device="cuda", dtype=dtype)[off:]
    da = flat.as_strided((21, I), (pitch, 1))
    da.copy_(d0)
    _check_all(gu, da)
    _check_all(gu[:1], da[:1])
    codes, scales = ops.checkpoint_rows(gu)
    want = _kept(gu)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,H", [(1, 1), (2, 8), (3, 31), (5, 32), (5, 33), (4, 72), (100, 200), (33, 257), (3, 7168), (500, 1500), (130, 4096), (70, 3001)])
def test_rows_in_8_bits(M, H, dtype):
    g = torch.Generator(device="cuda").manual_seed(M)
    x = (torch.randn(M, H, generator=g, device="cuda") * torch.exp(2 * torch.randn(M, 1, generator=g, device="cuda"))).to(dtype)
    x[:, ::7] *= 2.0 ** -9
    codes, scales = ops.checkpoint_rows(x)
    want = _kept(x)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    assert torch.equal(ops.restore_rows(codes, scales, dtype), want[2].to(dtype))
    # the next power of two above the largest is 64 to 128 steps of 1/64: half a step, one where 127.5 steps were cut
    v = torch.nn.functional.pad(x.double(), (0, -H % 32)).view(M, -1, 32)
    off = (torch.nn.functional.pad(want[2], (0, -H % 32)).view(M, -1, 32) - v).abs()
    assert (off <= v.abs().amax(2, keepdim=True) * 2.0 ** -6 + 2.0 ** -127).all()


def test_ties_clamps_and_extreme_groups():
    x = torch.zeros(8, 64, device="cuda")
    x[0, :4] = torch.tensor([1.0, 0.5 / 64, 1.5 / 64, 2.5 / 64])          # ties to even: 0, 2, 2
    x[1, :3] = torch.tensor([1.999, -1.999, 1.98])                        # past 127 steps
    x[2, 0] = 2.0 ** -126
    x[2, 1] = 2.0 ** -140
    x[3, 40] = 3.4e38
    x[3, 41] = -3.3e38
    x[4, 3], x[5, 33], x[6, 3] = float("nan"), float("inf"), -float("inf")
    x[4:7, 60] = 1.0
    codes, scales = ops.checkpoint_rows(x)
    want = _kept(x)
    fine = want[1] != 255
    assert torch.equal(scales, want[1])
    assert torch.equal(codes.view(8, 2, 32)[fine], want[0].view(8, 2, 32)[fine])
    assert codes[0, :4].tolist() == [64, 0, 2, 2] and codes[1, :3].tolist() == [127, -127, 127]
    for dtype in TYPES:
        assert _same(ops.restore_rows(codes, scales, dtype), want[2].to(dtype))


@pytest.mark.parametrize("H", [64, 61])
def test_every_byte_and_code_restores(H):
    codes = torch.arange(-128, 128, device="cuda").to(torch.int8).repeat(H)[:256 * H].view(256, H).contiguous()
    scales = torch.arange(256, device="cuda").to(torch.uint8)[:, None].repeat(1, 2).contiguous()
    want = codes.double() * _power(scales[:, :1].long() - 133)
    want[255] = float("nan")
    for dtype in TYPES:
        assert _same(ops.restore_rows(codes, scales, dtype), want.to(torch.float32).to(dtype))
    da = torch.ones(256, H, device="cuda")
    _, act = ops.swiglu_checkpoint_backward(da, codes.repeat(1, 2).contiguous(), scales.repeat(1, 2).contiguous())
    g = want[100:140]
    _check_act(act[100:140], torch.cat([g, g], 1))


def test_special_values_of_the_activation():
    gu = torch.tensor([[float("inf"), 0.0, float("nan"), 1.0, 100.0, -100.0, 1.0, 2.0]], device="cuda")    # gate, up: four each
    act = ops.swiglu(gu)
    assert act[0, 0] == float("inf") and act[0, 1] == 0 and act[0, 2].isnan() and act[0, 3] > 0
    rows, da = _inputs(300, 512, torch.bfloat16)
    clean = ops.swiglu_checkpoint(rows)
    rows[17, 600] = float("nan")
    act, codes, scales = ops.swiglu_checkpoint(rows)
    rest = torch.arange(300, device="cuda") != 17
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip((act, codes, scales), clean))
    dgu, again = ops.swiglu_checkpoint_backward(da, codes, scales)
    assert again[17, 88 - 24:88 + 8].isnan().all() and not again[rest].isnan().any() and not dgu[rest].isnan().any()


def test_gradient_against_differences():
    gu, da = _inputs(2, 9, torch.float32)
    got = ops.swiglu_backward(da, gu)
    f = lambda v: (torch.nn.functional.silu(v[:, :9]) * v[:, 9:] * da).sum()
    for i in range(18):
        d = torch.zeros(2, 18, dtype=torch.float64, device="cuda")
        d[1, i] = 1e-5
        # the differences are 1e-9 off, the gradient some ten roundings of terms of at most 30
        assert abs((f(gu.double() + d) - f(gu.double() - d)) / 2e-5 - got[1, i].double()) <= 1e-4


def test_streams_graphs_and_empty_batches():
    gu, da = _inputs(70, 264, torch.bfloat16)
    act, codes, scales = ops.swiglu_checkpoint(gu)
    dgu, again = ops.swiglu_checkpoint_backward(da, codes, scales)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a2, c2, s2 = ops.swiglu_checkpoint(gu, stream=s)
    d2, _ = ops.swiglu_checkpoint_backward(da, c2, s2, stream=s)
    r2 = ops.restore_rows(c2, s2[:, :0].new_full((70, 17), 130), torch.float32, stream=s)
    k2 = ops.checkpoint_rows(gu, stream=s)
    p2 = ops.swiglu_backward(da, gu, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a2, act) and torch.equal(d2, dgu) and torch.equal(r2, codes.float() * 0.125)
    assert all(torch.equal(a, b) for a, b in zip(k2, ops.checkpoint_rows(gu))) and torch.equal(p2, ops.swiglu_backward(da, gu))
    live = gu.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a3, c3, s3 = ops.swiglu_checkpoint(live)
        d3, g3 = ops.swiglu_checkpoint_backward(da, c3, s3)
        r3 = ops.restore_rows(*ops.checkpoint_rows(live), torch.bfloat16)
    g.replay()
    assert torch.equal(a3, act) and torch.equal(d3, dgu) and torch.equal(g3, again)
    live.copy_(gu.flip(0))
    g.replay()
    assert torch.equal(a3, act.flip(0)) and torch.equal(r3, ops.restore_rows(*ops.checkpoint_rows(gu), torch.bfloat16).flip(0))
    e, d = gu[:0], da[:0]
    act, codes, scales = ops.swiglu_checkpoint(e)
    assert act.shape == (0, 264) and codes.shape == (0, 528) and scales.shape == (0, 18)
    assert ops.swiglu(e).shape == (0, 264) and ops.swiglu_backward(d, e).shape == (0, 528)
    assert ops.swiglu_checkpoint_backward(d, codes, scales)[0].shape == (0, 528)
    assert ops.restore_rows(*ops.checkpoint_rows(e), torch.float16).shape == (0, 528)


@pytest.mark.parametrize("I", [8192, 8191])
def test_offsets_past_31_bits(I):
    M = 135000
    gu = torch.zeros(M, 2 * I, device="cuda", dtype=torch.bfloat16)
    tail, da = _inputs(3, I, torch.bfloat16)
    gu[-3:] = tail
    act, codes, scales = ops.swiglu_checkpoint(gu)
    _check_act(act[-3:], tail)
    want = torch.cat([_kept(tail[:, :I])[2], _kept(tail[:, I:])[2]], 1)
    act[-3:] = da
    dgu, again = ops.swiglu_checkpoint_backward(act, codes, scales)
    _check_grad(dgu[-3:], da, want)
    del dgu, again, act
    c, s = ops.checkpoint_rows(gu)
    assert torch.equal(ops.restore_rows(c, s, torch.bfloat16)[-3:], _kept(tail)[2].bfloat16())
