"""Layer norm, its FP8 form and its gradients against 64-bit formulas.

Bounds.  With u the unit roundoff of the output's type and e = 2^-24, sums of H terms in fp32 by
threads and a tree are at most c*e*sum|.| off, c = 64 (up to 32 terms a thread, 10 tree levels, the
roundings around them).  So mean is off by c*e*mean|x|, a centred value by that plus e|x|, rstd by
2c*e relative, and every output by its own rounding u|y| on top; sums over T rows by
(c + rows a block + 64)*e*sum|.|.
"""
import pytest
import torch

from combine_persistent_warp_gb300 import ops

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -10}
TINY16 = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -24}


def _inputs(T, H, dtype, wdtype, seed=0, mean=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return ((r(T, H) + mean).to(dtype), (1 + 0.1 * r(H)).to(wdtype), (0.1 * r(H)).to(wdtype), r(T, H).to(dtype))


def _ref(x, g, b, eps=1e-5):
    x = x.double()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = (c.square().mean(1) + eps).rsqrt()
    xh = c * rstd[:, None]
    y = xh
    if g is not None:
        y = y * g.double()
    if b is not None:
        y = y + b.double()
    # bounds of mean, xh and y before the last rounding
    em = 64 * E24 * x.abs().mean(1)
    exh = rstd[:, None] * (em[:, None] + 2 * E24 * x.abs()) + 130 * E24 * xh.abs()
    return y, mean, rstd, xh, em, exh


def _check_forward(x, g, b, got, eps=1e-5):
    y, mean, rstd = got
    ry, rm, rr, xh, em, exh = _ref(x, g, b, eps)
    gain = 1.0 if g is None else g.double().abs()
    assert ((mean.double() - rm).abs() <= em + 1e-30).all()
    # rstd: half the relative error of the variance, whose centred values carry the mean's error
    assert ((rstd.double() - rr).abs() <= rr * (130 * E24 + (em * rr).square() + 1e-30)).all()
    bound = exh * gain + 4 * E24 * (ry.abs() + 1) + U[y.dtype] * ry.abs() + TINY16[y.dtype]
    assert ((y.double() - ry).abs() <= bound).all()


CASES = [(1, 1), (1, 8), (3, 5), (2, 32), (7, 100), (5, 1000), (9, 1001), (4, 1024), (3, 2056), (130, 4096), (700, 1024),
         (2, 4097), (3, 7168), (1, 8191), (2, 8192), (2, 16384), (2, 16383), (1300, 264)]


@pytest.mark.parametrize("dtype,wdtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                          (torch.float32, torch.float32), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("T,H", CASES)
def test_forward(T, H, dtype, wdtype):
    x, g, b, _ = _inputs(T, H, dtype, wdtype)
    _check_forward(x, g, b, ops.layer_norm(x, g, b))


def test_forward_without_weight_or_bias_and_other_eps():
    x, g, b, _ = _inputs(33, 520, torch.bfloat16, torch.bfloat16)
    _check_forward(x, None, None, ops.layer_norm(x))
    _check_forward(x, g, None, ops.layer_norm(x, g, eps=0.5), eps=0.5)
    _check_forward(x, None, b, ops.layer_norm(x, None, b, eps=1e-2), eps=1e-2)


@pytest.mark.parametrize("H,off,pitch", [(512, 0, 1536), (512, 3, 1539), (1000, 8, 1016), (333, 1, 400)])
def test_strided_and_unaligned_rows(H, off, pitch):
    big, g, b, _ = _inputs(21, pitch, torch.bfloat16, torch.bfloat16)
    x = big[:, off:off + H]
    _check_forward(x, g[:H], b[:H], ops.layer_norm(x, g[:H].clone(), b[:H].clone()))
    _check_backward(x, g[:H].clone(), big.flip(0)[:, off:off + H])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H,off,pitch", [(1, 2049, 1, 2050), (3, 2049, 1, 2051), (700, 1500, 3, 1503), (5, 1025, 5, 1030), (2, 9001, 7, 9009),
                                           (4, 1030, 0, 1030), (3, 3000, 2, 3003)])
def test_long_unaligned_rows(T, H, off, pitch, dtype):
    """Rows that start before, on and after 16-byte boundaries, at both ends of the allocation."""
    flat = torch.randn(T * pitch + off, device="cuda").to(dtype)[off:].clone() if off == 0 else torch.randn(T * pitch + off, device="cuda").to(dtype)[off:]
    x = flat.as_strided((T, H), (pitch, 1))
    _, g, b, dy = _inputs(T, H, dtype, dtype)
    _check_forward(x, g, b, ops.layer_norm(x, g, b))
    _check_backward(x, g, dy)


@pytest.mark.parametrize("T,H", [(3042, 5888), (1300, 6016), (2500, 2952), (2500, 3064), (1300, 12288), (700, 4104)])
def test_every_block_size_of_the_persistent_kernels_launches(T, H):
    """Hidden sizes whose rings of rows take 48 KB of shared memory, a little less and more."""
    x, g, b, dy = _inputs(T, H, torch.bfloat16, torch.bfloat16)
    _check_forward(x, g, b, ops.layer_norm(x, g, b))
    _check_backward(x, g, dy)
    if H % 128 == 0:
        q, sf = ops.layer_norm_fp8(x, g, b)
        assert sf.isfinite().all() and (q.view(torch.float8_e4m3fn).float().abs().amax(1) <= 448).all()


@pytest.mark.parametrize("dtype,wdtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32), (torch.float32, torch.float32)])
@pytest.mark.parametrize("T,H,pitch,woff", [(5003, 1025, 1025, 0), (4901, 1031, 1039, 1), (2500, 2895, 2903, 3), (1300, 4091, 4091, 0),
                                            (1300, 8185, 8185, 5), (1250, 5004, 5012, 2), (3100, 2048, 2048, 1), (2500, 2003, 2006, 0)])
def test_long_batches_of_rows_off_the_boundaries(T, H, pitch, woff, dtype, wdtype):
    """Rows that lie alike in every tensor, and (the last) that do not; what lies between the rows and
    after the last one is NaN, and one row in the middle is: no other row may show it."""
    flat = torch.full((T * pitch,), float("nan"), device="cuda", dtype=dtype)
    x = flat.as_strided((T, H), (pitch, 1))
    v, g, b, dy = _inputs(T, H, dtype, wdtype)
    x.copy_(v)
    off = lambda t: torch.cat([t[:woff], t])[woff:]        # a vector that starts `woff` elements into its allocation
    g, b = off(g), off(b)
    _check_forward(x, g, b, ops.layer_norm(x, g, b))
    _check_backward(x, g, dy)
    clean = ops.layer_norm(x, g, b)
    dx = ops.layer_norm_backward(dy, x, g, clean[1], clean[2])[0]
    x[T // 2] = float("nan")
    y, mean, rstd = ops.layer_norm(x, g, b)
    rest = torch.arange(T, device="cuda") != T // 2
    assert y[T // 2].isnan().all() and torch.equal(y[rest], clean[0][rest]) and torch.equal(rstd[rest], clean[2][rest])
    assert torch.equal(ops.layer_norm_backward(dy, x, g, mean, rstd)[0][rest], dx[rest])


def test_large_mean_keeps_the_variance():
    x, g, b, _ = _inputs(16, 4096, torch.float32, torch.float32, mean=1000.0)
    y, _, _ = ops.layer_norm(x, g, b)
    ry = _ref(x, g, b)[0]
    # one rounding of a centred value of 1 beside a mean of 1000: 1000 * e; a one-pass variance loses 1e6 * e
    assert (y.double() - ry).abs().max() <= 64 * 1000 * E24 * 2


def test_constant_rows_and_special_values():
    x = torch.full((4, 1024), 3.0, device="cuda", dtype=torch.bfloat16)
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    y, mean, rstd = ops.layer_norm(x)
    assert (y[0] == 0).all() and (y[3] == 0).all() and mean[0] == 3.0
    assert y[1].isnan().all() and y[2].isnan().any()
    q, sf = ops.layer_norm_fp8(x)
    assert (q[0] == 0).all() and torch.equal(sf[0], torch.full_like(sf[0], 1e-4) / 448)
    assert (q[1].view(torch.float8_e4m3fn).float().isnan()).all()


def _check_backward(x, g, dy, param_dtype=None):
    y, mean, rstd = ops.layer_norm(x, g)
    dx, dg, db = ops.layer_norm_backward(dy, x, g, mean, rstd, param_dtype=param_dtype)
    _, _, rr, xh, _, exh = _ref(x, g, None)
    d = dy.double()
    a = d if g is None else d * g.double()
    m1, m2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    rdx = rr[:, None] * (a - m1 - xh * m2)
    T = x.shape[0]
    e_m1 = 64 * E24 * a.abs().mean(1, keepdim=True)
    e_m2 = 66 * E24 * (a * xh).abs().mean(1, keepdim=True) + (a.abs() * exh).mean(1, keepdim=True)
    e = rr[:, None] * (4 * E24 * (a.abs() + m1.abs() + (xh * m2).abs()) + e_m1 + xh.abs() * e_m2 + exh * m2.abs()) + 140 * E24 * rdx.abs()
    assert ((dx.double() - rdx).abs() <= e + U[dx.dtype] * rdx.abs() + TINY16[dx.dtype]).all()
    rdg, rdb = (d * xh).sum(0), d.sum(0)
    n = (128 + T / 152 + 64) * E24
    assert ((dg.double() - rdg).abs() <= n * (d * xh).abs().sum(0) + (d.abs() * exh).sum(0) + U[dg.dtype] * rdg.abs() + TINY16[dg.dtype]).all()
    assert ((db.double() - rdb).abs() <= n * d.abs().sum(0) + U[db.dtype] * rdb.abs() + TINY16[db.dtype]).all()
    assert dx.dtype == x.dtype and dg.dtype == db.dtype


@pytest.mark.parametrize("dtype,wdtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32),
                                          (torch.float32, torch.float32)])
@pytest.mark.parametrize("T,H", CASES)
def test_backward(T, H, dtype, wdtype):
    x, g, _, dy = _inputs(T, H, dtype, wdtype)
    _check_backward(x, g, dy)


def test_backward_without_weight():
    x, _, _, dy = _inputs(50, 640, torch.bfloat16, torch.bfloat16)
    _check_backward(x, None, dy)
    _check_backward(x, None, dy, torch.float32)


def test_backward_against_differences():
    """<gradient, direction> against central differences of the 64-bit forward's <y, dy>."""
    T, H, h = 6, 200, 1e-4
    x, g, b, dy = (v.float() for v in _inputs(T, H, torch.float32, torch.float32))
    _, mean, rstd = ops.layer_norm(x, g, b)
    dx, dg, db = ops.layer_norm_backward(dy, x, g, mean, rstd)
    gen = torch.Generator(device="cuda").manual_seed(9)
    f = lambda x, g, b: (_ref(x, g, b)[0] * dy.double()).sum()
    xd, gd, bd = x.double(), g.double(), b.double()
    for at, grad in ((0, dx), (1, dg), (2, db)):
        v = torch.randn(grad.shape, generator=gen, device="cuda", dtype=torch.double)
        p, m = [xd, gd, bd], [xd, gd, bd]
        p[at], m[at] = p[at] + h * v, m[at] - h * v
        diff = (f(*p) - f(*m)) / (2 * h)
        # h^2 truncation and fp32 gradients: 1e-5 of the product's scale
        assert abs((grad.double() * v).sum() - diff) <= 1e-5 * (grad.double() * v).norm() * grad.numel() ** 0.5


def test_empty_batch():
    x = torch.zeros(0, 256, device="cuda", dtype=torch.bfloat16)
    g = torch.ones(256, device="cuda", dtype=torch.bfloat16)
    y, mean, rstd = ops.layer_norm(x, g)
    assert y.shape == (0, 256) and mean.numel() == 0
    dx, dg, db = ops.layer_norm_backward(x, x, g, mean, rstd)
    assert dx.shape == (0, 256) and (dg == 0).all() and (db == 0).all()


def test_equal_bits_again_and_on_another_stream():
    x, g, b, dy = _inputs(2000, 1024, torch.bfloat16, torch.bfloat16)
    ref = ops.layer_norm(x, g, b)
    back = ops.layer_norm_backward(dy, x, g, *ref[1:])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ops.layer_norm(x, g, b, stream=s)
    again = ops.layer_norm_backward(dy, x, g, *got[1:], stream=s)
    s.synchronize()
    for u, v in zip(ref + back, got + again):
        assert torch.equal(u, v)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("T,H", [(1, 128), (3, 256), (128, 7168), (700, 4096), (2, 16384), (1, 384)])
def test_fp8_form(T, H, dtype, pow2):
    x, g, b, _ = _inputs(T, H, dtype, dtype)
    q, sf = ops.layer_norm_fp8(x, g, b, pow2_scales=pow2)
    y, _, _, _, _, exh = _ref(x, g, b)
    ey = (exh * g.double().abs() + 4 * E24 * (y.abs() + 1)).view(T, -1, 128)
    y = y.view(T, -1, 128)
    want = y.abs().amax(2).clamp_min(1e-4) / 448
    off = ey.amax(2) / 448 + 2 * E24 * want
    s = sf.double()
    if pow2:
        m, _ = torch.frexp(sf)
        assert (m == 0.5).all()
        # the smallest power of two at or above the scale, up to the scale's own error
        assert (s >= want - off).all() and (s / 2 < want + off).all()
    else:
        assert ((s - want).abs() <= off).all()
    # e4m3 keeps 3 bits of fraction: half a step is 2^-4 of the value, 2^-10 below the normal range
    v = q.view(torch.float8_e4m3fn).double().view(T, -1, 128)
    code = y / s[:, :, None]
    assert ((v - code).abs() <= code.abs() * 2.0 ** -4 + 2.0 ** -10 + (ey / s[:, :, None]) + 4 * E24 * code.abs()).all()
    # and nearly every code is the one that the same fp32 quotient rounds to
    z = (ops.layer_norm(x.float(), g.float(), b.float())[0].view(T, -1, 128) / sf[:, :, None]).to(torch.float8_e4m3fn)
    assert (z.view(torch.uint8).view(T, H) != q).float().mean() <= 1e-3


def test_fp8_form_refuses_unaligned_rows():
    x = torch.zeros(4, 300, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ops.MoeError):
        ops.layer_norm_fp8(x[:, 1:257])
    with pytest.raises(ops.MoeError):
        ops.layer_norm_fp8(torch.zeros(4, 200, device="cuda", dtype=torch.bfloat16))


def test_refusals_of_tensors():
    x, g, b, _ = _inputs(4, 256, torch.bfloat16, torch.bfloat16)
    with pytest.raises(TypeError):
        ops.layer_norm(x, g.half())
    with pytest.raises(TypeError):
        ops.layer_norm(x, g, b.float())
    with pytest.raises(ValueError):
        ops.layer_norm(x, g[:128])
    with pytest.raises(ValueError):
        ops.layer_norm(x.t())
    with pytest.raises(ValueError):
        ops.layer_norm(x[:1].expand(4, 256))
    with pytest.raises(TypeError):
        ops.layer_norm(x.double())
    with pytest.raises(ops.MoeError):
        ops.layer_norm(torch.zeros(2, 16392, device="cuda"))


def test_rows_past_32_bit_offsets():
    T, H = 300001, 7168          # 2.15e9 elements
    x = torch.zeros(T, H, device="cuda", dtype=torch.bfloat16)
    tail, g, b, _ = _inputs(5, H, torch.bfloat16, torch.bfloat16)
    x[-5:] = tail
    y, mean, rstd = ops.layer_norm(x, g, b)
    _check_forward(tail, g, b, (y[-5:], mean[-5:], rstd[-5:]))
    dx, dg, _ = ops.layer_norm_backward(x, x, g, mean, rstd)
    rdx, rdg, _ = ops.layer_norm_backward(tail, tail, g, mean[-5:].clone(), rstd[-5:].clone())
    assert torch.equal(dx[-5:], rdx)
