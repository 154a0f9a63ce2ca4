"""RMS norm with the residual's addition, its FP8 form and its gradients against 64-bit formulas.

Bounds.  With u half a step of the output's type relative to the value and e = 2^-24: sums of H terms in fp32, by
threads (at most 16 pairs) and a tree of at most 10 levels, are at most 64 e sum|.| off.  So the mean square is 64 e
relative off, rstd half of that and its own few roundings (40 e), y that, two products and its rounding; the
gradient's mean 64 e mean|a xh| and the products' 48 e; sums over T rows (T/100 + 128) e sum|.|, as no block has more than
T/100 rows one after another.
"""
import pytest
import torch

from combine_persistent_warp_gb300 import ops

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}   # half a step next to zero
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32), (torch.float32, torch.float32)]


def _inputs(T, H, dtype, wdtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return dict(x=r(T, H).to(dtype), r=(2 * r(T, H)).to(dtype), w=(1 + 0.1 * r(H)).to(wdtype), dy=r(T, H).to(dtype), dh=r(T, H).to(dtype))


def _sum(x, r):
    return x if r is None else (x.float() + r.float()).to(x.dtype)


def _ref(h, w, eps):
    h = h.double()
    rstd = (h.square().mean(1) + eps).rsqrt()
    xh = h * rstd[:, None]
    return rstd, xh, xh if w is None else xh * w.double()


def _check_forward(got, x, w, r, eps=1e-6):
    y, rstd, h = got
    assert torch.equal(h, _sum(x, r)) and (r is not None or h is x)
    rr, _, ry = _ref(h, w, eps)
    assert ((rstd.double() - rr).abs() <= 40 * E24 * rr).all()
    assert y.dtype == x.dtype and ((y.double() - ry).abs() <= (48 * E24 + U[y.dtype]) * ry.abs() + TINY[y.dtype]).all()


def _check_backward(got, dy, h, w, dh, rstd, eps=1e-6):
    dx, dw = got
    rr, xh, _ = _ref(h, w, eps)
    d = dy.double()
    a = d if w is None else d * w.double()
    m, ma = (a * xh).mean(1, keepdim=True), (a * xh).abs().mean(1, keepdim=True)
    core = (a - xh * m) * rr[:, None]
    ref = core if dh is None else core + dh.double()
    bound = rr[:, None] * (44 * E24 * a.abs() + xh.abs() * (m.abs() * 96 * E24 + 112 * E24 * ma)) + 2 * E24 * (core.abs() + ref.abs())
    assert ((dx.double() - ref).abs() <= bound + U[dx.dtype] * ref.abs() + TINY[dx.dtype]).all()
    if dw is not None:
        s = (d * xh).sum(0)
        assert ((dw.double() - s).abs() <= (h.shape[0] / 100 + 128 + 44) * E24 * (d * xh).abs().sum(0) + U[dw.dtype] * s.abs() + TINY[dw.dtype]).all()


CASES = [(1, 1), (1, 8), (3, 5), (2, 32), (7, 100), (5, 1000), (9, 1001), (4, 1024), (3, 2056), (130, 4096), (700, 1024), (2, 4097),
         (3, 7168), (1, 8191), (2, 8192), (2, 16384), (2, 16383), (1300, 264), (2500, 2003), (3042, 5888), (1300, 4104), (900, 12288),
         (305, 7168), (4000, 96), (6000, 1040), (2600, 1027)]


@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("T,H", CASES)
def test_forward_and_backward(T, H, dtype, wdtype):
    v = _inputs(T, H, dtype, wdtype)
    for r, dh in ((v["r"], v["dh"]), (None, None), (v["r"], None)):
        got = ops.rms_norm(v["x"], v["w"], residual=r)
        _check_forward(got, v["x"], v["w"], r)
        y, rstd, h = got
        _check_backward(ops.rms_norm_backward(v["dy"], h, v["w"], rstd, dh=dh), v["dy"], h, v["w"], dh, rstd)


def test_without_weight_other_eps_and_gradients_not_asked_for():
    v = _inputs(33, 520, torch.bfloat16, torch.bfloat16)
    _check_forward(ops.rms_norm(v["x"], None, 0.5, residual=v["r"]), v["x"], None, v["r"], 0.5)
    y, rstd, h = ops.rms_norm(v["x"], None)
    for pd in (None, torch.float32):
        dx, dw = ops.rms_norm_backward(v["dy"], h, None, rstd, param_dtype=pd)
        assert dw.dtype == (pd or torch.bfloat16)
        _check_backward((dx, dw), v["dy"], h, None, None, rstd)
    only, none = ops.rms_norm_backward(v["dy"], h, None, rstd, weight_grad=False)
    assert none is None and torch.equal(only, dx)


@pytest.mark.parametrize("T,H,off,pitch", [(21, 512, 0, 1536), (21, 512, 3, 1539), (21, 1000, 8, 1016), (21, 333, 1, 400), (3, 2049, 1, 2051),
                                           (1, 2049, 1, 2050), (3000, 1500, 3, 1503), (5, 1030, 0, 1030), (2600, 2048, 0, 4096)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_and_unaligned_rows(T, H, off, pitch, dtype):
    """Rows apart from each other and off the boundaries; what lies between them is NaN."""
    v = _inputs(T, H, dtype, dtype)

    def placed(t):
        flat = torch.full((T * pitch + off,), float("nan"), device="cuda", dtype=dtype)[off:]
        s = flat.as_strided((T, H), (pitch, 1))
        s.copy_(t)
        return s

    x, r, dy, dh = (placed(v[n]) for n in ("x", "r", "dy", "dh"))
    w = torch.cat([v["w"][:1], v["w"]])[1:]
    got = ops.rms_norm(x, w, residual=r)
    _check_forward(got, x, w, r)
    h = placed(got[2])
    _check_backward(ops.rms_norm_backward(dy, h, w, got[1], dh=dh), dy, h, w, dh, got[1])
    _check_forward(ops.rms_norm(x, w), x, w, None)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("T,H", [(1, 128), (128, 7168), (3, 1024), (40, 4096), (2500, 2048), (1, 16384), (700, 256), (1300, 8192)])
@pytest.mark.parametrize("dtype,wdtype", TYPES)
def test_fp8_form(T, H, dtype, wdtype, pow2):
    v = _inputs(T, H, dtype, wdtype)
    v["x"][0, :128] = 0
    v["r"][0, :128] = 0
    for r in (v["r"], None):
        q, sf, h = ops.rms_norm_fp8(v["x"], v["w"], residual=r, pow2_scales=pow2)
        assert torch.equal(h, _sum(v["x"], r))
        _, _, y = _ref(h, v["w"], 1e-6)
        want = y.abs().view(T, -1, 128).amax(2).clamp_min(1e-4) / 448
        if pow2:
            s = sf.double()
            assert (torch.frexp(sf)[0] == 0.5).all() and (s >= want * (1 - 52 * E24)).all() and (s < 2 * want * (1 + 52 * E24)).all()
        else:
            assert ((sf.double() - want).abs() <= 52 * E24 * want).all()
        back = q.view(torch.float8_e4m3fn).double().view(T, -1, 128) * sf.double()[:, :, None]
        # half a step of e4m3 (2^-4 of the value, 2^-10 of a scale next to zero), and the quotient's roundings
        ya = y.view(T, -1, 128)
        assert ((back - ya).abs() <= (2.0 ** -4 + 64 * E24) * ya.abs() + 2.0 ** -10 * sf.double()[:, :, None]).all()


def test_gradient_against_differences():
    v = _inputs(3, 24, torch.float32, torch.float32)
    x, r, w = v["x"].double(), v["r"].double(), v["w"].double()
    f = lambda x, r, w: ((x + r) * ((x + r).square().mean(1, keepdim=True) + 1e-6).rsqrt() * w * v["dy"]).sum() + ((x + r) * v["dh"]).sum()
    y, rstd, h = ops.rms_norm(v["x"], v["w"], residual=v["r"])
    dx, dw = ops.rms_norm_backward(v["dy"], h, v["w"], rstd, dh=v["dh"])
    step = 1e-5
    for i in range(24):
        d = torch.zeros_like(x)
        d[1, i] = step
        got = (f(x + d, r, w) - f(x - d, r, w)) / (2 * step)
        # differences in 64 bits are 1e-8 off; h is rounded to fp32, the gradient to 1e-5 of its parts
        assert abs(got - dx[1, i].double()) <= 1e-4
        d = torch.zeros_like(w)
        d[i] = step
        assert abs((f(x, r, w + d) - f(x, r, w - d)) / (2 * step) - dw[i].double()) <= 1e-4


def test_special_values_stay_in_their_rows():
    v = _inputs(3000, 2048, torch.bfloat16, torch.bfloat16)
    clean = ops.rms_norm(v["x"], v["w"], residual=v["r"])
    gclean = ops.rms_norm_backward(v["dy"], clean[2], v["w"], clean[1], dh=v["dh"])[0]
    x = v["x"].clone()
    x[7], x[11, 3], x[2999, 5] = float("nan"), float("inf"), -float("inf")
    bad = torch.zeros(3000, dtype=torch.bool, device="cuda")
    bad[[7, 11, 2999]] = True
    y, rstd, h = ops.rms_norm(x, v["w"], residual=v["r"])
    assert torch.equal(y[~bad], clean[0][~bad]) and torch.equal(rstd[~bad], clean[1][~bad])
    assert y[7].isnan().all() and rstd[11] == 0 and y[11, 3].isnan()
    dx, _ = ops.rms_norm_backward(v["dy"], h, v["w"], rstd, dh=v["dh"])
    assert torch.equal(dx[~bad], gclean[~bad])
    zero = torch.zeros(4, 256, device="cuda", dtype=torch.float16)
    y, rstd, _ = ops.rms_norm(zero)
    assert (y == 0).all() and ((rstd - 1000).abs() < 0.01).all()


def test_empty_batch_and_equal_bits():
    v = _inputs(4000, 2504, torch.bfloat16, torch.bfloat16)
    a, b = (ops.rms_norm(v["x"], v["w"], residual=v["r"]) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    ga, gb = (ops.rms_norm_backward(v["dy"], a[2], v["w"], a[1], dh=v["dh"]) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(ga, gb))
    e = v["x"][:0]
    y, rstd, h = ops.rms_norm(e, v["w"], residual=e)
    assert y.shape == h.shape == (0, 2504) and rstd.shape == (0,)
    dx, dw = ops.rms_norm_backward(e, e, v["w"], rstd)
    assert dx.shape == (0, 2504) and (dw == 0).all()
    q, sf, _ = ops.rms_norm_fp8(e[:, :128])
    assert q.shape == (0, 128) and sf.shape == (0, 1)


def test_other_stream_and_graph():
    v = _inputs(64, 1024, torch.bfloat16, torch.bfloat16)
    want = ops.rms_norm(v["x"], v["w"], residual=v["r"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ops.rms_norm(v["x"], v["w"], residual=v["r"], stream=s)
    back = ops.rms_norm_backward(v["dy"], got[2], v["w"], got[1], dh=v["dh"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = v["x"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, rstd, h = ops.rms_norm(x, v["w"], residual=v["r"])
        dx, dw = ops.rms_norm_backward(v["dy"], h, v["w"], rstd, dh=v["dh"])
        q = ops.rms_norm_fp8(x, v["w"], residual=v["r"])
    g.replay()
    assert torch.equal(y, want[0]) and torch.equal(dx, back[0]) and torch.equal(dw, back[1])
    x.copy_(v["dy"])
    g.replay()
    again = ops.rms_norm(v["dy"], v["w"], residual=v["r"])
    assert torch.equal(y, again[0]) and all(torch.equal(a, b) for a, b in zip(q, ops.rms_norm_fp8(v["dy"], v["w"], residual=v["r"])))


def test_offsets_past_31_bits():
    T, H = 140000, 16384
    x = torch.zeros(T, H, device="cuda", dtype=torch.bfloat16)
    tail = _inputs(3, H, torch.bfloat16, torch.bfloat16)
    x[-3:] = tail["x"]
    y, rstd, h = ops.rms_norm(x, tail["w"], residual=x)
    _check_forward((y[-3:], rstd[-3:], h[-3:]), tail["x"], tail["w"], tail["x"])
    dx, _ = ops.rms_norm_backward(x, h, tail["w"], rstd, dh=y)
    _check_backward((dx[-3:], None), tail["x"], h[-3:], tail["w"], y[-3:], rstd[-3:])
