"""What the operators of a block with RMS norms, scored routing and 8-bit checkpoints refuse, before any
CUDA call (no GPU needed), and the shape and type checks of their Python entry points."""
import ctypes

import pytest
import torch

from combine_persistent_warp_gb300 import native, ops

INVALID = 1
F32, BF16, F16 = native.F32, native.BF16, native.F16
P = 1 << 20          # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    return native.load()


def _rms(lib, T=4, H=256, x=P, ldx=256, r=P, ldr=256, dtype=BF16, w=P, w_dtype=BF16, eps=1e-6, h=P, y=P, rstd=P):
    return lib.moe_rms_norm(T, H, x, ldx, r, ldr, dtype, w, w_dtype, eps, h, y, rstd, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=(1 << 30) + 1), dict(H=0), dict(H=16385, ldx=16385, ldr=16385), dict(dtype=3), dict(dtype=-1), dict(w_dtype=F16),
    dict(ldx=255), dict(ldr=255), dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(y=None), dict(h=None), dict(x=P + 1),
    dict(r=P + 1), dict(h=P + 1), dict(y=P + 1), dict(rstd=P + 2), dict(w=P + 1)])
def test_rms_norm_refuses(lib, bad):
    assert _rms(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", [dict(H=192), dict(x=P + 8), dict(r=P + 8), dict(h=P + 8), dict(ldx=260), dict(ldr=260), dict(w=P + 4), dict(q=P + 8),
                                 dict(q=None), dict(sf=None), dict(sf=P + 2), dict(pow2=2), dict(pow2=-1), dict(h=None)])
def test_rms_norm_fp8_refuses(lib, bad):
    a = dict(T=4, H=256, x=P, ldx=256, r=P, ldr=256, w=P, pow2=0, h=P, q=P, sf=P) | bad
    assert lib.moe_rms_norm_fp8(a["T"], a["H"], a["x"], a["ldx"], a["r"], a["ldr"], BF16, a["w"], BF16, 1e-6, a["pow2"], a["h"],
                                a["q"], a["sf"], None) == INVALID


@pytest.mark.parametrize("bad", [dict(lddy=100), dict(ldh=100), dict(lddh=100), dict(dy=None), dict(h=None), dict(rstd=None), dict(dx=None),
                                 dict(dh=P + 1), dict(dweight=P + 1), dict(w_dtype=F16), dict(H=20000), dict(T=(1 << 30) + 1)])
def test_rms_norm_backward_refuses(lib, bad):
    a = dict(T=4, H=256, dy=P, lddy=256, h=P, ldh=256, dh=P, lddh=256, w=P, w_dtype=BF16, rstd=P, dx=P, dweight=P) | bad
    assert lib.moe_rms_norm_backward(a["T"], a["H"], a["dy"], a["lddy"], a["h"], a["ldh"], a["dh"], a["lddh"], BF16, a["w"], a["w_dtype"],
                                     a["rstd"], a["dx"], a["dweight"], P, 1 << 40, None) == INVALID
    n = ctypes.c_uint64()
    assert lib.moe_rms_norm_backward_workspace(4, 0, ctypes.byref(n)) == INVALID
    assert lib.moe_rms_norm_backward_workspace(4, 256, None) == INVALID


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=(1 << 30) + 1), dict(E=0), dict(E=1026, ld=1026), dict(topk=0), dict(topk=33), dict(ld=31), dict(dtype=3), dict(score=2),
    dict(score=-1), dict(groups=0), dict(groups=5), dict(groups=64, E=64, ld=64), dict(kept=0), dict(kept=5), dict(top=0), dict(top=3),
    dict(topk=17), dict(renorm=2), dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(logits=None), dict(idx=None),
    dict(w=None), dict(idx=P + 4), dict(w=P + 2), dict(logits=P + 2), dict(bias=P + 2)])
def test_route_scores_refuses(lib, bad):
    a = dict(T=4, E=32, topk=4, logits=P, ld=32, dtype=F32, score=0, bias=P, groups=4, kept=2, top=2, renorm=1, scale=1.0, idx=P, w=P) | bad
    assert lib.moe_route_scores(a["T"], a["E"], a["topk"], a["logits"], a["ld"], a["dtype"], a["score"], a["bias"], a["groups"], a["kept"],
                                a["top"], None, a["renorm"], a["scale"], a["idx"], a["w"], None) == INVALID


@pytest.mark.parametrize("bad", [dict(T=-1), dict(E=0), dict(topk=33), dict(ld=31), dict(dtype=3), dict(score=2), dict(renorm=2), dict(scale=0.0),
                                 dict(dw=None), dict(idx=None), dict(w=None), dict(logits=None), dict(logits=None, score=1, renorm=0), dict(d=None),
                                 dict(idx=P + 4), dict(d=P + 2)])
def test_route_scores_backward_refuses(lib, bad):
    a = dict(T=4, E=32, topk=4, dw=P, idx=P, w=P, logits=P, ld=32, dtype=F32, score=0, renorm=1, scale=1.0, d=P) | bad
    assert lib.moe_route_scores_backward(a["T"], a["E"], a["topk"], a["dw"], a["idx"], a["w"], a["logits"], a["ld"], a["dtype"], a["score"],
                                         a["renorm"], a["scale"], a["d"], None) == INVALID


@pytest.mark.parametrize("bad", [dict(M=-1), dict(M=(1 << 30) + 1), dict(I=0), dict(I=(1 << 20) + 1, ld=1 << 22), dict(ld=127), dict(dtype=4), dict(gu=None),
                                 dict(act=None), dict(gu=P + 1), dict(act=P + 1), dict(codes=None), dict(scales=None)])
def test_swiglu_refuses(lib, bad):
    a = dict(M=4, I=64, gu=P, ld=128, dtype=BF16, act=P, codes=P, scales=P) | bad
    assert lib.moe_swiglu(a["M"], a["I"], a["gu"], a["ld"], a["dtype"], a["act"], a["codes"], a["scales"], None) == INVALID


@pytest.mark.parametrize("bad", [dict(M=-1), dict(I=0), dict(ldd=63), dict(ldg=127), dict(dtype=4), dict(da=None), dict(dgu=None), dict(da=P + 1),
                                 dict(dgu=P + 1), dict(act=P + 1), dict(gu=P + 1), dict(gu=None), dict(codes=P, scales=P), dict(codes=P),
                                 dict(gu=None, scales=P)])
def test_swiglu_backward_refuses(lib, bad):
    a = dict(M=4, I=64, da=P, ldd=64, gu=P, ldg=128, codes=None, scales=None, dtype=BF16, dgu=P, act=P) | bad
    assert lib.moe_swiglu_backward(a["M"], a["I"], a["da"], a["ldd"], a["gu"], a["ldg"], a["codes"], a["scales"], a["dtype"], a["dgu"],
                                   a["act"], None) == INVALID


@pytest.mark.parametrize("bad", [dict(M=-1), dict(M=(1 << 30) + 1), dict(H=0), dict(H=(1 << 20) + 1, ld=1 << 21), dict(ld=63), dict(dtype=4), dict(x=None),
                                 dict(x=P + 1), dict(codes=None), dict(scales=None)])
def test_checkpoint_refuses(lib, bad):
    a = dict(M=4, H=64, x=P, ld=64, dtype=BF16, codes=P, scales=P) | bad
    assert lib.moe_checkpoint_rows(a["M"], a["H"], a["x"], a["ld"], a["dtype"], a["codes"], a["scales"], None) == INVALID
    if "ld" not in bad:
        assert lib.moe_restore_rows(a["M"], a["H"], a["codes"], a["scales"], a["dtype"], a["x"], None) == INVALID


def test_empty_batches_need_no_gpu(lib):
    assert _rms(lib, T=0, x=None, r=None, h=None, y=None, w=None) == 0
    assert lib.moe_rms_norm_fp8(0, 256, None, 256, None, 0, BF16, None, BF16, 1e-6, 0, None, None, None, None) == 0
    assert lib.moe_route_scores(0, 8, 2, None, 8, F32, 0, None, 1, 1, 2, None, 1, 1.0, None, None, None) == 0
    assert lib.moe_route_scores_backward(0, 8, 2, None, None, None, None, 8, F32, 0, 1, 1.0, None, None) == 0
    assert lib.moe_swiglu(0, 64, None, 128, BF16, None, None, None, None) == 0
    assert lib.moe_swiglu_backward(0, 64, None, 64, None, 128, None, None, BF16, None, None, None) == 0
    assert lib.moe_checkpoint_rows(0, 64, None, 64, BF16, None, None, None) == 0
    assert lib.moe_restore_rows(0, 64, None, None, BF16, None, None) == 0


def test_python_entry_points_check_shapes_and_types():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.rms_norm(x)
    with pytest.raises(ValueError, match=r"\[rows"):
        ops.rms_norm(x[0])
    with pytest.raises(TypeError, match="Long"):
        ops.rms_norm_fp8(x.long())
    with pytest.raises(TypeError, match="param_dtype"):
        ops.rms_norm_backward(x, x, None, x, param_dtype=torch.float16)
    with pytest.raises(ValueError, match="score"):
        ops.route_scores(torch.zeros(4, 8), 2, score="tanh")
    with pytest.raises(ValueError, match="CUDA"):
        ops.route_scores(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError, match=r"\[T, topk\]"):
        ops.route_scores_backward(x, x[0], x, x)
    with pytest.raises(ValueError, match="CUDA"):
        ops.swiglu(x)
    with pytest.raises(ValueError, match="CUDA"):
        ops.checkpoint_rows(x)
    with pytest.raises(ValueError, match="CUDA"):
        ops.restore_rows(x.to(torch.int8), x, torch.float32)
    with pytest.raises(TypeError, match="dtype"):
        ops.restore_rows(x, x, torch.int8)
    with pytest.raises(TypeError, match="tensor"):
        ops.swiglu_checkpoint([1.0])


def test_binding_constants_match_the_header():
    text = open(native.HEADER, encoding="utf-8").read()
    assert f"MOE_SCORE_SIGMOID = {native.SCORE_SIGMOID}" in text and f"MOE_SCORE_SOFTMAX = {native.SCORE_SOFTMAX}" in text
