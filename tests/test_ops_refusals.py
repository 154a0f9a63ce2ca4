"""What the operators around the expert layer refuse, before any CUDA call (no GPU needed), and the
shape and type checks of their Python entry points."""
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


def _layer_norm(lib, T=4, H=256, x=P, ldx=256, dtype=BF16, weight=P, bias=P, w_dtype=BF16, eps=1e-5, y=P, mean=P, rstd=P):
    return lib.moe_layer_norm(T, H, x, ldx, dtype, weight, bias, w_dtype, eps, y, mean, rstd, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=0), dict(H=16385, ldx=16385), dict(dtype=3), dict(dtype=-1), dict(w_dtype=F16), dict(w_dtype=7),
    dict(ldx=255), dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(y=None), dict(x=P + 1), dict(y=P + 1),
    dict(mean=P + 2), dict(rstd=P + 1), dict(weight=P + 1), dict(bias=P + 1)])
def test_layer_norm_refuses(lib, bad):
    assert _layer_norm(lib, **bad) == INVALID


def test_empty_batches_need_no_gpu(lib):
    assert _layer_norm(lib, T=0, x=None, y=None) == 0
    assert lib.moe_layer_norm_fp8(0, 256, None, 256, BF16, None, None, BF16, 1e-5, 0, None, None, None) == 0
    assert lib.moe_route_topk(0, 8, 2, None, 8, F32, None, 1, None, None, None) == 0
    assert lib.moe_route_topk_backward(0, 8, 2, None, None, None, None, 8, F32, 1, None, None) == 0
    assert lib.moe_gather_rows(0, 2, 64, 4, 0, None, 64, BF16, None, None, None, None) == 0
    assert lib.moe_combine_rows(0, 2, 64, 0, None, BF16, None, None, None, None) == 0
    assert lib.moe_grouped_mm(0, 4, 64, 64, None, 64, None, None, None, 64, BF16, None, 0, None) == 0
    assert lib.moe_grouped_mm_dx(0, 4, 64, 64, None, 64, None, None, None, 64, BF16, None, 0, None) == 0
    n = ctypes.c_uint64(1)
    assert lib.moe_grouped_mm_workspace(0, 4, 64, 64, ctypes.byref(n)) == 0 and n.value == 0


@pytest.mark.parametrize("bad", [
    dict(H=192), dict(x=P + 8), dict(ldx=260), dict(weight=P + 2), dict(bias=P + 4), dict(q=P + 8), dict(q=None),
    dict(sf=None), dict(sf=P + 2), dict(pow2=2), dict(pow2=-1)])
def test_layer_norm_fp8_refuses(lib, bad):
    a = dict(T=4, H=256, x=P, ldx=256, dtype=BF16, weight=P, bias=P, pow2=0, q=P, sf=P) | bad
    assert lib.moe_layer_norm_fp8(a["T"], a["H"], a["x"], a["ldx"], a["dtype"], a["weight"], a["bias"], BF16, 1e-5,
                                  a["pow2"], a["q"], a["sf"], None) == INVALID


@pytest.mark.parametrize("bad", [dict(lddy=100), dict(ldx=100), dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None),
                                 dict(dx=None), dict(dweight=P + 1), dict(dbias=P + 1), dict(w_dtype=F16), dict(H=20000)])
def test_layer_norm_backward_refuses(lib, bad):
    a = dict(T=4, H=256, dy=P, lddy=256, x=P, ldx=256, weight=P, w_dtype=BF16, mean=P, rstd=P, dx=P, dweight=P, dbias=P) | bad
    assert lib.moe_layer_norm_backward(a["T"], a["H"], a["dy"], a["lddy"], a["x"], a["ldx"], BF16, a["weight"], a["w_dtype"],
                                       a["mean"], a["rstd"], a["dx"], a["dweight"], a["dbias"], P, 1 << 40, None) == INVALID
    n = ctypes.c_uint64()
    assert lib.moe_layer_norm_backward_workspace(4, 0, ctypes.byref(n)) == INVALID
    assert lib.moe_layer_norm_backward_workspace(4, 256, None) == INVALID


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(E=0), dict(E=1025, ld=1025), dict(topk=0), dict(topk=33, E=64, ld=64), dict(topk=9), dict(ld=7), dict(dtype=3),
    dict(renorm=2), dict(logits=None), dict(idx=None), dict(w=None), dict(idx=P + 4), dict(w=P + 2), dict(logits=P + 2)])
def test_router_refuses(lib, bad):
    a = dict(T=4, E=8, topk=2, logits=P, ld=8, dtype=F32, renorm=1, idx=P, w=P) | bad
    assert lib.moe_route_topk(a["T"], a["E"], a["topk"], a["logits"], a["ld"], a["dtype"], None, a["renorm"], a["idx"],
                              a["w"], None) == INVALID
    a["logits"] = bad.get("logits", P)
    if "logits" in bad and bad["logits"] is None:
        a["renorm"] = 0        # the renormalised gradient does not read the logits
    assert lib.moe_route_topk_backward(a["T"], a["E"], a["topk"], P, a["idx"], a["w"], a["logits"], a["ld"], a["dtype"],
                                       a["renorm"], P, None) == INVALID


@pytest.mark.parametrize("bad", [dict(T=-1), dict(topk=0), dict(topk=33), dict(E=0), dict(E=1025), dict(T=1 << 30, topk=32),
                                 dict(idx=None), dict(offsets=None), dict(rows=None), dict(status=None), dict(idx=P + 4),
                                 dict(offsets=P + 2), dict(T=4096, topk=8, ws=None), dict(T=4096, topk=8, ws_bytes=100)])
def test_expert_order_refuses(lib, bad):
    a = dict(T=4, topk=2, E=8, idx=P, offsets=P, rows=P, status=P, ws=P, ws_bytes=1 << 40) | bad
    assert lib.moe_expert_order(a["T"], a["topk"], a["E"], a["idx"], a["offsets"], a["rows"], a["status"], a["ws"],
                                a["ws_bytes"], None) == INVALID


@pytest.mark.parametrize("bad", [dict(topk=0), dict(topk=33), dict(H=0), dict(M=-1), dict(M=1 << 31), dict(dtype=5), dict(ld=63),
                                 dict(x=P + 1), dict(out=P + 1), dict(out=None), dict(rows=P + 2), dict(rows=None)])
def test_rows_refuse(lib, bad):
    a = dict(T=4, topk=2, H=64, E=3, M=8, x=P, ld=64, dtype=BF16, rows=P, offsets=P, out=P) | bad
    assert lib.moe_gather_rows(a["T"], a["topk"], a["H"], a["E"], a["M"], a["x"], a["ld"], a["dtype"], a["rows"], P,
                               a["out"], None) == INVALID
    assert lib.moe_combine_rows_backward(a["T"], a["topk"], a["H"], a["E"], a["M"], a["x"], a["ld"], P, a["dtype"], a["rows"],
                                         P, P, a["out"], P, None) == INVALID
    if "ld" not in bad:
        assert lib.moe_combine_rows(a["T"], a["topk"], a["H"], a["M"], a["x"], a["dtype"], a["rows"], P, a["out"], None) == INVALID


@pytest.mark.parametrize("bad", [dict(M=-1), dict(M=1 << 31), dict(E=0), dict(E=1025), dict(N=0), dict(N=60), dict(K=4), dict(K=68),
                                 dict(N=(1 << 20) + 8), dict(dtype=F32), dict(dtype=4), dict(ld=56), dict(ld=260), dict(x=None),
                                 dict(x=P + 8), dict(w=None), dict(w=P + 8), dict(offsets=None), dict(offsets=P + 2),
                                 dict(out=None), dict(out=P + 8)])
def test_grouped_refuse(lib, bad):
    a = dict(M=16, E=4, N=64, K=64, x=P, ld=64, w=P, offsets=P, out=P, dtype=BF16) | bad
    args = (a["M"], a["E"], a["N"], a["K"], a["x"], a["ld"], a["w"], a["offsets"], a["out"], 64, a["dtype"], None, 0, None)
    assert lib.moe_grouped_mm(*args) == INVALID
    assert lib.moe_grouped_mm_dx(*args) == INVALID
    assert lib.moe_grouped_mm_dw(a["M"], a["E"], a["N"], a["K"], a["x"], a["ld"], a["w"], 64, a["offsets"], a["out"], a["dtype"],
                                 a["dtype"], 0, P, 1 << 20, None) == INVALID


def test_grouped_dw_refuses_types(lib):
    def dw(dtype, out, acc):
        return lib.moe_grouped_mm_dw(16, 4, 64, 64, P, 64, P, 64, P, P, dtype, out, acc, ws, ws_bytes, None)
    ws, ws_bytes = P, 4 * 256
    assert dw(BF16, F16, 0) == INVALID and dw(F16, BF16, 0) == INVALID and dw(BF16, BF16, 2) == INVALID
    for ws, ws_bytes in ((None, 4 * 256), (P + 64, 4 * 256)):
        assert dw(BF16, BF16, 0) == INVALID
    for call in (lib.moe_grouped_mm_workspace, lib.moe_grouped_mm_dw_workspace):
        assert call(16, 0, 64, 64, ctypes.byref(ctypes.c_uint64())) == INVALID
        assert call(16, 8, 60, 64, ctypes.byref(ctypes.c_uint64())) == INVALID
        assert call(16, 8, 64, 64, None) == INVALID


def test_more_rows_than_31_bits_hold_are_refused(lib):
    n, big = ctypes.c_uint64(), (1 << 30) + 1
    assert _layer_norm(lib, T=big) == INVALID
    assert lib.moe_layer_norm_backward_workspace(big, 256, ctypes.byref(n)) == INVALID
    assert lib.moe_route_topk(big, 8, 2, P, 8, F32, None, 1, P, P, None) == INVALID
    assert lib.moe_expert_order_workspace(1 << 28, 5, 8, ctypes.byref(n)) == INVALID
    assert lib.moe_gather_rows(4, 2, 64, 3, big, P, 64, BF16, P, P, P, None) == INVALID
    assert lib.moe_combine_rows(big, 2, 64, 8, P, BF16, P, P, P, None) == INVALID
    assert lib.moe_grouped_mm_workspace(big, 4, 64, 64, ctypes.byref(n)) == INVALID


def test_python_entry_points_check_shapes_and_types():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.layer_norm(x)
    with pytest.raises(ValueError, match=r"\[rows"):
        ops.layer_norm(x[0])
    with pytest.raises(ValueError, match="CUDA"):
        ops.route_topk(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError, match=r"\[T, topk\]"):
        ops.expert_order(torch.zeros(4, dtype=torch.int64), 8)
    with pytest.raises(TypeError, match="float32"):
        ops.grouped_mm(x.float(), x.float()[None], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        ops.combine_rows(x.long(), torch.zeros(4, 2, dtype=torch.int32))


def test_rows_longer_than_31_bits_hold_are_refused(lib):
    big = (1 << 30) + 1
    assert lib.moe_gather_rows(4, 2, big, 3, 8, P, big, BF16, P, P, P, None) == INVALID
    assert lib.moe_combine_rows(4, 2, big, 8, P, BF16, P, P, P, None) == INVALID
    assert lib.moe_combine_rows_backward(4, 2, big, 3, 8, P, big, P, BF16, P, P, P, P, P, None) == INVALID
