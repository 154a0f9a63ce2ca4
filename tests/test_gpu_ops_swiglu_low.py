"""SwiGLU where the logistic function of the gate is no normal number (gates from -87.4 to -88.7): with a large `up` the
products are ordinary numbers.

Bounds as in test_gpu_ops_swiglu: the logistic function (1.5 |g| + 8) e relative off, e = 2^-24, and here half a step of 2^-149 of
a value above 2^-128 more, 2^-22 relative; the products after it four roundings.
"""
import pytest
import torch

from combine_persistent_warp_gb300 import ops

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133}


def _near(got, ref, g, dtype):
    assert (got.double() - ref).abs().le(((1.5 * g.abs() + 14) * E24 + 2.0 ** -22 + U[dtype]) * ref.abs() + TINY[dtype]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("I", [64, 40, 33, 257])
def test_gates_whose_logistic_function_is_subnormal(I, dtype):
    gates = torch.tensor([-86.0, -87.0, -87.5, -88.0, -88.5], device="cuda").repeat_interleave(6)
    ups = torch.tensor([1.0, -3.0, 1e10, 1e30, 1e38, -2e38], device="cuda").repeat(5)
    g = gates[:, None].expand(30, I).to(dtype)
    u = (ups[:, None] * (1 + 0.25 * torch.rand(30, I, generator=torch.Generator(device="cuda").manual_seed(I), device="cuda"))).to(dtype)
    gu, da = torch.cat([g, u], 1).contiguous(), torch.ones(30, I, device="cuda", dtype=dtype)
    da[:, 1::2] = -0.5
    gd, ud, d = g.double(), u.double(), da.double()
    s = torch.sigmoid(gd)
    act = ops.swiglu(gu)
    _near(act, gd * s * ud, gd, dtype)
    again, codes, scales = ops.swiglu_checkpoint(gu)
    assert torch.equal(act, again)
    dg, du = ops.swiglu_backward(da, gu).chunk(2, 1)
    _near(du, d * gd * s, gd, dtype)
    _near(dg, d * ud * s * (1 + gd * (1 - s)), gd, dtype)
    # from 8 bits: gates on whole steps (of 1) and ups as they are kept
    whole = torch.cat([gates[:, None].round().expand(30, I).to(dtype), u], 1).contiguous()
    act, codes, scales = ops.swiglu_checkpoint(whole)
    kept = ops.restore_rows(*ops.checkpoint_rows(whole[:, I:].contiguous()), torch.float32).double()
    gd = whole[:, :I].double()
    s = torch.sigmoid(gd)
    dgu, again = ops.swiglu_checkpoint_backward(da, codes, scales)
    dg, du = dgu.chunk(2, 1)
    _near(again, gd * s * kept, gd, dtype)
    _near(du, d * gd * s, gd, dtype)
    _near(dg, d * kept * s * (1 + gd * (1 - s)), gd, dtype)
