"""The RMS norm's gradients in each of the forms that long batches of short rows go through, against 64-bit formulas.

The bounds are those of test_gpu_ops_rms; here too no block has more than T/100 rows one after another.
"""
import pytest
import torch

import test_gpu_ops_rms as rms
from combine_persistent_warp_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,wdtype", rms.TYPES)
@pytest.mark.parametrize("T,H", [(6000, 520), (6000, 577), (6000, 701), (6001, 1001), (6000, 1023), (6000, 1024), (9000, 600), (9000, 1016), (700, 1001),
                                 (6000, 576), (6000, 512)])
def test_long_batches_of_short_rows(T, H, dtype, wdtype):
    v = rms._inputs(T, H, dtype, wdtype)
    y, rstd, h = got = ops.rms_norm(v["x"], v["w"], residual=v["r"])
    rms._check_forward(got, v["x"], v["w"], v["r"])
    for dh in (v["dh"], None):
        both = ops.rms_norm_backward(v["dy"], h, v["w"], rstd, dh=dh)
        rms._check_backward(both, v["dy"], h, v["w"], dh, rstd)
        only, none = ops.rms_norm_backward(v["dy"], h, v["w"], rstd, dh=dh, weight_grad=False)
        assert none is None and torch.equal(only, both[0])


@pytest.mark.parametrize("T,H,off,pitch", [(6000, 1001, 0, 1009), (6000, 1001, 8, 1009), (6000, 701, 0, 1405), (6000, 701, 3, 704), (6000, 1024, 0, 1040),
                                           (6000, 1024, 1, 1025), (5000, 640, 8, 648)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_long_batches_of_short_strided_rows(T, H, off, pitch, dtype):
    """What lies between the rows is NaN."""
    v = rms._inputs(T, H, dtype, dtype)

    def placed(t):
        flat = torch.full((T * pitch + off,), float("nan"), device="cuda", dtype=dtype)[off:]
        s = flat.as_strided((T, H), (pitch, 1))
        s.copy_(t)
        return s

    dy, dh = placed(v["dy"]), placed(v["dh"])
    _, rstd, h = ops.rms_norm(v["x"], v["w"], residual=v["r"])
    h = placed(h)
    w = torch.cat([v["w"][:1], v["w"]])[1:]
    for up in (dh, None):
        rms._check_backward(ops.rms_norm_backward(dy, h, w, rstd, dh=up), dy, h, w, up, rstd)
