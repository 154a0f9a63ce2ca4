"""Rows with offsets that no expert_order makes: nothing outside the tensors is written."""
import pytest
import torch

from combine_persistent_warp_gb300 import native, ops

pytestmark = pytest.mark.gpu
CODE = {torch.float32: 0, torch.bfloat16: 1}


@pytest.mark.parametrize("H", [64, 70])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("end", [-(1 << 31), -5, 12, 13, 1 << 30, (1 << 31) - 200, (1 << 31) - 1])
def test_offsets_that_lie_are_kept_inside(H, dtype, end):
    T, k = 6, 2
    M = T * k
    torch.manual_seed(0)
    x, y = torch.randn(T, H, device="cuda").to(dtype), torch.randn(M, H, device="cuda").to(dtype)
    order = ops.expert_order(torch.zeros(T, k, dtype=torch.int64, device="cuda"), 1)
    w = torch.rand(T, k, device="cuda")
    lie = torch.tensor([0, end], dtype=torch.int32, device="cuda")
    guarded = torch.full((M + 2000, H), 7.0, dtype=dtype, device="cuda")
    out = guarded[1000:1000 + M]
    lib, s, q = native.load(), torch.cuda.current_stream().cuda_stream, lambda t: t.data_ptr()
    dw = torch.empty(T, k, device="cuda")
    assert lib.moe_gather_rows(T, k, H, 1, M, q(x), H, CODE[dtype], q(order.rows), q(lie), q(out), s) == 0
    assert (guarded[:1000] == 7).all() and (guarded[1000 + M:] == 7).all()
    if end >= M:
        assert torch.equal(out, ops.gather_rows(x, order.rows, order.offsets))
    out.fill_(7)
    assert lib.moe_combine_rows_backward(T, k, H, 1, M, q(x), H, q(y), CODE[dtype], q(order.rows), q(w), q(lie), q(out), q(dw), s) == 0
    assert (guarded[:1000] == 7).all() and (guarded[1000 + M:] == 7).all()
    if end >= M:
        assert torch.equal(out, ops.combine_rows_backward(x, y, order.rows, w, order.offsets)[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [1, 2, 3, 5, 6, 7, 10, 13, 18, 21, 22])
def test_combine_of_short_rows_near_the_matrix_ends(H, dtype):
    """Every row of y by itself, first to last, for rows shorter than the vectors that move them."""
    M = 64
    torch.manual_seed(H)
    rows = torch.arange(M, dtype=torch.int32, device="cuda")[:, None].contiguous()
    buf = torch.full((M * H + 16,), float("nan"), dtype=dtype, device="cuda")
    lib, s = native.load(), torch.cuda.current_stream().cuda_stream
    for at in range(0, 8):
        y = buf[at:at + M * H].view(M, H)
        buf.fill_(float("nan"))
        y.copy_(torch.randn(M, H, device="cuda"))
        out = torch.zeros(M, H, dtype=dtype, device="cuda")
        assert lib.moe_combine_rows(M, 1, H, M, y.data_ptr(), CODE[dtype], rows.data_ptr(), None, out.data_ptr(), s) == 0
        assert torch.equal(out, y)
