"""A group of as many rows as a call may have."""
import pytest
import torch

from combine_persistent_warp_gb300 import ops

pytestmark = pytest.mark.gpu


def test_weight_gradient_of_one_group_of_2_to_the_30_rows():
    """One of 128 experts has every row, so that its tile is not split and takes some seconds: longer than
    a wait of the kernel has by itself.  Few rows are not zero, at both ends; their sums are exact."""
    M, E, n = 1 << 30, 128, 8
    dy, x = (torch.zeros(M, n, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    at = torch.tensor([0, 1, M // 2, M - 65, M - 1], device="cuda")
    torch.manual_seed(0)
    dy[at], x[at] = (torch.randint(-8, 9, (5, n), device="cuda").bfloat16() for _ in range(2))
    off = torch.full((E + 1,), M, dtype=torch.int32, device="cuda")
    off[:4] = 0                                       # expert 3 has them all
    dw = ops.grouped_mm_dw(dy, x, off, dtype=torch.float32)
    assert ops.get_error() == 0
    assert torch.equal(dw[3], dy[at].float().t() @ x[at].float())
    assert not dw[:3].any() and not dw[4:].any()
