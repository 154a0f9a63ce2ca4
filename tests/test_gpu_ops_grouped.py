"""Grouped products by expert, forward and both gradients, against 64-bit products.

Bound: the tensor core adds 16 products at a time to an fp32 sum by truncation, so a sum of n
products is at most (n/16 + 2) * 2^-22 * sum|a*b| off (2^-23 for the sum's own truncation a step,
as much for the products' alignment), and the result is rounded once more to the output's type.
"""
import pytest
import torch

from combine_persistent_warp_gb300 import ops

pytestmark = pytest.mark.gpu
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -10}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -24}


def _offsets(sizes):
    return torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def _case(sizes, N, K, dtype, extra=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)
    M = sum(sizes) + extra
    return r(M, K), r(len(sizes), N, K) * 0.25, r(M, N), _offsets(sizes)


def _bounded(got, ref, mag, n):
    u = U[got.dtype]
    e = (n / 16 + 2) * 2.0 ** -22 * mag + u * ref.abs() + TINY[got.dtype]
    assert ((got.double() - ref).abs() <= e).all()


def _check(x, w, dy, off, dw_dtype=None):
    o = off.tolist()
    M, (E, N, K) = x.shape[0], w.shape
    D = torch.double
    y, dx = ops.grouped_mm(x, w, off), ops.grouped_mm_dx(dy, w, off)
    dw = ops.grouped_mm_dw(dy, x, off, dtype=dw_dtype)
    assert ops.get_error() == 0
    assert y.shape == (M, N) and dx.shape == (M, K) and dw.shape == (E, N, K)
    for e in range(E):
        s = slice(o[e], o[e + 1])
        xe, we, de = x[s].to(D), w[e].to(D), dy[s].to(D)
        _bounded(y[s], xe @ we.t(), xe.abs() @ we.abs().t(), K)
        _bounded(dx[s], de @ we, de.abs() @ we.abs(), N)
        _bounded(dw[e], de.t() @ xe, de.abs().t() @ xe.abs(), o[e + 1] - o[e])
    assert (y[o[-1]:] == 0).all() and (dx[o[-1]:] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes,N,K", [
    ([1], 8, 8), ([1], 256, 64), ([5, 0, 1], 264, 200), ([64, 128], 128, 256), ([256], 256, 256), ([257, 255], 512, 136),
    ([0, 0, 0], 64, 64), ([16, 17, 15, 31, 33], 72, 520), ([300, 1, 0, 700, 513], 320, 448), ([1000], 1032, 1096),
    ([2, 0, 3, 1] * 40, 136, 104), ([512] * 3, 384, 128)])
def test_products(sizes, N, K, dtype):
    _check(*_case(sizes, N, K, dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes,N,K", [
    ([1], 256, 4096), ([3, 0, 40], 136, 2056), ([200], 520, 1544), ([5] * 9, 64, 7168), ([3000], 264, 136), ([900, 0, 4001], 72, 200),
    ([2000, 33], 2056, 64)])
def test_products_split_along_the_contraction(sizes, N, K, dtype):
    """Few tiles and a long contraction, with rows of no expert: sums of parts."""
    x, w, dy, off = _case(sizes, N, K, dtype, extra=3)
    _check(x, w, dy, off)
    _check(x, w, dy, off, torch.float32)
    acc = torch.randn(len(sizes), N, K, device="cuda").to(dtype)
    got = ops.grouped_mm_dw(dy, x, off, out=acc.clone(), accumulate=True)
    assert torch.equal(got, (acc.float() + ops.grouped_mm_dw(dy, x, off, dtype=torch.float32)).to(dtype))
    out = torch.full((x.shape[0], N + 24), 5.0, device="cuda", dtype=dtype)
    assert torch.equal(ops.grouped_mm(x, w, off, out=out[:, 8:8 + N]), ops.grouped_mm(x, w, off)) and (out[:, :8] == 5).all()


def test_missing_workspace_is_refused():
    import ctypes
    from combine_persistent_warp_gb300 import native
    lib, n = native.load(), ctypes.c_uint64()
    assert lib.moe_grouped_mm_workspace(16, 1, 256, 4096, ctypes.byref(n)) == 0 and n.value > 0
    x, w, dy, off = _case([16], 256, 4096, torch.bfloat16)
    out = torch.empty(16, 256, device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(n.value, device="cuda", dtype=torch.uint8)
    args = (16, 1, 256, 4096, x.data_ptr(), 4096, w.data_ptr(), off.data_ptr(), out.data_ptr(), 256, native.BF16)
    for p, size in ((None, n.value), (ws.data_ptr(), n.value - 1), (ws.data_ptr() + 64, n.value)):
        assert lib.moe_grouped_mm(*args, p, size, None) == 1
    assert lib.moe_grouped_mm_dw_workspace(16, 1, 256, 4096, ctypes.byref(n)) == 0 and n.value >= 256
    dw = torch.empty(1, 256, 4096, device="cuda", dtype=torch.bfloat16)
    assert lib.moe_grouped_mm_dw(16, 1, 256, 4096, dy.data_ptr(), 256, x.data_ptr(), 4096, off.data_ptr(), dw.data_ptr(), native.BF16,
                                 native.BF16, 0, ws.data_ptr(), n.value - 1, None) == 1


def test_ragged_groups_of_every_remainder():
    sizes = list(range(0, 70)) + [127, 129, 191, 193, 255, 257, 272, 289, 320]
    _check(*_case(sizes, 64, 72, torch.bfloat16))


def test_rows_of_no_expert_are_zero_and_not_read():
    x, w, dy, off = _case([30, 0, 50], 128, 192, torch.bfloat16, extra=41)
    x[80:], dy[80:] = float("nan"), float("inf")
    _check(x, w, dy, off)


def test_a_neighbour_groups_values_do_not_leak():
    """NaN and infinity in one expert's rows and weights stay in its own results."""
    x, w, dy, off = _case([37, 21, 40], 96, 80, torch.bfloat16)      # N, K and sizes that end inside tiles
    clean = [ops.grouped_mm(x, w, off), ops.grouped_mm_dx(dy, w, off), ops.grouped_mm_dw(dy, x, off)]
    x[37:58], dy[37:58] = float("nan"), float("inf")
    w[1] = float("nan")
    got = [ops.grouped_mm(x, w, off), ops.grouped_mm_dx(dy, w, off), ops.grouped_mm_dw(dy, x, off)]
    for i in range(2):
        assert torch.equal(got[i][:37], clean[i][:37]) and torch.equal(got[i][58:], clean[i][58:])
        assert got[i][37:58].isnan().all()
    assert torch.equal(got[2][0], clean[2][0]) and torch.equal(got[2][2], clean[2][2]) and got[2][1].isnan().all()


def test_strided_rows_and_given_outputs():
    x, w, dy, off = _case([20, 70], 128, 64, torch.bfloat16)
    wide_x = torch.full((90, 200), float("nan"), device="cuda", dtype=torch.bfloat16)
    wide_dy = torch.full((90, 400), float("nan"), device="cuda", dtype=torch.bfloat16)
    wide_x[:, 8:72], wide_dy[:, 16:144] = x, dy
    xs, dys = wide_x[:, 8:72], wide_dy[:, 16:144]
    out = torch.full((90, 160), 7.0, device="cuda", dtype=torch.bfloat16)
    got = ops.grouped_mm(xs, w, off, out=out[:, 24:152])
    assert torch.equal(got, ops.grouped_mm(x, w, off)) and (out[:, :24] == 7).all() and (out[:, 152:] == 7).all()
    assert torch.equal(ops.grouped_mm_dx(dys, w, off), ops.grouped_mm_dx(dy, w, off))
    assert torch.equal(ops.grouped_mm_dw(dys, xs, off), ops.grouped_mm_dw(dy, x, off))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,K", [(136, 264), (512, 320)])
def test_weight_gradient_types_and_accumulation(dtype, N, K):
    x, w, dy, off = _case([100, 0, 33], N, K, dtype)
    full = ops.grouped_mm_dw(dy, x, off, dtype=torch.float32)
    assert torch.equal(full.to(dtype), ops.grouped_mm_dw(dy, x, off))
    for kind in (torch.float32, dtype):
        base = torch.randn(3, N, K, device="cuda").to(kind)
        acc = base.clone()
        assert ops.grouped_mm_dw(dy, x, off, out=acc, accumulate=True) is acc
        assert torch.equal(acc, (base.float() + full).to(kind))
        assert torch.equal(acc[1], base[1])


def test_offsets_that_lie_are_kept_inside():
    x, w, dy, off = _case([40, 40], 64, 64, torch.bfloat16)
    for bad in ([-5, 40, 80], [0, 90, 60], [0, 40, 1 << 30], [0, -7, 80]):
        o = torch.tensor(bad, dtype=torch.int32, device="cuda")
        seq = torch.tensor(bad).clamp(0, 80).cummax(0).values.int().cuda()
        for f, a in ((ops.grouped_mm, (x, w)), (ops.grouped_mm_dx, (dy, w)), (ops.grouped_mm_dw, (dy, x))):
            assert torch.equal(f(*a, o), f(*a, seq))
    late = torch.tensor([10, 40, 80], dtype=torch.int32, device="cuda")      # rows before the first expert
    y = ops.grouped_mm(x, w, late)
    assert (y[:10] == 0).all() and torch.equal(y[40:], ops.grouped_mm(x, w, off)[40:])


def test_gradients_against_differences():
    h = 1e-4
    x, w, dy, off = _case([9, 0, 22], 40, 56, torch.float16)
    o = off.tolist()
    dx, dw = ops.grouped_mm_dx(dy, w, off), ops.grouped_mm_dw(dy, x, off, dtype=torch.float32)

    def f(x, w):
        return sum(((x[o[e]:o[e + 1]] @ w[e].t()) * dy[o[e]:o[e + 1]].double()).sum() for e in range(3))

    g = torch.Generator(device="cuda").manual_seed(3)
    vx = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.double)
    vw = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.double)
    xd, wd = x.double(), w.double()
    for grad, v, diff, u in ((dx, vx, (f(xd + h * vx, wd) - f(xd - h * vx, wd)) / (2 * h), 2.0 ** -10),
                             (dw, vw, (f(xd, wd + h * vw) - f(xd, wd - h * vw)) / (2 * h), 2.0 ** -18)):
        assert abs((grad.double() * v).sum() - diff) <= u * (grad.double() * v).abs().sum() + 1e-6


def test_empty_batch_and_equal_bits_again():
    x, w, dy, off = _case([0, 0], 64, 72, torch.bfloat16)
    assert ops.grouped_mm(x, w, off).shape == (0, 64)
    assert (ops.grouped_mm_dw(dy, x, off) == 0).all()
    keep = torch.ones(2, 64, 72, device="cuda")
    assert (ops.grouped_mm_dw(dy, x, off, out=keep, accumulate=True) == 1).all()
    x, w, dy, off = _case([513, 100, 300], 520, 264, torch.bfloat16)
    for f, a in ((ops.grouped_mm, (x, w)), (ops.grouped_mm_dx, (dy, w)), (ops.grouped_mm_dw, (dy, x))):
        first = f(*a, off)
        assert all(torch.equal(first, f(*a, off)) for _ in range(3))


def test_another_stream_and_a_graph():
    x, w, dy, off = _case([70, 60], 256, 128, torch.bfloat16)
    ref = ops.grouped_mm(x, w, off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ops.grouped_mm(x, w, off, stream=s)
    s.synchronize()
    assert torch.equal(got, ref)
    out = torch.zeros_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.grouped_mm(x, w, off, out=out)
    x.copy_(torch.randn_like(x))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ops.grouped_mm(x, w, off))


def test_results_past_32_bit_offsets():
    sizes, N, K = [300000, 230001], 4096, 64            # out: 2.17e9 elements
    x, w, _, off = _case(sizes, N, K, torch.bfloat16)
    y = ops.grouped_mm(x, w, off)
    D = torch.double
    for a in (0, 299990, 300000, 529990):
        s = slice(a, a + 10)
        e = 0 if a < 300000 else 1
        _bounded(y[s], x[s].to(D) @ w[e].to(D).t(), x[s].to(D).abs() @ w[e].to(D).abs().t(), K)


def test_refusals_of_tensors():
    x, w, dy, off = _case([4, 4], 64, 64, torch.bfloat16)
    with pytest.raises(TypeError):
        ops.grouped_mm(x, w.half(), off)
    with pytest.raises(ValueError):
        ops.grouped_mm(x[:, :56], w, off)
    with pytest.raises(ValueError):
        ops.grouped_mm(x, w, off[:2])
    with pytest.raises(TypeError):
        ops.grouped_mm(x, w, off.long())
    with pytest.raises(ValueError):
        ops.grouped_mm(x, w.transpose(1, 2), off)
    with pytest.raises(ops.MoeError):
        ops.grouped_mm(torch.zeros(4, 60, device="cuda").half(), torch.zeros(2, 64, 60, device="cuda").half(), off)
    with pytest.raises(ops.MoeError):                    # rows that start off a 16-byte boundary
        ops.grouped_mm(torch.zeros(8, 72, device="cuda", dtype=torch.bfloat16)[:, 4:68], w, off)
    with pytest.raises(ValueError):
        ops.grouped_mm_dw(dy, x, off, accumulate=True)
    with pytest.raises(TypeError):
        ops.grouped_mm_dw(dy, x, off, dtype=torch.float16)
