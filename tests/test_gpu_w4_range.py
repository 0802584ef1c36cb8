"""4-bit weights against bf16 x of any magnitude: the products are taken in f16, and so are scaled."""
import pytest
import torch

import block_reference as R
import dense_reference as D
from mixture_experts_forward_moe_gb300 import binding as B
from test_gpu_block_ops import BF, rand
from test_gpu_dense_block import weights4

pytestmark = pytest.mark.gpu

MAGNITUDES = [1.0, 1e-2, 6e-5, 3e5, 1e-6, 1e-20, 3e10, 1e-36, 1e30, 3e37, 1.0]


def rows_of(T, K, seed, magnitudes):
    x = rand(T, K, seed=seed, dtype=torch.float32)
    m = torch.tensor([magnitudes[(i + T) % len(magnitudes)] for i in range(T)], device="cuda")
    x = x * m[:, None]
    x[T // 2, : K // 3] *= 1e-9  # and within a row
    return x.to(BF)


def sums64(x, w):
    """(x w^T, bound): K/16 + 32 additions of a step each, and x in f16: 2^-25 off in a row whose
    largest value is 0.5 or more, and 2^-39 of that value in any."""
    x = x.cpu().double()
    z, off = D.product64(x, w)
    top = x.abs().amax(dim=1, keepdim=True)
    less = torch.where(top >= 0.5, (2.0 ** -39 * top).clamp(min=2.0 ** -25), 2.0 ** -39 * top)
    return z, off + less * w.abs().sum(1) + 4 * R.F32 * z.abs()


# T, N, K: the streamed rows, whose x is staged in one or several chunks, and tiles; K in one and in
# several parts, with an end inside a block
SIZES = [(1, 70, 160), (1, 33, 40000), (4, 300, 4096), (7, 130, 18432), (11, 260, 7168), (16, 64, 2080),
         (20, 500, 4096), (70, 64, 18464), (140, 130, 96)]


@pytest.mark.parametrize("T,N,K", SIZES)
def test_rows_of_any_magnitude(T, N, K, cuda_device):
    codes, scales, alpha = weights4(N, K, seed=2)
    alpha = alpha / (K ** 0.5 * 64)
    w = D.weights64(codes, scales, alpha.cpu())
    x = rows_of(T, K, 1, MAGNITUDES)
    out = B.moe_linear_w4a16(x, codes, scales, alpha)
    z, off = sums64(x, w)
    assert bool((z.abs().amax(dim=1) < 3e38).all())
    R.assert_within(out, z, D.rounded(z, off, BF), "out")
    assert torch.equal(out, B.moe_linear_w4a16(x, codes, scales, alpha))
    one = B.moe_linear_w4a16(x[:1].contiguous(), codes, scales, alpha)
    R.assert_within(one, z[:1], D.rounded(z[:1], off[:1], BF), "one row")


@pytest.mark.parametrize("T,F,K", [(1, 70, 160), (5, 130, 7168), (16, 64, 2080), (40, 64, 4128)])
def test_gated_rows_of_any_magnitude(T, F, K, cuda_device):
    codes, scales, alpha = weights4(2 * F, K, seed=2)
    alpha = alpha / (K ** 0.5 * 64)
    w = D.weights64(codes, scales, alpha.cpu())
    x = rows_of(T, K, 1, [1.0, 1e-2, 6e-5, 3e5, 1e-6, 1e-12, 3e10])
    z, off = sums64(x, w)
    g, u, og, ou = z[:, :F], z[:, F:], off[:, :F], off[:, F:]
    a = R.act64(g, "silu")
    h = a * u
    bound = 1.2 * og * (u.abs() + ou) + a.abs() * ou + D.EVAL * h.abs()
    # g - e^-g of a gate next to 0 is good to a step of 1/2, which `h` has in its own measure
    R.assert_within(B.moe_gated_linear_w4a16(x, codes, scales, alpha), h, D.rounded(h, bound, BF), "out")


@pytest.mark.parametrize("T", [3, 7, 12, 20, 70])
def test_a_rows_scale_is_its_own(T, cuda_device):
    """Whatever lies in one row, the others' results keep their bits."""
    N, K = 100, 1056
    codes, scales, alpha = weights4(N, K, seed=2)
    x = rows_of(T, K, 1, [1.0, 1e-3, 2.0, 30.0])
    x[0] *= 1e-4
    want = B.moe_linear_w4a16(x, codes, scales, alpha)
    row = T - 2
    rest = [i for i in range(T) if i != row]
    for bad in (1e38, 1e-38, 0.0, float("inf"), float("nan")):
        y = x.clone()
        y[row] = (y[row].float() * bad).to(BF)
        got = B.moe_linear_w4a16(y, codes, scales, alpha)
        assert torch.equal(got[rest], want[rest]), bad
        if bad != bad or bad == float("inf"):
            assert not bool(torch.isfinite(got[row]).any())
        if bad == 0.0:
            assert not bool(got[row].any())
    B.get_device_status(B.call_workspace(cuda_device))
