"""Sizes next to 2^31: rows, columns and reduction lengths that a 32-bit sum with a tile's size would
pass.  A few rows at the start, the middle and the end are compared with 64 bits."""
import pytest
import torch

import block_reference as R
from mixture_experts_forward_moe_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
FAR = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def room(cuda_device):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GB of device memory")
    yield
    torch.cuda.empty_cache()


def spots(n, width=300):
    return [slice(0, width), slice(n // 2, n // 2 + width), slice(n - width, n)]


def normal(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(rows, cols, dtype=BF, device="cuda").normal_(generator=g)


def test_block_norm_of_rows_next_to_2_31(cuda_device):
    y = normal(FAR, 8, 1)
    wq = torch.full((8,), 0.5, dtype=BF, device="cuda")
    s, _ = B.moe_block_norm(y, post_weight=wq, pre_norm=False, eps=1e-5)
    for at in spots(FAR):
        c = y[at].cpu().double()
        args = (c, None, 1.0, wq.cpu().double(), None, True, False, 1.0, 0.0, 1e-5)
        R.assert_within(s[at], R.norm64(*args)[0], R.norm_bounds(*args, BF)[0], str(at))


def test_block_norm_gradients_of_rows_next_to_2_31(cuda_device):
    y, dr = normal(FAR, 8, 1), normal(FAR, 8, 2)
    got = B.moe_block_norm_bwd(dr, None, y, pre_norm=False, eps=1e-5)
    for at in spots(FAR):
        ref, mag = R.norm_bwd64(dr[at].cpu().double(), None, y[at].cpu().double(), None, 1.0, None,
                                None, True, False, 1.0, 0.0, 1e-5)
        R.assert_within(got["d_branch"][at], ref["branch"],
                        R.grad_bound(ref["branch"], mag["branch"], BF), str(at))


@pytest.mark.parametrize("N", [8, 5])  # whole vectors of outputs, and one by one
def test_linear_of_rows_next_to_2_31(N, cuda_device):
    x, w, r = normal(FAR, 8, 1), normal(N, 8, 2), normal(FAR, N, 3)
    want = [R.linear64(x[at], w, None, "none", r[at], BF) for at in spots(FAR)]
    B.moe_linear(x, w, residual=r, out=r)
    assert B.get_device_status(B.call_workspace(cuda_device)) == B.MOE_OK
    for at, (ref, bound) in zip(spots(FAR), want):
        R.assert_within(r[at], ref, bound, str(at))


@pytest.mark.parametrize("T", [1, 3])
def test_linear_of_columns_next_to_2_31(T, cuda_device):
    x, w = normal(T, 8, 1), normal(FAR, 8, 2)
    out = B.moe_linear(x, w, activation="relu2")
    assert B.get_device_status(B.call_workspace(cuda_device)) == B.MOE_OK
    for at in spots(FAR):
        ref, bound = R.linear64(x, w[at], None, "relu2", None, BF)
        R.assert_within(out[:, at], ref, bound, str(at))


# Ones (and halves): a lane's or an accumulator's sums are multiples of their last bit's weight below
# 2^24 of it, so exact; the last of eight parts and their sums round, ten times at most.
@pytest.mark.parametrize("T", [1, 2])
def test_linear_of_a_reduction_next_to_2_31(T, cuda_device):
    K = 2 ** 31 - 8
    x = torch.ones(T, K, dtype=BF, device="cuda")
    w = torch.ones(3, K, dtype=BF, device="cuda")
    w[1] = 0.5
    out = B.moe_linear(x, w, out_dtype=torch.float32)
    assert B.get_device_status(B.call_workspace(cuda_device)) == B.MOE_OK
    ref = torch.tensor([1.0, 0.5, 1.0], dtype=torch.float64) * K
    assert (out.cpu().double() / ref - 1).abs().max() <= 10 * R.F32
