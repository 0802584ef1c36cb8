"""f32 results of long sums: where the tensor cores' truncation shows (positive operands, whose
partial sums all grow one way), and every option beside them."""
import pytest
import torch

import block_reference as R
from mixture_experts_forward_moe_gb300 import binding as B
from test_gpu_block_ops import BF, HF, rand

pytestmark = pytest.mark.gpu

BLOCKS = 8  # 64-k blocks that one accumulator meets at most


# The sum of an accumulator after j of its J = 4 BLOCKS MMAs is j / J of its last one, and each MMA
# cuts it to 24 bits: by half a step on average, and a step is at most 2^-23 of it.  The average
# loss is then at most sum_j (j / J) / 2 = (J + 1) / 4 steps.  Accumulators and parts are added in
# f32 rounded to nearest, which leaves no average; one more step is allowed for it.  Chains of two
# and three times the blocks lost 16.6 and 32 to 37 steps.  (bf16: the products' 16 bits are whole.
# f16's have 22, some of which the tensor cores cut as well, so this does not bound them.)
@pytest.mark.parametrize("T,N,K", [
    (128, 128, 32768), (128, 128, 51200), (65, 256, 25600), (100, 100, 49152),  # few tiles, long K
    (16, 19584, 7168), (32, 19584, 7168), (64, 19584, 7168),  # so many tiles that K stays whole
    (7, 26000, 18432),
    (64, 7168, 7168), (300, 128, 32768), (300, 512, 7168), (5, 256, 7168),
])
def test_f32_sums_lose_no_more_than_short_accumulators(T, N, K, cuda_device):
    g = torch.Generator(device="cuda").manual_seed(T + N + K)
    x = torch.randn(T, K, generator=g, device="cuda").abs().to(BF)
    w = (torch.randn(N, K, generator=g, device="cuda").abs() * K ** -0.5).to(BF)
    out = B.moe_linear(x, w, out_dtype=torch.float32)
    assert B.get_device_status(B.call_workspace(cuda_device)) == B.MOE_OK
    z = x.double() @ w.double().T
    lost = float(((z - out.double()) / z).mean()) * 2.0 ** 23
    assert abs(lost) <= (4 * BLOCKS + 1) / 4 + 1, lost


# so long that accumulators are added while others fill, ragged, with everything in the epilogue
LONG = [(5, 130, 24576, HF, "silu", True, True), (20, 257, 20488, BF, "gelu_tanh", True, False),
        (60, 100, 18440, HF, "relu2", False, True), (100, 64, 32768, BF, "none", True, True),
        (3, 19600, 2056, BF, "none", True, True)]


@pytest.mark.parametrize("T,N,K,dtype,act,bias,res", LONG)
def test_long_f32_sums(T, N, K, dtype, act, bias, res, cuda_device):
    x, w = rand(T, K, seed=1, dtype=dtype), rand(N, K, seed=2, std=K ** -0.5, dtype=dtype)
    b = rand(N, seed=3, dtype=dtype) if bias else None
    r = rand(T, N, seed=4) if res else None
    ws = B.new_workspace(256, cuda_device)
    kw = dict(bias=b, activation=act, residual=r, out_dtype=torch.float32, workspace=ws)
    out, again = B.moe_linear(x, w, **kw), B.moe_linear(x, w, **kw)
    assert torch.equal(out, again) and B.get_device_status(ws) == B.MOE_OK
    ref, bound = R.linear64(x, w, b, act, r, torch.float32)
    R.assert_within(out, ref, bound, "linear")


def test_long_f32_sums_that_give_up(cuda_device):
    x, w = rand(16, 32768, seed=1, dtype=BF), rand(300, 32768, seed=2, std=0.01, dtype=BF)
    ws = B.new_workspace(256, cuda_device)
    kw = dict(out_dtype=torch.float32, workspace=ws)
    want = B.moe_linear(x, w, **kw)
    torch.cuda.synchronize()
    old = B.set_wait_limit_ns(0)
    try:
        B.moe_linear(x, w, **kw)
        got = B.get_device_status(ws)
    finally:
        B.set_wait_limit_ns(old)
    assert got == B.MOE_ERR_TIMEOUT
    assert torch.equal(B.moe_linear(x, w, **kw), want) and B.get_device_status(ws) == B.MOE_OK
