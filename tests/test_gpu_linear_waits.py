"""Waits of the dense product that give up, in each of its tensor-core forms: reported, and the next
call is right.  The wait limit is 0, so that the first look that finds nothing landed gives up;
nothing hangs."""
import pytest
import torch

import block_reference as R
from mixture_experts_forward_moe_gb300 import binding as B
from test_gpu_block_ops import BF, HF, rand

pytestmark = pytest.mark.gpu


# K short enough that every copy is on its way before anything is waited for, and longer
@pytest.mark.parametrize("T,N,K,dtype,f32", [
    (12, 256, 192, BF, False), (30, 256, 8, HF, False), (40, 512, 256, BF, True),
    (12, 256, 4096, HF, True), (60, 130, 2048, BF, False),   # one-CTA tiles, K split or not
    (300, 2048, 512, BF, False), (300, 1024, 4096, HF, False), (300, 1024, 4096, BF, True),
    (300, 5000, 328, BF, True),                               # pairs, 128 columns
    (1000, 5000, 1032, BF, False), (1300, 6152, 136, HF, False),  # pairs, 256 columns
])
def test_a_wait_that_gives_up_in_every_form(T, N, K, dtype, f32, cuda_device):
    x, w = rand(T, K, seed=1, dtype=dtype), rand(N, K, seed=2, std=K ** -0.5, dtype=dtype)
    odt = torch.float32 if f32 else dtype
    ws = B.new_workspace(256, cuda_device)
    kw = dict(out_dtype=torch.float32 if f32 else None, workspace=ws)
    want = B.moe_linear(x, w, **kw)
    torch.cuda.synchronize()
    old = B.set_wait_limit_ns(0)
    try:
        for _ in range(2):
            B.moe_linear(x, w, **kw)
            assert B.get_device_status(ws) == B.MOE_ERR_TIMEOUT  # synchronises, clears
    finally:
        B.set_wait_limit_ns(old)
    got = B.moe_linear(x, w, **kw)
    assert torch.equal(got, want) and B.get_device_status(ws) == B.MOE_OK
    ref, bound = R.linear64(x, w, None, "none", None, odt)
    R.assert_within(got, ref, bound, "linear")
