"""Waits of the grouped GEMMs that give up when K is so short that every copy is on its way before
anything is waited for: reported, and the next call is right.  The wait limit is 0, so that the first
look that finds nothing landed gives up; nothing hangs."""
import pytest
import torch

from helpers import run_fused
from mixture_experts_forward_moe_gb300 import binding as B
from mixture_experts_forward_moe_gb300 import inputs

pytestmark = pytest.mark.gpu


def gives_up(call, ws):
    want = call().clone()
    assert B.get_device_status(ws) == B.MOE_OK
    old = B.set_wait_limit_ns(0)
    try:
        for _ in range(2):
            call()
            assert B.get_device_status(ws) == B.MOE_ERR_TIMEOUT  # synchronises, clears
    finally:
        B.set_wait_limit_ns(old)
    assert torch.equal(call(), want)
    assert B.get_device_status(ws) == B.MOE_OK


# the direct path, token rows, the SM-pair down projection (at least 96 rows per expert), and the
# NVFP4 forms of the first two and of gathered rows
@pytest.mark.parametrize("T,E,H,F,weights", [
    (4, 16, 256, 64, "bf16"), (96, 16, 256, 64, "bf16"), (600, 8, 256, 128, "bf16"),
    (4, 16, 256, 128, "nvfp4"), (96, 16, 256, 128, "nvfp4"), (300, 8, 256, 128, "nvfp4"),
])
def test_a_short_grouped_gemm_that_gives_up(T, E, H, F, weights, cuda_device):
    w = inputs.Workload("short-waits", T=T, H=H, E=E, F=F, top_k=4, S=64, weights=weights)
    d = inputs.generate(w, seed=5, device=cuda_device)
    prob = B.make_problem(w.T, w.H, w.E, w.F, w.top_k, w.dtype, w.scoring_func, w.renormalize,
                          w.num_expert_group, w.topk_group, w.routed_scaling_factor, w.S)
    ws = B.new_workspace(B.workspace_size(prob), cuda_device)
    gives_up(lambda: run_fused(w, d, workspace=ws), ws)


@pytest.mark.parametrize("E,max_m,K,N,total", [(5, 16, 128, 128, 9), (3, 144, 384, 256, 200),
                                               (4, 256, 512, 256, 600)])
def test_a_short_fp8_gemm_that_gives_up(E, max_m, K, N, total, cuda_device):
    w = inputs.Fp8GemmWorkload("t", E=E, max_m=max_m, K=K, N=N, total=total)
    d = inputs.generate_fp8_gemm(w, seed=E + K, device=cuda_device)
    ws = B.new_workspace(1 << 20, cuda_device)
    gives_up(lambda: B.moe_grouped_gemm_fp8(d["a"], d["a_scale"], d["b"], d["b_scale"], d["meta"],
                                            workspace=ws), ws)
