"""The scratch of calls without a workspace: no place for an x that comes in 16 bits, and given back."""
import ctypes

import pytest
import torch

from mixture_experts_forward_moe_gb300 import binding as B
from test_gpu_block_ops import BF, rand

pytestmark = pytest.mark.gpu

T, K, N = 2048, 1032, 272  # F = 136


def tensors():
    return (rand(T, K, seed=1, dtype=BF), rand(N, K, seed=2, std=K ** -0.5, dtype=BF),
            rand(T, N, seed=3, dtype=BF), rand(T, N // 2, seed=4, dtype=BF))


def test_what_calls_hold(cuda_device):
    x, w, dy, dh = tensors()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lin, gated = B.Linear(T, N, K, 0, 0, 0), B.GatedLinear(T, K, N // 2, 0, 0)
    L = B.lib()
    small = max(int(L.moe_linear_bwd_workspace_size_x16(ctypes.byref(lin))),
                int(L.moe_gated_linear_bwd_workspace_size_x16(ctypes.byref(gated))))
    B.release_call_workspaces()
    got = B.moe_linear_bwd(dy, x, w, stream=s), B.moe_gated_linear_bwd(dh, x, w, stream=s)
    assert B.call_workspace(cuda_device, stream=s).numel() == small
    with torch.cuda.stream(s):
        x8 = B.moe_checkpoint(x)
    B.moe_linear_bwd(dy, x8, w, stream=s)
    full = int(L.moe_linear_bwd_workspace_size(ctypes.byref(lin)))
    assert B.call_workspace(cuda_device, stream=s).numel() == full > max(small, T * K * 2)
    s.synchronize()
    # in a workspace of just that size, whose end is kept
    for desc, call, want in ((lin, lambda ws: B.moe_linear_bwd(dy, x, w, workspace=ws), got[0]),
                             (gated, lambda ws: B.moe_gated_linear_bwd(dh, x, w, workspace=ws), got[1])):
        fn = "moe_linear_bwd" if desc is lin else "moe_gated_linear_bwd"
        n = int(getattr(L, fn + "_workspace_size_x16")(ctypes.byref(desc)))
        whole = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        whole[:256] = 0
        again = call(whole[:n])
        assert all(torch.equal(again[k], want[k]) for k in want)
        assert bool((whole[n:] == 0xFF).all()) and B.get_device_status(whole[:n]) == B.MOE_OK


def test_scratch_is_given_back(cuda_device):
    x, w, dy, _ = tensors()
    x8 = B.moe_checkpoint(x)
    B.release_call_workspaces()
    torch.cuda.synchronize()
    want = B.moe_linear_bwd(dy, x8, w)
    held = torch.cuda.memory_allocated()
    B.release_call_workspaces()  # the call may still run: the stream's order keeps it whole
    assert torch.cuda.memory_allocated() <= held - T * K * 2
    filler = [torch.full((T * K * 2,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(4)]
    again = B.moe_linear_bwd(dy, x8, w)
    torch.cuda.synchronize()
    assert all(torch.equal(again[k], want[k]) for k in want) and len(filler) == 4
    assert B.get_device_status(B.call_workspace(cuda_device)) == B.MOE_OK
    B.release_call_workspaces()
    assert B.get_device_status(B.call_workspace(cuda_device)) == B.MOE_OK
