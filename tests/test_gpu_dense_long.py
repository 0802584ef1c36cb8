"""Products of a long K, whose accumulators are added up on the way: captured, repeated, and with waits
that give up."""
import ctypes

import pytest
import torch

from mixture_experts_forward_moe_gb300 import binding as B
from test_gpu_block_ops import HF
from test_gpu_dense_block import weights4
from test_gpu_dense_large import normal
from test_gpu_dense_use import same

pytestmark = pytest.mark.gpu


def size(fn, desc):
    return int(getattr(B.lib(), fn + "_workspace_size")(ctypes.byref(desc)))


def gated(T, H, F):
    return (normal(T, H, seed=1), normal(2 * F, H, seed=2, std=H ** -0.5), normal(T, F, seed=3),
            B.GatedLinear(T, H, F, 0, 0))


def call_of(name):
    """(a call that takes a workspace, the bytes that it needs)."""
    if name in ("gated", "gated_bwd"):  # tiles of 256 rows, whole ones and split ones, ragged ends
        x, w, dh, desc = gated(2500, 16392, 1096)
        if name == "gated":
            return lambda ws=None: B.moe_gated_linear(x, w, workspace=ws), size("moe_gated_linear", desc)
        return (lambda ws=None: B.moe_gated_linear_bwd(dh, x, w, want_out=True, workspace=ws),
                size("moe_gated_linear_bwd", desc))
    if name == "linear_bwd":
        T, N, K = 20011, 2312, 2312
        dy, x, w = normal(T, N, seed=1), normal(T, K, seed=2), normal(N, K, seed=3)
        return (lambda ws=None: B.moe_linear_bwd(dy, x, w, want_bias=True, workspace=ws),
                size("moe_linear_bwd", B.Linear(T, N, K, 0, 0, 0)))
    if name == "few":
        x, w, _, desc = gated(40, 262152, 72)
        return lambda ws=None: B.moe_gated_linear(x, w, workspace=ws), size("moe_gated_linear", desc)
    T, K = (16, 300000 // 32 * 32) if name == "w4_rows" else (40, 300000 // 32 * 32)
    codes, scales, alpha = weights4(70, K, seed=1)
    x, alpha = normal(T, K, seed=2).to(HF), alpha / K
    return (lambda ws=None: B.moe_linear_w4a16(x, codes, scales, alpha, workspace=ws),
            size("moe_linear_w4a16", B.Linear(T, 70, K, B.MOE_F16, 0, 0)))


@pytest.mark.parametrize("name", ["gated", "gated_bwd", "linear_bwd", "few", "w4_rows", "w4_tiles"])
def test_captured_and_repeated(name, cuda_device):
    call, bytes_ = call_of(name)
    want = call()
    ws = torch.full((bytes_ + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    assert same(call(ws[:bytes_]), want)
    assert bool((ws[bytes_:] == 0xFF).all()) and B.get_device_status(ws[:bytes_]) == B.MOE_OK
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", ["gated", "gated_bwd", "linear_bwd", "few", "w4_tiles"])
def test_a_wait_that_gives_up(name, cuda_device):
    """The wait limit is 0, so that the first look that finds nothing landed gives up; nothing hangs."""
    call, bytes_ = call_of(name)
    ws = B.new_workspace(bytes_)
    want = call(ws)
    torch.cuda.synchronize()
    old = B.set_wait_limit_ns(0)
    try:
        for _ in range(2):
            call(ws)
            assert B.get_device_status(ws) == B.MOE_ERR_TIMEOUT  # synchronises, clears
    finally:
        B.set_wait_limit_ns(old)
    assert same(call(ws), want) and B.get_device_status(ws) == B.MOE_OK
