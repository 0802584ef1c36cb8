"""Calls of the dense feed-forward block without rows are checked as others are."""
import pytest
import torch

from mixture_experts_forward_moe_gb300 import binding as B
from test_gpu_block_ops import BF, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [0, 4])
@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("H,F,act", [(60, 40, "silu"), (64, 44, "silu"), (64, 40, "relu2")])
def test_refusals_without_rows(T, save, H, F, act, cuda_device):
    x, w = torch.zeros(T, H, dtype=BF, device="cuda"), rand(2 * F, H, seed=1, dtype=BF)
    with pytest.raises(B.MoeError):
        B.moe_gated_linear(x, w, activation=act, save=save)
    d_out = torch.zeros(T, F, dtype=BF, device="cuda")
    with pytest.raises(B.MoeError):
        B.moe_gated_linear_bwd(d_out, x, w, activation=act)


def test_a_short_workspace_without_rows(cuda_device):
    x, w = torch.zeros(0, 64, dtype=BF, device="cuda"), rand(80, 64, seed=1, dtype=BF)
    short = torch.zeros(128, dtype=torch.uint8, device="cuda")
    for save in (False, True):
        with pytest.raises(B.MoeError, match="workspace"):
            B.moe_gated_linear(x, w, save=save, workspace=short)
