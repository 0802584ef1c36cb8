"""How the gate of the norm between two blocks is told apart: batches of no rows, and of as many
rows as channels."""
import pytest
import torch

from mixture_experts_forward_moe_gb300 import binding as B
from test_gpu_block_ops import BF, HF, norm_inputs, rand

pytestmark = pytest.mark.gpu

CHANNEL_GRADS = ("d_post_weight", "d_pre_weight")


@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
def test_no_rows_with_any_gate(gate, cuda_device):
    d = norm_inputs(0, 64, BF, gate, True, True, 0.0, True)
    s, h = B.moe_block_norm(**d)
    assert s.shape == h.shape == (0, 64)
    got = B.moe_block_norm_bwd(torch.empty_like(s), torch.empty_like(s), **d)
    for k in CHANNEL_GRADS + (("d_gate",) if gate == "channel" else ()):
        assert got[k].shape == (64,) and (got[k] == 0).all(), k
    if gate in ("token", "element"):
        assert got["d_gate"].shape == d["gate"].shape
