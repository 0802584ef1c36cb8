"""Sums of the dense feed-forward block: checkpoints as close to those of 64 bits as an f32 product's."""
import pytest
import torch

import dense_reference as D
from mixture_experts_forward_moe_gb300 import binding as B
from test_gpu_block_ops import BF, HF

pytestmark = pytest.mark.gpu


def randn(*shape, seed, dtype, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def neighbours(z, want):
    """Values of the checkpoint of `z` (64 bits) that are not those of `want`."""
    return int((D.checkpoint64(z)[0] != want).sum())


# T, H, F: K of a few blocks to many; the last one's tiles are all split along K
@pytest.mark.parametrize("T,H,F,dtype", [
    (65536, 136, 640, BF), (32768, 264, 1280, HF), (16384, 512, 2560, BF), (8192, 2056, 2560, BF),
    (4096, 7168, 2048, BF), (512, 7168, 2304, HF),
])
def test_saved_values_next_to_a_border(T, H, F, dtype, cuda_device):
    """A sum that is a little off falls on the other side of a border between E4M3 values now and
    then.  That may happen as often as to the sums of an f32 product, within three standard deviations
    of the difference of two such counts (each has the root of itself)."""
    x, w = randn(T, H, seed=1, dtype=dtype), randn(2 * F, H, seed=2, std=H ** -0.5, dtype=dtype)
    _, gate, up = B.moe_gated_linear(x, w, save=True)
    mine = plain = 0
    for part, saved in ((w[:F], gate), (w[F:], up)):
        for i in range(0, T, 4096):
            rows = slice(i, min(i + 4096, T))
            want = D.checkpoint64(x[rows].double() @ part.double().T)[0]
            got = B.moe_checkpoint_restore(B.Fp8Checkpoint(saved.codes[rows], saved.scale[rows], F),
                                           BF).double()
            mine += int((got != want).sum())
            plain += neighbours((x[rows].float() @ part.float().T).double(), want)
    assert mine <= plain + 3 * (2 * plain) ** 0.5, (mine, plain)
