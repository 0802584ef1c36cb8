"""Gates far out in the dense feed-forward block's gradients: what they are worth there, and that the
block computed again is the block that was computed."""
import pytest
import torch

import block_reference as R
import dense_reference as D
from mixture_experts_forward_moe_gb300 import binding as B
from test_gpu_block_ops import BF, rand

pytestmark = pytest.mark.gpu

GATES = [-3e38, -1e20, -1e12, -1e4, -300.0, -120.0, -100.0, -90.0, -81.0, -79.0, -60.0, -45.0, -41.0,
         -39.0, -30.0, -20.0, -11.0, -9.75, -9.5, -8.0, -7.5, -7.0, -1.0, 0.0, 1.0, 7.5, 9.5, 12.5,
         41.0, 81.0, 300.0, 1e4, 1e12, 1e20]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("saved", [False, True])
def test_gradients_of_far_gates(act, saved, cuda_device):
    T, H, F = len(GATES), 16, 8
    x = torch.zeros(T, H)
    x[:, 0], x[:, 1] = torch.tensor(GATES), 1.0
    w = torch.zeros(2 * F, H)
    w[:F, 0] = w[F:, 1] = 1.0  # gate = x0, up = 1
    x, w = x.to(BF).cuda(), w.to(BF).cuda()
    dh = rand(T, F, seed=1, dtype=BF)
    g = x[:, :1].double().cpu().expand(T, F)
    if saved:
        gate = B.moe_checkpoint(x[:, :1].expand(T, F).contiguous())
        up = B.moe_checkpoint(torch.ones(T, F, dtype=BF, device="cuda"))
        got = B.moe_gated_linear_bwd(dh, x, w, act, gate=gate, up=up, want_out=True)
        g = D.restore64(gate.codes, gate.scale, F)
    else:
        got = B.moe_gated_linear_bwd(dh, x, w, act, want_out=True)
    a, s, d = R.act64(g, act), D.slope64(g, act), dh.double().cpu()
    # e^-v is good to 2^-19 and to a rounding of v log2 e, 2^-24 of it, which it magnifies by v; past
    # v = 80 the slope's tail stays where it is, and below 1e-38 are subnormals that may be 0
    v = (g if act == "silu" else 1.6 * (g + 0.044715 * g ** 3)).abs().clamp(max=100)
    near, far = 2.0 ** -19 + v * 2.0 ** -22, 2.0 ** -100
    R.assert_within(got["out"], a, R.half_step(a, BF) + near * a.abs() + far, "out")
    # d_x0 = sum dh s, d_x1 = sum dh a: of terms that are rounded to bf16 before
    for col, t in ((0, d * s), (1, d * a)):
        ref = t.sum(1)
        bound = ((2.0 ** -8 + 2 * near) * t.abs() + far * d.abs()).sum(1)
        R.assert_within(got["d_x"][:, col], ref, bound + R.half_step(ref, BF) * (1 + 2.0 ** -7), f"d_x{col}")


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_the_block_computed_again(act, cuda_device):
    """Gates of all magnitudes: the gradient's `out` is the forward's, within a rounding of each."""
    T, H, F = 200, 264, 136
    x, w = rand(T, H, seed=1, dtype=BF), rand(2 * F, H, seed=2, dtype=BF)
    w[:F] = (w[:F].float() * torch.logspace(-2, 25, F, device="cuda")[:, None]).to(BF)
    w[F:] *= H ** -0.5
    dh = rand(T, F, seed=3, dtype=BF)
    out = B.moe_gated_linear(x, w, activation=act).double().cpu()
    again = B.moe_gated_linear_bwd(dh, x, w, act, want_x=False, want_w=False, want_out=True)["out"]
    near = 2.0 ** -8 + 100 * 2.0 ** -21
    R.assert_within(again, out, near * out.abs() + 2.0 ** -100, "out")
