"""The example of a dense feed-forward block: it runs, its gradients are those of the block in 64 bits
at the checkpoints that it keeps, and its 4-bit form is the block of the decoded weights."""
import os
import sys

import pytest
import torch

import block_reference as R
import dense_reference as D
from mixture_experts_forward_moe_gb300 import binding as B

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import dense_feed_forward as ex  # noqa: E402

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def d64(t):
    return t.detach().cpu().double()


def test_it_runs(cuda_device):
    p, history = ex.train(cuda_device, steps=4, report=lambda s: None)
    assert len(history) == 4 and all(torch.isfinite(torch.tensor(history)))
    assert torch.isfinite(p["w_gate_up"]).all() and torch.isfinite(p["w_down"]).all()


def test_gradients(cuda_device):
    p = ex.problem(cuda_device, T=300, H=264, F=136)
    w = ex.sixteen(p)
    y, kept = ex.forward(p, w)
    err = (y.float() - p["target"].float()).to(BF)
    got = ex.gradients(w, kept, err)
    # the block in 64 bits behind the checkpoints, whose values are what the backward goes by
    h, g, u = (D.restore64(c.codes, c.scale, c.C) for c in (kept["h"], kept["gate"], kept["up"]))
    dy, wd, wgu = d64(err), d64(w["w_down"]), d64(w["w_gate_up"])
    da, off = D.product64(dy, wd.T.contiguous())
    e_da = D.rounded(da, off, BF)
    zero = torch.zeros_like(g)
    ref = D.gated_bwd64(da, h, wgu, g, u, zero, zero, "silu", BF)
    # what d_a's rounding adds to d_gate and d_up, and with them to the products
    a, s = D.act64(g, "silu"), D.slope64(g, "silu")
    e_d = 1.01 * torch.cat([e_da * (u * s).abs(), e_da * a.abs()], dim=1)
    want, bound = ref["d_x"]
    R.assert_within(got["h"], want, 1.01 * (bound + e_d @ wgu.abs()), "h")
    want, bound = ref["d_w"]
    R.assert_within(got["w_gate_up"], want, 1.01 * (bound + e_d.T @ h.abs()), "w_gate_up")
    act, e_act = ref["out"]
    want, off = D.product64(dy.T.contiguous(), act.T.contiguous())
    R.assert_within(got["w_down"], want, 1.01 * (D.rounded(want, off, BF) + dy.abs().T @ e_act),
                    "w_down")


def test_gradients_against_differences(cuda_device):
    """Along a random direction of the weights the 64-bit loss at what the backward goes by changes
    by the gradient's share, which is that of the checkpointed block: the checkpoints of gate and up
    are taken as fixed offsets of their sums."""
    p = ex.problem(cuda_device, T=120, H=136, F=72)
    w = ex.sixteen(p)
    y, kept = ex.forward(p, w)
    err = (y.float() - p["target"].float()).to(BF)
    got = ex.gradients(w, kept, err)
    h, g, u = (D.restore64(c.codes, c.scale, c.C) for c in (kept["h"], kept["gate"], kept["up"]))
    F = g.shape[1]
    w0, wd0, dy = d64(w["w_gate_up"]), d64(w["w_down"]), d64(err)
    gen = torch.Generator().manual_seed(7)
    v = torch.randn(w0.shape, generator=gen, dtype=torch.float64)
    vd = torch.randn(wd0.shape, generator=gen, dtype=torch.float64)

    def loss(t):  # linear in y, whose gradient is d_y
        z = t * (h @ v.T)
        a = D.act64(g + z[:, :F], "silu") * (u + z[:, F:])
        return float((dy * (a @ (wd0 + t * vd).T)).sum())

    t = 1e-4
    slope = (loss(t) - loss(-t)) / (2 * t)
    mine = float((d64(got["w_gate_up"]) * v).sum() + (d64(got["w_down"]) * vd).sum())
    # each gradient value is off by roundings of its factors to 16 bits (2^-8 a step at most, four in
    # a row: d_a, d_gate, a, itself), all with signs of their own: the sum against random directions
    # is off by that share of the norm, six standard deviations of it
    norm = float((d64(got["w_gate_up"]).square().sum() + d64(got["w_down"]).square().sum()).sqrt())
    third = 1e-6 * norm  # what the central difference leaves out: t^2 of a third derivative
    assert abs(mine - slope) <= 6 * 4 * 2.0 ** -8 * norm + third


def test_four_bits(cuda_device):
    p = ex.problem(cuda_device, T=40, H=256, F=160)
    gate_up, down = ex.four_bits(p["w_gate_up"]), ex.four_bits(p["w_down"])
    for T in (1, 5, 40):
        x = p["x"][:T].contiguous()
        out = ex.decode(x, p["norm"], gate_up, down)
        _, h = B.moe_block_norm(x, pre_weight=p["norm"], post_norm=False, want_stream=False)
        a, e_a = D.w4_gated64(h, D.weights64(*gate_up[:2], gate_up[2].cpu()), "silu")
        w = D.weights64(*down[:2], down[2].cpu())
        z, off = D.product64(a, w.contiguous())
        want = z + d64(x)
        # a is rounded to bf16 (within e_a) and taken in f16, 2^-25 off at most
        err = 1.01 * off + (e_a + 2.0 ** -25) @ w.abs().T + 4 * R.F32 * want.abs()
        R.assert_within(out, want, D.rounded(want, err, BF), "decode")
        assert B.get_device_status(B.call_workspace(cuda_device)) == B.MOE_OK
