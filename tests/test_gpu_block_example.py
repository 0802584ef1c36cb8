"""The example that runs the operators around the routed experts together: its loss falls, and its
gradient of the gate's weights is that of the losses it prints."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import router_training as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def test_router_training_lowers_its_losses(cuda_device):
    history = ex.train(cuda_device, steps=12, report=lambda s: None)
    total = [a + b for a, b in history]
    assert total[-1] < total[0] and history[-1][1] < history[0][1]


def test_gate_gradient_points_down(cuda_device):
    """Along the gradient the loss changes by |gradient|^2 per unit, as far as the routes stay the
    same and 16-bit rows and logits' inputs can tell."""
    p = ex.problem(cuda_device)
    f = ex.forward(p, p["w_gate"])
    # the balance term alone is smooth in f32 while the ids do not change
    coef, ids = f["balance"]["coef"], f["ids"]
    grad = ex.B.moe_router_bwd(f["logits"], ids, coef=coef, seq_offsets=p["offsets"])
    h = 1e-3 / float(grad.norm())
    up, down = (float((ex.B.moe_balance_loss(f["logits"] + s * h * grad, ids, ex.COEFF,
                                             seq_offsets=p["offsets"])["loss"]).double())
                for s in (1, -1))
    want = float(grad.double().square().sum())
    # central difference: f32 losses of about 0.1 are good to 1e-8, the step is 1e-3 / |grad|
    assert abs((up - down) / (2 * h) - want) <= 1e-8 * 2 / h + 1e-3 * want
    g = ex.gate_gradient(p, f)
    assert torch.isfinite(g).all() and float(g.norm()) > 0
