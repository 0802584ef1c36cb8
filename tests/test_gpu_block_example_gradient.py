"""The gate's gradient in the example of router training: route weights of zero, and the gradient
of the losses it prints."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import router_training as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def test_gate_gradient_with_route_weights_of_zero(cuda_device):
    p = ex.problem(cuda_device)
    f = ex.forward(p, 400 * p["w_gate"])
    assert (f["w"] == 0).any() and (f["w"] > 0.99).any()
    assert torch.isfinite(ex.gate_gradient(p, f)).all()


def losses64(p, f, w_gate, rows):
    """The losses of the block in 64 bits with the routes (and so the counts) held fixed; `rows`
    [T, k, H]: the experts' outputs of each token's routes, without their weights."""
    ids = f["ids"].long()
    logits = f["h"].double() @ w_gate.T + p["bias"].double()
    w = torch.softmax(logits.gather(1, ids), dim=1)
    y = (w[:, :, None] * rows).sum(1)

    def norm(v, weight):
        return v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * weight.double()

    stream = p["x"].double() + p["scale"].double() * norm(y, p["post"])
    fit = 0.5 * (norm(stream, p["nxt"]) - p["target"].double()).square().mean()
    seq = torch.bucketize(torch.arange(len(ids), device=ids.device), p["offsets"][1:-1].long(),
                          right=True)
    balance = (f["balance"]["coef"].double()[seq] * torch.softmax(logits, dim=1)).sum()
    return fit, balance


# Between the experts' rows and d loss / d w there are four roundings to bf16 (y, the normed rows, their
# gradient, y's gradient), each off by at most half a step, 2^-8; the gradient of a renormalised
# weight is a difference of two such sums.
def test_gate_gradient_is_that_of_the_losses(cuda_device):
    p = ex.problem(cuda_device)
    f = ex.forward(p, p["w_gate"])
    T, k = f["w"].shape
    rows = f["rows"][f["inv"].long()].view(T, k, -1).double() / f["w"].double()[:, :, None]
    w_gate = p["w_gate"].to(torch.bfloat16).double().requires_grad_(True)
    fit, balance = losses64(p, f, w_gate, rows)
    shown = ex.losses(p, f)
    assert abs(shown[0] - float(fit.detach())) <= 2.0 ** -7 * shown[0]
    assert abs(shown[1] - float(balance.detach())) <= 2.0 ** -16 * shown[1]
    want = torch.autograd.grad(fit + balance, w_gate)[0]
    got = ex.gate_gradient(p, f).double()
    assert float((got - want).norm() / want.norm()) <= 2 * 4 * 2.0 ** -8
