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
