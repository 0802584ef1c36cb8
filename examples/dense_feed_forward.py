"""A dense feed-forward block, as the layers before the first Mixture-of-Experts layer and the shared
experts are: trained with 8 bits kept per activation, then served with 4-bit weights.

  h             = norm(x)
  a, gate, up   = moe_gated_linear(h, w_gate_up, save=True)   gate and up stay as 8-bit checkpoints
  y             = moe_linear(a, w_down, residual=x)
  loss          = mean |y - target|^2 / 2

Between the forward and the backward lie the checkpoints of h, gate and up, a byte per value: `a`
is computed again from them.  Back:

  d_a           = moe_linear_bwd(d_y, w_down)                 the gradient of a
  d_h, d_w, a   = moe_gated_linear_bwd(d_a, h, gate, up)
  d_w_down      = moe_linear_bwd(d_y, a)

Serving a token takes the same weights in NVFP4: moe_gated_linear_w4a16, moe_linear_w4a16.

    python examples/dense_feed_forward.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mixture_experts_forward_moe_gb300 import binding as B  # noqa: E402
from mixture_experts_forward_moe_gb300 import inputs  # noqa: E402

BF = torch.bfloat16


def problem(device, T=500, H=512, F=384):
    """Weights (f32 masters), one batch of ragged length, and what the block should learn."""
    g = torch.Generator(device=device).manual_seed(0)

    def randn(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device=device) * std + mean

    x = randn(T, H).to(BF)
    return dict(x=x, norm=randn(H, std=0.05, mean=1.0).to(BF),
                w_gate_up=randn(2 * F, H, std=H ** -0.5), w_down=randn(H, F, std=F ** -0.5),
                target=(x.float() + randn(T, H, std=0.5)).to(BF))


def forward(p, w):
    """(y, what the backward needs); w: the weights in 16 bits."""
    _, h = B.moe_block_norm(p["x"], pre_weight=p["norm"], post_norm=False, want_stream=False)
    a, gate, up = B.moe_gated_linear(h, w["w_gate_up"], save=True)
    y = B.moe_linear(a, w["w_down"], residual=p["x"])
    return y, dict(h=B.moe_checkpoint(h), gate=gate, up=up)


def gradients(w, kept, d_y):
    """{name: gradient in 16 bits} of the weights, and of h."""
    d_a = B.moe_linear_bwd(d_y, None, w["w_down"], want_w=False)["d_x"]
    g = B.moe_gated_linear_bwd(d_a, kept["h"], w["w_gate_up"], gate=kept["gate"], up=kept["up"],
                               want_out=True)
    d_w_down = B.moe_linear_bwd(d_y, g["out"], w["w_down"], want_x=False)["d_w"]
    return dict(w_gate_up=g["d_w"], w_down=d_w_down, h=g["d_x"])


def sixteen(p):
    return {k: p[k].to(BF) for k in ("w_gate_up", "w_down")}


def train(device, steps=20, rate=100.0, report=print):
    p = problem(device)
    history = []
    for step in range(steps):
        w = sixteen(p)
        y, kept = forward(p, w)
        err = y.float() - p["target"].float()
        history.append(float(0.5 * err.square().mean()))
        report(f"step {step:3d}  loss {history[-1]:.5f}")
        # the loss's gradient is O(1/n): the 16-bit gradients carry it times n
        g = gradients(w, kept, err.to(BF))
        for k in w:
            p[k] = p[k] - rate / err.numel() * g[k].float()
    return p, history


def four_bits(w):
    """(codes, scales, alpha) of one matrix, as the calls take them."""
    codes, scales, alpha = inputs.quantize_nvfp4(w)
    return codes, scales, torch.tensor([alpha], device=w.device)


def decode(x, norm, gate_up, down):
    """One or a few tokens through the block with 4-bit weights."""
    _, h = B.moe_block_norm(x, pre_weight=norm, post_norm=False, want_stream=False)
    a = B.moe_gated_linear_w4a16(h, *gate_up)
    return B.moe_linear_w4a16(a, *down, residual=x)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    p, _ = train(torch.device("cuda:0"), ap.parse_args().steps)
    y, _ = forward(p, sixteen(p))
    out = decode(p["x"][:1].contiguous(), p["norm"], four_bits(p["w_gate_up"]),
                 four_bits(p["w_down"]))
    rel = float((out.float() - y[:1].float()).norm() / (y[:1].float() - p["x"][:1].float()).norm())
    print(f"one token with 4-bit weights: off by {rel:.3f} of what the block adds")
