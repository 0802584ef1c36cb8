"""A Mixture-of-Experts block between two blocks, and the training of its router with the experts
held fixed: every operator around the routed experts, as they are used together.

  logits  = moe_linear(h, w_gate)                        f32, for the router
  ids, w  = moe_route(logits)
  y       = the experts, combined with w                 (staged: their rows give w's gradient)
  stream, normed = moe_block_norm(y, residual=x)         the next block's input
  loss    = mean |normed - target|^2 / 2 + moe_balance_loss(logits, ids)

and back: moe_block_norm_bwd gives the gradient of y, its products with the experts' rows that of
the route weights, moe_router_bwd that of the logits, and w_gate takes a step.  Serving needs the
forward half alone, with fused_moe_fwd in place of the staged calls (the two agree, which is
checked here).

    python examples/router_training.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mixture_experts_forward_moe_gb300 import binding as B  # noqa: E402
from mixture_experts_forward_moe_gb300 import inputs  # noqa: E402

COEFF = 0.1  # weight of the balance loss


def problem(device, T=512, H=512, E=32, F=256, k=4):
    """The block's weights and one packed batch of ragged sequences."""
    d = inputs.generate(inputs.Workload("router-training", T=T, H=H, E=E, F=F, top_k=k), 0, device)
    g = torch.Generator(device=device).manual_seed(1)

    def randn(*shape, std=1.0, mean=0.0):
        t = torch.randn(shape, generator=g, device=device) * std + mean
        return t.to(torch.bfloat16)

    return dict(
        x=d["hidden_states"], w_gate_up=d["w_gate_up"], w_down=d["w_down"], k=k,
        # a few experts start out with most of the tokens
        w_gate=randn(E, H, std=H ** -0.5).float()
        + 0.02 * torch.randn(E, 1, generator=g, device=device),
        bias=randn(E, std=0.5), scale=randn(H, std=0.05, mean=0.3),
        pre=randn(H, std=0.05, mean=1.0), post=randn(H, std=0.05, mean=1.0),
        nxt=randn(H, std=0.05, mean=1.0), target=randn(T, H),
        offsets=torch.tensor([0, T // 5, T // 2, T], dtype=torch.int32, device=device))


def forward(p, w_gate):
    """The block; returns what the backward needs too."""
    _, h = B.moe_block_norm(p["x"], pre_weight=p["pre"], post_norm=False, want_stream=False)
    logits = B.moe_linear(h, w_gate.to(torch.bfloat16), bias=p["bias"], out_dtype=torch.float32)
    ids, w = B.moe_route(logits, p["k"])
    T, E = logits.shape
    s = B.moe_align_sort(ids, E)
    act = B.moe_gemm1_swiglu(h, s["sorted_ids"], s["offsets"], p["w_gate_up"], p["k"])
    rows = B.moe_gemm2(act, s["sorted_ids"], s["offsets"], w, p["w_down"], T, p["k"])
    y = B.moe_combine(rows, s["inv_route"], T, p["k"])
    norm = dict(branch=y, residual=p["x"], gate=p["scale"], gate_kind="channel",
                post_weight=p["post"], pre_weight=p["nxt"])
    _, normed = B.moe_block_norm(**norm, want_stream=False)
    balance = B.moe_balance_loss(logits, ids, COEFF, seq_offsets=p["offsets"])
    return dict(h=h, logits=logits, ids=ids, w=w, rows=rows, inv=s["inv_route"], y=y, norm=norm,
                normed=normed, balance=balance)


def losses(p, f):
    fit = 0.5 * (f["normed"].float() - p["target"].float()).square().mean()
    return float(fit), float(f["balance"]["loss"])


def gate_gradient(p, f):
    """d loss / d w_gate [E, H] f32."""
    n = f["normed"].numel()
    # the fit's gradient is O(1/n): the 16-bit gradients carry it times n
    d_normed = (f["normed"].float() - p["target"].float()).to(torch.bfloat16)
    d_y = B.moe_block_norm_bwd(None, d_normed, **f["norm"])["d_branch"].float()
    T, k = f["w"].shape
    # the rows carry their route's weight; one of 0 (a far logit) leaves its logit's gradient, the
    # weight times a difference, at 0 whatever its row is
    w = f["w"][:, :, None]
    per_route = f["rows"][f["inv"].long()].view(T, k, -1) / torch.where(w == 0, 1, w)
    d_w = torch.einsum("tkh,th->tk", per_route, d_y) / n
    d_logits = B.moe_router_bwd(f["logits"], f["ids"], d_w.contiguous(), f["balance"]["coef"],
                                seq_offsets=p["offsets"])
    return d_logits.t() @ f["h"].float()


def train(device, steps=20, rate=30.0, report=print):
    p = problem(device)
    w_gate = p["w_gate"]
    history = []
    for step in range(steps):
        f = forward(p, w_gate)
        if step == 0:  # the fused forward is the same block
            fused = B.fused_moe_fwd(f["h"], f["logits"], p["w_gate_up"], p["w_down"], p["k"])
            off = (fused.float() - f["y"].float()).abs().max() / f["y"].float().abs().max()
            assert float(off) < 2.0 ** -7, float(off)
        history.append(losses(p, f))
        load = f["balance"]["counts"].sum(0).float()
        report(f"step {step:3d}  fit {history[-1][0]:.5f}  balance {history[-1][1]:.5f}  "
               f"busiest expert {float(load.max() / load.mean()):.2f}x the mean")
        w_gate = w_gate - rate * gate_gradient(p, f)
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    train(torch.device("cuda:0"), ap.parse_args().steps)
