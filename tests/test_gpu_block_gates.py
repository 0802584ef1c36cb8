"""How the gate of the norm between two blocks is told apart: batches of no rows, and of as many
rows as channels."""
import pytest
import torch

import block_reference as R
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


@pytest.mark.parametrize("dtype", [BF, HF])
def test_as_many_rows_as_channels(dtype, cuda_device):
    n, eps = 64, 1e-6
    d = norm_inputs(n, n, dtype, "none", True, True, 0.0, True)
    g = rand(n, seed=3, std=0.3, mean=0.6, dtype=dtype)
    dr, dh = rand(n, n, seed=6, dtype=dtype), rand(n, n, seed=7, dtype=dtype)
    # a gate of n values says neither
    with pytest.raises(ValueError, match="gate_kind"):
        B.moe_block_norm(**{**d, "gate": g})
    with pytest.raises(ValueError, match="gate_kind"):
        B.moe_block_norm_bwd(dr, dh, **{**d, "gate": g})
    c = {k: None if v is None else v.cpu().double() for k, v in d.items()}
    wide = {"token": g[:, None], "channel": g[None, :]}
    for kind in ("token", "channel"):
        args = (c["branch"], c["residual"], wide[kind].cpu().double().expand(n, n),
                c["post_weight"], c["pre_weight"], True, True, 1.0, 0.0, eps)
        # [T, 1] is per token at any size
        forms = [(g, kind)] + ([(g[:, None].contiguous(), None)] if kind == "token" else [])
        for gate, said in forms:
            kw = {**d, "gate": gate, "gate_kind": said, "eps": eps}
            out = B.moe_block_norm(**kw)
            for got, ref, bound in zip(out, R.norm64(*args), R.norm_bounds(*args, dtype)):
                R.assert_within(got, ref, bound, kind)
            grads = B.moe_block_norm_bwd(dr, dh, **kw)
            ref, mag = R.norm_bwd64(dr.cpu().double(), dh.cpu().double(), *args)
            for k, v in (("d_branch", "branch"), ("d_residual", "residual")):
                R.assert_within(grads[k], ref[v], R.grad_bound(ref[v], mag[v], dtype), k)
            over = 1 if kind == "token" else 0
            r, m = ref["gate"].sum(over), mag["gate"].sum(over)
            assert grads["d_gate"].shape == gate.shape
            R.assert_within(grads["d_gate"].view(n), r, R.grad_bound(r, m, dtype, n), "d_gate")


def test_gate_kind_goes_with_the_shape(cuda_device):
    d = norm_inputs(48, 64, BF, "none", True, True, 0.0, True)
    shapes = {"channel": (64,), "token": (48, 1), "element": (48, 64)}
    for kind, shape in shapes.items():
        g = rand(*shape, seed=3, dtype=BF)
        want = B.moe_block_norm(**{**d, "gate": g})
        got = B.moe_block_norm(**{**d, "gate": g}, gate_kind=kind)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), kind
        for other in set(shapes) - {kind}:
            with pytest.raises(ValueError, match="gate"):
                B.moe_block_norm(**{**d, "gate": g}, gate_kind=other)
    flat = rand(48, seed=3, dtype=BF)
    want = B.moe_block_norm(**{**d, "gate": flat[:, None].contiguous()})
    assert all(torch.equal(a, b) for a, b in zip(B.moe_block_norm(**{**d, "gate": flat}), want))
    with pytest.raises(ValueError, match="gate"):
        B.moe_block_norm(**d, gate_kind="channel")  # no gate
    with pytest.raises(ValueError, match="gate_kind"):
        B.moe_block_norm(**{**d, "gate": flat}, gate_kind="row")
