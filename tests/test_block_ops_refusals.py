"""Argument checks of the operators around the routed experts, before any launch (CPU only: the
pointers here are never dereferenced), and their plain forms against differences."""
import ctypes

import pytest
import torch

import block_reference as R
from mixture_experts_forward_moe_gb300 import binding as B

D = 1 << 20  # an address on a 256-byte boundary
BAD, UNSUP, SHORT = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE_TOO_SMALL


def linear(ptrs=None, ws=256, **kw):
    base = dict(T=4, N=8, K=16, dtype=0, activation=0, out_f32=0)
    base.update(kw)
    a = dict(x=D, w=D, bias=None, res=None, out=D, ws=D)
    a.update(ptrs or {})
    return B.lib().moe_linear(ctypes.byref(B.Linear(**base)), a["x"], a["w"], a["bias"], a["res"],
                              a["out"], a["ws"], ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(N=0), BAD), (dict(K=0), BAD), (dict(K=12), UNSUP),
    (dict(dtype=2), BAD), (dict(activation=4), BAD), (dict(activation=-1), BAD),
    (dict(ptrs=dict(x=None)), BAD), (dict(ptrs=dict(w=None)), BAD),
    (dict(ptrs=dict(out=None)), BAD), (dict(ptrs=dict(ws=None)), BAD),
    (dict(ptrs=dict(x=D + 2)), BAD), (dict(ptrs=dict(bias=D + 8)), BAD),
    (dict(ptrs=dict(res=D + 4)), BAD), (dict(ptrs=dict(out=D + 2)), BAD),
    (dict(ws=255), SHORT), (dict(T=0, ptrs=dict(x=None, out=None)), B.MOE_OK),
])
def test_linear_refusals(kw, code):
    assert linear(**kw) == code


def norm_fwd(ptrs=None, **kw):
    base = dict(T=4, H=64, dtype=0, gate=0, post_norm=1, pre_norm=1, residual_scale=1.0,
                weight_offset=0.0, eps=1e-6)
    base.update(kw)
    a = dict(y=D, x=None, g=None, wq=None, wp=None, r=D, h=D)
    a.update(ptrs or {})
    return B.lib().moe_block_norm_fwd(ctypes.byref(B.BlockNorm(**base)), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(H=0), BAD), (dict(H=60), UNSUP), (dict(H=16392), UNSUP),
    (dict(dtype=5), BAD), (dict(gate=4), BAD), (dict(gate=1), BAD),
    (dict(ptrs=dict(g=D)), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(residual_scale=float("inf")), BAD), (dict(weight_offset=float("nan")), BAD),
    (dict(ptrs=dict(y=None)), BAD), (dict(ptrs=dict(h=None)), BAD),
    (dict(pre_norm=0), BAD), (dict(post_norm=0, ptrs=dict(wq=D)), BAD),
    (dict(pre_norm=0, ptrs=dict(wp=D, h=None)), BAD),
    (dict(ptrs=dict(y=D + 2)), BAD), (dict(ptrs=dict(x=D + 8)), BAD),
    (dict(ptrs=dict(r=D + 2)), BAD), (dict(ptrs=dict(wp=D + 4)), BAD),
    (dict(T=0), B.MOE_OK),
])
def test_block_norm_refusals(kw, code):
    assert norm_fwd(**kw) == code


def norm_bwd(ptrs=None, ws=1 << 30, **kw):
    base = dict(T=4, H=64, dtype=0, gate=0, post_norm=1, pre_norm=1, residual_scale=1.0,
                weight_offset=0.0, eps=1e-6)
    base.update(kw)
    a = dict(dr=D, dh=D, y=D, x=None, g=None, wq=None, wp=None, dy=D, dx=D, dg=None, dwq=None,
             dwp=None, ws=D)
    a.update(ptrs or {})
    return B.lib().moe_block_norm_bwd(ctypes.byref(B.BlockNorm(**base)), *a.values(), ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(H=12), UNSUP), (dict(ptrs=dict(y=None)), BAD),
    (dict(ptrs=dict(dh=None)), BAD), (dict(pre_norm=0), BAD), (dict(ptrs=dict(dg=D)), BAD),
    (dict(ptrs=dict(dwq=D)), BAD), (dict(ptrs=dict(dwp=D)), BAD),
    (dict(ptrs=dict(ws=None)), BAD), (dict(ptrs=dict(dr=D + 2)), BAD),
    (dict(ptrs=dict(dy=D + 8)), BAD), (dict(ws=256), SHORT),
])
def test_block_norm_bwd_refusals(kw, code):
    assert norm_bwd(**kw) == code


def prob(**kw):
    base = dict(T=8, H=8, E=16, F=8, top_k=2)
    base.update(kw)
    return B.make_problem(**base)


def balance(ptrs=None, n=1, coeff=1.0, ws=1 << 30, **kw):
    a = dict(x=D, ids=D, off=None, loss=D, counts=D, live=D, sums=D, coef=D, ws=D)
    a.update(ptrs or {})
    return B.lib().moe_balance_loss_fwd(ctypes.byref(prob(**kw)), n, coeff, *a.values(), ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), BAD), (dict(n=2), BAD), (dict(n=(1 << 20) + 1, ptrs=dict(off=D)), UNSUP),
    (dict(top_k=17), BAD), (dict(E=1025), UNSUP), (dict(ep_num_local=4), UNSUP),
    (dict(coeff=float("nan")), BAD), (dict(ptrs=dict(x=None)), BAD),
    (dict(ptrs=dict(ids=None)), BAD), (dict(ptrs=dict(loss=None)), BAD),
    (dict(ptrs=dict(coef=None)), BAD), (dict(ptrs=dict(ws=None)), BAD),
    (dict(ptrs=dict(x=D + 4)), BAD), (dict(ptrs=dict(sums=D + 8)), BAD), (dict(ws=256), SHORT),
])
def test_balance_loss_refusals(kw, code):
    assert balance(**kw) == code


def router(ptrs=None, n=1, **kw):
    a = dict(x=D, ids=D, dw=None, coef=None, off=None, dl=None, out=D)
    a.update(ptrs or {})
    return B.lib().moe_router_bwd(ctypes.byref(prob(**kw)), n, *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), BAD), (dict(n=3), BAD), (dict(ep_num_local=4), UNSUP), (dict(T=-1), BAD),
    (dict(ptrs=dict(x=None)), BAD), (dict(ptrs=dict(out=None)), BAD),
    (dict(ptrs=dict(out=D + 4)), BAD), (dict(ptrs=dict(coef=D + 8)), BAD),
    (dict(T=0, ptrs=dict(x=None, ids=None, out=None)), B.MOE_OK),
])
def test_router_bwd_refusals(kw, code):
    assert router(**kw) == code


def test_workspace_sizes():
    L = B.lib()
    assert L.moe_linear_workspace_size(ctypes.byref(B.Linear(4, 8, 16, 0, 0, 0))) == 256
    assert L.moe_linear_workspace_size(ctypes.byref(B.Linear(4, 8, 12, 0, 0, 0))) == 0
    assert L.moe_block_norm_bwd_workspace_size(
        ctypes.byref(B.BlockNorm(4, 60, 0, 0, 1, 1, 1.0, 0.0, 1e-6))) == 0
    n = L.moe_block_norm_bwd_workspace_size(
        ctypes.byref(B.BlockNorm(4, 64, 0, 0, 1, 1, 1.0, 0.0, 1e-6)))
    assert n >= 256 + 4 * 3 * 64 * 4 and n % 256 == 0
    p = prob()
    assert L.moe_balance_loss_workspace_size(ctypes.byref(p), 0) == 0
    assert L.moe_balance_loss_workspace_size(ctypes.byref(p), 300) > \
        L.moe_balance_loss_workspace_size(ctypes.byref(p), 1) > 256


def test_binding_refuses_host_and_mismatched_tensors():
    x = torch.zeros(2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.moe_linear(x, x)
    with pytest.raises(ValueError, match="activation"):
        B.moe_linear(x, x, activation="tanh")
    with pytest.raises(ValueError, match="dtype"):
        B.moe_linear(x.float(), x.float())
    with pytest.raises(ValueError, match="out_dtype"):
        B.moe_linear(x, x, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="dimensions"):
        B.moe_block_norm(x[0])
    with pytest.raises(ValueError, match="dimensions"):
        B.moe_balance_loss(x.float(), x[0].int(), 1.0)


def test_plain_norm_gradients_against_differences():
    """The formulas of the norm's gradients are those of its plain form."""
    g = torch.Generator().manual_seed(0)
    T, H, eps = 3, 16, 1e-5

    def r(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    y, x, gate, wq, wp, dr, dh = r(T, H), r(T, H), r(T, H), r(H), r(H), r(T, H), r(T, H)

    def total(y, x, gate, wq, wp):
        s, h = R.norm64(y, x, gate, wq, wp, True, True, 0.7, 1.0, eps)
        return (s * dr).sum() + (h * dh).sum()

    ref, _ = R.norm_bwd64(dr, dh, y, x, gate, wq, wp, True, True, 0.7, 1.0, eps)
    got = [ref["branch"], ref["residual"], ref["gate"], ref["post"].sum(0), ref["pre"].sum(0)]
    ins = [y, x, gate, wq, wp]
    for i, d in enumerate(got):
        for _ in range(4):
            v = r(*ins[i].shape)
            h = 1e-6
            up, down = (total(*[t + s * h * v if j == i else t for j, t in enumerate(ins)])
                        for s in (1, -1))
            assert abs(float((up - down) / (2 * h) - (d * v).sum())) < 1e-6, i
