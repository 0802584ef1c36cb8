"""Argument checks of the dense feed-forward block, before any launch (CPU only: the pointers here are
never dereferenced), and its plain forms against differences and against torch's E4M3."""
import ctypes

import pytest
import torch

import dense_reference as D
from block_reference import act64
from mixture_experts_forward_moe_gb300 import binding as B

P = 1 << 20  # an address on a 256-byte boundary
OK, BAD, UNSUP, SHORT = (B.MOE_OK, B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED,
                         B.MOE_ERR_WORKSPACE_TOO_SMALL)
BIG = 1 << 40


def gated_desc(**kw):
    base = dict(T=40, H=64, F=48, dtype=0, activation=0)
    base.update(kw)
    return B.GatedLinear(**base)


def call(fn, desc, names, ptrs, ws):
    a = dict.fromkeys(names.split(), P)
    a.update(ptrs or {})
    return getattr(B.lib(), fn)(ctypes.byref(desc), *a.values(), ws, None)


def gated(ptrs=None, ws=BIG, **kw):
    p = dict(gc=None, gs=None, uc=None, us=None)
    p.update(ptrs or {})
    return call("moe_gated_linear", gated_desc(**kw), "x w out gc gs uc us ws", p, ws)


SIZES = [
    (dict(T=-1), BAD), (dict(H=0), BAD), (dict(F=0), BAD), (dict(dtype=2), BAD),
    (dict(activation=3), BAD), (dict(activation=-1), BAD), (dict(activation=2), UNSUP),
    (dict(H=60), UNSUP), (dict(F=44), UNSUP), (dict(F=1 << 30), UNSUP),
]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(ptrs=dict(x=None)), BAD), (dict(ptrs=dict(w=None)), BAD),
    (dict(ptrs=dict(out=None)), BAD), (dict(ptrs=dict(ws=None)), BAD),
    (dict(ptrs=dict(gc=P)), BAD), (dict(ptrs=dict(gc=P, gs=P)), BAD),
    (dict(ptrs=dict(uc=P, us=P)), BAD), (dict(ptrs=dict(gc=P, uc=P, us=P)), BAD),
    (dict(ptrs=dict(x=P + 2)), BAD), (dict(ptrs=dict(w=P + 8)), BAD),
    (dict(ptrs=dict(gc=P, gs=P + 4, uc=P, us=P)), BAD),
    (dict(ws=255), SHORT), (dict(T=0, ptrs=dict(x=None, out=None)), OK),
])
def test_gated_refusals(kw, code):
    assert gated(**kw) == code


def gated_bwd(ptrs=None, ws=BIG, **kw):
    p = dict(xc=None, xs=None, gc=None, gs=None, uc=None, us=None)
    p.update(ptrs or {})
    return call("moe_gated_linear_bwd", gated_desc(**kw),
                "dy x xc xs w gc gs uc us dx dw out ws", p, ws)


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(ptrs=dict(dy=None)), BAD), (dict(ptrs=dict(x=None)), BAD),
    (dict(ptrs=dict(w=None)), BAD), (dict(ptrs=dict(ws=None)), BAD),
    (dict(ptrs=dict(xc=P, xs=P)), BAD), (dict(ptrs=dict(x=None, xc=P)), BAD),
    (dict(ptrs=dict(gc=P, gs=P)), BAD), (dict(ptrs=dict(gc=P, gs=P, uc=P)), BAD),
    # with the checkpoints of gate and up x is for d_w alone
    (dict(ptrs=dict(x=None, gc=P, gs=P, uc=P, us=P)), BAD),
    (dict(ptrs=dict(x=None, gc=P, gs=P, uc=P, us=P, dx=None, dw=None, out=None)), OK),
    (dict(ptrs=dict(x=None, dx=None, dw=None, out=None)), BAD),
    (dict(ptrs=dict(dx=None, dw=None, out=None)), OK),
    (dict(ptrs=dict(dw=P + 8)), BAD), (dict(ptrs=dict(dx=P + 2)), BAD),
    (dict(ws=1024), SHORT), (dict(T=0, ptrs=dict(dy=None, x=None, dw=None)), OK),
])
def test_gated_bwd_refusals(kw, code):
    assert gated_bwd(**kw) == code


def linear_bwd(ptrs=None, ws=BIG, **kw):
    base = dict(T=40, N=48, K=64, dtype=0, activation=0, out_f32=0)
    base.update(kw)
    p = dict(xc=None, xs=None)
    p.update(ptrs or {})
    return call("moe_linear_bwd", B.Linear(**base), "dy x xc xs w dx dw db ws", p, ws)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(N=0), BAD), (dict(K=0), BAD), (dict(K=12), UNSUP),
    (dict(dtype=3), BAD), (dict(activation=4), BAD), (dict(activation=1), UNSUP),
    (dict(out_f32=1), UNSUP), (dict(ptrs=dict(dy=None)), BAD), (dict(ptrs=dict(x=None)), BAD),
    (dict(ptrs=dict(w=None)), BAD), (dict(ptrs=dict(ws=None)), BAD),
    (dict(ptrs=dict(xc=P, xs=P)), BAD), (dict(ptrs=dict(x=None, xs=P)), BAD),
    (dict(ptrs=dict(dy=P + 2)), BAD), (dict(ptrs=dict(db=P + 8)), BAD), (dict(ws=512), SHORT),
    (dict(ptrs=dict(dx=None, dw=None, db=None, x=None, w=None)), OK),
    (dict(T=0, ptrs=dict(dy=None, x=None, dw=None, db=None)), OK),
])
def test_linear_bwd_refusals(kw, code):
    assert linear_bwd(**kw) == code


@pytest.mark.parametrize("T,C,dtype,ptrs,code", [
    (-1, 64, 0, {}, BAD), (4, 0, 0, {}, BAD), (4, 64, 2, {}, BAD), (4, 60, 0, {}, UNSUP),
    (4, 64, 0, dict(a=None), BAD), (4, 64, 0, dict(b=None), BAD), (4, 64, 0, dict(c=None), BAD),
    (4, 64, 0, dict(a=P + 8), BAD), (4, 64, 0, dict(b=P + 4), BAD),
    (0, 64, 0, dict(a=None, b=None, c=None), OK),
])
@pytest.mark.parametrize("fn", ["moe_checkpoint", "moe_checkpoint_restore"])
def test_checkpoint_refusals(fn, T, C, dtype, ptrs, code):
    a = dict(a=P, b=P, c=P)
    a.update(ptrs)
    assert getattr(B.lib(), fn)(T, C, dtype, *a.values(), None) == code


def linear_w4(ptrs=None, ws=256, **kw):
    base = dict(T=4, N=5, K=64, dtype=0, activation=0, out_f32=0)
    base.update(kw)
    p = dict(bias=None, res=None)
    p.update(ptrs or {})
    return call("moe_linear_w4a16", B.Linear(**base), "x codes scales alpha bias res out ws", p, ws)


def gated_w4(ptrs=None, ws=256, **kw):
    base = dict(T=4, F=5, H=64)
    base.update({{"N": "F", "K": "H"}.get(k, k): v for k, v in kw.items()})
    return call("moe_gated_linear_w4a16", gated_desc(**base), "x codes scales alpha out ws", ptrs, ws)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(N=0), BAD), (dict(K=0), BAD), (dict(K=48), UNSUP),
    (dict(dtype=2), BAD), (dict(activation=9), BAD), (dict(T=(1 << 20) + 1), UNSUP),
    (dict(ptrs=dict(x=None)), BAD), (dict(ptrs=dict(codes=None)), BAD),
    (dict(ptrs=dict(scales=None)), BAD), (dict(ptrs=dict(alpha=None)), BAD),
    (dict(ptrs=dict(out=None)), BAD), (dict(ptrs=dict(ws=None)), BAD),
    (dict(ptrs=dict(codes=P + 8)), BAD), (dict(ptrs=dict(scales=P + 2)), BAD),
    (dict(ptrs=dict(out=P + 2)), BAD), (dict(ws=255), SHORT),
    (dict(T=0, ptrs=dict(x=None, out=None)), OK),
])
def test_w4_refusals(kw, code):
    assert linear_w4(**kw) == code
    assert gated_w4(**kw) == code


def test_w4_refusals_of_one_form():
    assert linear_w4(out_f32=1) == UNSUP
    assert linear_w4(ptrs=dict(bias=P + 2)) == BAD and linear_w4(ptrs=dict(res=P + 4)) == BAD
    assert gated_w4(activation=2) == UNSUP and gated_w4(F=1 << 30) == UNSUP


def test_workspace_sizes():
    L = B.lib()
    g = gated_desc(T=512, H=512, F=256)
    assert L.moe_gated_linear_workspace_size(ctypes.byref(g)) >= 256
    # d_gate, d_up and x in 16 bits at least
    assert L.moe_gated_linear_bwd_workspace_size(ctypes.byref(g)) >= 512 * (4 * 256 + 2 * 512)
    lin = B.Linear(T=100, N=13, K=64, dtype=0, activation=0, out_f32=0)
    assert L.moe_linear_bwd_workspace_size(ctypes.byref(lin)) >= 100 * (2 * 16 + 2 * 64)
    for fn, bad in (("moe_gated_linear", gated_desc(H=7)), ("moe_gated_linear_bwd", gated_desc(T=-1)),
                    ("moe_gated_linear_w4a16", gated_desc(H=16)),
                    ("moe_linear_bwd", B.Linear(1, 8, 7, 0, 0, 0)),
                    ("moe_linear_w4a16", B.Linear(1, 8, 8, 0, 0, 0))):
        assert getattr(L, fn + "_workspace_size")(ctypes.byref(bad)) == 0


# ---------------------------------------------------------------------------- the binding's checks
def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="activation"):
        B.moe_gated_linear(x, w, activation="relu")
    with pytest.raises(ValueError, match="activation"):
        B.moe_linear_w4a16(x, w, w, w, activation="tanh")
    with pytest.raises(ValueError, match="CUDA"):
        B.moe_gated_linear(x, w)
    with pytest.raises(ValueError, match="together"):
        B.moe_gated_linear_bwd(x, x, w, gate=B.Fp8Checkpoint(x, x, 64))
    with pytest.raises(TypeError, match="Fp8Checkpoint"):
        B.moe_gated_linear_bwd(x, x, w, gate=x, up=x)
    with pytest.raises(TypeError, match="Fp8Checkpoint"):
        B.moe_checkpoint_restore(x)
    with pytest.raises(ValueError, match="dtype"):
        B.moe_checkpoint_restore(B.Fp8Checkpoint(x, x, 64), torch.float32)
    with pytest.raises(TypeError, match="Tensor"):
        B.moe_linear_bwd(x, 3, w)


# ------------------------------------------------------------------------- the plain forms here
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_slope_against_differences(act):
    z = torch.linspace(-30, 30, 4001, dtype=torch.float64)
    h = 1e-5
    d = (act64(z + h, act) - act64(z - h, act)) / (2 * h)
    # a central difference is off by h^2/6 of a third derivative below 10, and by rounding
    assert float((D.slope64(z, act) - d).abs().max()) < 1e-8


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_gradients_against_automatic_ones(act):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 7, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(6, 7, generator=g, dtype=torch.float64, requires_grad=True)
    dh = torch.randn(5, 3, generator=g, dtype=torch.float64)
    z = x @ w.T
    h = act64(z[:, :3], act) * z[:, 3:]
    want = torch.autograd.grad(h, [x, w], dh)
    with torch.no_grad():
        zero = torch.zeros(5, 3, dtype=torch.float64)
        got = D.gated_bwd64(dh, x, w, z[:, :3], z[:, 3:], zero, zero, act, torch.float64)
    assert torch.allclose(got["d_x"][0], want[0], rtol=1e-12, atol=1e-12)
    assert torch.allclose(got["d_w"][0], want[1], rtol=1e-12, atol=1e-12)


def test_e4m3_against_torch():
    codes = torch.arange(256, dtype=torch.uint8).view(2, 128)
    v = codes.view(torch.float8_e4m3fn).double()
    mine = D.restore64(codes, torch.ones(2, 1), 128)
    assert torch.equal(mine.nan_to_num(), v.nan_to_num())
    assert torch.equal(torch.isnan(mine), torch.isnan(v))
    x = torch.randn(10000, generator=torch.Generator().manual_seed(1)) * 60
    x = torch.cat([x, x * 2.0 ** -8]).clamp(-448, 448)
    assert torch.equal(D.e4m3_64(x.double()), x.to(torch.float8_e4m3fn).double())
