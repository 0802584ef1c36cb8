"""Workspaces of the dense block's gradients: x in 16 bits has no place there unless a checkpoint is
restored to it (CPU: nothing is wanted of the calls, which check their workspace all the same)."""
import ctypes

import pytest

from mixture_experts_forward_moe_gb300 import binding as B
from test_dense_refusals import OK, P, SHORT, gated_bwd, gated_desc, linear_bwd


def sizes(fn, desc):
    return [int(getattr(B.lib(), f"{fn}_workspace_size{k}")(ctypes.byref(desc))) for k in ("", "_x16")]


def up(n):
    return (n + 255) // 256 * 256


@pytest.mark.parametrize("T,wide", [(0, 64), (40, 64), (300, 1032), (4096, 2048), (32768, 18432)])
def test_sizes(T, wide):
    x = up(T * wide * 2)
    place = x if x > 1 << 20 else 0  # up to a megabyte there is one size
    full, small = sizes("moe_gated_linear_bwd", gated_desc(T=T, H=wide, F=48))
    assert full - small == place and small >= 256 + T * 2 * 48 * 2
    full, small = sizes("moe_linear_bwd", B.Linear(T, 50, wide, 0, 0, 0))
    assert full - small == place and small >= 256 + T * 56 * 2


NONE = dict(dx=None, dw=None)
CKPT = dict(x=None, xc=P, xs=P)


def test_what_a_call_needs():
    kw = dict(T=4096, H=2048, F=48)
    full, small = sizes("moe_gated_linear_bwd", gated_desc(**kw))
    nothing = dict(NONE, out=None)
    assert gated_bwd(ws=small, ptrs=nothing, **kw) == OK
    assert gated_bwd(ws=small - 1, ptrs=nothing, **kw) == SHORT
    assert gated_bwd(ws=full, ptrs=dict(nothing, **CKPT), **kw) == OK
    assert gated_bwd(ws=full - 1, ptrs=dict(nothing, **CKPT), **kw) == SHORT
    # with gate and up saved x is for d_w alone
    saved = dict(gc=P, gs=P, uc=P, us=P)
    assert gated_bwd(ws=small, ptrs=dict(nothing, **CKPT, **saved), **kw) == OK
    assert gated_bwd(ws=small, ptrs=dict(CKPT, **saved), **kw) == SHORT

    kw = dict(T=4096, N=50, K=2048)
    full, small = sizes("moe_linear_bwd", B.Linear(*kw.values(), 0, 0, 0))
    nothing = dict(NONE, db=None)
    assert linear_bwd(ws=small, ptrs=nothing, **kw) == OK
    assert linear_bwd(ws=small - 1, ptrs=nothing, **kw) == SHORT
    assert linear_bwd(ws=small, ptrs=dict(nothing, **CKPT), **kw) == OK  # x is not read
    assert linear_bwd(ws=small, ptrs=CKPT, **kw) == SHORT
    assert linear_bwd(ws=full - 1, ptrs=CKPT, **kw) == SHORT


def test_sizes_of_what_is_refused():
    assert sizes("moe_gated_linear_bwd", gated_desc(H=7)) == [0, 0]
    assert sizes("moe_linear_bwd", B.Linear(1, 8, 7, 0, 0, 0)) == [0, 0]
