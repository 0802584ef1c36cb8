"""Argument checks of the norm's gate, before any launch (CPU only: the pointers are never
dereferenced): a gate of no elements has no address."""
import ctypes

import pytest

from mixture_experts_forward_moe_gb300 import binding as B

D = 1 << 20  # an address on a 256-byte boundary
NONE, CHANNEL, TOKEN, ELEMENT = range(4)


def shape(T, gate):
    return B.BlockNorm(T, 64, 0, gate, 1, 1, 1.0, 0.0, 1e-6)


def forward(T, gate, g):
    y = D if T else None
    return B.lib().moe_block_norm_fwd(ctypes.byref(shape(T, gate)), y, None, g, None, None, y, y,
                                      None)


def backward(T, gate, g):
    # no output is wanted: nothing is launched for no rows
    y = D if T else None
    return B.lib().moe_block_norm_bwd(ctypes.byref(shape(T, gate)), y, y, y, None, g, None, None,
                                      None, None, None, None, None, D, 1 << 30, None)


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("T,gate,g,code", [
    (0, NONE, None, B.MOE_OK), (0, NONE, D, B.MOE_ERR_INVALID_ARG),
    (0, CHANNEL, D, B.MOE_OK), (0, CHANNEL, None, B.MOE_ERR_INVALID_ARG),
    (0, TOKEN, None, B.MOE_OK), (0, TOKEN, D, B.MOE_OK),
    (0, ELEMENT, None, B.MOE_OK), (0, ELEMENT, D, B.MOE_OK),
    (4, TOKEN, None, B.MOE_ERR_INVALID_ARG), (4, ELEMENT, None, B.MOE_ERR_INVALID_ARG),
    (4, CHANNEL, None, B.MOE_ERR_INVALID_ARG), (4, NONE, D, B.MOE_ERR_INVALID_ARG),
])
def test_gate_goes_with_its_kind(call, T, gate, g, code):
    assert call(T, gate, g) == code
