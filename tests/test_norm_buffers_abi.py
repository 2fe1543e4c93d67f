"""mp_block_norm_bwd refuses results that would overwrite one another or what is still to be read."""
from __future__ import annotations

import ctypes

import pytest

from tests import test_norm_layer_abi as abi
from unpermute_routing_indices_gb300 import _build, _lib

A, B, C = (ctypes.c_void_p(0x100000 * i) for i in (1, 2, 3))   # never dereferenced
INVALID, WORKSPACE = -1, -2


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


@pytest.mark.parametrize("new,code", [
    # `workspace` is left out: what passes the checks of buffers stops there
    (dict(g_x=A, g_residual=A), INVALID),                                  # they differ by the norm after the block,
    (dict(g_x=A, g_residual=A, post_weight=None, gate=B, gate_form=1), INVALID),   # by the gate,
    (dict(g_x=A, g_residual=A, post_weight=None, scale=0.5), INVALID),     # by the scale
    (dict(g_x=A, g_residual=A, post_weight=None), WORKSPACE),              # they are the same values
    (dict(g_x=A, g_residual=B), WORKSPACE),
    (dict(gate=C, gate_form=3, g_gate=A, g_x=A), INVALID),
    (dict(gate=C, gate_form=3, g_gate=A, g_x=B, g_residual=A), INVALID),
    (dict(gate=C, gate_form=3, g_gate=C, g_x=B, g_residual=A), WORKSPACE),
    (dict(x=A, g_x=B, g_residual=A), INVALID),                             # x is read after g_residual is written
    (dict(x=A, g_x=B, g_residual=A, post_weight=None), WORKSPACE),         # not read at all
    (dict(gate=A, gate_form=3, g_x=B, g_residual=A), INVALID),             # so is the gate
    (dict(x=A, gate=B, gate_form=3, g_x=A, g_residual=C), WORKSPACE),
    (dict(gate=B, gate_form=3, g_x=B, g_residual=C), WORKSPACE),
    (dict(g_x=B, g_post_weight=A, g_pre_weight=A), INVALID),               # vectors that the rows share
    (dict(g_x=B, g_pre_weight=A, g_pre_bias=A), INVALID),
    (dict(g_x=B, gate=C, gate_form=1, g_gate=A, g_post_weight=A), INVALID),
    (dict(g_x=B, gate=C, gate_form=1, g_gate=A, g_post_weight=C), WORKSPACE),
])
def test_block_norm_bwd_buffers(lib, new, code):
    base = {**abi.BWD, "g_pre_weight": ctypes.c_void_p(0x900000), "workspace": None}
    assert lib.mp_block_norm_bwd(*abi.changed(base, **new).values()) == code
