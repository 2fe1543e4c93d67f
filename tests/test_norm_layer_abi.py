"""The norms' and the whole layer's entry points reject bad arguments on the host, before
any launch; the formulas that the GPU tests compare with, against differences."""
from __future__ import annotations

import ctypes

import pytest
import torch

import unpermute_routing_indices_gb300 as mp
from tests import norm_util as nu
from unpermute_routing_indices_gb300 import _build, _lib

FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: every call fails validation
OTHER = ctypes.c_void_p(0x2000)
INVALID, WORKSPACE, UNSUPPORTED = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


def changed(base, **new):
    assert set(new) <= set(base)
    return {**base, **new}


NORM = dict(x=FAKE, residual=FAKE, T=4, H=64, dtype=0, kind=0, eps=1e-6, post_weight=FAKE, post_bias=None,
            gate=None, gate_form=0, scale=1.0, pre_weight=FAKE, pre_bias=None, s=FAKE, y=OTHER, stats=None,
            status=None, stream=None)


@pytest.mark.parametrize("new,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=32769), UNSUPPORTED), (dict(T=2 ** 31), UNSUPPORTED),
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(kind=2), INVALID), (dict(kind=-1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(x=None), INVALID), (dict(s=None), INVALID), (dict(y=None), INVALID),
    (dict(s=OTHER), INVALID),   # one buffer for both
    (dict(gate_form=4), INVALID), (dict(gate_form=1), INVALID), (dict(gate=FAKE), INVALID),
    (dict(post_weight=None, pre_weight=None, y=None), INVALID), (dict(pre_weight=None), INVALID),
    (dict(pre_weight=None, pre_bias=FAKE, y=None), INVALID), (dict(post_weight=None, post_bias=FAKE), INVALID),
    (dict(post_weight=None, s=None), INVALID),                       # a residual changes the stream
    (dict(post_weight=None, residual=None, s=None, scale=0.5), INVALID),
    (dict(stats=ctypes.c_void_p(0x1004)), INVALID),
    (dict(T=0, x=None, s=None, y=None, pre_weight=None, post_weight=None), 0),
])
def test_block_norm_rejects(lib, new, code):
    assert lib.mp_block_norm(*changed(NORM, **new).values()) == code


BWD = dict(g_s=FAKE, g_y=FAKE, x=FAKE, s=FAKE, stats=FAKE, T=4, H=64, dtype=0, kind=0, post_weight=FAKE,
           post_bias=None, gate=None, gate_form=0, scale=1.0, pre_weight=FAKE, g_x=FAKE, g_residual=None,
           g_gate=None, g_post_weight=None, g_post_bias=None, g_pre_weight=FAKE, g_pre_bias=None, grad_dtype=2,
           workspace=FAKE, workspace_bytes=1 << 30, status=None, stream=None)


@pytest.mark.parametrize("new,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=32769), UNSUPPORTED), (dict(T=2 ** 31), UNSUPPORTED),
    (dict(dtype=5), INVALID), (dict(kind=3), INVALID), (dict(grad_dtype=1), INVALID), (dict(grad_dtype=3), INVALID),
    (dict(dtype=2, grad_dtype=0), INVALID), (dict(stats=None), INVALID), (dict(s=None), INVALID),
    (dict(x=None), INVALID), (dict(g_y=None), INVALID), (dict(g_gate=FAKE), INVALID),
    (dict(gate=FAKE, gate_form=0), INVALID), (dict(gate_form=3), INVALID), (dict(post_weight=None, pre_weight=None), INVALID),
    (dict(pre_weight=None, g_s=None, g_y=None, g_pre_weight=None), INVALID),
    (dict(pre_weight=None, g_y=None), INVALID), (dict(pre_weight=None, g_pre_weight=None), INVALID),
    (dict(post_weight=None, g_post_weight=FAKE), INVALID), (dict(post_weight=None, g_post_bias=FAKE), INVALID),
    (dict(stats=ctypes.c_void_p(0x1008)), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=255), WORKSPACE),
    (dict(workspace=ctypes.c_void_p(0x1004)), WORKSPACE),
    (dict(T=0, g_pre_weight=None, g_s=None, g_y=None, x=None, s=None, stats=None), 0),
])
def test_block_norm_bwd_rejects(lib, new, code):
    assert lib.mp_block_norm_bwd(*changed(BWD, **new).values()) == code


LAYER = dict(x=FAKE, router=FAKE, router_dtype=2, bias=None, w1=FAKE, b1=None, w2=FAKE, b2=None, T=4, E=64, K=8,
             H=64, F=64, O=64, act=5, score=0, n_groups=1, topk_groups=1, group_top=1, renorm=1, scale=1.0,
             idx=FAKE, weights=FAKE, y=FAKE, workspace=FAKE, workspace_bytes=1 << 40, status=None, stream=None)


@pytest.mark.parametrize("new,code", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(K=0), INVALID), (dict(K=65), INVALID),
    (dict(H=0), INVALID), (dict(F=0), INVALID), (dict(O=0), INVALID), (dict(T=65), UNSUPPORTED),
    (dict(E=1025), UNSUPPORTED), (dict(K=33), UNSUPPORTED), (dict(H=65537), UNSUPPORTED),
    (dict(F=65537), UNSUPPORTED), (dict(O=65537), UNSUPPORTED), (dict(act=6), INVALID), (dict(act=-1), INVALID),
    (dict(score=2), INVALID), (dict(router_dtype=3), INVALID), (dict(n_groups=3), INVALID),
    (dict(n_groups=64, topk_groups=8), UNSUPPORTED), (dict(n_groups=8, topk_groups=9), INVALID),
    (dict(group_top=3), INVALID), (dict(x=None), INVALID), (dict(router=None), INVALID), (dict(w1=None), INVALID),
    (dict(w2=None), INVALID), (dict(idx=None), INVALID), (dict(weights=None), INVALID), (dict(y=None), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=100), WORKSPACE),
    (dict(workspace=ctypes.c_void_p(0x1008)), WORKSPACE),
    (dict(T=0, x=None, w1=None, idx=None, workspace=None, workspace_bytes=0), 0),
])
def test_moe_layer_rejects(lib, new, code):
    assert lib.mp_moe_layer(*changed(LAYER, **new).values()) == code


def test_workspace_sizes(lib):
    assert lib.mp_moe_layer_workspace_size(0, 4, 2, 8, 8, 8) >= 256
    assert lib.mp_moe_layer_workspace_size(65, 128, 8, 64, 64, 64) == 0
    assert lib.mp_moe_layer_workspace_size(4, 128, 0, 64, 64, 64) == 0
    assert lib.mp_moe_layer_workspace_size(64, 1024, 32, 65536, 65536, 65536) > 0
    assert lib.mp_block_norm_bwd_workspace_size(0, 64) >= 256
    assert lib.mp_block_norm_bwd_workspace_size(100, 64) % 256 == 0
    assert lib.mp_block_norm_bwd_workspace_size(-1, 64) == 0 and lib.mp_block_norm_bwd_workspace_size(1, 40000) == 0


def test_binding_wants_cuda_tensors():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        mp.mp_block_norm(x, pre_weight=torch.ones(8))
    with pytest.raises(ValueError, match="CUDA"):
        mp.mp_moe_layer(x.bfloat16(), torch.zeros(4, 8), torch.zeros(4, 8, 8).bfloat16(),
                        torch.zeros(4, 8, 4).bfloat16(), 2)
    with pytest.raises(TypeError):
        mp.mp_block_norm(torch.zeros(2, 8, dtype=torch.float64), pre_weight=torch.ones(8))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
def test_formulas_against_differentiation(kind, gate):
    """The gradients' formulas against autograd and against central differences, in 64 bits."""
    t, how = nu.make(4, 12, torch.float64, kind=kind, post=True, gate=gate, bias=True, scale=0.7, seed=5,
                     device="cpu")
    leaves = {k: None if v is None else v.clone().requires_grad_() for k, v in t.items()}
    s, y, stats, _, _ = nu.forward(leaves, how)
    g_s, g_y = nu.rows(4, 12, torch.float64, 1, "cpu"), nu.rows(4, 12, torch.float64, 2, "cpu")
    there = [k for k in nu.NAMES if leaves[k] is not None]
    grads = dict(zip(there, torch.autograd.grad([s, y], [leaves[k] for k in there], [g_s, g_y])))
    formulas = nu.backward(t, how, g_s, g_y, s.detach(), stats.detach())

    def loss(v):
        s, y, *_ = nu.forward(v, how)
        return float((s * g_s).sum() + (y * g_y).sum())
    for k in there:
        assert torch.allclose(formulas[k][0].view_as(grads[k]), grads[k], rtol=1e-9, atol=1e-9)
        d = torch.randn(t[k].shape, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
        h = 1e-5
        slope = (loss({**t, k: t[k] + h * d}) - loss({**t, k: t[k] - h * d})) / (2 * h)
        assert abs(slope - float((grads[k] * d).sum())) < 1e-6 * (1 + abs(slope))
