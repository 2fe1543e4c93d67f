"""The router's and the experts' entry points reject bad arguments on the host,
before any launch (no GPU needed; nothing here reaches a kernel)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import unpermute_routing_indices_gb300 as mp
from unpermute_routing_indices_gb300 import _build, _lib

FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: every call fails validation
INVALID, UNSUPPORTED = -1, -3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


def changed(base, **new):
    return {**base, **new}


ROUTE = dict(logits=FAKE, dtype=2, bias=None, T=4, E=64, K=8, score=0, n_groups=1, topk_groups=1,
             group_top=1, renorm=1, scale=1.0, idx=FAKE, weights=FAKE, stream=None)


@pytest.mark.parametrize("new,code", [
    (dict(T=-1), INVALID), (dict(K=0), INVALID), (dict(K=65), INVALID), (dict(E=0), INVALID),
    (dict(score=2), INVALID), (dict(score=-1), INVALID), (dict(dtype=3), INVALID),
    (dict(K=33), UNSUPPORTED), (dict(E=1025), UNSUPPORTED), (dict(T=2 ** 31), UNSUPPORTED),
    (dict(n_groups=0), INVALID), (dict(n_groups=3), INVALID),
    (dict(n_groups=64, topk_groups=8), UNSUPPORTED),
    (dict(n_groups=8, topk_groups=9), INVALID), (dict(n_groups=16, topk_groups=1), INVALID),
    (dict(group_top=0), INVALID), (dict(group_top=3), INVALID),
    (dict(logits=None), INVALID), (dict(idx=None), INVALID), (dict(weights=None), INVALID),
    (dict(T=0, logits=None, idx=None, weights=None), 0),
])
def test_route_rejects(lib, new, code):
    assert lib.mp_route(*changed(ROUTE, **new).values()) == code


ROUTE_BWD = dict(g=FAKE, logits=FAKE, dtype=0, idx=FAKE, T=4, E=64, K=8, score=1, renorm=1,
                 scale=1.0, g_logits=FAKE, stream=None)


@pytest.mark.parametrize("new,code", [
    (dict(T=-1), INVALID), (dict(K=0), INVALID), (dict(score=7), INVALID), (dict(dtype=-1), INVALID),
    (dict(K=33), UNSUPPORTED), (dict(E=2000), UNSUPPORTED),
    (dict(g=None), INVALID), (dict(idx=None), INVALID), (dict(g_logits=None), INVALID),
    (dict(T=0, g=None, logits=None, idx=None, g_logits=None), 0),
])
def test_route_bwd_rejects(lib, new, code):
    assert lib.mp_route_bwd(*changed(ROUTE_BWD, **new).values()) == code


GEMM = dict(x=FAKE, w=FAKE, offsets=FAKE, R=8, E=4, N=64, K=64, bias=None, act=0, residual=None,
            out=FAKE, save=0, z=None, z_exp=None, status=None, stream=None)


@pytest.mark.parametrize("new,code", [
    (dict(R=-1), INVALID), (dict(E=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID),
    (dict(E=1025), UNSUPPORTED), (dict(R=2 ** 31), UNSUPPORTED), (dict(N=2 ** 23), UNSUPPORTED),
    (dict(K=2 ** 23), UNSUPPORTED),
    (dict(act=6), INVALID), (dict(act=-1), INVALID), (dict(act=5, N=63), INVALID),
    (dict(save=3), INVALID), (dict(save=1), INVALID), (dict(save=2, z=FAKE), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(offsets=None), INVALID),
    (dict(out=None), INVALID),
    (dict(R=0, x=None, w=None, out=None), 0),
])
def test_expert_gemm_rejects(lib, new, code):
    assert lib.mp_expert_gemm(*changed(GEMM, **new).values()) == code


DGRAD = dict(g=FAKE, w=FAKE, offsets=FAKE, R=8, E=4, N=64, K=64, act=5, save=2, z=FAKE,
             z_exp=FAKE, g_x=FAKE, h=None, status=None, stream=None)


@pytest.mark.parametrize("new,code", [
    (dict(R=-1), INVALID), (dict(K=0), INVALID), (dict(E=5000), UNSUPPORTED),
    (dict(act=9), INVALID), (dict(save=0), INVALID), (dict(save=4), INVALID),
    (dict(act=0), INVALID),                       # no activation: nothing saved to read
    (dict(act=0, save=0, h=FAKE), INVALID),       # nor anything to compute again
    (dict(z=None), INVALID), (dict(z_exp=None), INVALID), (dict(g=None), INVALID),
    (dict(g_x=None), INVALID), (dict(R=0, g=None, w=None, g_x=None), 0),
])
def test_expert_dgrad_rejects(lib, new, code):
    assert lib.mp_expert_dgrad(*changed(DGRAD, **new).values()) == code


WGRAD = dict(g=FAKE, x=FAKE, offsets=FAKE, R=8, E=4, N=64, K=64, dtype=0, accumulate=0, g_w=FAKE,
             g_bias=None, status=None, stream=None)


@pytest.mark.parametrize("new,code", [
    (dict(R=-1), INVALID), (dict(N=0), INVALID), (dict(E=1025), UNSUPPORTED),
    (dict(dtype=1), INVALID), (dict(accumulate=1), INVALID), (dict(g_w=None), INVALID),
    (dict(offsets=None), INVALID), (dict(g=None), INVALID), (dict(x=None), INVALID),
])
def test_expert_wgrad_rejects(lib, new, code):
    assert lib.mp_expert_wgrad(*changed(WGRAD, **new).values()) == code


MLP = dict(x=FAKE, w1=FAKE, b1=None, w2=FAKE, b2=None, offsets=FAKE, R=8, E=4, H=64, F=32, O=64,
           act=5, h=FAKE, y=FAKE, save=0, z=None, z_exp=None, status=None, stream=None)


@pytest.mark.parametrize("new,code", [
    (dict(R=-1), INVALID), (dict(F=0), INVALID), (dict(F=2 ** 22), INVALID), (dict(act=0), INVALID),
    (dict(act=6), INVALID), (dict(h=None), INVALID), (dict(x=None), INVALID), (dict(w1=None), INVALID),
    (dict(save=1), INVALID), (dict(H=0), INVALID), (dict(E=1025), UNSUPPORTED),
    (dict(w2=None), INVALID), (dict(y=None), INVALID), (dict(O=0), INVALID),
    (dict(R=0, x=None, w1=None, w2=None, h=None, y=None), 0),
])
def test_expert_mlp_rejects(lib, new, code):
    assert lib.mp_expert_mlp(*changed(MLP, **new).values()) == code


MLP_BWD = dict(g_y=FAKE, x=FAKE, w1=FAKE, w2=FAKE, offsets=FAKE, R=8, E=4, H=64, F=32, O=64, act=5,
               save=1, z=FAKE, z_exp=None, g_z=FAKE, h=FAKE, g_x=FAKE, g_w1=FAKE, g_b1=None,
               g_w2=FAKE, g_b2=None, status=None, stream=None)


@pytest.mark.parametrize("new,code", [
    (dict(R=-1), INVALID), (dict(F=0), INVALID), (dict(O=0), INVALID), (dict(act=0), INVALID),
    (dict(save=0), INVALID), (dict(save=2), INVALID), (dict(z=None), INVALID), (dict(g_y=None), INVALID),
    (dict(g_z=None), INVALID), (dict(h=None), INVALID), (dict(offsets=None), INVALID),
    (dict(w1=None), INVALID), (dict(w2=None), INVALID),
    (dict(E=5000), UNSUPPORTED),
])
def test_expert_mlp_bwd_rejects(lib, new, code):
    assert lib.mp_expert_mlp_bwd(*changed(MLP_BWD, **new).values()) == code


def test_status_bits_have_names():
    assert mp.status_bits(0x80 | 0x100) == {"bad_offsets", "stalled"}


def test_the_binding_refuses_what_is_not_on_a_gpu():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    offsets = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mp.mp_expert_gemm(x, w, offsets)
    with pytest.raises(ValueError, match="CUDA"):
        mp.mp_expert_dgrad(x, w, offsets)
    with pytest.raises(ValueError, match="CUDA"):
        mp.mp_expert_wgrad(x, x, offsets)
    with pytest.raises(ValueError, match="CUDA"):
        mp.mp_route(x.float(), 4)
    with pytest.raises(TypeError):
        mp.mp_route(x.int(), 4)


def test_expert_mlp_refuses_unknown_forms():
    from unpermute_routing_indices_gb300 import autograd as ag
    with pytest.raises(ValueError, match="activation"):
        ag.expert_mlp(None, None, None, None, act="none")
    with pytest.raises(ValueError, match="checkpoint"):
        ag.expert_mlp(None, None, None, None, checkpoint="int4")
