"""A block as a model stacks it: norm, router, experts, combine, norm after with gate, scale
and residual, norm before the next; trained, and asked for single tokens."""
from __future__ import annotations

import os
import sys

import pytest
import torch

import unpermute_routing_indices_gb300 as mp
from tests import norm_util as nu
from unpermute_routing_indices_gb300 import autograd as ag

pytestmark = pytest.mark.gpu
E, K, H, F = 16, 4, 256, 128


def parameters(seed):
    r = lambda *s, **k: nu.rows(*s, torch.bfloat16, seed + len(s) + k.pop("n", 0), **k)  # noqa: E731
    return dict(pre=r(1, H, n=1, mean=1.0, std=0.2)[0], post=r(1, H, n=2, mean=1.0, std=0.2)[0],
                next=r(1, H, n=3, mean=1.0, std=0.2)[0], gate=r(1, H, n=4, mean=0.5, std=0.3)[0],
                router=nu.rows(E, H, torch.float32, seed + 5, mean=0.0, std=H ** -0.5),
                w1=r(E * 2 * F, H, n=6, mean=0.0, std=H ** -0.5).view(E, 2 * F, H),
                w2=r(E * H, F, n=7, mean=0.0, std=F ** -0.5).view(E, H, F))


def block(x, p, idx=None):
    """(s, y) of one block on the stream x, through the differentiable forms."""
    _, n = ag.block_norm(x, pre_weight=p["pre"])
    logits = n.float() @ p["router"].t()
    i, w = ag.route(logits, K, score="sigmoid")
    rows, _, d = ag.permute(n, i, E)
    out = ag.unpermute(ag.expert_mlp(rows, d, p["w1"], p["w2"]), d, w)
    return ag.block_norm(out, x, post_weight=p["post"], gate=p["gate"], scale=0.5, pre_weight=p["next"]), i


def plain(x, p, idx):
    """The same in 64 bits, with the given choice."""
    def rms(v, w):
        return v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * w
    n = rms(x, p["pre"])
    s = torch.sigmoid(n @ p["router"].t()).gather(1, idx.long())
    w = s / s.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for k in range(K):
        z = torch.einsum("th,tfh->tf", n, p["w1"][idx[:, k].long()])
        h = torch.nn.functional.silu(z[:, :F]) * z[:, F:]
        out = out + w[:, k:k + 1] * torch.einsum("tf,thf->th", h, p["w2"][idx[:, k].long()])
    s = x + 0.5 * p["gate"] * rms(out, p["post"])
    return s, rms(s, p["next"])


def test_a_training_step():
    """Results and gradients against the block in 64 bits.  On the way to a gradient at most a
    dozen tensors are rounded to bf16, by 2^-8 of each value at most: 12/256 in norm, and
    as much again for what the norms' divisions make of it."""
    T = 96
    p = parameters(3)
    leaves = {k: v.clone().requires_grad_() for k, v in p.items()}
    x = nu.rows(T, H, torch.bfloat16, 50, mean=0.1).requires_grad_()
    (s, y), idx = block(x, leaves)
    g_s, g_y = nu.rows(T, H, torch.bfloat16, 51, mean=0.0), nu.rows(T, H, torch.bfloat16, 52, mean=0.0)
    got = torch.autograd.grad([s, y], [x, *leaves.values()], [g_s, g_y])
    wide = {k: v.double().requires_grad_() for k, v in p.items()}
    x64 = x.detach().double().requires_grad_()
    s64, y64 = plain(x64, wide, idx)
    want = torch.autograd.grad([s64, y64], [x64, *wide.values()], [g_s.double(), g_y.double()])
    for name, a, b in zip(["s", "y", "x", *p], [s, y, *got], [s64, y64, *want]):
        off = float((a.double() - b).norm() / b.norm())
        assert off <= 24 / 256, (name, off)


@pytest.mark.parametrize("T", [1, 5, 64])
def test_single_tokens(T):
    """norm, layer, norm for the tokens of answers beside the calls of the training step."""
    p = parameters(9)
    x = nu.rows(T, H, torch.bfloat16, T, mean=0.1)
    (want_s, want_y), idx = block(x, p)
    _, n, _ = mp.mp_block_norm(x, pre_weight=p["pre"])
    out, i, w = mp.mp_moe_layer(n, p["router"], p["w1"], p["w2"], K, score="sigmoid")
    s, y, _ = mp.mp_block_norm(out, x, post_weight=p["post"], gate=p["gate"], scale=0.5, pre_weight=p["next"])
    exact_s, exact_y = plain(x.double(), {k: v.double() for k, v in p.items()}, i)
    same = (i == idx).all(1)        # fp32 logits of another order of sums may turn a near choice
    assert int((~same).sum()) <= 1
    for a, b, c in ((s, exact_s, want_s), (y, exact_y, want_y)):
        assert float((a.double() - b).norm() / b.norm()) <= 8 / 256
        assert float((a[same].double() - c[same].double()).norm() / c.double().norm()) <= 16 / 256


@pytest.mark.parametrize("T", [1, 7, 64])
def test_the_example_layer(T):
    """Its answers to few tokens, beside the calls for many."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_layer
    layer = moe_layer.MoeLayer.make(256, 64, 16, 4, seed=3)
    layer.bias += torch.linspace(-0.1, 0.1, 16, device="cuda")
    x = nu.rows(T, 256, torch.bfloat16, T, mean=0.0)
    y, idx, w = mp.mp_moe_layer(x, layer.router, layer.w1, layer.w2, 4, score="sigmoid", bias=layer.bias)
    want, bound = nu.layer(x, layer.w1, layer.w2, None, None, "swiglu", idx, w)
    nu.within(layer.answer_few(x), want, bound)
    assert torch.equal(layer.answer_few(x), y)
    assert float((layer.answer(x).double() - want).norm() / want.norm()) <= 4 * 2.0 ** -8


def test_captured_answers():
    """Eight steps of an answer in one graph, each fed by the last, replayed with new tokens."""
    p = parameters(4)
    x = nu.rows(2, H, torch.bfloat16, 1, mean=0.1)
    ws = torch.empty(mp.mp_moe_layer_workspace_size(2, E, K, H, F, H), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def steps(v):
        for _ in range(8):
            _, n, _ = mp.mp_block_norm(v, pre_weight=p["pre"], status=status)
            out, _, _ = mp.mp_moe_layer(n, p["router"], p["w1"], p["w2"], K, workspace=ws, status=status)
            v, _, _ = mp.mp_block_norm(out, v, post_weight=p["post"], scale=0.1, status=status)
        return v
    steps(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = steps(x)
    for seed in (5, 6):
        x.copy_(nu.rows(2, H, torch.bfloat16, seed, mean=0.1))
        graph.replay()
        assert torch.equal(got, steps(x))
    assert int(status) == 0


def test_a_captured_training_step():
    p = {k: v.clone().requires_grad_() for k, v in parameters(8).items()}
    x = nu.rows(32, H, torch.bfloat16, 50, mean=0.1)
    g = [nu.rows(32, H, torch.bfloat16, 51, mean=0.0), nu.rows(32, H, torch.bfloat16, 52, mean=0.0)]

    def step():
        (s, y), _ = block(x, p)
        return torch.autograd.grad([s, y], list(p.values()), g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.copy_(nu.rows(32, H, torch.bfloat16, 60, mean=0.1))
    graph.replay()
    torch.cuda.synchronize()
    want = step()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
