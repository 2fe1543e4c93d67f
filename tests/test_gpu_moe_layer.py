"""The example layer: its forward pass and gradients against 64 bits, its single-token
path against its batch path, and a training run that learns."""
from __future__ import annotations

import os
import sys

import pytest
import torch

from tests.gpu_util import DEV

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
pytestmark = pytest.mark.gpu
BF16 = torch.finfo(torch.bfloat16).eps / 2


def plain(layer, x):
    """The layer in 64 bits, token by token: (y, the magnitudes it is the sum of)."""
    logits = (x.float() @ layer.router.t()).double()
    s = torch.sigmoid(logits)
    idx = (s + layer.bias.double()).sort(dim=1, descending=True, stable=True).indices[:, :layer.topk]
    w = s.gather(1, idx)
    w = w / w.sum(1, keepdim=True)
    y, size = torch.zeros_like(x, dtype=torch.float64), torch.zeros_like(x, dtype=torch.float64)
    for k in range(layer.topk):
        w1, w2 = layer.w1[idx[:, k]].double(), layer.w2[idx[:, k]].double()
        z = torch.einsum("th,tfh->tf", x.double(), w1)
        a, b = z.chunk(2, 1)
        h = a * torch.sigmoid(a) * b
        y += w[:, k:k + 1] * torch.einsum("tf,thf->th", h, w2)
        size += w[:, k:k + 1] * torch.einsum("tf,thf->th", h.abs(), w2.abs())
    return y, size


@pytest.mark.parametrize("T", [1, 7, 300])
def test_layer_against_64_bits(T):
    """h, each expert's row and y are rounded to bf16: 2^-8 of the magnitudes summed,
    three times; fp32 sums of 64 and 256 terms are far below."""
    import moe_layer
    layer = moe_layer.MoeLayer.make(256, 64, 16, 4, seed=3)
    layer.bias += torch.linspace(-0.1, 0.1, 16, device=DEV)
    x = torch.randn(T, 256, device=DEV).bfloat16()
    y, size = plain(layer, x)
    got = layer.answer(x)
    assert ((got.double() - y).abs() <= 3.1 * BF16 * size).all()
    trained, counts = layer.train_step(x)
    assert torch.equal(trained, got) and int(counts.sum()) == 4 * T
    one = torch.cat([layer.answer(x[t:t + 1]) for t in range(min(T, 20))])
    assert ((one.double() - y[:20]).abs() <= 3.1 * BF16 * size[:20]).all()


def test_training_learns_and_balances():
    import moe_layer
    layer, teacher, losses, loads = moe_layer.train(steps=60, T=1024)
    assert torch.isfinite(losses).all()
    assert losses[-5:].mean() < 0.8 * losses[:5].mean()
    assert loads[-5:].mean() < loads[:5].mean() + 0.2
