"""What the differentiable forms hand to the entry points, with stand-ins for those (no
GPU needed)."""
from __future__ import annotations

import pytest
import torch

from unpermute_routing_indices_gb300 import autograd as ag


@pytest.fixture
def calls(monkeypatch):
    """The keyword arguments of each call of the layer's two entry points."""
    seen = []

    def forward(rows, w1, w2, offsets, b1=None, b2=None, **how):
        seen.append(how)
        z = None if how["save"] == "none" else torch.zeros(rows.shape[0], w1.shape[1])
        return rows @ torch.ones(rows.shape[1], w2.shape[1]), z, None

    def backward(g_y, rows, w1, w2, offsets, z, z_exp=None, **how):
        seen.append(how)
        made = (torch.ones_like(rows), torch.ones_like(w1), torch.ones_like(w2), None, None)
        return tuple(t if need else None for t, need in zip(made, how["need"]))
    monkeypatch.setattr(ag, "mp_expert_mlp", forward)
    monkeypatch.setattr(ag, "mp_expert_mlp_bwd", backward)
    return seen


def layer(requires_grad=True):
    x, w1, w2 = torch.randn(5, 4), torch.randn(2, 6, 4), torch.randn(2, 4, 3)
    return [t.requires_grad_(requires_grad) for t in (x, w1, w2)], torch.tensor([0, 2, 5])


def test_expert_mlp_hands_the_status_word_on(calls):
    (x, w1, w2), offsets = layer()
    status = torch.zeros(1, dtype=torch.int32)
    y = ag.expert_mlp(x, offsets, w1, w2, status=status)
    y.sum().backward()
    assert len(calls) == 2 and all(how["status"] is status for how in calls)
    ag.expert_mlp(x, offsets, w1, w2).sum().backward()
    assert all(how["status"] is None for how in calls[2:])


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_expert_mlp_keeps_nothing_without_a_backward_pass(calls, mode):
    """Evaluating a trained layer, or one whose tensors require nothing."""
    (x, w1, w2), offsets = layer()
    with mode():
        assert not ag.expert_mlp(x, offsets, w1, w2).requires_grad
    tensors, _ = layer(requires_grad=False)
    ag.expert_mlp(tensors[0], offsets, *tensors[1:])
    assert [how["save"] for how in calls] == ["none", "none"]


@pytest.mark.parametrize("which", range(5))
@pytest.mark.parametrize("checkpoint", ["e4m3", "bf16"])
def test_expert_mlp_keeps_what_a_backward_pass_needs(calls, which, checkpoint):
    (x, w1, w2), offsets = layer(requires_grad=False)
    tensors = [x, w1, w2, torch.zeros(2, 6), torch.zeros(2, 4)]
    tensors[which].requires_grad_()
    y = ag.expert_mlp(x, offsets, w1, w2, *tensors[3:], checkpoint=checkpoint)
    assert y.requires_grad and calls[0]["save"] == checkpoint
