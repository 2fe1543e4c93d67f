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


def test_expert_mlp_rounds_to_8_bits_only_if_asked(calls):
    (x, w1, w2), offsets = layer()
    ag.expert_mlp(x, offsets, w1, w2)
    assert calls[0]["save"] == "bf16"


def stand_ins(monkeypatch):
    """The other entry points on the CPU, as far as their types go: every result is a
    linear form of the floating-point arguments (so gradients depend on them)."""
    def make(shapes):
        def call(*args, **how):
            given = [a.detach().float().sum() for a in (*args, *how.values())
                     if torch.is_tensor(a) and a.is_floating_point()]
            made = tuple(torch.zeros(shape, dtype=torch.int32) if kind is int else torch.ones(shape) * sum(given)
                         for shape, kind in shapes)
            return made if len(made) > 1 else made[0]
        return call
    rows, tokens, slots = (6, 4), (3, 4), (3, 2)
    for name, shapes in dict(
            mp_permute=[(rows, float), ((6,), float)], mp_permute_bwd=[(tokens, float), (slots, float)],
            mp_unpermute=[(tokens, float)], mp_unpermute_ep=[(tokens, float)],
            mp_unpermute_bwd=[(rows, float), (slots, float)],
            mp_topk_softmax=[(slots, int), (slots, float)], mp_topk_softmax_bwd=[((3, 5), float)],
            mp_route=[(slots, int), (slots, float)], mp_route_bwd=[((3, 5), float)],
            mp_sort_chunks_pad=[((8, 4), float), ((8,), float), ((8,), int), ((3,), int)],
            mp_sort_chunks_pad_bwd=[(rows, float)],
            mp_unpad_restore=[(rows, float)], mp_unpad_restore_bwd=[((8, 4), float)],
            ).items():
        monkeypatch.setattr(ag, name, make(shapes))
    restored = ag.mp_unpad_restore_bwd
    monkeypatch.setattr(ag, "mp_unpad_restore_bwd", lambda *args: (restored(*args), None))
    monkeypatch.setattr(ag, "mp_zero_rows_from", lambda buffer, first: buffer)


def leaf(*shape):
    return torch.randn(*shape, requires_grad=True)


def expert_mlp():
    (x, w1, w2), offsets = layer()
    return ag.expert_mlp(x, offsets, w1, w2), x


def route():
    logits = leaf(3, 5)
    return ag.route(logits, 2)[1], logits


def topk_softmax():
    logits = leaf(3, 5)
    return ag.topk_softmax(logits, 2)[1], logits


def permute():
    x = leaf(3, 4)
    return ag._Permute.apply(x, leaf(3, 2), torch.zeros(3, 2), torch.zeros(1), 6)[0], x


def unpermute():
    rows = leaf(6, 4)
    return ag._Unpermute.apply(rows, leaf(3, 2), torch.zeros(3, 2), torch.zeros(1), None), rows


def sort_chunks_pad():
    x = leaf(6, 4)
    return ag.sort_chunks_pad(x, None, None, 2, 4, 8)[0], x


def unpad_restore():
    padded = leaf(8, 4)
    return ag.unpad_restore(padded, torch.zeros(8), 6)[0], padded


FORMS = [expert_mlp, route, topk_softmax, permute, unpermute, sort_chunks_pad, unpad_restore]


@pytest.mark.parametrize("form", FORMS, ids=lambda f: f.__name__)
def test_gradients_of_gradients_are_refused(calls, monkeypatch, form):
    """Not left out of the sum: a second backward pass that reaches a gradient of these
    raises; one that does not reach it, and the gradient's own values, are there."""
    stand_ins(monkeypatch)
    result, x = form()
    scale = torch.ones(result.shape, requires_grad=True)     # the gradient given depends on it
    g, = torch.autograd.grad((result * scale).sum(), x, create_graph=True)
    assert g.requires_grad and g.shape == x.shape
    again, = torch.autograd.grad((x ** 2).sum(), x)
    assert torch.equal(again, 2 * x.detach())
    with pytest.raises(RuntimeError, match="gradients of gradients"):
        ((g ** 2).sum() + (x ** 2).sum()).backward()
    result, x = form()
    plain, = torch.autograd.grad((result * scale.detach()).sum(), x)
    assert not plain.requires_grad and plain.shape == g.shape


@pytest.mark.parametrize("form", [expert_mlp, route, unpermute], ids=lambda f: f.__name__)
def test_gradients_that_depend_on_what_was_kept_are_refused(calls, monkeypatch, form):
    """The same where the gradient given depends on nothing, but the result does on the
    inputs (weights, logits, rows and probabilities)."""
    stand_ins(monkeypatch)
    result, x = form()
    g, = torch.autograd.grad(result.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="gradients of gradients"):
        ((g ** 2).sum() + (x ** 2).sum()).backward()


@pytest.mark.parametrize("form", [permute, sort_chunks_pad, unpad_restore], ids=lambda f: f.__name__)
def test_gradients_that_depend_on_nothing_are_final(monkeypatch, form):
    """Gradients of a reordering are constant where the gradient given is: there is
    nothing to leave out."""
    stand_ins(monkeypatch)
    result, x = form()
    g, = torch.autograd.grad(result.sum(), x, create_graph=True)
    assert not g.requires_grad
    ((g ** 2).sum() + (x ** 2).sum()).backward()
    assert torch.equal(x.grad, 2 * x.detach())
