"""The router's groups at their edges: groups of one expert, and scores that round to one
value, which logits tell apart where there is no bias."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import unpermute_routing_indices_gb300 as mp
from tests.gpu_util import DEV
from tests.test_gpu_route import choose, logits_of, scores

pytestmark = pytest.mark.gpu


def route(l, K, bias, **how):
    bt = None if bias is None else torch.from_numpy(bias).to(DEV)
    return mp.mp_route(torch.from_numpy(l).to(DEV), K, bias=bt, **how)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("E,keep,K,top", [(8, 4, 3, 1), (8, 4, 3, 2), (32, 9, 8, 2), (32, 32, 8, 1), (5, 2, 2, 2),
                                          (2, 1, 1, 1), (1, 1, 1, 2)])
def test_groups_of_one_expert(score, with_bias, E, keep, K, top):
    """n_groups == E: the choice, weights and all, of no groups."""
    T = 100
    l = logits_of(T, E, E + keep).cpu().numpy()
    l[40:] = np.round(l[40:] * 2) / 2              # ties
    l[50:60] = 45 + l[50:60]                       # sigmoids that are 1 in 64 bits
    l[60:70, ::2] = -np.inf
    bias = (0.1 * np.random.default_rng(E).standard_normal(E)).astype(np.float32) if with_bias else None
    idx, w = route(l, K, bias, score=score, n_groups=E, topk_groups=keep, group_top=top)
    same_idx, same_w = route(l, K, bias, score=score)
    assert torch.equal(idx, same_idx) and torch.equal(w, same_w)
    l64 = l.astype(np.float64)
    s, usable = scores(l64, score)
    want = choose(l64, s, usable, K, None if bias is None else bias.astype(np.float64), 1, 1, 1)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)


@pytest.mark.parametrize("score,shift", [("sigmoid", 45.0), ("softmax", -800.0)])
@pytest.mark.parametrize("G,keep,E,K", [(1, 1, 64, 6), (8, 3, 64, 6), (4, 2, 128, 8), (6, 2, 24, 5)])
def test_scores_that_round_to_one_value(score, shift, G, keep, E, K):
    """Sigmoids that are 1, and softmax terms that are 0, in 64 bits too: without a bias
    the logits decide between experts, and between groups by their best one."""
    T = 60
    l = logits_of(T, E, G + E).cpu().numpy() + np.float32(shift)
    if score == "softmax":
        l[:, 5] = 0                                # all the others' terms are below 2^-1074
    idx, _ = route(l, K, None, score=score, n_groups=G, topk_groups=keep)
    l64 = l.astype(np.float64)
    want = choose(l64, l64, np.ones_like(l64, dtype=bool), K, None, G, keep, 1)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)
