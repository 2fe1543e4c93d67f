"""The router with scores, balance bias and renormalised weights against its
definition in 64 bits: choices equal, weights and gradients within bounds
derived from the roundings.

Weights: expf and the divisions are within 2 and 1 ulp (2^-23 and 2^-24), the
argument l - max is rounded once (2^-24 |l - max|, at most 30 here), sums of n
terms add n 2^-24: W = (32 + 30 + 8) 2^-24 relative covers the K <= 32 picks, and
(E/32 + 5) more the sum over all experts.
Gradients: sums of products of the weights, each term within the same relative
error plus its own, so 4 W times the sum of the magnitudes; a 16-bit result is
off by half a step more."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import unpermute_routing_indices_gb300 as mp
from unpermute_routing_indices_gb300 import autograd as ag
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


def scores(l, score):
    """(scores, usable) of float64 logits."""
    usable = ~np.isnan(l) & (l > -np.inf)
    l = np.where(usable, np.minimum(l, np.finfo(np.float32).max), -np.inf)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            s = 1 / (1 + np.exp(-l))
        else:
            m = l.max(1, keepdims=True)
            s = np.exp(l - np.where(np.isfinite(m), m, 0))
            s = s / np.maximum(s.sum(1, keepdims=True), 1e-300)
    return np.where(usable, s, 0), usable


def choose(l, s, usable, K, bias, G, keep, top):
    """The definition, token by token, in Python's own order."""
    T, E = l.shape
    idx = np.full((T, K), -1, np.int32)
    for t in range(T):
        c = s[t] if bias is None else s[t] + bias
        live = [e for e in range(E) if usable[t, e] and (bias is None or bias[e] > -np.inf)]
        if G > 1:
            n = E // G
            worth = {}
            for g in range(G):
                best = sorted((c[e] for e in live if e // n == g), reverse=True)[:top]
                if best:
                    worth[g] = sum(best)
            kept = sorted(worth, key=lambda g: (-worth[g], g))[:keep]
            live = [e for e in live if e // n in kept]
        by = l[t] if bias is None else c
        live.sort(key=lambda e: (-by[e], e))
        idx[t, :min(K, len(live))] = live[:K]
    return idx


def weights(s, l, idx, score, renorm, scale):
    """Weights and the magnitude they are compared by; empty slots 0."""
    at = np.maximum(idx, 0)
    w = np.where(idx >= 0, np.take_along_axis(s, at, 1), 0)
    if renorm:
        lw = np.where(idx >= 0, np.take_along_axis(l, at, 1), -np.inf)
        m = lw.max(1, keepdims=True)
        low = m < -30                # every score underflows together: the ratio is exp's
        if score == "softmax" or low.any():
            with np.errstate(invalid="ignore"):
                e = np.where(idx >= 0, np.exp(lw - np.where(np.isfinite(m), m, 0)), 0)
            w = np.where(low | (score == "softmax"), e, w)
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    return scale * w


def logits_of(T, E, seed, dtype=torch.float32, kind="normal"):
    rng = np.random.default_rng(seed)
    if kind == "ties":
        a = rng.integers(-3, 4, (T, E)) / 2
    else:
        a = rng.standard_normal((T, E)) * 1.5
    return torch.from_numpy(a.astype(np.float32)).to(DEV).to(dtype)


CASES = [
    # T, E, K, score, dtype, bias, groups, keep, group_top, renorm, scale, kind
    (1, 1, 1, "softmax", torch.float32, False, 1, 1, 1, True, 1.0, "normal"),
    (1, 64, 6, "softmax", torch.float32, False, 1, 1, 1, True, 1.0, "normal"),
    (37, 64, 6, "sigmoid", torch.float32, True, 1, 1, 1, True, 1.0, "normal"),
    (513, 128, 8, "softmax", torch.bfloat16, False, 1, 1, 1, False, 1.0, "normal"),
    (300, 128, 8, "softmax", torch.float16, True, 1, 1, 1, False, 2.5, "normal"),
    (1025, 256, 8, "sigmoid", torch.float32, True, 8, 4, 2, True, 2.5, "normal"),
    (200, 256, 8, "sigmoid", torch.bfloat16, False, 8, 4, 2, True, 1.0, "normal"),
    (200, 256, 8, "softmax", torch.float32, True, 8, 3, 2, True, 1.0, "normal"),
    (100, 96, 5, "sigmoid", torch.float32, True, 6, 2, 1, False, 1.0, "normal"),
    (100, 96, 16, "softmax", torch.float32, False, 6, 2, 2, False, 1.0, "ties"),
    (100, 160, 7, "sigmoid", torch.float32, True, 5, 3, 2, True, 1.0, "ties"),
    (64, 40, 5, "sigmoid", torch.float32, False, 8, 8, 1, True, 1.0, "ties"),
    (33, 1024, 32, "softmax", torch.float32, True, 32, 8, 2, True, 1.0, "normal"),
    (33, 1000, 8, "sigmoid", torch.bfloat16, True, 1, 1, 1, True, 1.0, "normal"),
    (65, 8, 8, "sigmoid", torch.float32, True, 2, 2, 2, False, 1.0, "ties"),
    (40, 512, 9, "softmax", torch.float16, False, 16, 4, 1, False, 1.0, "normal"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d-E%d-K%d-%s" % c[:4])
def test_route_and_its_gradient(case):
    T, E, K, score, dtype, with_bias, G, keep, top, renorm, scale, kind = case
    lt = logits_of(T, E, T + E + K, dtype, kind)
    rng = np.random.default_rng(5)
    bias = rng.standard_normal(E).astype(np.float32) * 0.1 if with_bias else None
    if with_bias and kind == "ties":
        bias = np.round(bias * 4).astype(np.float32) / 4
    bt = None if bias is None else torch.from_numpy(bias).to(DEV)
    how = dict(score=score, renorm=renorm, scale=scale)
    idx, w = mp.mp_route(lt, K, bias=bt, n_groups=G, topk_groups=keep, group_top=top, **how)
    l = lt.double().cpu().numpy()
    s, usable = scores(l, score)
    want = choose(l, s, usable, K, None if bias is None else bias.astype(np.float64), G, keep, top)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)
    W = (70 + E / 32 + 5) * 2.0 ** -24
    exact = weights(s, l, want, score, renorm, scale)
    assert np.all(np.abs(w.cpu().numpy() - exact) <= W * np.abs(exact) + 1e-37)

    g = rng.standard_normal((T, K)).astype(np.float32)
    got = mp.mp_route_bwd(torch.from_numpy(g).to(DEV), lt, idx, **how)
    assert got.dtype == dtype
    formula, size = gradient(s, want, g.astype(np.float64), score, renorm, scale)
    half = 0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    low = torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    assert np.all(np.abs(got.double().cpu().numpy() - formula)
                  <= 4 * W * size + half * np.abs(formula) + low)


def gradient(s, idx, g, score, renorm, scale):
    """(gradient, sum of the magnitudes it is made of), from the definition."""
    at = np.maximum(idx, 0)
    picked = np.where(idx >= 0, np.take_along_axis(s, at, 1), 0)
    g = np.where(idx >= 0, g, 0) * scale
    if renorm:
        S = np.maximum(picked.sum(1, keepdims=True), 1e-300)
        p = picked / S
        mean, amean = (g * p).sum(1, keepdims=True), (np.abs(g) * p).sum(1, keepdims=True)
        u, a = (g - mean) / S, (np.abs(g) + amean) / S
    else:
        u, a = g, np.abs(g)
    du, da = np.zeros_like(s), np.zeros_like(s)
    for t in range(s.shape[0]):
        for k in range(idx.shape[1]):
            if idx[t, k] >= 0:
                du[t, idx[t, k]] += u[t, k]
                da[t, idx[t, k]] += a[t, k]
    if score == "sigmoid":
        return du * s * (1 - s), da * s
    return (s * (du - (du * s).sum(1, keepdims=True)),
            s * (da + (da * s).sum(1, keepdims=True)))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(score, renorm):
    """<gradient, d> is the difference of the 64-bit loss along d, up to the
    gradient's own error and the third derivatives (below step^2)."""
    T, E, K, scale, step = 20, 48, 5, 1.5, 1e-4
    lt = logits_of(T, E, 3)
    idx, _ = mp.mp_route(lt, K, score=score, renorm=renorm, scale=scale)
    rng = np.random.default_rng(4)
    g = rng.standard_normal((T, K)).astype(np.float32)
    got = mp.mp_route_bwd(torch.from_numpy(g).to(DEV), lt, idx, score=score, renorm=renorm,
                          scale=scale).double().cpu().numpy()
    at, l = idx.cpu().numpy(), lt.double().cpu().numpy()
    d = rng.standard_normal((T, E))

    def loss(x):
        return (weights(scores(x, score)[0], x, at, score, renorm, scale) * g).sum()
    difference = (loss(l + step * d) - loss(l - step * d)) / (2 * step)
    _, size = gradient(scores(l, score)[0], at, g.astype(np.float64), score, renorm, scale)
    bound = 4 * 80 * 2.0 ** -24 * (size * np.abs(d)).sum() + 30 * step ** 2 * np.abs(g).sum()
    assert abs((got * d).sum() - difference) <= bound


def test_scores_next_to_each_other():
    """Sigmoids that fp32 rounds to 1, and sums with the bias that differ by
    less than fp32 holds, are told apart as 64 bits do."""
    E, K = 64, 8
    rng = np.random.default_rng(8)
    l = (20 + rng.permutation(E)[None, :] * 0.01 + np.zeros((50, 1))).astype(np.float32)
    l[25:] = rng.standard_normal((25, E)).astype(np.float32)
    bias = np.full(E, 0.25, np.float32)
    for t in range(25, 50):       # pairs a step of fp32 apart, in turned order
        l[t, 1::2] = np.nextafter(l[t, 0::2], np.float32(np.inf))
    idx, _ = mp.mp_route(torch.from_numpy(l).to(DEV), K, score="sigmoid",
                         bias=torch.from_numpy(bias).to(DEV))
    s, usable = scores(l.astype(np.float64), "sigmoid")
    want = choose(l.astype(np.float64), s, usable, K, bias.astype(np.float64), 1, 1, 1)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("E,top,copies", [(32, 2, 1), (32, 1, 1), (128, 2, 1), (128, 2, 2), (96, 1, 2)])
def test_groups_next_to_each_other(score, with_bias, E, top, copies):
    """Groups whose worths differ by a step of one logit, at the border of those
    kept: two of them, and three."""
    G, K, T = 4, 6, 200
    n = E // G
    rng = np.random.default_rng(E + top + copies)
    l = rng.standard_normal((T, G, n)).astype(np.float32)
    bias = (0.05 * rng.standard_normal((G, n))).astype(np.float32)
    l[:, 0] += 3                                   # kept in any case
    for g in range(2, 2 + copies):                 # the copies of group 1, a step off
        l[:, g] = l[:, 1]
        bias[g] = bias[1]
        t = np.arange(T)
        best = np.argmax(l[:, g] + 4 * bias[g], axis=1)
        l[t, g, best] = np.nextafter(l[t, g, best], np.where(t % 3 == g % 3, np.float32(9), np.float32(-9)))
    l[:, 2 + copies:] -= 3
    l, bias = l.reshape(T, E), bias.reshape(E)
    idx, _ = mp.mp_route(torch.from_numpy(l).to(DEV), K, score=score, n_groups=G, topk_groups=2,
                         group_top=top, bias=torch.from_numpy(bias).to(DEV) if with_bias else None)
    s, usable = scores(l.astype(np.float64), score)
    want = choose(l.astype(np.float64), s, usable, K, bias.astype(np.float64) if with_bias else None,
                  G, 2, top)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)


@pytest.mark.parametrize("step", [1, 3, 40])
def test_picks_next_to_each_other(step):
    """Runs of scores a few steps of fp32 apart around the last place."""
    E, K, T = 96, 8, 300
    rng = np.random.default_rng(step)
    l = rng.standard_normal((T, E)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    c = 1 / (1 + np.exp(-l.astype(np.float64))) + bias
    order = np.argsort(-c, axis=1)
    for t in range(T):
        at = order[t, K - 1]
        for i in range(1 + t % 3):                 # the next one, two, three
            e = order[t, K + i]
            target = c[t, at] - bias[e] + (rng.integers(-step, step + 1)) * 2.0 ** -25
            target = min(max(target, 1e-3), 1 - 1e-3)
            l[t, e] = np.float32(np.log(target / (1 - target)))
    idx, _ = mp.mp_route(torch.from_numpy(l).to(DEV), K, score="sigmoid",
                         bias=torch.from_numpy(bias).to(DEV))
    s, usable = scores(l.astype(np.float64), "sigmoid")
    want = choose(l.astype(np.float64), s, usable, K, bias.astype(np.float64), 1, 1, 1)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("groups", [(1, 1, 1), (4, 2, 2)])
def test_unavailable_experts(score, renorm, groups):
    """-inf and NaN logits and -inf biases are never picked; slots left over are
    empty, weigh nothing and give no gradient; the type's lowest value is
    picked last; +inf counts as the largest."""
    E, K = 32, 6
    G, keep, top = groups
    l = logits_of(12, E, 6).cpu().numpy()
    l[0] = -np.inf
    l[1] = np.nan
    l[2] = -np.inf
    l[2, 5] = 0.5                              # one left
    l[3, ::2] = -np.inf
    l[4, 3:] = np.finfo(np.float32).min        # the lowest finite value
    l[5, 7] = np.inf
    l[6, 1:9] = np.nan
    l[7, :] = np.finfo(np.float32).min
    l[8, 8:] = -np.inf                         # three of four groups gone
    l[9] = -200.0 + np.arange(E) % 5           # every sigmoid below fp32
    bias = np.zeros(E, np.float32)
    bias[4] = -np.inf
    bias[9] = np.nan
    lt, bt = torch.from_numpy(l).to(DEV), torch.from_numpy(bias).to(DEV)
    how = dict(score=score, renorm=renorm)
    idx, w = mp.mp_route(lt, K, bias=bt, n_groups=G, topk_groups=keep, group_top=top, **how)
    l64 = l.astype(np.float64)
    s, usable = scores(l64, score)
    want = choose(np.minimum(l64, np.finfo(np.float32).max), s, usable, K,
                  np.where(np.isnan(bias), -np.inf, bias).astype(np.float64), G, keep, top)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)
    got = w.cpu().numpy()
    assert np.isfinite(got).all() and (got[want < 0] == 0).all()
    if renorm:
        left = (want >= 0).any(1)
        np.testing.assert_allclose(got[left].sum(1), 1, atol=40 * 2.0 ** -24)
    g = mp.mp_route_bwd(torch.ones_like(w), lt, idx, **how).cpu().numpy()
    assert np.isfinite(g).all()
    assert (g[0] == 0).all() and (g[1] == 0).all()


def test_empty_and_refused():
    lt = torch.empty((0, 64), device=DEV)
    idx, w = mp.mp_route(lt, 4)
    assert idx.shape == (0, 4) and w.shape == (0, 4)
    lt = logits_of(4, 64, 1)
    with pytest.raises(mp.MPError):
        mp.mp_route(lt, 65)
    with pytest.raises(ValueError):
        mp.mp_route(lt, 4, score="tanh")
    with pytest.raises(ValueError):
        mp.mp_route(lt, 4, bias=torch.zeros(63, device=DEV))
    with pytest.raises(TypeError):
        mp.mp_route(lt, 4, bias=torch.zeros(64, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        mp.mp_route(lt.t(), 4)


def test_autograd_route():
    lt = logits_of(50, 64, 2).requires_grad_()
    idx, w = ag.route(lt, 6, score="sigmoid", scale=2.0)
    g = torch.randn_like(w)
    w.backward(g)
    want = mp.mp_route_bwd(g, lt.detach(), idx, score="sigmoid", scale=2.0)
    assert torch.equal(lt.grad, want) and not idx.requires_grad
