"""The experts' calls at edges of their contract: a residual that is the result's own
buffer, a contraction that takes longer than a wait may last without progress, rows
before the first expert's, the status word through autograd,
no rows, the order of sums."""
from __future__ import annotations

import pytest
import torch

import unpermute_routing_indices_gb300 as mp
from tests.gpu_util import DEV, status_word
from unpermute_routing_indices_gb300 import _lib
from unpermute_routing_indices_gb300 import autograd as ag
from tests.test_gpu_expert import COUNTS, GATED, normal, offsets_of

pytestmark = pytest.mark.gpu


# counts, N, K, activation, elements that the bases are moved by
IN_PLACE = [
    ("big", 640, 192, "none", 0),                  # whole tiles, stored by TMA
    ("long", 512, 320, "silu", 0),
    ("long", 2 * 1012, 776, "swiglu", 0),          # pairs of CTAs
    ("long", 2050, 1000, "none", 0),
    ("long", 2 * 264, 200, "swiglu", 8),           # 16-byte, not 32-byte aligned rows
    ("many", 101, 200, "relu", 0),                 # rows off 16 bytes: neighbours share sectors
    ("big", 2 * 129, 1031, "swiglu", 0),           # the load warps
    ("big", 514, 130, "none", 1),
    ("one expert", 328, 6344, "gelu", 0),          # split contractions
    ("first empty", 261, 2056, "none", 0),
    ("tokens", 2 * 264, 1032, "swiglu", 0),        # few rows, split
    ("tokens", 130, 512, "none", 0),
    ("few each", 131, 64, "none", 0),              # few rows, whole
]


@pytest.mark.parametrize("case", IN_PLACE, ids=lambda c: "%s-N%d-K%d-%s-s%d" % c)
def test_residual_in_place(case):
    """out may be the residual itself: the same bits as with a buffer of its own, and
    the rows that no expert has stay."""
    name, N, K, act, shift = case
    counts, more = COUNTS[name], 3
    E, R = len(counts), sum(counts) + more
    offsets = offsets_of(counts)
    F = N // 2 if act in GATED else N
    x, w = normal(R, K, seed=1, shift=shift), normal(E, N, K, seed=2, std=K ** -0.5, shift=shift)
    bias, residual = normal(E, N, seed=3), normal(R, F, seed=4, shift=shift)
    want = normal(R, F, seed=4, shift=shift)
    mp.mp_expert_gemm(x, w, offsets, bias=bias, act=act, residual=residual, out=want)
    for _ in range(3):
        both = normal(R, F, seed=4, shift=shift)
        got, _, _ = mp.mp_expert_gemm(x, w, offsets, bias=bias, act=act, residual=both, out=both)
        assert got is both and torch.equal(both, want)
    assert torch.equal(want[R - more:], residual[R - more:])


def test_a_long_contraction_is_no_stall():
    """360 million rows of one expert of 128, 1 x 1: 5.6 million slices of one tile, which
    take 5 s on one SM, longer than the 4 s that a wait lasts when nothing moves.  The
    sums are of three ones: exact."""
    R, E = 360_000_000, 128
    offsets = torch.full((E + 1,), R, dtype=torch.int32, device=DEV)
    offsets[0] = 0
    g = torch.zeros((R, 1), dtype=torch.bfloat16, device=DEV)
    x = torch.ones((R, 1), dtype=torch.bfloat16, device=DEV)
    for row in (0, R // 2 + 3, R - 1):
        g[row] = 1
    status = status_word()
    g_w, _ = mp.mp_expert_wgrad(g, x, offsets, dtype=torch.float32, status=status)
    assert int(status) == 0
    assert g_w[0].item() == 3.0 and (g_w[1:] == 0).all()


@pytest.mark.parametrize("before,counts,after", [(7, [30, 0, 41], 5), (3, [1, 2, 0], 0), (200, [500, 900], 0),
                                                 (1200, [2300, 1900, 2100], 77), (64, [0, 0], 6)])
@pytest.mark.parametrize("H,F", [(136, 72), (33, 40), (264, 136)])
def test_rows_before_the_first_expert(before, counts, after, H, F):
    """Offsets may begin past row 0 (a part of the experts, with all the rows): the rows
    before them are zero in the layer's result and gradient, whatever the buffers held,
    and the others what a call on them alone gives."""
    E, n = len(counts), sum(counts)
    R, offsets = before + n + after, offsets_of(counts) + before
    x, g = normal(R, H, seed=1), normal(R, H, seed=2)
    w1, w2 = normal(E, 2 * F, H, seed=3, std=0.1), normal(E, H, F, seed=4, std=0.1)
    none = torch.ones(R, dtype=torch.bool, device=DEV)
    none[before:before + n] = False
    x[none], g[none] = float("nan"), float("inf")
    y, g_x = (torch.full((R, H), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    h, g_z = (torch.empty((R, k), dtype=torch.bfloat16, device=DEV) for k in (F, 2 * F))
    z = torch.empty((R, 2 * F), dtype=torch.bfloat16, device=DEV)
    status, lib = status_word(), _lib.load()
    stream = torch.cuda.current_stream().cuda_stream

    def p(t):
        return t.data_ptr()
    assert lib.mp_expert_mlp(p(x), p(w1), None, p(w2), None, p(offsets), R, E, H, F, H, mp.ACTS["swiglu"], p(h),
                             p(y), mp.SAVES["bf16"], p(z), None, p(status), stream) == 0
    assert lib.mp_expert_mlp_bwd(p(g), p(x), p(w1), p(w2), p(offsets), R, E, H, F, H, mp.ACTS["swiglu"],
                                 mp.SAVES["bf16"], p(z), None, p(g_z), None, p(g_x), None, None, None, None,
                                 p(status), stream) == 0
    assert int(status) == 0
    assert (y[none] == 0).all() and (g_x[none] == 0).all()
    assert torch.isfinite(y.float()).all() and torch.isfinite(g_x.float()).all()
    assert (y[~none] != 7.0).any(1).all() and (g_x[~none] != 7.0).any(1).all()
    out = torch.full((R, 2 * F), 7.0, dtype=torch.bfloat16, device=DEV)
    mp.mp_expert_gemm(x, w1, offsets, out=out)
    assert (out[none] == 7.0).all() and torch.equal(out[~none], z[~none])


def test_status_through_autograd():
    """Offsets that fall set their bit in the forward and in the backward pass of the
    layer's differentiable form; good ones set none."""
    R, H, F = 100, 64, 32
    x, w1 = normal(R, H, seed=1).requires_grad_(), normal(4, 2 * F, H, seed=2).requires_grad_()
    w2, g = normal(4, H, F, seed=3).requires_grad_(), normal(R, H, seed=4)
    for falling in (True, False):
        offsets = torch.tensor([0, 30, 20 if falling else 40, 90, 100], dtype=torch.int32, device=DEV)
        status = status_word()
        y = ag.expert_mlp(x, offsets, w1, w2, status=status)
        expected = {"bad_offsets"} if falling else set()
        assert mp.status_bits(int(status)) == expected
        status.zero_()
        torch.autograd.grad(y, [x, w1, w2], g)
        assert mp.status_bits(int(status)) == expected


def test_no_rows_through_autograd():
    """No rows at all: empty results, zero gradients of the weights."""
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV, requires_grad=True)
    w1, w2 = normal(3, 64, 64, seed=1).requires_grad_(), normal(3, 64, 32, seed=2).requires_grad_()
    b1, b2 = normal(3, 64, seed=3).requires_grad_(), normal(3, 64, seed=4).requires_grad_()
    for checkpoint in ("e4m3", "bf16"):
        y = ag.expert_mlp(x, offsets_of([0, 0, 0]), w1, w2, b1, b2, checkpoint=checkpoint)
        assert y.shape == (0, 64)
        g_x, *others = torch.autograd.grad(y, [x, w1, w2, b1, b2], torch.empty_like(y))
        assert g_x.shape == (0, 64) and all((g == 0).all() for g in others)


# Two loads of the same experts with the same sum; N, K: few rows whole and split, tiles
# whole and split, the load warps, pairs of CTAs
LOADS = [
    ([5, 9, 2, 0, 16], [0, 3, 20, 8, 1], 264, 512),
    ([1, 0, 1, 2], [2, 2, 0, 0], 136, 2048),
    ([300, 513, 128, 1000], [600, 41, 1200, 100], 640, 192),
    ([70, 30], [1, 99], 264, 4104),
    ([70, 300], [200, 170], 259, 1031),
    ([1500, 700, 1031], [31, 2500, 700], 2048, 768),
]


@pytest.mark.parametrize("one,two,N,K", LOADS)
def test_a_row_does_not_depend_on_its_place(one, two, N, K):
    """In calls of the same sizes a row of an expert has the same bits wherever it stands
    and whatever the loads are."""
    E, R = len(one), sum(one)
    assert sum(two) == R
    pool = [normal(max(a, b, 1), K, seed=10 + e) for e, (a, b) in enumerate(zip(one, two))]
    pool_g = [normal(max(a, b, 1), N, seed=50 + e) for e, (a, b) in enumerate(zip(one, two))]
    w = normal(E, N, K, seed=2, std=K ** -0.5)
    got = []
    for counts in (one, two):
        x, g = (torch.cat([p[e][:n] for e, n in enumerate(counts)]) for p in (pool, pool_g))
        offsets = offsets_of(counts)
        got.append((offsets.tolist(), mp.mp_expert_gemm(x, w, offsets, act="silu")[0],
                    mp.mp_expert_dgrad(g, w, offsets)[0]))
    (at1, *first), (at2, *second) = got
    for a, b in zip(first, second):
        for e in range(E):
            n = min(one[e], two[e])
            assert torch.equal(a[at1[e]:at1[e] + n], b[at2[e]:at2[e] + n])
