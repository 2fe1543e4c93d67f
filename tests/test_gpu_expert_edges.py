"""The experts' calls at edges of their contract: a residual that is the result's own
buffer, a contraction that takes longer than a wait may last without progress."""
from __future__ import annotations

import pytest
import torch

import unpermute_routing_indices_gb300 as mp
from tests.gpu_util import DEV, status_word
from tests.test_gpu_expert import COUNTS, GATED, normal, offsets_of

pytestmark = pytest.mark.gpu


# counts, N, K, activation, elements that the bases are moved by
IN_PLACE = [
    ("big", 640, 192, "none", 0),                  # whole tiles, stored by TMA
    ("long", 512, 320, "silu", 0),
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
