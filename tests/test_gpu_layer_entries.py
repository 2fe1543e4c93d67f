"""mp_moe_layer where experts have more tokens than an entry holds: few experts, whose tokens are taken 16 at a
time, and many, 32 at a time, on both sides of where the one form follows the other."""
from __future__ import annotations

import pytest
import torch

from tests import norm_util as nu
from tests.test_gpu_layer import check, weights_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,K,H,F", [
    (9, 1, 1, 72, 40), (16, 1, 1, 72, 40), (17, 2, 2, 136, 64), (33, 3, 2, 200, 72), (48, 8, 4, 264, 128), (64, 8, 8, 512, 96),
    (64, 16, 8, 256, 64), (63, 31, 12, 136, 72), (64, 31, 31, 136, 40), (24, 32, 16, 128, 64), (25, 32, 16, 128, 64),
    (64, 32, 13, 264, 72), (64, 33, 20, 101, 67), (64, 31, 20, 101, 67), (64, 64, 32, 128, 40)])
def test_more_tokens_than_an_entry(T, E, K, H, F):
    for act, biases in (("swiglu", True), ("relu", False)):
        x = nu.rows(T, H, torch.bfloat16, T + E, mean=0.0)
        check(x, weights_of(E, H, F, H, act, H + F, biases), K, act)
