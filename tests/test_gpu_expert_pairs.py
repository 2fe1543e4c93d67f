"""Products and gradients large enough for pairs of CTAs: at least 384 rows an expert (512
in weight gradients), contractions of 768 (row gradients 640), and as many tiles as SMs.
The checks and bounds are those of the small ones."""
from __future__ import annotations

import pytest
import torch

from tests import test_gpu_expert as small
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

MORE = {"mixed": [640, 601, 1024, 577, 3], "equal": [768, 768, 768, 768]}


@pytest.fixture(autouse=True)
def counts(monkeypatch):
    for name, n in MORE.items():
        monkeypatch.setitem(small.COUNTS, name, n)


def in_pairs(name, tile_rows, cols, rows, depth, least_depth):
    n = MORE.get(name) or small.COUNTS[name]
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    return sum(n) >= rows * len(n) and depth >= least_depth and \
        -(-cols // 256) * (tile_rows or sum(n) // 128) >= sms


# as small.PRODUCTS
PRODUCTS = [
    ("long", 2048, 768, "none", False, False, 0),
    ("long", 2 * 1012, 776, "swiglu", True, True, 0),
    ("long", 2050, 1000, "gelu", True, False, 0),
    ("long, one empty", 2 * 640, 768, "geglu", False, True, 0),
    ("mixed", 2088, 1032, "relu", True, True, 8),
    ("equal", 2 * 1032, 1088, "swiglu", False, False, 0),
]


@pytest.mark.parametrize("save", ["none", "bf16", "e4m3"])
@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: "%s-N%d-K%d-%s" % c[:4])
def test_product(case, save):
    assert in_pairs(case[0], 0, case[1], 384, case[2], 768)
    small.test_product(case, save)


# as small.DGRADS
DGRADS = [
    ("long", 648, 2048, "none", None),
    ("long", 776, 2056, "swiglu", "e4m3"),
    ("long, one empty", 640, 1304, "geglu", "bf16"),
    ("mixed", 1000, 2000, "gelu", "e4m3"),
    ("equal", 1088, 2040, "silu", "bf16"),
]


@pytest.mark.parametrize("case", DGRADS, ids=lambda c: "%s-N%d-K%d-%s-%s" % c)
def test_row_gradient(case):
    assert in_pairs(case[0], 0, case[2], 384, case[1], 640)
    small.test_row_gradient(case)


# as small.WGRADS
WGRADS = [
    ("long", 1032, 1800, True), ("long, one empty", 1024, 1800, False), ("mixed", 648, 1544, True),
    ("equal", 768, 1792, True), ("deep", 1544, 3400, True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", WGRADS, ids=lambda c: "%s-N%d-K%d-%d" % c)
def test_weight_gradient(case, dtype):
    name, N, K, _ = case
    E = len(MORE.get(name) or small.COUNTS[name])
    assert in_pairs(name, E * -(-N // 128), K, 512, 1, 0)
    small.test_weight_gradient(case, dtype)
