"""mp_block_norm_bwd over so many rows that each group of threads takes several: sums over the
rows, of every kind and in every layout, against the formulas in 64 bits."""
from __future__ import annotations

import pytest
import torch

import unpermute_routing_indices_gb300 as mp
from tests import norm_util as nu

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def moved(v, off):
    """The same values `off` values into a buffer that starts on 16 bytes."""
    big = torch.empty(v.numel() + off, dtype=v.dtype, device="cuda")
    big[off:] = v.flatten()
    return big[off:].view(v.shape)


def check(T, H, dtype, kind="layer", gate="channel", seed=0, off=0):
    t, how = nu.make(T, H, dtype, kind=kind, post=True, gate=gate, scale=0.7, bias=True, seed=seed)
    if off:
        t = {k: moved(v, off) for k, v in t.items()}
    args = {k: t[k] for k in nu.NAMES[2:]}
    s, y, stats = mp.mp_block_norm(t["x"], t["residual"], with_stats=True, **args, **how)
    nu.check_forward(t, how, s, y, stats)
    g_s, g_y = nu.rows(T, H, dtype, seed + 9, mean=0.0), nu.rows(T, H, dtype, seed + 10, mean=0.1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mp.mp_block_norm_bwd(g_s, g_y, t["x"], s, stats, grad_dtype=torch.float32, status=status, kind=kind,
                               scale=how["scale"], **args)
    nu.check_backward(t, how, g_s, g_y, s, stats, got)
    assert int(status) == 0


@pytest.mark.parametrize("T,H,off", [
    (2500, 245, 0), (2600, 250, 0), (2600, 255, 0), (2600, 256, 0), (2600, 256, 1), (5000, 127, 0), (5000, 128, 0),
    (5000, 128, 3), (10000, 63, 0), (10000, 64, 2), (20000, 32, 0), (20000, 32, 1), (20001, 31, 0), (40000, 13, 0),
    (40000, 16, 1), (152 * 600, 1, 0)])
@pytest.mark.parametrize("gate", ["channel", "element"])
def test_narrow_fp32(T, H, off, gate):
    """Rows of less than a warp's 32 x 16 values, where sums of several groups fill shared memory."""
    check(T, H, torch.float32, gate=gate, seed=T + H, off=off)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["channel", "token", "element"])
@pytest.mark.parametrize("T,H,dtype", [(4099, 4096, "bf16"), (4099, 1009, "fp16"), (40000, 64, "bf16"), (20011, 264, "fp32"),
                                       (3001, 2048, "fp32"), (5003, 4097, "bf16"), (30011, 33, "fp16"), (2203, 8192, "bf16")])
def test_sums_over_many_rows(T, H, dtype, kind, gate):
    """Biases' and a channel gate's sums beside the weights', each group of threads over 2 to 30 rows."""
    check(T, H, DT[dtype], kind, gate, seed=H)


@pytest.mark.parametrize("gate", ["channel", "element"])
@pytest.mark.parametrize("T,H,dtype", [(400, 8200, "bf16"), (403, 8201, "fp16"), (460, 16384, "bf16"), (333, 16385, "fp32"),
                                       (320, 32768, "fp16"), (310, 32767, "bf16"), (412, 7168, "fp32"), (409, 7173, "fp32"),
                                       (460, 5640, "fp32"), (460, 6300, "fp32")])
def test_sums_of_wide_rows(T, H, dtype, gate):
    """Rows too wide to be staged, or just not, 3 or 4 of each CTA."""
    check(T, H, DT[dtype], gate=gate, seed=H)
