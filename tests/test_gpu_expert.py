"""The experts' products, their gradients and the 8-bit checkpoint against plain
64-bit implementations.

Bounds.  A product of K terms summed in fp32, in any order and with truncating
adds, is off by at most K 2^-23 sum|x w| (Z below); adding the bias 2^-24 more
of the result.  An activation with slopes up to 1.13 passes that on; fast exp
and division add 2^-18 of the magnitude.  The result is rounded once to bf16:
half a step, 2^-8 of it.  The checkpoint's codes are off by half a step of e4m3,
2^-4 of the value or 2^-10 of the unit.  Gradients are tested on given
checkpoints, whose values are exact."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import unpermute_routing_indices_gb300 as mp
from unpermute_routing_indices_gb300 import autograd as ag
from tests.gpu_util import DEV, status_word

pytestmark = pytest.mark.gpu

BF16 = torch.finfo(torch.bfloat16).eps / 2
GATED = ("geglu", "swiglu")
SLOPE = 1.13


def normal(*shape, seed, std=1.0, shift=0):
    """bf16 values; with `shift`, from the middle of a buffer, so that the first
    element lies `shift` elements past a 256-byte boundary."""
    g = torch.Generator().manual_seed(seed)
    t = (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).to(DEV)
    if not shift:
        return t
    room = torch.zeros(t.numel() + shift, dtype=t.dtype, device=DEV)
    room[shift:] = t.flatten()
    return room[shift:].view(t.shape)


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)


def act64(z, act):
    """(act(z), slope of the inner function) and the parts, in 64 bits."""
    if act in GATED:
        a, b = z.chunk(2, 1)
        f, d = act64(a, "silu" if act == "swiglu" else "gelu")
        return f * b, (f, d, b)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * (1 - q)
    if act == "gelu":
        # (1 + tanh u) / 2 is sigmoid(2u), which keeps its digits where tanh is near -1.
        c = 2 * (2 / np.pi) ** 0.5
        q = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return z * q, q + z * q * (1 - q) * c * (1 + 0.134145 * z ** 2)
    return z, torch.ones_like(z)


def rows64(x, w, offsets, turned=False):
    """(x w[e]^T or x w[e], the same of magnitudes), in 64 bits."""
    edges = offsets.tolist()
    n = w.shape[2] if turned else w.shape[1]
    out, size = (torch.zeros(x.shape[0], n, dtype=torch.float64, device=DEV) for _ in range(2))
    for e, (a, b) in enumerate(zip(edges, edges[1:])):
        m = w[e].double() if turned else w[e].double().T
        out[a:b], size[a:b] = x[a:b].double() @ m, x[a:b].double().abs() @ m.abs()
    return out, size


def expert_of_row(offsets, R):
    return torch.searchsorted(offsets[1:].contiguous(), torch.arange(R, device=DEV, dtype=torch.int32),
                              right=True)


def decode(z, z_exp, parts):
    """The values of a checkpoint, and the unit of each."""
    v, x = z.float(), z_exp.float() - 127
    F = v.shape[1] // parts
    unit = torch.exp2(x).view(-1, parts, z_exp.shape[1] // parts).repeat_interleave(32, 2)[..., :F]
    unit = unit.reshape(v.shape).double()
    return v.double() * unit, unit


COUNTS = {
    "one row": [1],
    "one expert": [70],
    "many": [3, 0, 64, 1, 0, 129, 65, 0],
    "first empty": [0, 0, 257, 31],
    "tokens": [0, 1, 0, 1, 1, 0, 0, 1],
    "few each": [5, 9, 2, 8, 3, 16, 17, 1],
    "big": [300, 513, 128, 1000],
    "long": [1500, 700, 1031],       # enough rows an expert for pairs of CTAs, all three ragged
    "long, one empty": [2111, 0, 1985],
    "single long": [5001],           # few tiles: split contractions, ragged at the end
    "two, short and long": [3, 2500],
    "deep": [13001],                 # contractions over rows in 8 parts
    "deep, one short": [9000, 3, 0],
}

# counts, N (columns of w), K, activation, bias, residual, shift of x
PRODUCTS = [
    ("one row", 8, 8, "none", False, False, 0),
    ("one row", 1, 1, "none", True, True, 0),
    ("many", 64, 64, "none", False, False, 0),
    ("many", 96, 136, "gelu", True, False, 0),
    ("many", 2 * 40, 72, "swiglu", True, True, 0),
    ("many", 2 * 33, 37, "geglu", True, False, 0),
    ("many", 101, 200, "relu", False, True, 0),
    ("first empty", 257, 520, "silu", True, True, 0),
    ("first empty", 2 * 200, 264, "swiglu", False, False, 0),
    ("tokens", 2 * 264, 1032, "swiglu", True, True, 0),
    ("tokens", 130, 512, "none", False, True, 0),
    ("few each", 384, 256, "gelu", False, False, 0),
    ("few each", 2 * 136, 640, "geglu", True, False, 0),
    ("one expert", 512, 2048, "silu", False, False, 0),
    ("big", 2 * 256, 576, "swiglu", True, False, 0),
    ("big", 640, 192, "none", True, True, 0),
    ("many", 64, 64, "gelu", True, False, 1),      # 2-byte aligned rows
    ("many", 128, 128, "silu", True, True, 8),     # 16-byte, not 32-byte aligned
    ("long", 2 * 136, 200, "swiglu", True, True, 0),
    ("long", 264, 320, "gelu", False, True, 0),
    ("long, one empty", 2 * 256, 128, "geglu", False, False, 0),
    ("two, short and long", 2 * 72, 1032, "swiglu", True, True, 0),
    ("single long", 40, 4096, "gelu", True, False, 0),
    # Few tiles and a long contraction, in 2, 4 and 8 parts
    ("many", 264, 1672, "relu", True, True, 0),
    ("first empty", 2 * 136, 4104, "swiglu", True, True, 0),
    ("first empty", 520, 3400, "gelu", False, True, 0),
    ("one expert", 2 * 72, 8200, "geglu", True, False, 0),
    ("one expert", 328, 6344, "none", True, True, 8),
    # Widths and bases that are no multiples of 16 bytes, whole and in parts
    ("big", 2 * 129, 1031, "swiglu", True, True, 0),
    ("big", 514, 130, "none", True, True, 1),
    ("first empty", 261, 2050, "gelu", True, False, 0),
    ("one expert", 2 * 70, 6001, "geglu", False, True, 0),
    ("one expert", 200, 4096, "silu", True, False, 3),
]


@pytest.mark.parametrize("save", ["none", "bf16", "e4m3"])
@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: "%s-N%d-K%d-%s-s%d" % (c[:4] + c[6:]))
def test_product(case, save):
    name, N, K, act, with_bias, with_residual, shift = case
    counts = COUNTS[name]
    E, R = len(counts), sum(counts)
    offsets = offsets_of(counts)
    parts = 2 if act in GATED else 1
    F = N // parts
    x, w = normal(R, K, seed=1, shift=shift), normal(E, N, K, seed=2, std=K ** -0.5, shift=shift)
    bias = normal(E, N, seed=3, std=0.3) if with_bias else None
    residual = normal(R, F, seed=4, shift=shift) if with_residual else None
    out, z, z_exp = mp.mp_expert_gemm(x, w, offsets, bias=bias, act=act, residual=residual, save=save)
    z64, size = rows64(x, w, offsets)
    if with_bias:
        b = bias[expert_of_row(offsets, R)].double()
        z64, size = z64 + b, size + b.abs()
    Z = (K + 2) * 2.0 ** -23 * size
    y, parted = act64(z64, act)
    if act in GATED:
        f, _, u = parted
        off = SLOPE * Z[:, :F] * (u.abs() + Z[:, F:]) + f.abs() * Z[:, F:]
    else:
        off = SLOPE * Z
    off = off + 2.0 ** -18 * y.abs()
    if with_residual:
        r = residual.double()
        off, y = off + 2.0 ** -24 * (y.abs() + r.abs()), y + r
    assert ((out.double() - y).abs() <= off * (1 + BF16) + BF16 * y.abs() + 1e-38).all()
    if save == "none":
        assert z is None and z_exp is None
    elif save == "bf16":
        assert z_exp is None
        assert ((z.double() - z64).abs() <= Z * (1 + BF16) + BF16 * z64.abs()).all()
    else:
        v, unit = decode(z, z_exp, parts)
        near = Z + torch.maximum(2.0 ** -4 * (z64.abs() + Z), 2.0 ** -10 * unit)
        assert ((v - z64).abs() <= near).all()
        # The unit is the smallest that brings the block's largest to 448.
        pad = torch.nn.functional.pad
        blocks = -(-F // 32)
        big = pad(z64.abs().view(R, parts, F), (0, blocks * 32 - F)).view(R, -1, 32).amax(2)
        slack = pad(Z.view(R, parts, F), (0, blocks * 32 - F)).view(R, -1, 32).amax(2)
        u = torch.exp2(z_exp.double() - 127)
        assert (big - slack <= 448 * u).all()
        assert ((big + slack > 224 * u) | (z_exp == 1)).all()


# counts, N, K, activation, checkpoint
DGRADS = [
    ("one row", 8, 8, "none", None),
    ("one row", 1, 1, "silu", "bf16"),
    ("many", 64, 64, "none", None),
    ("many", 136, 96, "gelu", "e4m3"),
    ("many", 200, 40, "swiglu", "e4m3"),
    ("many", 37, 33, "geglu", "e4m3"),
    ("first empty", 520, 257, "relu", "bf16"),
    ("first empty", 264, 200, "swiglu", "bf16"),
    ("tokens", 1032, 264, "swiglu", "e4m3"),
    ("few each", 256, 384, "silu", "e4m3"),
    ("big", 576, 256, "geglu", "e4m3"),
    ("big", 192, 640, "none", None),
    ("big", 256, 328, "swiglu", "bf16"),
    ("long", 192, 264, "swiglu", "e4m3"),
    ("long, one empty", 320, 136, "none", None),
    ("two, short and long", 1544, 72, "geglu", "e4m3"),
    ("many", 1672, 264, "gelu", "e4m3"),
    ("first empty", 4104, 136, "swiglu", "bf16"),
    ("one expert", 8200, 72, "geglu", "e4m3"),
    ("one expert", 6344, 328, "none", None),
    ("big", 515, 203, "swiglu", "bf16"),
    ("many", 1034, 131, "gelu", "e4m3"),
    ("one expert", 4099, 130, "geglu", "e4m3"),
]


def checkpoint_of(R, F, act, save, seed):
    """A checkpoint of normal values as mp_expert_gemm writes one: (z, z_exp, values)."""
    parts = 2 if act in GATED else 1
    x = normal(R, 64, seed=seed)
    w = normal(1, parts * F, 64, seed=seed + 1, std=0.2)
    _, z, z_exp = mp.mp_expert_gemm(x, w, offsets_of([R]), act=act, save=save)
    return z, z_exp, z.double() if save == "bf16" else decode(z, z_exp, parts)[0]


@pytest.mark.parametrize("case", DGRADS, ids=lambda c: "%s-N%d-K%d-%s-%s" % c)
def test_row_gradient(case):
    name, N, K, act, save = case
    counts = COUNTS[name]
    E, R = len(counts), sum(counts)
    offsets = offsets_of(counts)
    g, w = normal(R, N, seed=5), normal(E, N, K, seed=6, std=N ** -0.5)
    t, size = rows64(g, w, offsets, turned=True)
    Z = (N + 2) * 2.0 ** -23 * size
    if act == "none":
        got, h = mp.mp_expert_dgrad(g, w, offsets)
        assert h is None
        want, off = t, Z
    else:
        z, z_exp, v = checkpoint_of(R, K, act, save, 7)
        got, h = mp.mp_expert_dgrad(g, w, offsets, act=act, z=z, z_exp=z_exp, with_h=True)
        alone, none = mp.mp_expert_dgrad(g, w, offsets, act=act, z=z, z_exp=z_exp)
        assert none is None and torch.equal(alone, got)
        y, parted = act64(v, act)
        fast = 2.0 ** -17
        if act in GATED:
            f, d, u = parted
            want = torch.cat([t * u * d, t * f], 1)
            # act and its slope: 2^-17 of the terms they are made of (at most 1.2 for
            # the slope's, by |z| s (1-s) u' <= 0.6)
            off = torch.cat([Z * u.abs() * SLOPE + fast * 1.2 * (t.abs() + Z) * u.abs(),
                             Z * f.abs() + fast * (t.abs() + Z) * f.abs()], 1)
        else:
            want, off = t * parted, Z * SLOPE + fast * 1.2 * (t.abs() + Z)
        assert ((h.double() - y).abs() <= (BF16 + 2.0 ** -17) * y.abs() + 1e-38).all()
    assert ((got.double() - want).abs() <= off * (1 + BF16) + BF16 * want.abs() + 1e-38).all()


# counts, N, K, bias
WGRADS = [
    ("one row", 8, 8, True), ("one row", 1, 1, True), ("many", 64, 64, False),
    ("many", 136, 72, True), ("many", 33, 37, True), ("first empty", 264, 520, True),
    ("first empty", 257, 128, False), ("tokens", 128, 264, True), ("few each", 256, 384, True),
    ("big", 192, 576, True), ("big", 520, 264, False), ("one expert", 384, 512, True),
    ("long", 264, 520, True), ("long, one empty", 136, 264, False), ("long", 512, 256, False),
    ("single long", 136, 264, True), ("single long", 24, 1000, True), ("two, short and long", 264, 72, True),
    ("deep", 136, 264, True), ("deep", 8, 1000, True), ("deep, one short", 264, 72, True),
    ("deep, one short", 136, 520, False),
    ("big", 203, 515, True), ("deep", 33, 130, True), ("deep, one short", 130, 259, True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", WGRADS, ids=lambda c: "%s-N%d-K%d-%d" % c)
def test_weight_gradient(case, dtype):
    name, N, K, with_bias = case
    counts = COUNTS[name]
    E, R = len(counts), sum(counts)
    offsets = offsets_of(counts)
    g, x = normal(R, N, seed=8), normal(R, K, seed=9)
    # What lies past the experts' rows is not read, whatever it holds.
    spare = torch.full((3, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    gs, xs = torch.cat([g, spare]), torch.cat([x, spare[:, :1].expand(3, K)])
    g_w, g_b = mp.mp_expert_wgrad(gs, xs, offsets, with_bias=with_bias, dtype=dtype)
    half = BF16 if dtype == torch.bfloat16 else 2.0 ** -24
    base = {}
    for e, n in enumerate(counts):
        a = int(offsets[e])
        ge, xe = g[a:a + n].double(), x[a:a + n].double()
        off = (n + 2) * 2.0 ** -23 * (ge.abs().T @ xe.abs())
        want = base[e] = ge.T @ xe
        assert ((g_w[e].double() - want).abs() <= off + half * want.abs()).all()
        if with_bias:
            off, want = (n + 2) * 2.0 ** -24 * ge.abs().sum(0), ge.sum(0)
            assert ((g_b[e].double() - want).abs() <= off + half * want.abs()).all()
        if n == 0:
            assert (g_w[e] == 0).all()
    if dtype == torch.float32:
        old = torch.randn(E, N, K, device=DEV)
        acc, old_b = old.clone(), torch.randn(E, N, device=DEV)
        acc_b = old_b.clone()
        mp.mp_expert_wgrad(g, x, offsets, with_bias=with_bias, accumulate=True, g_w=acc,
                           g_bias=acc_b if with_bias else None)
        assert torch.equal(acc, old + g_w)
        if with_bias:
            assert torch.equal(acc_b, old_b + g_b)


@pytest.mark.parametrize("N,K", [(136, 72), (64, 264), (33, 37)])
def test_rows_past_the_last_expert_stay(N, K):
    counts, more = [5, 0, 40], 9
    R = sum(counts) + more
    offsets = offsets_of(counts)
    x, w = normal(R, K, seed=1), normal(3, N, K, seed=2)
    x[sum(counts):] = float("nan")
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV)
    mp.mp_expert_gemm(x, w, offsets, out=out)
    want, _, _ = mp.mp_expert_gemm(x[:sum(counts)].contiguous(), w, offsets)
    assert (out[sum(counts):] == 7.0).all() and torch.equal(out[:sum(counts)], want)
    g = normal(R, N, seed=3)
    g[sum(counts):] = float("inf")
    g_x = torch.full((R, K), 7.0, dtype=torch.bfloat16, device=DEV)
    mp.mp_expert_dgrad(g, w, offsets, g_x=g_x)
    assert (g_x[sum(counts):] == 7.0).all() and torch.isfinite(g_x.float()).all()


@pytest.mark.parametrize("counts", [[5, 0, 40], [0, 0, 0], [300, 700, 900], [2500]])
@pytest.mark.parametrize("H,F", [(136, 72), (33, 40), (264, 37)])
def test_mlp_zeroes_what_is_past_the_last_expert(counts, H, F):
    E, more = len(counts), 13
    R, offsets = sum(counts) + more, offsets_of(counts)
    x, g = normal(R, H, seed=1), normal(R, H, seed=2)
    w1, w2 = normal(E, F, H, seed=3, std=0.1), normal(E, H, F, seed=4, std=0.1)
    junk = torch.full((R, 1000), float("nan"), dtype=torch.bfloat16, device=DEV)
    del junk                                     # new buffers are likely to hold it
    y, z, z_exp = mp.mp_expert_mlp(x, w1, w2, offsets, act="silu", save="e4m3")
    g_x = mp.mp_expert_mlp_bwd(g, x, w1, w2, offsets, z, z_exp, act="silu")[0]
    n = sum(counts)
    assert (y[n:] == 0).all() and (g_x[n:] == 0).all()
    assert torch.isfinite(y.float()).all() and torch.isfinite(g_x.float()).all()


@pytest.mark.parametrize("N,K", [(64, 64), (264, 520), (33, 37)])
def test_a_row_does_not_see_its_neighbours(N, K):
    """NaN and infinity stay in the row they are in, and the weight gradient of
    an expert does not see the rows of the others."""
    counts = [20, 45, 3, 130]
    R, offsets = sum(counts), offsets_of(counts)
    x, w = normal(R, K, seed=1), normal(4, N, K, seed=2)
    clean, _, _ = mp.mp_expert_gemm(x, w, offsets, act="silu")
    bad = x.clone()
    rows = torch.tensor([19, 20, 64, 65, 197], device=DEV)
    bad[rows[::2]] = float("nan")
    bad[rows[1::2], 1] = float("inf")
    out, z, z_exp = mp.mp_expert_gemm(bad, w, offsets, act="silu", save="e4m3")
    good = torch.ones(R, dtype=torch.bool, device=DEV)
    good[rows] = False
    assert torch.equal(out[good], clean[good])
    assert not torch.isfinite(out[rows].float()).any(1).all() or N == 0
    assert torch.isnan(z.float()[rows]).all() and torch.isfinite(z.float()[good]).all()
    g = normal(R, N, seed=3)
    ref, _ = mp.mp_expert_wgrad(g, x, offsets)
    x2 = x.clone()
    x2[offsets[1]:offsets[2]] = float("nan")
    g2 = g.clone()
    g2[offsets[1]:offsets[2]] = float("inf")
    got, _ = mp.mp_expert_wgrad(g2, x2, offsets)
    for e in (0, 2, 3):
        assert torch.equal(got[e], ref[e])


@pytest.mark.parametrize("N,K", [(64, 64), (33, 37)])
def test_offsets_that_fall_or_leave_the_rows(N, K):
    """They are clamped, flagged, and lead nowhere else."""
    R = 100
    x, w, g = normal(R, K, seed=1), normal(4, N, K, seed=2), normal(R, N, seed=3)
    given = torch.tensor([-5, 30, 20, 90, 5000], dtype=torch.int32, device=DEV)
    clamped = torch.tensor([0, 30, 30, 90, 100], dtype=torch.int32, device=DEV)
    for call in (lambda o, s: mp.mp_expert_gemm(x, w, o, status=s)[0],
                 lambda o, s: mp.mp_expert_dgrad(g, w, o, status=s)[0],
                 lambda o, s: mp.mp_expert_wgrad(g, x, o, status=s)[0]):
        bad, fine = status_word(), status_word()
        assert torch.equal(call(given, bad), call(clamped, fine))
        assert mp.status_bits(int(bad)) == {"bad_offsets"} and int(fine) == 0


def test_no_rows():
    w = normal(3, 64, 64, seed=1)
    empty = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    offsets = offsets_of([0, 0, 0])
    assert mp.mp_expert_gemm(empty, w, offsets)[0].shape == (0, 64)
    assert mp.mp_expert_dgrad(empty, w, offsets)[0].shape == (0, 64)
    g_w, g_b = mp.mp_expert_wgrad(empty, empty, offsets, with_bias=True)
    assert (g_w == 0).all() and (g_b == 0).all()
    x = normal(10, 64, seed=2)           # rows, but no expert has any
    out = torch.full((10, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    mp.mp_expert_gemm(x, w, offsets, out=out)
    assert (out == 3.0).all()
    g_w, g_b = mp.mp_expert_wgrad(x, x, offsets, with_bias=True)
    assert (g_w == 0).all() and (g_b == 0).all()


def test_checkpoint_of_special_values():
    """Zero rows, the smallest and largest values, and what is not finite."""
    R, N = 6, 64
    x = torch.zeros((R, 8), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((1, N, 8), dtype=torch.bfloat16, device=DEV)
    w[0, :, 0] = 1
    x[1, 0], x[2, 0], x[3, 0], x[4, 0], x[5, 0] = 1e-38, 3e38, float("inf"), float("nan"), -449.0
    out, z, z_exp = mp.mp_expert_gemm(x, w, offsets_of([R]), act="relu", save="e4m3")
    v, _ = decode(z, z_exp, 1)
    assert (v[0] == 0).all() and (out[0] == 0).all()
    assert ((v[1] - x[1, 0].double()).abs() <= 2.0 ** -4 * x[1, 0].double() + 2.0 ** -136).all()
    assert ((v[2] - x[2, 0].double()).abs() <= 2.0 ** -4 * x[2, 0].double()).all()
    assert torch.isnan(v[3]).all() and torch.isnan(v[4]).all()
    assert (v[5] == -448.0).all()
    g, w2 = normal(R, 16, seed=1), normal(1, 16, N, seed=2)
    g_z, h = mp.mp_expert_dgrad(g, w2, offsets_of([R]), act="silu", z=z, z_exp=z_exp, with_h=True)
    assert torch.isnan(g_z[3:5].float()).all() and torch.isfinite(g_z[:3].float()).all()
    assert torch.isfinite(g_z[5].float()).all() and (h[5] == 0).all() and (h[0] == 0).all()


@pytest.mark.parametrize("checkpoint", ["bf16", "e4m3"])
@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_expert_mlp_is_its_calls(act, checkpoint):
    counts, H, F, more = [30, 0, 200, 7], 136, 72, 5
    two = 2 if act in GATED else 1
    R, offsets = sum(counts) + more, offsets_of(counts)
    x, g = normal(R, H, seed=1).requires_grad_(), normal(R, H, seed=2)
    w1 = normal(4, two * F, H, seed=3, std=0.1).requires_grad_()
    w2 = normal(4, H, F, seed=4, std=0.1).requires_grad_()
    b1 = normal(4, two * F, seed=5).requires_grad_()
    b2 = normal(4, H, seed=6).requires_grad_()
    y = ag.expert_mlp(x, offsets, w1, w2, b1, b2, act=act, checkpoint=checkpoint)
    got = torch.autograd.grad(y, [x, w1, w2, b1, b2], g)
    with torch.no_grad():
        h, z, z_exp = mp.mp_expert_gemm(x, w1, offsets, bias=b1, act=act, save=checkpoint)
        want = mp.mp_expert_gemm(h, w2, offsets, bias=b2)[0]
        g_z, h = mp.mp_expert_dgrad(g, w2, offsets, act=act, z=z, z_exp=z_exp, with_h=True)
        g_x = mp.mp_expert_dgrad(g_z, w1, offsets)[0]
        g_w2, g_b2 = mp.mp_expert_wgrad(g, h, offsets, with_bias=True)
        g_w1, g_b1 = mp.mp_expert_wgrad(g_z, x, offsets, with_bias=True)
    n = sum(counts)
    assert torch.equal(y[:n], want[:n]) and (y[n:] == 0).all()
    assert torch.equal(got[0][:n], g_x[:n]) and (got[0][n:] == 0).all()
    for a, b in zip(got[1:], (g_w1, g_w2, g_b1, g_b2)):
        assert torch.equal(a, b)
    # Only what is asked for.
    y = ag.expert_mlp(x.detach(), offsets, w1.detach(), w2, act=act, checkpoint=checkpoint)
    y.backward(g)
    assert w2.grad is not None
    with torch.no_grad():
        assert not ag.expert_mlp(x, offsets, w1, w2, act=act).requires_grad


@pytest.mark.parametrize("act", ["swiglu", "geglu", "silu", "gelu"])
def test_expert_mlp_gradient_against_differences(act):
    """Along a direction d the 64-bit loss changes by <gradient, d>.  The kept
    product is bf16 (off by 2^-8), h and g_z are rounded to bf16 once, the
    gradient too: 4 roundings of 2^-8 of the magnitudes the gradient is made of,
    which the 64-bit gradient of magnitudes bounds."""
    counts, H, F = [9, 0, 14], 24, 16
    two = 2 if act in GATED else 1
    R, offsets = sum(counts), offsets_of(counts)
    x, g = normal(R, H, seed=1).requires_grad_(), normal(R, H, seed=2)
    w1 = normal(3, two * F, H, seed=3, std=0.2).requires_grad_()
    w2 = normal(3, H, F, seed=4, std=0.3).requires_grad_()
    y = ag.expert_mlp(x, offsets, w1, w2, act=act, checkpoint="bf16")
    grads = torch.autograd.grad(y, [x, w1, w2], g)

    def loss(x, w1, w2):
        z, _ = rows64(x, w1, offsets)
        return (rows64(act64(z, act)[0], w2, offsets)[0] * g.double()).sum()
    at = [t.detach().double() for t in (x, w1, w2)]
    # Magnitudes: |g||w2| through slopes of at most 1.13 and factors of |u|, |f|.
    z, zs = rows64(*at[:2], offsets)
    t = rows64(g.double().abs(), at[2].abs(), offsets, turned=True)[0]
    if act in GATED:
        f, u = z[:, :F].abs(), z[:, F:].abs()
        gz = torch.cat([t * u * SLOPE + t * 0.6 * u, t * f + t * SLOPE * f], 1)
        h = f * u
    else:
        gz, h = t * SLOPE + t * z.abs(), z.abs()
    sizes = [rows64(gz, at[1].abs(), offsets, turned=True)[0], torch.zeros_like(at[1]),
             torch.zeros_like(at[2])]
    edges = offsets.tolist()
    for e, (a, b) in enumerate(zip(edges, edges[1:])):
        sizes[1][e] = gz[a:b].T @ at[0][a:b].abs()
        sizes[2][e] = g[a:b].double().abs().T @ h[a:b]
    step = 1e-5
    gen = torch.Generator().manual_seed(9)
    for k in range(3):
        d = torch.randn(at[k].shape, generator=gen, dtype=torch.float64).to(DEV)
        up, down = list(at), list(at)
        up[k], down[k] = at[k] + step * d, at[k] - step * d
        difference = (loss(*up) - loss(*down)) / (2 * step)
        bound = 4 * 2.0 ** -8 * (sizes[k] * d.abs()).sum()
        assert (difference - (grads[k].double() * d).sum()).abs() <= bound
        # The bound above adds all errors up; they are independent, so the
        # root of their squares (6 of them) is what they come to.
        assert (difference - (grads[k].double() * d).sum()).abs() <= \
            6 * 4 * 2.0 ** -8 * (sizes[k] * d).square().sum().sqrt()


@pytest.mark.parametrize("counts", ["few each", "many", "long"])
def test_captured_and_replayed(counts):
    """The calls in a CUDA graph, replayed with other rows and other offsets in the
    same buffers, give what eager calls give."""
    counts = COUNTS[counts]
    E, R, H, F = len(counts), sum(counts), 136, 72
    first, second = offsets_of(counts), offsets_of(counts[::-1])
    x, g = normal(R, H, seed=1), normal(R, H, seed=2)
    w1, w2 = normal(E, 2 * F, H, seed=3, std=0.1), normal(E, H, F, seed=4, std=0.1)
    b1, l = normal(E, 2 * F, seed=5), torch.randn(R, E, device=DEV)
    offsets = first.clone()

    def calls():
        idx, weights = mp.mp_route(l, 1, score="sigmoid")
        y, z, z_exp = mp.mp_expert_mlp(x, w1, w2, offsets, b1, save="e4m3")
        grads = mp.mp_expert_mlp_bwd(g, x, w1, w2, offsets, z, z_exp, need=(True,) * 5)
        return [idx, weights, mp.mp_route_bwd(weights, l, idx, score="sigmoid"), y, *grads]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    for o, seed in ((second, 11), (first, 12)):
        offsets.copy_(o)
        x.copy_(normal(R, H, seed=seed))
        l.copy_(torch.randn(R, E, device=DEV))
        graph.replay()
        got = [t.clone() for t in outs]
        for a, b in zip(got, calls()):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """Calls on two streams, started together again and again, give what they give
    alone (the persistent kernels share SMs and tensor memory)."""
    counts = COUNTS["long"]
    R, offsets = sum(counts), offsets_of(counts)
    small = offsets_of(COUNTS["few each"])
    x, w, g = normal(R, 256, seed=1), normal(3, 512, 256, seed=2), normal(R, 512, seed=3)
    xs, ws = normal(sum(COUNTS["few each"]), 512, seed=4), normal(8, 384, 512, seed=5)
    want = [mp.mp_expert_gemm(x, w, offsets)[0], mp.mp_expert_wgrad(g, x, offsets)[0],
            mp.mp_expert_gemm(xs, ws, small, act="silu")[0], mp.mp_expert_dgrad(g, w, offsets)[0]]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(30):
        with torch.cuda.stream(streams[0]):
            got.append((0, mp.mp_expert_gemm(x, w, offsets)[0]))
            got.append((2, mp.mp_expert_gemm(xs, ws, small, act="silu")[0]))
        with torch.cuda.stream(streams[1]):
            got.append((1, mp.mp_expert_wgrad(g, x, offsets)[0]))
            got.append((2, mp.mp_expert_gemm(xs, ws, small, act="silu")[0]))
            got.append((3, mp.mp_expert_dgrad(g, w, offsets)[0]))
    torch.cuda.synchronize()
    for k, t in got:
        assert torch.equal(t, want[k])


def test_repeated_calls_are_equal():
    counts = COUNTS["big"]
    R, offsets = sum(counts), offsets_of(counts)
    x, w, g = normal(R, 576, seed=1), normal(4, 512, 576, seed=2), normal(R, 512, seed=3)
    once = [mp.mp_expert_gemm(x, w, offsets, act="swiglu")[0], mp.mp_expert_dgrad(g, w, offsets)[0],
            *mp.mp_expert_wgrad(g, x, offsets, with_bias=True)]
    for _ in range(5):
        again = [mp.mp_expert_gemm(x, w, offsets, act="swiglu")[0],
                 mp.mp_expert_dgrad(g, w, offsets)[0],
                 *mp.mp_expert_wgrad(g, x, offsets, with_bias=True)]
        for a, b in zip(once, again):
            assert torch.equal(a, b)


def test_buffers_past_two_thirty_one_elements():
    """Rows whose offsets need 64 bits: the last ones come out right."""
    R, K, N = 540_000, 4096, 64
    offsets = torch.tensor([0, 1000, R], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.empty((R, K), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    w = normal(2, N, K, seed=2, std=K ** -0.5)
    tail = slice(R - 700, R)
    out, _, _ = mp.mp_expert_gemm(x, w, offsets)
    want, size = x[tail].double() @ w[1].double().T, x[tail].double().abs() @ w[1].double().abs().T
    bound = (K + 2) * 2.0 ** -23 * size * (1 + BF16) + BF16 * want.abs()
    assert ((out[tail].double() - want).abs() <= bound).all()
    # The gradient of the weights of an expert whose rows all lie past 2^31 elements.
    offsets = torch.tensor([0, R - 700, R], dtype=torch.int32, device=DEV)
    gy = normal(R, N, seed=3)
    g_w, g_b = mp.mp_expert_wgrad(gy, x, offsets, with_bias=True)
    want = gy[tail].double().T @ x[tail].double()
    size = gy[tail].double().abs().T @ x[tail].double().abs()
    assert ((g_w[1].double() - want).abs() <= 702 * 2.0 ** -23 * size + BF16 * want.abs()).all()
    want, size = gy[tail].double().sum(0), gy[tail].double().abs().sum(0)
    assert ((g_b[1].double() - want).abs() <= 702 * 2.0 ** -24 * size + BF16 * want.abs()).all()
    del x
    g_x, _ = mp.mp_expert_dgrad(gy, w, offsets)
    want, size = gy[tail].double() @ w[1].double(), gy[tail].double().abs() @ w[1].double().abs()
    bound = (N + 2) * 2.0 ** -23 * size * (1 + BF16) + BF16 * want.abs()
    assert ((g_x[tail].double() - want).abs() <= bound).all()


def test_refusals():
    x, w = normal(10, 64, seed=1), normal(3, 64, 64, seed=2)
    offsets = offsets_of([3, 3, 4])
    with pytest.raises(ValueError):
        mp.mp_expert_gemm(x, w, offsets[:-1])
    with pytest.raises(TypeError):
        mp.mp_expert_gemm(x, w, offsets.long())
    with pytest.raises(ValueError):
        mp.mp_expert_gemm(x[:, :32], w, offsets)
    with pytest.raises(ValueError):
        mp.mp_expert_gemm(x, w.transpose(1, 2), offsets)
    with pytest.raises(TypeError):
        mp.mp_expert_gemm(x.half(), w, offsets)
    with pytest.raises(ValueError):
        mp.mp_expert_gemm(x, w, offsets, act="tanh")
    with pytest.raises(ValueError):
        mp.mp_expert_gemm(x, w, offsets, save="int8")
    with pytest.raises(ValueError):
        mp.mp_expert_gemm(x, w[:, :63].contiguous(), offsets, act="swiglu")
    with pytest.raises(ValueError):
        mp.mp_expert_gemm(x, w, offsets, z=x)
    with pytest.raises(ValueError):
        mp.mp_expert_dgrad(x, w, offsets, act="silu")
    with pytest.raises(ValueError):
        mp.mp_expert_dgrad(x, w, offsets, h=x)
    with pytest.raises(ValueError):
        mp.mp_expert_dgrad(x, w, offsets, act="swiglu", z=x)
    with pytest.raises(TypeError):
        mp.mp_expert_wgrad(x, x, offsets, dtype=torch.float16)
    with pytest.raises(ValueError):
        mp.mp_expert_wgrad(x, x, offsets, accumulate=True)
