"""Results of the norms and their gradients in the buffers of inputs, as the header allows, bit by bit beside
separate buffers: rows by bulk copies, by vectors, from anywhere, narrow ones, and rows that are not staged."""
from __future__ import annotations

import pytest
import torch

import unpermute_routing_indices_gb300 as mp
from tests import norm_util as nu
from unpermute_routing_indices_gb300 import _lib

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GATES = dict(none=0, channel=1, token=2, element=3)
# more rows than a wave of groups holds, so that rows are copied while earlier ones are written
SHAPES = [(700, 4096, "bf16"), (400, 1024, "fp32"), (3000, 264, "fp16"), (9000, 40, "bf16"), (900, 1009, "bf16"),
          (3000, 101, "fp32"), (310, 8200, "bf16"), (310, 8201, "fp16"), (310, 7176, "fp32")]


def ptr(t):
    return None if t is None else t.data_ptr()


def backward(c, how, gate, stats, out, ws):
    """Through the C entry point; c: the inputs, out: where results go."""
    T, H = c["x"].shape
    code = _lib.load().mp_block_norm_bwd(
        ptr(c["g_s"]), ptr(c["g_y"]), ptr(c["x"]), ptr(c["s"]), ptr(stats), T, H, mp.DTYPES[c["x"].dtype],
        mp.NORMS[how["kind"]], ptr(c["post_weight"]), ptr(c["post_bias"]), ptr(c["gate"]), GATES[gate], how["scale"],
        ptr(c["pre_weight"]), ptr(out["g_x"]), ptr(out["g_residual"]), ptr(out["g_gate"]), ptr(out["post_weight"]),
        ptr(out["post_bias"]), ptr(out["pre_weight"]), ptr(out["pre_bias"]), mp.DTYPES[c["x"].dtype], ptr(ws), ws.numel(),
        None, torch.cuda.current_stream().cuda_stream)
    assert code == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,H,dtype", SHAPES)
@pytest.mark.parametrize("gate", ["channel", "token", "element"])
def test_gradients_in_place(T, H, dtype, gate):
    t, how = nu.make(T, H, DT[dtype], kind="layer", post=True, gate=gate, scale=0.7, bias=True, seed=T)
    t["s"], _, stats = mp.mp_block_norm(t["x"], t["residual"], with_stats=True, **{k: t[k] for k in nu.NAMES[2:]}, **how)
    t["g_s"], t["g_y"] = nu.rows(T, H, DT[dtype], 1, mean=0.0), nu.rows(T, H, DT[dtype], 2, mean=0.1)
    ws = torch.empty(mp.mp_block_norm_bwd_workspace_size(T, H), dtype=torch.uint8, device="cuda")

    def fresh():
        c = {k: None if v is None else v.clone() for k, v in t.items()}
        out = {k: torch.empty_like(t[k]) for k in nu.NAMES[3:]}
        out.update(g_x=torch.empty_like(t["x"]), g_residual=torch.empty_like(t["x"]), g_gate=torch.empty_like(t["gate"]))
        return c, out
    c, want = fresh()
    backward(c, how, gate, stats, want, ws)
    for g_residual, g_x in (("g_s", "x"), ("g_y", "s"), ("s", "g_y"), (None, "g_s"), ("g_s", "gate")):
        if g_x == "gate" and gate != "element":
            continue
        c, out = fresh()
        if g_residual is not None:
            out["g_residual"] = c[g_residual]
        out["g_x"] = c[g_x]
        if g_x != "gate":
            out["g_gate"] = c["gate"]
        backward(c, how, gate, stats, out, ws)
        for k in want:
            assert torch.equal(out[k], want[k]), (g_residual, g_x, k)


@pytest.mark.parametrize("T,H,dtype", SHAPES)
def test_results_in_place(T, H, dtype):
    t, how = nu.make(T, H, DT[dtype], kind="layer", post=True, gate="element", scale=0.7, bias=True, seed=T)
    s, y, stats = mp.mp_block_norm(t["x"], t["residual"], with_stats=True, **{k: t[k] for k in nu.NAMES[2:]}, **how)
    for a, b in (("x", "residual"), ("residual", "gate"), ("gate", "x"), ("residual", "x")):
        c = {k: v.clone() for k, v in t.items()}
        s1, y1, st1 = mp.mp_block_norm(c["x"], c["residual"], with_stats=True, s=c[a], y=c[b],
                                       **{k: c[k] for k in nu.NAMES[2:]}, **how)
        assert s1 is c[a] and y1 is c[b] and torch.equal(s1, s) and torch.equal(y1, y) and torch.equal(st1, stats)
