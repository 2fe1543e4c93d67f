"""What the router and the experts' entry points promise beside their values: nothing
written outside the outputs, no device memory allocated, operands of any base, values
that are not finite kept in their rows, calls from several host threads at once."""
from __future__ import annotations

import os
import sys
import threading

import pytest
import torch

import unpermute_routing_indices_gb300 as mp
from unpermute_routing_indices_gb300 import _lib
from tests.gpu_util import DEV, status_word
from tests.test_gpu_expert import (COUNTS, GATED, act64, checkpoint_of, normal, offsets_of, rows64, BF16,
                                   SLOPE)
from tests.test_gpu_guards import Guarded

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


class Bytes:
    """A tensor of a one-byte type between guards."""

    def __init__(self, shape, dtype):
        n = shape[0] * shape[1]
        self.base = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=DEV)
        self.t = self.base[256:256 + n].view(dtype).view(shape)
        self.n = n

    def guards_intact(self):
        return bool((self.base[:256] == 0xA5).all()) and bool((self.base[256 + self.n:] == 0xA5).all())


# counts, H, F, activation, checkpoint: the tensor-core form with and without TMA, split
# contractions, few rows, pairs of CTAs
LAYERS = [
    ("many", 136, 72, "swiglu", "e4m3"), ("many", 37, 33, "geglu", "e4m3"), ("many", 131, 70, "gelu", "bf16"),
    ("big", 264, 136, "swiglu", "bf16"), ("tokens", 520, 264, "swiglu", "e4m3"), ("few each", 101, 64, "silu", "bf16"),
    ("one expert", 2048, 40, "relu", "e4m3"), ("long", 264, 200, "geglu", "e4m3"), ("deep", 72, 40, "gelu", "bf16"),
]


def layer_call(name, H, F, act, save, buffer, byte_buffer):
    """mp_expert_mlp, its backward pass and the single products and gradients, every output
    made by `buffer`; (a function that issues the calls, the outputs' owners)."""
    counts, more = COUNTS[name], 9
    E, R = len(counts), sum(counts) + more
    P = 2 * F if act in GATED else F
    offsets = offsets_of(counts) + 4
    x, g = normal(R, H, seed=1), normal(R, H, seed=2)
    w1, w2 = normal(E, P, H, seed=3, std=0.1), normal(E, H, F, seed=4, std=0.1)
    b1, b2, residual = normal(E, P, seed=5), normal(E, H, seed=6), normal(R, F, seed=7)
    own = {k: buffer(s, torch.bfloat16) for k, s in dict(
        h=(R, F), y=(R, H), g_z=(R, P), g_x=(R, H), g_w1=(E, P, H), g_w2=(E, H, F), g_b1=(E, P), g_b2=(E, H),
        out=(R, F), d_x=(R, P), d_h=(R, F), w_w=(E, H, F), w_b=(E, H)).items()}
    own |= {k: buffer(s, torch.float32) for k, s in dict(f_w=(E, H, F), f_b=(E, H)).items()}
    z = buffer((R, P), torch.bfloat16) if save == "bf16" else byte_buffer((R, P), torch.float8_e4m3fn)
    own["z"] = z
    z_exp = None
    if save == "e4m3":
        own["z_exp"] = byte_buffer((R, P // F * -(-F // 32)), torch.uint8)
        z_exp = own["z_exp"].t
    status, lib, t = status_word(), _lib.load(), {k: v.t for k, v in own.items()}

    def p(v):
        return None if v is None else v.data_ptr()

    def run():
        s = torch.cuda.current_stream().cuda_stream
        assert lib.mp_expert_mlp(p(x), p(w1), p(b1), p(w2), p(b2), p(offsets), R, E, H, F, H, mp.ACTS[act], p(t["h"]),
                                 p(t["y"]), mp.SAVES[save], p(t["z"]), p(z_exp), p(status), s) == 0
        assert lib.mp_expert_mlp_bwd(p(g), p(x), p(w1), p(w2), p(offsets), R, E, H, F, H, mp.ACTS[act],
                                     mp.SAVES[save], p(t["z"]), p(z_exp), p(t["g_z"]), p(t["d_h"]), p(t["g_x"]),
                                     p(t["g_w1"]), p(t["g_b1"]), p(t["g_w2"]), p(t["g_b2"]), p(status), s) == 0
        mp.mp_expert_gemm(x, w1, offsets, bias=b1, act=act, residual=residual, save=save, out=t["out"],
                          z=t["z"], z_exp=z_exp, status=status)
        mp.mp_expert_dgrad(g, w2, offsets, act=act, z=t["z"], z_exp=z_exp, g_x=t["d_x"], h=t["d_h"], status=status)
        mp.mp_expert_wgrad(g, residual, offsets, g_w=t["w_w"], g_bias=t["w_b"], status=status)
        for accumulate in (False, True):
            mp.mp_expert_wgrad(g, residual, offsets, g_w=t["f_w"], g_bias=t["f_b"], accumulate=accumulate,
                               status=status)
    return run, own, status, offsets


@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "%s-H%d-F%d-%s-%s" % c)
def test_expert_calls_stay_inside_their_outputs(case):
    run, own, status, offsets = layer_call(*case, Guarded, Bytes)
    run()
    torch.cuda.synchronize()
    assert int(status) == 0
    for name, buffer in own.items():
        assert buffer.guards_intact(), name
    first, last = int(offsets[0]), int(offsets[-1])
    for name in ("h", "g_z", "out", "d_x", "d_h"):      # rows without an expert are left
        there = own[name].sentinel()
        assert bool(there[:first].all()) and bool(there[last:].all()), name
        assert not bool(there[first:last].any()), name


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,K,G,keep", [(333, 128, 8, 1, 1), (257, 256, 8, 8, 4), (99, 37, 5, 1, 1),
                                          (50, 1000, 9, 10, 3), (1, 8, 2, 8, 2)])
def test_route_stays_inside_its_outputs(T, E, K, G, keep, dtype):
    logits = normal(T, E, seed=T).to(dtype)
    bias = torch.linspace(-0.1, 0.1, E, device=DEV)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            idx, w = Guarded((T, K), torch.int32), Guarded((T, K), torch.float32)
            mp.mp_route(logits, K, score=score, renorm=renorm, bias=bias, n_groups=G, topk_groups=keep, group_top=2,
                        idx=idx.t, weights=w.t)
            assert idx.guards_intact() and w.guards_intact()
            base = torch.full((T * E + 512,), -12288.0, dtype=dtype, device=DEV)
            mp.mp_route_bwd(torch.ones(T, K, device=DEV), logits, idx.t, score=score, renorm=renorm,
                            g_logits=base[256:256 + T * E].view(T, E))
            assert bool((base[:256] == -12288.0).all()) and bool((base[256 + T * E:] == -12288.0).all())
            assert not bool((base[256:256 + T * E] == -12288.0).any())


def test_route_and_expert_calls_allocate_no_device_memory():
    class Plain:
        def __init__(self, shape, dtype):
            self.t = torch.zeros(shape, dtype=torch.uint8 if dtype.itemsize == 1 else dtype, device=DEV).view(dtype)
    runs = [layer_call(*case, Plain, Plain)[0] for case in LAYERS]
    logits, bias = normal(700, 128, seed=1).float(), torch.zeros(128, device=DEV)
    idx = torch.empty((700, 8), dtype=torch.int32, device=DEV)
    w, g_logits = torch.empty((700, 8), device=DEV), torch.empty_like(logits)

    def run():
        mp.mp_route(logits, 8, score="sigmoid", bias=bias, idx=idx, weights=w)
        mp.mp_route_bwd(w, logits, idx, score="sigmoid", g_logits=g_logits)
        for r in runs:
            r()
    run()                                   # loads the kernels
    torch.cuda.synchronize()
    free0, _ = torch.cuda.mem_get_info(DEV)
    used0 = torch.cuda.memory_allocated(DEV)
    for _ in range(3):
        run()
    torch.cuda.synchronize()
    free1, _ = torch.cuda.mem_get_info(DEV)
    assert torch.cuda.memory_allocated(DEV) == used0
    assert free1 == free0, f"device free memory changed by {free0 - free1} bytes"


@pytest.mark.parametrize("shift", [1, 2, 3, 8])
@pytest.mark.parametrize("name,N,K", [("many", 64, 128), ("big", 136, 72), ("long", 192, 264), ("deep, one short", 72, 40),
                                      ("few each", 33, 37)])
def test_gradients_of_operands_off_their_grid(name, N, K, shift):
    """Rows, weights, the kept product and every result begin `shift` elements past a
    256-byte boundary.  Bounds as in the tests of the gradients themselves."""
    counts = COUNTS[name]
    E, R, offsets = len(counts), sum(counts), offsets_of(counts)
    g, w = normal(R, N, seed=5, shift=shift), normal(E, N, K, seed=6, std=N ** -0.5, shift=shift)
    x = normal(R, K, seed=9, shift=shift)

    def moved(*shape, dtype=torch.bfloat16):
        n = 1
        for k in shape:
            n *= k
        return torch.zeros(n + shift, dtype=dtype, device=DEV)[shift:].view(shape)
    t, size = rows64(g, w, offsets, turned=True)
    Z = (N + 2) * 2.0 ** -23 * size
    got, _ = mp.mp_expert_dgrad(g, w, offsets, g_x=moved(R, K))
    assert ((got.double() - t).abs() <= Z * (1 + BF16) + BF16 * t.abs() + 1e-38).all()

    for act, save in (("silu", "bf16"), ("gelu", "e4m3")):
        z, z_exp, v = checkpoint_of(R, K, act, save, 7)
        zs = moved(R, K) if save == "bf16" else moved(R, K, dtype=torch.uint8).view(torch.float8_e4m3fn)
        zs.view(torch.uint8).copy_(z.view(torch.uint8))
        if z_exp is not None:
            z_exp = moved(*z_exp.shape, dtype=torch.uint8).copy_(z_exp)
        got, h = mp.mp_expert_dgrad(g, w, offsets, act=act, z=zs, z_exp=z_exp, g_x=moved(R, K), h=moved(R, K))
        y, slope = act64(v, act)
        want, off = t * slope, Z * SLOPE + 2.0 ** -17 * 1.2 * (t.abs() + Z)
        assert ((got.double() - want).abs() <= off * (1 + BF16) + BF16 * want.abs() + 1e-38).all()
        assert ((h.double() - y).abs() <= (BF16 + 2.0 ** -17) * y.abs() + 1e-38).all()

    for dtype, half in ((torch.bfloat16, BF16), (torch.float32, 2.0 ** -24)):
        g_w, g_b = mp.mp_expert_wgrad(g, x, offsets, g_w=moved(E, N, K, dtype=dtype), g_bias=moved(E, N, dtype=dtype))
        for e, n in enumerate(counts):
            a = int(offsets[e])
            ge, xe = g[a:a + n].double(), x[a:a + n].double()
            want, off = ge.T @ xe, (n + 2) * 2.0 ** -23 * (ge.abs().T @ xe.abs())
            assert ((g_w[e].double() - want).abs() <= off + half * want.abs()).all()
            want, off = ge.sum(0), (n + 2) * 2.0 ** -24 * ge.abs().sum(0)
            assert ((g_b[e].double() - want).abs() <= off + half * want.abs()).all()


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("N,K", [(64, 64), (264, 520), (33, 37)])
def test_what_is_not_finite_fills_its_row(N, K, act):
    """Every element of a row with a NaN or an infinity in it (the weights have no zeros)
    is not finite, in the result, and the rows beside it are finite."""
    counts = [20, 45, 3, 130]
    R, offsets = sum(counts), offsets_of(counts)
    x, w = normal(R, K, seed=1), normal(4, N, K, seed=2)
    w[w == 0] = 1
    rows = torch.tensor([19, 20, 64, 65, 197], device=DEV)
    x[rows[::2], K // 2] = float("nan")
    x[rows[1::2], 1] = float("inf")
    out, _, _ = mp.mp_expert_gemm(x, w, offsets, act=act)
    good = torch.ones(R, dtype=torch.bool, device=DEV)
    good[rows] = False
    assert torch.isnan(out[rows[::2]].float()).all() and torch.isfinite(out[good].float()).all()
    # silu of -inf is 0 * inf
    assert not torch.isfinite(out[rows[1::2]].float()).any()


def test_host_threads_at_once():
    """Calls of four host threads, each on its own stream, give what they give alone."""
    jobs = []
    for name, N, K in (("many", 64, 128), ("big", 264, 136), ("few each", 130, 512), ("many", 37, 41)):
        counts = COUNTS[name]
        offsets = offsets_of(counts)
        x, w = normal(sum(counts), K, seed=1), normal(len(counts), N, K, seed=2)
        g, logits = normal(sum(counts), N, seed=3), normal(sum(counts), 64, seed=4).float()

        def job(offsets=offsets, x=x, w=w, g=g, logits=logits):
            return [mp.mp_expert_gemm(x, w, offsets, act="silu")[0], mp.mp_expert_dgrad(g, w, offsets)[0],
                    mp.mp_expert_wgrad(g, x, offsets)[0], *mp.mp_route(logits, 6, score="sigmoid")]
        jobs.append(job)
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    failures = []

    def thread(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = jobs[k]()
                torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                failures.append(f"job {k} differs")
        except Exception as error:   # noqa: BLE001
            failures.append(repr(error))
    threads = [threading.Thread(target=thread, args=(k,)) for k in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures


def test_balance_evens_the_load():
    """From a router that prefers some experts, the bias brings the largest load down to
    within a third of the mean on the same tokens (from more than twice)."""
    import moe_layer
    layer = moe_layer.MoeLayer.make(256, 32, 16, 4, seed=3)
    layer.bias += torch.linspace(-0.3, 0.3, 16, device=DEV)
    x = torch.randn(4096, 256, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).bfloat16()

    def load():
        idx, _ = mp.mp_route(x.float() @ layer.router.t(), 4, score="sigmoid", bias=layer.bias)
        return torch.bincount(idx.flatten(), minlength=16)
    before = load()
    for _ in range(200):
        layer.balance(load(), 4e-3)
    mean = 4096 * 4 / 16
    assert before.max() > 2 * mean and load().max() < 1.33 * mean
