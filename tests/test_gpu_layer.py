"""mp_moe_layer against the layer in 64 bits: choice, weights, results; sizes that fill no
tile, tensors that start anywhere, empty slots, many tokens for one expert."""
from __future__ import annotations

import itertools
import math
import threading

import pytest
import torch

import unpermute_routing_indices_gb300 as mp
from tests import norm_util as nu

pytestmark = pytest.mark.gpu


def weights_of(E, H, F, O, act, seed, biases=False, router=torch.float32):
    P = 2 * F if act in ("swiglu", "geglu") else F
    t = dict(router=nu.rows(E, H, router, seed, mean=0.0, std=H ** -0.5),
             w1=nu.rows(E * P, H, torch.bfloat16, seed + 1, mean=0.0, std=H ** -0.5).view(E, P, H),
             w2=nu.rows(E * O, F, torch.bfloat16, seed + 2, mean=0.0, std=F ** -0.5).view(E, O, F), b1=None, b2=None)
    if biases:
        t["b1"] = nu.rows(E, P, torch.bfloat16, seed + 3, mean=0.1, std=0.3)
        t["b2"] = nu.rows(E, O, torch.bfloat16, seed + 4, mean=-0.1, std=0.3)
    return t


def check(x, t, K, act, out=None, **how):
    y, idx, w = out if out is not None else mp.mp_moe_layer(x, t["router"], t["w1"], t["w2"], K, b1=t["b1"],
                                                            b2=t["b2"], act=act, **how)
    want_idx, want_w = nu.choice(nu.logits(x, t["router"]), K, **how)
    assert torch.equal(idx, want_idx)
    # expf and a division of fp32 logits: a few roundings, and those of |l| in the exponent
    nu.within(w, want_w, (16 + 2 * 20) * nu.U32 * want_w.abs())
    want, bound = nu.layer(x, t["w1"], t["w2"], t["b1"], t["b2"], act, idx, w)
    nu.within(y, want, bound, "y")
    return y, idx, w


SIZES = [  # T, E, K, H, F, O
    (1, 1, 1, 1, 1, 1), (1, 4, 4, 8, 8, 8), (1, 16, 4, 256, 128, 256), (2, 8, 2, 64, 32, 40),
    (1, 64, 6, 2048, 1024, 2048), (7, 40, 3, 1001, 333, 1001), (8, 32, 8, 520, 264, 512),
    (16, 8, 2, 1024, 512, 1024), (33, 6, 6, 136, 72, 200), (64, 64, 6, 512, 256, 512), (64, 2, 1, 264, 96, 17),
    (64, 1, 1, 128, 64, 128), (3, 300, 10, 96, 40, 96), (5, 1024, 32, 72, 16, 64), (64, 40, 32, 40, 24, 48),
    (9, 16, 4, 1000, 1000, 1000), (1, 3, 2, 4099, 17, 5), (4, 12, 2, 7168, 24, 16), (2, 4, 1, 16, 4100, 24),
    (12, 5, 3, 2050, 1022, 2046), (1, 2, 1, 40000, 64, 40),
    (2, 3, 2, 65536, 16, 8), (2, 3, 2, 8, 65536, 8), (3, 3, 2, 16, 8, 65536),   # the widest
    (64, 1024, 32, 24, 16, 40), (64, 170, 32, 40, 24, 40),                      # the largest tables
]


@pytest.mark.parametrize("T,E,K,H,F,O", SIZES)
def test_sizes(T, E, K, H, F, O):
    for act, biases in (("swiglu", False), ("gelu", True)):
        x = nu.rows(T, H, torch.bfloat16, T + H, mean=0.0)
        check(x, weights_of(E, H, F, O, act, H + F, biases), K, act)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "geglu", "swiglu"])
@pytest.mark.parametrize("biases", [False, True])
def test_activations(act, biases):
    for T, H, F in ((1, 128, 72), (20, 200, 65)):
        x = nu.rows(T, H, torch.bfloat16, 5, mean=0.0)
        check(x, weights_of(8, H, F, H, act, 6, biases), 3, act)


@pytest.mark.parametrize("score,bias,groups,renorm", list(itertools.product(
    ["softmax", "sigmoid"], [False, True], [(1, 1, 1), (8, 4, 2), (4, 2, 1)], [True, False])))
def test_choices(score, bias, groups, renorm):
    E, H = 64, 136
    for router, T in itertools.product((torch.bfloat16, torch.float16, torch.float32), (1, 29)):
        t = weights_of(E, H, 24, 32, "silu", 3, router=router)
        x = nu.rows(T, H, torch.bfloat16, 8, mean=0.0)
        b = nu.rows(1, E, torch.float32, 9, mean=0.0, std=0.1)[0] if bias else None
        check(x, t, 5, "silu", score=score, bias=b, n_groups=groups[0], topk_groups=groups[1],
              group_top=groups[2], renorm=renorm, scale=2.5)


def test_logits_that_differ_in_the_last_place():
    """Two routers' rows whose sums differ by less than fp32 sums in any order could tell, and
    equal ones: the choice is that of the exact logits, ties to the lower expert."""
    H, E = 4096, 32
    g = torch.Generator().manual_seed(3)
    row = torch.randn(H, generator=g)
    router = row.repeat(E, 1)
    x = torch.randn(1, H, generator=g).bfloat16().cuda()
    for e in range(E):                      # the same values, one of them a step up or down
        at = int(torch.randint(H, (1,), generator=g))
        router[e, at] = torch.nextafter(router[e, at], torch.tensor(math.inf if e % 3 else -math.inf))
    t = weights_of(E, H, 8, 8, "silu", 1)
    t["router"] = router.cuda()
    check(x, t, 8, "silu")
    t["router"] = row.repeat(E, 1).cuda()
    _, idx, _ = check(x, t, 8, "silu")
    assert idx.tolist() == [list(range(8))]


def test_same_expert_for_every_token():
    """All tokens through few experts: 64 rows of one."""
    H, E = 256, 16
    t = weights_of(E, H, 128, 256, "swiglu", 4)
    t["router"][3:] = -t["router"][2]
    t["router"][:2] = t["router"][2] * 0.5
    for T in (8, 9, 33, 64):
        x = t["router"][2].bfloat16() * 16 + nu.rows(T, H, torch.bfloat16, T, mean=0.0, std=0.1)
        check(x.bfloat16(), t, 3, "swiglu")


def test_empty_slots_and_tokens_that_are_not_finite():
    """An expert with a bias of -inf cannot be chosen; logits that are NaN leave a token without
    experts, whose result is zero, and the others as they were."""
    H, E = 128, 6
    t = weights_of(E, H, 64, 96, "swiglu", 7, biases=True)
    x = nu.rows(5, H, torch.bfloat16, 2, mean=0.0)
    bias = torch.zeros(E, device="cuda")
    bias[1:] = -math.inf
    y, idx, w = mp.mp_moe_layer(x, t["router"], t["w1"], t["w2"], 3, b1=t["b1"], b2=t["b2"], bias=bias)
    assert bool((idx[:, 0] == 0).all()) and bool((idx[:, 1:] == -1).all())
    assert bool((w[:, 0] == 1).all()) and bool((w[:, 1:] == 0).all())
    want, bound = nu.layer(x, t["w1"], t["w2"], t["b1"], t["b2"], "swiglu", idx, w)
    nu.within(y, want, bound)
    bias[:] = -math.inf
    y, idx, w = mp.mp_moe_layer(x, t["router"], t["w1"], t["w2"], 3, b1=t["b1"], b2=t["b2"], bias=bias)
    assert bool((idx == -1).all()) and bool((y == 0).all())
    plain = mp.mp_moe_layer(x, t["router"], t["w1"], t["w2"], 3, b1=t["b1"], b2=t["b2"])
    x2 = x.clone()
    x2[1, 5] = float("nan")
    got = mp.mp_moe_layer(x2, t["router"], t["w1"], t["w2"], 3, b1=t["b1"], b2=t["b2"])
    for a, b in zip(got, plain):
        assert torch.equal(a[[0, 2, 3, 4]], b[[0, 2, 3, 4]])
    assert got[1][1].tolist() == [-1] * 3 and bool((got[0][1] == 0).all())


def test_weights_that_are_not_finite_reach_their_tokens_alone():
    H, E, F = 192, 8, 64
    t = weights_of(E, H, F, 128, "silu", 7)
    x = nu.rows(12, H, torch.bfloat16, 2, mean=0.0)
    y, idx, w = mp.mp_moe_layer(x, t["router"], t["w1"], t["w2"], 2, act="silu")
    e = int(idx[0, 0])
    t["w2"][e, 5, 3] = float("nan")
    t["w1"][e, 9] = float("inf")
    y2, _, _ = mp.mp_moe_layer(x, t["router"], t["w1"], t["w2"], 2, act="silu")
    hit = (idx == e).any(1)
    assert torch.equal(y2[~hit], y[~hit]) and bool(torch.isnan(y2[hit][:, 5]).all())


@pytest.mark.parametrize("T,H,F", [(3, 256, 128), (17, 264, 100), (2, 333, 77)])
@pytest.mark.parametrize("shift", [1, 2, 3, 4, 5, 7])
def test_tensors_that_start_anywhere(T, H, F, shift):
    """Views off 16 bytes at both ends of their buffers, guards around the results."""
    t = weights_of(5, H, F, H, "geglu", 13, biases=True)
    x = nu.rows(T, H, torch.bfloat16, 6, mean=0.0)

    def moved(v, off):
        big = torch.full((v.numel() + off,), 7, dtype=v.dtype, device="cuda")
        big[off:] = v.flatten()
        return big[off:].view(v.shape)
    m = {k: moved(v, (shift + i) % 8) for i, (k, v) in enumerate(t.items())}
    big = torch.full((T * H + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = big[shift:shift + T * H].view(T, H)
    out = mp.mp_moe_layer(moved(x, shift), m["router"], m["w1"], m["w2"], 2, b1=m["b1"], b2=m["b2"], act="geglu", y=y)
    check(x, t, 2, "geglu", out)
    assert bool((big[:shift] == 7).all()) and bool((big[shift + T * H:] == 7).all())


def test_no_tokens_and_a_dirty_workspace():
    t = weights_of(4, 64, 32, 64, "swiglu", 1)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    y, idx, w = mp.mp_moe_layer(x, t["router"], t["w1"], t["w2"], 2)
    assert y.shape == (0, 64) and idx.shape == (0, 2)
    x = nu.rows(9, 64, torch.bfloat16, 1, mean=0.0)
    want = mp.mp_moe_layer(x, t["router"], t["w1"], t["w2"], 2)
    n = mp.mp_moe_layer_workspace_size(9, 4, 2, 64, 32, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for fill in (0, 255, 127):
        ws = torch.full((n + 256,), fill, dtype=torch.uint8, device="cuda")
        got = mp.mp_moe_layer(x, t["router"], t["w1"], t["w2"], 2, workspace=ws[:n], status=status)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool((ws[n:] == fill).all())
    assert int(status) == 0


def test_a_token_does_not_depend_on_the_others():
    t = weights_of(16, 512, 256, 512, "swiglu", 21, biases=True)
    for T in (4, 40):
        x = nu.rows(T, 512, torch.bfloat16, T, mean=0.0)
        y, idx, w = mp.mp_moe_layer(x, t["router"], t["w1"], t["w2"], 4, b1=t["b1"], b2=t["b2"])
        order = torch.randperm(T, generator=torch.Generator().manual_seed(1)).cuda()
        other = x[order].clone()
        other[0] = other[1]
        y2, idx2, w2 = mp.mp_moe_layer(other, t["router"], t["w1"], t["w2"], 4, b1=t["b1"], b2=t["b2"])
        assert torch.equal(y2[1:], y[order][1:]) and torch.equal(idx2[1:], idx[order][1:])
        assert torch.equal(w2[1:], w[order][1:])


def test_graph_streams_and_repeats():
    t = weights_of(24, 1024, 256, 1024, "swiglu", 2)
    x = nu.rows(6, 1024, torch.bfloat16, 3, mean=0.0)

    def call(ws=None):
        return mp.mp_moe_layer(x, t["router"], t["w1"], t["w2"], 4, workspace=ws)
    want = [v.clone() for v in call()]
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
    torch.cuda.synchronize()
    side, results = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(5):
        for q in side:
            with torch.cuda.stream(q):
                results.append(call())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in results for a, b in zip(r, want))
    # two graphs that share a workspace, replayed one after the other
    ws = torch.empty(mp.mp_moe_layer_workspace_size(6, 24, 4, 1024, 256, 1024), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                out = call(ws)
        graphs.append(g)
        outs.append(out)
    x.copy_(nu.rows(6, 1024, torch.bfloat16, 4, mean=0.0))
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    want = call()
    assert all(torch.equal(a, b) for out in outs for a, b in zip(out, want))


def test_weights_past_32_bits():
    """Experts whose weights lie beyond 2^32 values; the others' are not read."""
    E, H, F = 10, 4096, 65536
    gen = torch.Generator(device="cuda").manual_seed(5)
    t = dict(w1=torch.full((E, 2 * F, H), float("nan"), dtype=torch.bfloat16, device="cuda"),
             w2=torch.full((E, H, F), float("nan"), dtype=torch.bfloat16, device="cuda"), b1=None, b2=None,
             router=nu.rows(E, H, torch.float32, 1, mean=0.0, std=H ** -0.5))
    for e in (8, 9):
        t["w1"][e].normal_(0.0, H ** -0.5, generator=gen)
        t["w2"][e].normal_(0.0, F ** -0.5, generator=gen)
    bias = torch.zeros(E, device="cuda")
    bias[8:] = 100.0
    x = nu.rows(2, H, torch.bfloat16, 3, mean=0.0)
    y, idx, _ = check(x, t, 2, "swiglu", bias=bias)
    assert bool((idx >= 8).all()) and bool(y.isfinite().all())


def test_two_host_threads():
    t = weights_of(24, 512, 96, 512, "swiglu", 2)
    norm = nu.rows(1, 512, torch.bfloat16, 9, mean=1.0)[0]
    x = nu.rows(6, 512, torch.bfloat16, 3, mean=0.0)

    def call():
        s, n, _ = mp.mp_block_norm(x, pre_weight=norm)
        y, idx, w = mp.mp_moe_layer(n, t["router"], t["w1"], t["w2"], 4)
        return mp.mp_block_norm(y, s, post_weight=norm)[0], idx, w
    want = call()
    torch.cuda.synchronize()
    results, errors = [], []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                mine = [call() for _ in range(30)]
                torch.cuda.current_stream().synchronize()
            results.extend(mine)
        except Exception as e:   # noqa: BLE001 - told to the test below
            errors.append(e)
    threads = [threading.Thread(target=work) for _ in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors and len(results) == 60
    assert all(torch.equal(a, b) for r in results for a, b in zip(r, want))


def test_beside_the_chain():
    """The layer and the calls that it stands for: the same choice, results within both bounds."""
    t = weights_of(32, 512, 128, 512, "swiglu", 5)
    x = nu.rows(48, 512, torch.bfloat16, 1, mean=0.0)
    y, idx, w = check(x, t, 4, "swiglu")
    idx2, w2 = mp.mp_route(nu.logits(x, t["router"]), 4)
    assert torch.equal(idx, idx2) and torch.equal(w, w2)
    rim, _, _, offsets = mp.mp_build_map(idx, 32)
    rows, _ = mp.mp_permute(x, rim)
    out, _, _ = mp.mp_expert_mlp(rows, t["w1"], t["w2"], offsets)
    chain = mp.mp_unpermute(out, rim, w)
    # the chain keeps h as one bf16 value
    want, bound = nu.layer(x, t["w1"], t["w2"], None, None, "swiglu", idx, w, kept=2.0 ** -8)
    each = torch.zeros_like(want)
    for k in range(4):
        ek = idx[:, k:k + 1]
        yk, _ = nu.layer(x, t["w1"], t["w2"], None, None, "swiglu", ek, torch.ones_like(w[:, :1]))
        each += w[:, k:k + 1].double() * yk.abs()
    nu.within(chain, want, bound + 2.0 ** -8 * 1.1 * each)   # the chain rounds each expert's result
