"""mp_block_norm and its gradients against the formulas in 64 bits: types, norms, gates,
widths that fill no vector, strides of nothing, rows of one value, empty inputs."""
from __future__ import annotations

import itertools

import pytest
import torch

import unpermute_routing_indices_gb300 as mp
from tests import norm_util as nu
from unpermute_routing_indices_gb300 import autograd as ag

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 64), (2, 1000), (7, 1009), (33, 520), (152, 128), (305, 40),
          (3, 2816), (2, 7168), (1, 8200), (2, 16384), (2, 32768), (1, 32767), (700, 33)]


def both(t, how, dtype, seed=50, with_gs=True, **kw):
    s, y, stats = mp.mp_block_norm(t["x"], t["residual"], with_stats=True,
                                   **{k: t[k] for k in nu.NAMES[2:]}, **how)
    nu.check_forward(t, how, s, y, stats)
    T, H = t["x"].shape
    g_s = nu.rows(T, H, dtype, seed, mean=0.0) if with_gs or t["pre_weight"] is None else None
    g_y = nu.rows(T, H, dtype, seed + 1, mean=0.1) if t["pre_weight"] is not None else None
    back = dict(how)
    back.pop("eps")
    got = mp.mp_block_norm_bwd(g_s, g_y, t["x"], s, stats, **{k: t[k] for k in nu.NAMES[2:]}, **back, **kw)
    nu.check_backward(t, how, g_s, g_y, s, stats, got)
    return s, y, stats, got


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,H", SHAPES)
def test_before_a_block(T, H, dtype):
    t, how = nu.make(T, H, DT[dtype], seed=T + H)
    both(t, how, DT[dtype])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,H", SHAPES)
def test_between_blocks_layer_norm(T, H, dtype):
    t, how = nu.make(T, H, DT[dtype], kind="layer", post=True, gate="channel", scale=0.5, bias=True, seed=T * H)
    both(t, how, DT[dtype])


@pytest.mark.parametrize("post,pre", [(False, True), (True, False), (True, True)])
@pytest.mark.parametrize("kind,gate,residual", list(itertools.product(
    ["rms", "layer"], ["none", "channel", "token", "element"], [False, True])))
def test_every_form(kind, gate, residual, post, pre):
    for T, H, dtype, bias, scale in ((37, 264, torch.bfloat16, False, 1.0), (19, 101, torch.float16, True, 0.22),
                                     (9, 1032, torch.float32, True, -1.5)):
        t, how = nu.make(T, H, dtype, kind=kind, post=post, pre=pre, residual=residual, gate=gate,
                         scale=scale, bias=bias, seed=H)
        both(t, how, dtype)
        both(t, how, dtype, with_gs=False, grad_dtype=torch.float32)


@pytest.mark.parametrize("H", [64, 4096, 4097])
def test_many_rows(H):
    t, how = nu.make(4099 if H > 64 else 40000, H, torch.bfloat16, post=True, gate="token", seed=H)
    both(t, how, torch.bfloat16)


def test_rows_far_from_zero():
    """A mean that is large beside the deviation: deviations are taken from the mean."""
    for dtype, mean in ((torch.float32, 300.0), (torch.bfloat16, 40.0)):
        t, how = nu.make(16, 2048, dtype, kind="layer", residual=False, seed=3)
        t["x"] = nu.rows(16, 2048, dtype, 4, mean=mean)
        s, y, stats = mp.mp_block_norm(t["x"], pre_weight=t["pre_weight"], with_stats=True, **how)
        assert s is t["x"]
        v = t["x"].double()
        want = (v - v.mean(1, keepdim=True)) / (v.var(1, unbiased=False, keepdim=True) + how["eps"]).sqrt() \
            * t["pre_weight"].double()
        # the mean is off by a few roundings of it, and by its sum's tree
        nu.within(y, want, nu.half(dtype) * want.abs() + nu.terms(2048) * nu.U32 * (mean + 5) * stats[:, 3:].double()
                  * t["pre_weight"].double().abs() * (1 + want.abs()))


def test_rows_of_one_value_and_of_zeros():
    x = torch.zeros(4, 512, device="cuda", dtype=torch.bfloat16)
    x[1], x[2] = 3.0, -0.25
    w = torch.full((512,), 2.0, device="cuda", dtype=torch.bfloat16)
    _, y, stats = mp.mp_block_norm(x, pre_weight=w, kind="layer", eps=1e-5, with_stats=True)
    assert bool((y == 0).all()) and torch.equal(stats[:, 2], x[:, 0].float())
    _, y, _ = mp.mp_block_norm(x, pre_weight=w, eps=1e-6)
    assert bool((y[0] == 0).all()) and bool((y[1] == 2).all())
    g = torch.ones_like(x)
    g_x = mp.mp_block_norm_bwd(None, g, x, x, stats, pre_weight=w, kind="layer")[0]
    assert bool((g_x == 0).all())      # constant gradients have no effect on a layer norm


def test_what_is_not_finite_stays_in_its_row():
    t, how = nu.make(6, 520, torch.bfloat16, post=True, gate="channel", bias=True, seed=9)
    want = mp.mp_block_norm(t["x"], t["residual"], with_stats=True, **{k: t[k] for k in nu.NAMES[2:]}, **how)
    t["x"] = t["x"].clone()
    t["x"][2, 17], t["x"][4, 0] = float("nan"), float("inf")
    got = mp.mp_block_norm(t["x"], t["residual"], with_stats=True, **{k: t[k] for k in nu.NAMES[2:]}, **how)
    keep = [0, 1, 3, 5]
    for a, b in zip(got, want):
        assert torch.equal(a[keep], b[keep]) and not bool(torch.isfinite(a[[2, 4]].float()).all())
    assert bool(torch.isnan(got[0][2]).all()) and bool(torch.isnan(got[1][2]).all())


@pytest.mark.parametrize("H", [1024, 1009, 4096, 6144])
def test_a_row_does_not_depend_on_the_others(H):
    t, how = nu.make(611, H, torch.bfloat16, kind="layer", post=True, gate="element", bias=True, seed=2)
    s, y, stats = mp.mp_block_norm(t["x"], t["residual"], with_stats=True, **{k: t[k] for k in nu.NAMES[2:]}, **how)
    for at in (0, 7, 301, 610):
        part = {k: v[at:at + 1].clone() if v is not None and v.dim() == 2 else v for k, v in t.items()}
        s1, y1, st1 = mp.mp_block_norm(part["x"], part["residual"], with_stats=True,
                                       **{k: part[k] for k in nu.NAMES[2:]}, **how)
        assert torch.equal(s1[0], s[at]) and torch.equal(y1[0], y[at]) and torch.equal(st1[0], stats[at])


@pytest.mark.parametrize("H", [48, 1009, 4096])
@pytest.mark.parametrize("into", ["x", "residual", "gate"])
def test_in_place(H, into):
    t, how = nu.make(333, H, torch.bfloat16, post=True, gate="element", seed=11)
    args = {k: t[k] for k in nu.NAMES[2:]}
    s, y, stats = mp.mp_block_norm(t["x"], t["residual"], with_stats=True, **args, **how)
    other = {"x": "residual", "residual": "gate", "gate": "x"}[into]
    c = {k: None if v is None else v.clone() for k, v in t.items()}
    s1, y1, st1 = mp.mp_block_norm(c["x"], c["residual"], with_stats=True, s=c[into], y=c[other],
                                   **{k: c[k] for k in nu.NAMES[2:]}, **how)
    assert s1 is c[into] and torch.equal(s1, s) and torch.equal(y1, y) and torch.equal(st1, stats)


@pytest.mark.parametrize("shift", [1, 2, 3, 4, 6])
@pytest.mark.parametrize("H", [64, 1001, 4096])
def test_tensors_that_start_anywhere(H, shift):
    """Views off 16 bytes, with guards around each result.  A row's values lie over other threads
    there, so its sums are added in another order: the bound is that of any order."""
    T, dtype = 70, torch.bfloat16
    t, how = nu.make(T, H, dtype, kind="layer", post=True, gate="element", bias=True, seed=5)
    plain = mp.mp_block_norm(t["x"], t["residual"], with_stats=True, **{k: t[k] for k in nu.NAMES[2:]}, **how)

    def moved(v, off):
        if v is None:
            return None
        big = torch.full((v.numel() + 64,), 7.0, dtype=v.dtype, device="cuda")
        big[off:off + v.numel()] = v.flatten()
        return big[off:off + v.numel()].view(v.shape)
    m = {k: moved(v, shift + i % 3) for i, (k, v) in enumerate(t.items())}
    s, y = moved(t["x"], shift), moved(t["x"], shift + 1)
    got = mp.mp_block_norm(m["x"], m["residual"], with_stats=True, s=s, y=y, **{k: m[k] for k in nu.NAMES[2:]}, **how)
    nu.check_forward(t, how, *got)
    for v, off in ((s, shift), (y, shift + 1)):
        base = v._base if v._base is not None else v
        whole = base.flatten()
        assert bool((whole[:off] == 7).all()) and bool((whole[off + T * H:] == 7).all())
    g_s, g_y = nu.rows(T, H, dtype, 1), nu.rows(T, H, dtype, 2)
    back = dict(how)
    back.pop("eps")
    got = mp.mp_block_norm_bwd(moved(g_s, shift), moved(g_y, shift + 2), m["x"], moved(plain[0], 1), plain[2],
                               **{k: m[k] for k in nu.NAMES[2:]}, **back)
    nu.check_backward(t, how, g_s, g_y, plain[0], plain[2], got)


def test_no_rows():
    x = torch.empty(0, 40, device="cuda")
    w = torch.ones(40, device="cuda")
    s, y, stats = mp.mp_block_norm(x, x, pre_weight=w, with_stats=True)
    assert s.shape == y.shape == (0, 40)
    got = mp.mp_block_norm_bwd(x, x, x, s, stats, pre_weight=w, pre_bias=w)
    assert bool((got[5] == 0).all()) and bool((got[6] == 0).all()) and got[0].shape == (0, 40)


def test_gradients_that_are_not_wanted():
    t, how = nu.make(50, 256, torch.bfloat16, post=True, gate="channel", bias=True, seed=8)
    args = {k: t[k] for k in nu.NAMES[2:]}
    s, y, stats = mp.mp_block_norm(t["x"], t["residual"], with_stats=True, **args, **how)
    g_s, g_y = nu.rows(50, 256, torch.bfloat16, 1), nu.rows(50, 256, torch.bfloat16, 2)
    back = dict(how)
    back.pop("eps")
    whole = mp.mp_block_norm_bwd(g_s, g_y, t["x"], s, stats, **args, **back)
    for i in range(7):
        need = [j == i for j in range(7)]
        got = mp.mp_block_norm_bwd(g_s, g_y, t["x"], s, stats, need=need, **args, **back)
        for j, (a, b) in enumerate(zip(got, whole)):
            assert (a is None) if j != i else torch.equal(a, b)


@pytest.mark.parametrize("dtype", DT)
def test_autograd_against_torch(dtype):
    """Gradients through the Functions against differentiation of the forms in 64 bits."""
    for gate, kind in (("channel", "rms"), ("token", "layer"), ("element", "rms")):
        t, how = nu.make(21, 136, DT[dtype], kind=kind, post=True, gate=gate, bias=True, scale=0.7, seed=31)
        leaves = {k: v.clone().requires_grad_() for k, v in t.items()}
        s, y = ag.block_norm(leaves["x"], leaves["residual"], **{k: leaves[k] for k in nu.NAMES[2:]}, **how)
        g_s, g_y = nu.rows(21, 136, DT[dtype], 1), nu.rows(21, 136, DT[dtype], 2)
        got = torch.autograd.grad([s, y], list(leaves.values()), [g_s, g_y])
        wide = {k: v.double().requires_grad_() for k, v in t.items()}
        s64, y64, _, _, _ = nu.forward(wide, how)
        want = torch.autograd.grad([s64, y64], list(wide.values()), [g_s.double(), g_y.double()])
        stats = mp.mp_block_norm(t["x"], t["residual"], with_stats=True, **{k: t[k] for k in nu.NAMES[2:]}, **how)[2]
        sizes = nu.backward(t, how, g_s, g_y, s.detach(), stats)
        for name, a, b in zip(leaves, got, want):
            # the kept s is rounded: half a step of it moves hat by that times rstd
            _, size, n = sizes[name]
            slack = 40 * nu.half(DT[dtype]) * size
            nu.within(a, b.view_as(a), nu.half(DT[dtype]) * b.view_as(a).abs() + slack.view_as(a) + 1e-5 * size.view_as(a), name)


def test_autograd_forms():
    x = nu.rows(8, 64, torch.float32, 1).requires_grad_()
    w = torch.ones(64, device="cuda", requires_grad=True)
    s, y = ag.block_norm(x, pre_weight=w)
    assert s is x
    (g,) = torch.autograd.grad((y * y).sum() + s.sum(), x)
    v = x.detach().double().requires_grad_()
    y64 = v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt()
    (want,) = torch.autograd.grad((y64 * y64).sum() + v.sum(), v)
    assert bool(((g.double() - want).abs() <= 1e-5 * (1 + want.abs())).all())
    # only one of the results goes on
    r = nu.rows(8, 64, torch.float32, 2).requires_grad_()
    s, y = ag.block_norm(x, r, pre_weight=w)
    g1 = torch.autograd.grad(s.sum(), [x, r, w], retain_graph=True)
    assert bool((g1[0] == 1).all()) and bool((g1[1] == 1).all()) and bool((g1[2] == 0).all())
    g2 = torch.autograd.grad(y.sum(), [x, r, w])
    assert torch.equal(g2[0], g2[1])
    with torch.no_grad():
        assert not ag.block_norm(x, r, pre_weight=w)[1].requires_grad
    s, y = ag.block_norm(x, r, pre_weight=w)
    (g,) = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="gradients of gradients"):
        torch.autograd.grad(g.sum(), x)


def test_gradients_against_differences():
    """Central differences of the fp32 results along a direction d, by steps of h: off by
    h^2/6 times the third derivative (order 1 for these rows, times |d|^3) and the
    results' roundings over 2h."""
    t, how = nu.make(5, 96, torch.float32, kind="layer", post=True, gate="channel", bias=True, scale=0.8, seed=77)
    g_s, g_y = nu.rows(5, 96, torch.float32, 1), nu.rows(5, 96, torch.float32, 2)

    def loss(v):
        s, y, _ = mp.mp_block_norm(v["x"], v["residual"], **{k: v[k] for k in nu.NAMES[2:]}, **how)
        return float((s.double() * g_s.double()).sum() + (y.double() * g_y.double()).sum())
    s, y, stats = mp.mp_block_norm(t["x"], t["residual"], with_stats=True, **{k: t[k] for k in nu.NAMES[2:]}, **how)
    back = dict(how)
    back.pop("eps")
    grads = mp.mp_block_norm_bwd(g_s, g_y, t["x"], s, stats, **{k: t[k] for k in nu.NAMES[2:]}, **back)
    h = 2.0 ** -6
    for i, (name, g) in enumerate(zip(nu.NAMES, grads)):
        d = nu.rows(1, t[name].numel(), torch.float32, 90 + i, mean=0.0)[0].view_as(t[name])
        d = d / d.norm()
        up = loss({**t, name: t[name] + h * d})
        down = loss({**t, name: t[name] - h * d})
        along = float((g.double() * d.double()).sum())
        scale = float(g_s.norm() + 2 * g_y.norm())
        rounding = nu.U32 * 40 * float(g_s.abs().sum() + 3 * g_y.abs().sum()) / (2 * h)
        assert abs((up - down) / (2 * h) - along) <= h * h * scale + rounding, name


@pytest.mark.parametrize("H", [512, 1009])
def test_graph_streams_and_repeats(H):
    t, how = nu.make(1000, H, torch.bfloat16, post=True, gate="channel", seed=21)
    args = {k: t[k] for k in nu.NAMES[2:]}
    back = dict(how)
    back.pop("eps")
    g_s, g_y = nu.rows(1000, H, torch.bfloat16, 1), nu.rows(1000, H, torch.bfloat16, 2)

    def step():
        s, y, stats = mp.mp_block_norm(t["x"], t["residual"], with_stats=True, **args, **how)
        return [s, y, stats, *(g for g in mp.mp_block_norm_bwd(g_s, g_y, t["x"], s, stats, **args, **back)
                               if g is not None)]
    want = [v.clone() for v in step()]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
    side = [torch.cuda.Stream() for _ in range(2)]
    results = []
    torch.cuda.synchronize()
    for q in side:
        with torch.cuda.stream(q):
            results.append([step() for _ in range(3)])
    torch.cuda.synchronize()
    for r in itertools.chain(*results):
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    t["x"].copy_(nu.rows(1000, H, torch.bfloat16, 99))
    graph.replay()
    torch.cuda.synchronize()
    fresh = step()
    assert all(torch.equal(a, b) for a, b in zip(out, fresh))
    assert not torch.equal(out[0], want[0])


@pytest.mark.parametrize("T,H", [(1048580, 4096), (1048581, 4097)])
def test_rows_past_32_bits(T, H):
    """Rows beyond 2^32 values, beside the same rows alone."""
    assert (T - 3) * H > 2 ** 32
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_()
    w, v = (nu.rows(1, H, torch.bfloat16, i, mean=1.0)[0] for i in (1, 2))
    ends = torch.tensor([0, 1, T - 3, T - 2, T - 1], device="cuda")
    few = x[ends].contiguous()
    s, y, stats = mp.mp_block_norm(x, x, post_weight=w, pre_weight=v, scale=0.5, with_stats=True)
    s1, y1, stats1 = mp.mp_block_norm(few, few, post_weight=w, pre_weight=v, scale=0.5, with_stats=True)
    for a, b in ((s, s1), (y, y1), (stats, stats1)):
        assert torch.equal(a[ends], b)
    need = (True, True, False, False, False, False, False)
    g = mp.mp_block_norm_bwd(y, x, x, s, stats, post_weight=w, pre_weight=v, scale=0.5, need=need)
    g1 = mp.mp_block_norm_bwd(y1, few, few, s1, stats1, post_weight=w, pre_weight=v, scale=0.5, need=need)
    for a, b in zip(g[:2], g1[:2]):
        assert torch.equal(a[ends], b)
