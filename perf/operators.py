"""Cases of the expert layer's operators: the router, the experts' matrix
products with their epilogue, their gradients, and the training step of a
two-product expert with its activations kept in 8 bits.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, 64 for the router's choices) or, with ``own`` set, through this
repository's entry points.  ``exact`` computes it from the definitions in 64
bits.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 32          # columns of a row that share one exponent in an 8-bit checkpoint
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _route(T, E, K, score, dtype="float32", bias=False, groups=1, keep=1, group_top=1,
           renorm=True, scale=1.0, train=True):
    return dict(op="route", T=T, E=E, K=K, score=score, dtype=dtype, bias=bias, groups=groups,
                keep=keep, group_top=group_top, renorm=renorm, scale=scale, train=train)


def _product(op, R, E, n, k, act="none", bias=False, residual=False, saved="none"):
    return dict(op=op, R=R, E=E, n=n, k=k, act=act, bias=bias, residual=residual, saved=saved)


def _step(R, E, H, F, act, bias):
    return dict(op="step", R=R, E=E, H=H, F=F, act=act, bias=bias)


def listed():
    return [
        # the router of one token while an answer is written: latency alone
        dict(name="route one token", **_route(1, 64, 6, "softmax", train=False)),
        # a training batch whose choice is balanced by a bias and limited to groups
        dict(name="route sigmoid groups", **_route(32768, 256, 8, "sigmoid", bias=True, groups=8,
                                                   keep=4, group_top=2, scale=2.5)),
        # a training batch with 16-bit logits (many ties) and raw softmax weights
        dict(name="route softmax bf16", **_route(16383, 128, 8, "softmax", dtype="bfloat16",
                                                 renorm=False)),
        # one token's experts: each weight is read for a single row
        dict(name="product one token", **_product("product", 8, 128, 2048, 4096, "swiglu")),
        # 64 sequences being answered together, the second product of their experts
        dict(name="product 64 tokens", **_product("product", 384, 64, 2048, 1024, bias=True,
                                                  residual=True)),
        # widths and rows that fill no tile
        dict(name="product odd", **_product("product", 2999, 40, 1009, 1000, "gelu", bias=True)),
        # a long prompt's first product
        dict(name="product prompt", **_product("product", 131072, 128, 2048, 4096, "swiglu")),
        # the gradient back through the second product and the gated activation before it
        dict(name="dgrad activation", **_product("dgrad", 65536, 64, 4096, 1024, "swiglu",
                                                 saved="bfloat16")),
        # weight gradients of many experts with few rows each: their bytes count
        dict(name="wgrad many experts", **_product("wgrad", 32768, 256, 1024, 2048, bias=True)),
        # weight gradients of few experts with many rows each: the products count
        dict(name="wgrad few experts", **_product("wgrad", 16385, 8, 4096, 4096)),
        # a whole training step of the experts, activations kept in 8 bits: a mid layer
        dict(name="step mid", **_step(24576, 64, 2048, 1024, "swiglu", False)),
        # the same of a small layer with biases, at widths that fill no tile
        dict(name="step small", **_step(701, 32, 520, 264, "gelu", True)),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "product", "product", "dgrad", "wgrad", "step"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _between(rng, 8, 512 // groups)
        keep = rng.randint(max(1, (groups + 1) // 2), groups)
        K = rng.randint(1, min(16, keep * (E // groups)))
        T = _between(rng, 1, min(32768, 32768 * 256 // E))
        return _route(T, E, K, rng.choice(["softmax", "sigmoid"]),
                      dtype=rng.choice(["float32", "bfloat16", "float16"]),
                      bias=rng.random() < 0.5, groups=groups, keep=keep,
                      group_top=rng.choice([1, 2]) if groups > 1 else 1,
                      renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                      train=rng.random() < 0.7)
    E = _between(rng, 1, 256)
    wide = 8 * _between(rng, 8, 512)
    most = int(2 ** 31 / E)                     # weights of all experts: 4 GB at most
    narrow = 8 * _between(rng, 8, max(8, min(256, most // wide // 8)))
    R = _between(rng, 1, 32768)
    if op == "step":
        F = max(64, narrow // 2 // 8 * 8)
        wide = 8 * max(8, min(wide // 8, most // (2 * F) // 8))
        return _step(min(R, 24576), E, min(wide, 2048), F,
                     rng.choice(["swiglu", "geglu", "gelu", "relu", "silu"]), rng.random() < 0.5)
    if op == "product":
        act = rng.choice(["none", "swiglu", "geglu", "gelu", "relu", "silu"])
        n = narrow - rng.choice([0, 0, 1, 3]) if act not in ("swiglu", "geglu") else narrow
        return _product(op, R, E, n, wide, act, bias=rng.random() < 0.5,
                        residual=rng.random() < 0.3)
    if op == "dgrad":
        return _product(op, R, E, wide, narrow, rng.choice(["none", "swiglu", "gelu", "silu"]),
                        saved="bfloat16")
    return _product(op, R, E, narrow, wide, bias=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

GATED = ("swiglu", "geglu")


def _rows_of_experts(g, R, E, dev):
    """Where each expert's rows start, the experts drawn with unequal weights
    (every eighth one gets none); a few rows go to experts of their own, as
    one token's do."""
    if R <= E // 2:
        e = torch.randperm(E, generator=g, device=dev)[:R]
    else:
        w = torch.exp(0.3 * torch.randn(E, generator=g, device=dev))
        if E >= 16:
            w[torch.randperm(E, generator=g, device=dev)[:E // 8]] = 0
        e = torch.multinomial(w, R, replacement=True, generator=g)
    counts = torch.bincount(e, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    offsets[1:] = counts.cumsum(0).to(torch.int32)
    return offsets, counts


def _plan(offsets, counts, R):
    """The plan of the plain form: the experts that have rows, and the rows of
    each in a table as long as the longest."""
    experts = counts.nonzero().flatten()
    longest = int(counts.max())
    i = torch.arange(longest, device=counts.device)
    there = i[None, :] < counts[experts][:, None]
    at = (offsets[:-1].long()[experts][:, None] + i[None, :]).clamp(max=R - 1)
    return dict(experts=experts, at=at, there=there, rows=there.flatten().nonzero().flatten())


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    s = dict(case=case)
    if case["op"] == "route":
        T, E, K = case["T"], case["E"], case["K"]
        taste = 0.5 * torch.randn(E, generator=g, device=dev)
        s["logits"] = (torch.randn(T, E, generator=g, device=dev) + taste).to(
            getattr(torch, case["dtype"]))
        s["bias"] = -0.05 * taste + 0.01 * torch.randn(E, generator=g, device=dev) \
            if case["bias"] else None
        s["g_w"] = torch.randn(T, K, generator=g, device=dev) if case["train"] else None
        return s
    R, E = case["R"], case["E"]
    s["offsets"], counts = _rows_of_experts(g, R, E, dev)
    s["plan"] = _plan(s["offsets"], counts, R)
    if case["op"] == "step":
        H, F = case["H"], case["F"]
        two = 2 if case["act"] in GATED else 1
        s["x"] = normal(R, H).requires_grad_()
        s["w1"] = normal(E, two * F, H, std=H ** -0.5).requires_grad_()
        s["w2"] = normal(E, H, F, std=F ** -0.5).requires_grad_()
        s["b1"] = normal(E, two * F, std=0.1).requires_grad_() if case["bias"] else None
        s["b2"] = normal(E, H, std=0.1).requires_grad_() if case["bias"] else None
        s["g_y"] = normal(R, H)
        return s
    n, k, act = case["n"], case["k"], case["act"]
    if case["op"] == "product":
        s["x"] = normal(R, k)
        s["w"] = normal(E, n, k, std=k ** -0.5)
        s["bias"] = normal(E, n, std=0.1) if case["bias"] else None
        s["residual"] = normal(R, n // 2 if act in GATED else n) if case["residual"] else None
    elif case["op"] == "dgrad":
        s["g"] = normal(R, n)
        s["w"] = normal(E, n, k, std=n ** -0.5)
        s["z"] = None if act == "none" else normal(R, 2 * k if act in GATED else k)
    else:
        s["g"] = normal(R, n)
        s["x"] = normal(R, k)
    return s


def work(case):
    """Bytes: each input that the operator needs read once, each output
    written once."""
    if case["op"] == "route":
        T, E, K = case["T"], case["E"], case["K"]
        size = 4 if case["dtype"] == "float32" else 2
        b = T * E * size + T * K * 8
        if case["train"]:
            dense = case["score"] == "softmax" and not case["renorm"]
            b += T * K * 8 + T * E * size + (T * E * size if dense else T * K * size)
        return dict(bytes=b, flops=10 * T * E * (2 if case["train"] else 1))
    R, E = case["R"], case["E"]
    busy = min(R, E)
    if case["op"] == "step":
        H, F = case["H"], case["F"]
        n1 = F * (2 if case["act"] in GATED else 1)
        weights = n1 * H + H * F
        b = 2 * (2 * busy * weights + E * weights) + 2 * R * H * 5 + 2 * R * n1
        return dict(bytes=b, flops=6 * R * weights)
    n, k, act = case["n"], case["k"], case["act"]
    if case["op"] == "product":
        m = n // 2 if act in GATED else n
        b = 2 * (R * k + busy * n * k + R * m * (2 if case["residual"] else 1))
    elif case["op"] == "dgrad":
        z = 0 if act == "none" else 2 * k if act in GATED else k
        b = 2 * (R * n + busy * n * k + R * (2 * z + k if z else k))
    else:
        b = 2 * (R * (n + k) + E * n * k + (E * n if case["bias"] else 0))
    return dict(bytes=b, flops=2 * R * n * k)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    return {"route": _run_route, "product": _run_product, "dgrad": _run_dgrad,
            "wgrad": _run_wgrad, "step": _run_step}[case["op"]](state, case)


def _run_route(s, c):
    how = dict(score=c["score"], renorm=c["renorm"], scale=c["scale"])
    if own:
        import unpermute_routing_indices_gb300 as mp
        idx, w = mp.mp_route(s["logits"], c["K"], bias=s["bias"], n_groups=c["groups"],
                             topk_groups=c["keep"], group_top=c["group_top"], **how)
        if not c["train"]:
            return idx, w
        return idx, w, mp.mp_route_bwd(s["g_w"], s["logits"], idx, **how)
    idx = _choose(s, c)
    z = s["logits"].float()
    at = idx.long()
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-z))
    else:
        e = torch.exp(z - z.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    picked = score.gather(1, at)
    total = picked.sum(1, keepdim=True) if c["renorm"] else 1.0
    p = picked / total
    w = c["scale"] * p
    if not c["train"]:
        return idx, w
    g = c["scale"] * s["g_w"]
    if c["renorm"]:
        g = (g - (g * p).sum(1, keepdim=True)) / total
    if c["score"] == "sigmoid":
        at_picks = g * picked * (1 - picked)
        g_logits = torch.zeros_like(z).scatter_(1, at, at_picks)
    else:
        g_score = torch.zeros_like(z).scatter_(1, at, g)
        g_logits = score * (g_score - (g * picked).sum(1, keepdim=True))
    return idx, w, g_logits.to(s["logits"].dtype)


def _choose(s, c):
    """The experts of each token, in 64 bits: two scores may lie next to each other."""
    z = s["logits"].double()
    T, E = z.shape
    if c["score"] == "sigmoid":
        value = 1 / (1 + torch.exp(-z))
    else:
        e = torch.exp(z - z.amax(1, keepdim=True))
        value = e / e.sum(1, keepdim=True)
    if s["bias"] is not None:
        value = value + s["bias"].double()
    else:
        value = z                               # the scores rise with the logits
    if c["groups"] > 1:
        in_group = value.view(T, c["groups"], -1).sort(2, descending=True).values
        best = in_group[:, :, 0]
        if c["group_top"] == 2:
            if s["bias"] is None:               # sums are of scores, not of logits
                score = 1 / (1 + torch.exp(-z)) if c["score"] == "sigmoid" else \
                    e / e.sum(1, keepdim=True)
                in_group = score.view(T, c["groups"], -1).sort(2, descending=True).values
                best = in_group[:, :, 0]
            best = best + in_group[:, :, 1]
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        mask = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        value = value.masked_fill(~mask.repeat_interleave(E // c["groups"], 1), -math.inf)
    return value.sort(dim=1, descending=True, stable=True).indices[:, :c["K"]].int()


def _act(z, act):
    """act(z) of 32-bit values; gated forms take the gate's columns, then the others."""
    if act in GATED:
        a, b = z.chunk(2, -1)
        return _act(a, "silu" if act == "swiglu" else "gelu") * b
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        t = 1 / (1 + torch.exp(-z))
        return t * (1 + z * (1 - t))
    t = torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * 0.7978845608028654 * (1 + 0.134145 * z * z)


def _act_grad(z, act, g):
    if act in GATED:
        a, b = z.chunk(2, -1)
        inner = "silu" if act == "swiglu" else "gelu"
        return torch.cat([g * b * _act_slope(a, inner), g * _act(a, inner)], -1)
    return g * _act_slope(z, act)


def _table(x, p):
    """Rows of x as [experts with rows, longest, width], zero where there is none."""
    return x[p["at"]].float() * p["there"][:, :, None]


def _untable(t, p):
    return t.flatten(0, 1)[p["rows"]]


def _rows_product(x, w, bias, p):
    """x w[e]^T + b[e] of a table of rows, for the experts that have rows."""
    z = torch.bmm(x, w[p["experts"]].float().transpose(1, 2))
    return z if bias is None else z + bias[p["experts"]].float()[:, None, :]


def _weight_grad(g, x, p, E):
    t = torch.bmm(g.transpose(1, 2), x)
    out = torch.zeros((E, *t.shape[1:]), dtype=torch.bfloat16, device=t.device)
    out[p["experts"]] = t.to(torch.bfloat16)
    return out


def _bias_grad(g, p, E):
    out = torch.zeros((E, g.shape[2]), dtype=torch.bfloat16, device=g.device)
    out[p["experts"]] = g.sum(1).to(torch.bfloat16)
    return out


def _run_product(s, c):
    if own:
        import unpermute_routing_indices_gb300 as mp
        return mp.mp_expert_gemm(s["x"], s["w"], s["offsets"], bias=s["bias"], act=c["act"],
                                 residual=s["residual"])[0]
    p = s["plan"]
    out = _untable(_act(_rows_product(_table(s["x"], p), s["w"], s["bias"], p), c["act"]), p)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return out.to(torch.bfloat16)


def _run_dgrad(s, c):
    if own:
        import unpermute_routing_indices_gb300 as mp
        return [t for t in mp.mp_expert_dgrad(s["g"], s["w"], s["offsets"], act=c["act"],
                                              z=s["z"], with_h=c["act"] != "none")
                if t is not None]
    p = s["plan"]
    g = _untable(torch.bmm(_table(s["g"], p), s["w"][p["experts"]].float()), p)
    if s["z"] is None:
        return [g.to(torch.bfloat16)]
    z = s["z"].float()
    return [_act_grad(z, c["act"], g).to(torch.bfloat16), _act(z, c["act"]).to(torch.bfloat16)]


def _run_wgrad(s, c):
    if own:
        import unpermute_routing_indices_gb300 as mp
        return [t for t in mp.mp_expert_wgrad(s["g"], s["x"], s["offsets"], with_bias=c["bias"])
                if t is not None]
    p, E = s["plan"], c["E"]
    g = _table(s["g"], p)
    out = [_weight_grad(g, _table(s["x"], p), p, E)]
    return out + [_bias_grad(g, p, E)] if c["bias"] else out


def _eight_bits(z):
    """z as an 8-bit checkpoint holds it: e4m3 values times a power of two for
    each BLOCK columns, the smallest that brings the largest to 448 at most."""
    n = z.shape[-1]
    pad = -n % BLOCK
    b = torch.nn.functional.pad(z, (0, pad)).unflatten(-1, (-1, BLOCK))
    big = b.abs().amax(-1, keepdim=True)
    f, e = torch.frexp(big / E4M3_MAX)
    e = torch.where(f == 0.5, e - 1, e).clamp(-126, 127)
    unit = torch.ldexp(torch.ones_like(big), e)
    b = (b / unit).to(torch.float8_e4m3fn).float() * unit
    return b.flatten(-2)[..., :n]


def _run_step(s, c):
    leaves = [t for t in (s["x"], s["w1"], s["w2"], s["b1"], s["b2"]) if t is not None]
    if own:
        from unpermute_routing_indices_gb300 import autograd as ag
        y = ag.expert_mlp(s["x"], s["offsets"], s["w1"], s["w2"], s["b1"], s["b2"],
                          act=c["act"], checkpoint="e4m3")
        return [y, *torch.autograd.grad(y, leaves, s["g_y"])]
    with torch.no_grad():
        p, E, act = s["plan"], c["E"], c["act"]
        x, g = _table(s["x"], p), _table(s["g_y"], p)
        z = _rows_product(x, s["w1"], s["b1"], p)
        y = _rows_product(_act(z, act), s["w2"], s["b2"], p)
        if act in GATED:
            z = torch.cat([_eight_bits(t) for t in z.chunk(2, -1)], -1)
        else:
            z = _eight_bits(z)
        h = _act(z, act) * p["there"][:, :, None]
        g_z = _act_grad(z, act, torch.bmm(g, s["w2"][p["experts"]].float()))
        g_x = torch.bmm(g_z, s["w1"][p["experts"]].float())
        out = [_untable(y, p).to(torch.bfloat16), _untable(g_x, p).to(torch.bfloat16),
               _weight_grad(g_z, x, p, E), _weight_grad(g, h, p, E)]
        if s["b1"] is not None:
            out += [_bias_grad(g_z, p, E), _bias_grad(g, p, E)]
        return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"route": _exact_route, "product": _exact_product, "dgrad": _exact_dgrad,
                "wgrad": _exact_wgrad, "step": _exact_step}[case["op"]](s, case)


def _exact_route(s, c):
    l = s["logits"].double()
    T, E = l.shape
    score = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    by = score if s["bias"] is None else score + s["bias"].double()
    allowed = torch.ones_like(by, dtype=torch.bool)
    if c["groups"] > 1:
        size = E // c["groups"]
        worth = by.view(T, c["groups"], size).topk(c["group_top"], 2).values.sum(2)
        rank = ((worth[:, None, :] > worth[:, :, None]).sum(2))
        rank += torch.tril(worth[:, None, :] == worth[:, :, None], -1).sum(2)
        allowed = (rank < c["keep"])[:, :, None].expand(-1, -1, size).reshape(T, E)
    left = torch.where(allowed, by, -math.inf)
    if s["bias"] is None:
        left = torch.where(allowed, l, -math.inf)
    picks = []
    for _ in range(c["K"]):
        top = left.amax(1, keepdim=True)
        first = (left == top).to(torch.int32).argmax(1, keepdim=True)
        picks.append(first)
        left = left.scatter(1, first, -math.inf)
    at = torch.cat(picks, 1)
    chosen = score.gather(1, at)
    norm = chosen.sum(1, keepdim=True) if c["renorm"] else torch.ones_like(chosen[:, :1])
    w = c["scale"] * chosen / norm
    if not c["train"]:
        return at.int(), w
    u = s["g_w"].double() * c["scale"] / norm
    if c["renorm"]:
        u = u - (u * chosen).sum(1, keepdim=True) / norm
    dense = torch.zeros_like(score).scatter_(1, at, u)
    if c["score"] == "sigmoid":
        g = dense * score * (1 - score)
    else:
        g = score * dense - score * (dense * score).sum(1, keepdim=True)
    return at.int(), w, g


def _segments(s):
    edges = s["offsets"].tolist()
    return [(e, a, b) for e, (a, b) in enumerate(zip(edges, edges[1:])) if b > a]


def _exact_rows(s, x, w, bias=None, turned=False):
    """Each row times its expert's weights, in 64 bits."""
    out = torch.zeros((x.shape[0], w.shape[2] if turned else w.shape[1]), dtype=torch.float64,
                      device=x.device)
    for e, a, b in _segments(s):
        m = w[e].double()
        out[a:b] = x[a:b].double() @ (m if turned else m.T)
        if bias is not None:
            out[a:b] += bias[e].double()
    return out


def _exact_weights(s, g, x, E):
    out = torch.zeros((E, g.shape[1], x.shape[1]), dtype=torch.float64, device=x.device)
    for e, a, b in _segments(s):
        out[e] = g[a:b].double().T @ x[a:b].double()
    return out


def _exact_sums(s, g, E):
    out = torch.zeros((E, g.shape[1]), dtype=torch.float64, device=g.device)
    for e, a, b in _segments(s):
        out[e] = g[a:b].double().sum(0)
    return out


def _exact_h(z, act):
    """(act(z), its derivative) of an ungated activation, in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.relu(z), (z > 0).double()
    if act == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * (1 - q)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return z / 2 * (1 + t), (1 + t) / 2 + z / 2 * (1 - t ** 2) * c * (1 + 3 * 0.044715 * z ** 2)


def _exact_act(z, act, g=None):
    """act(z), and with g its gradient."""
    if act in GATED:
        n = z.shape[1] // 2
        f, df = _exact_h(z[:, :n], "silu" if act == "swiglu" else "gelu")
        h = f * z[:, n:]
        return h if g is None else (h, torch.cat([g * z[:, n:] * df, g * f], 1))
    f, df = _exact_h(z, act)
    return f if g is None else (f, g * df)


def _exact_product(s, c):
    out = _exact_act(_exact_rows(s, s["x"], s["w"], s["bias"]), c["act"])
    return out if s["residual"] is None else out + s["residual"].double()


def _exact_dgrad(s, c):
    g = _exact_rows(s, s["g"], s["w"], turned=True)
    if s["z"] is None:
        return [g]
    h, g_z = _exact_act(s["z"].double(), c["act"], g)
    return [g_z, h]


def _exact_wgrad(s, c):
    out = [_exact_weights(s, s["g"], s["x"], c["E"])]
    return out + [_exact_sums(s, s["g"], c["E"])] if c["bias"] else out


def _exact_e4m3(z):
    """z rounded as an 8-bit checkpoint, by the formula: 3 bits after the
    leading one, exponents from -6, ties to even."""
    out = torch.empty_like(z)
    for a in range(0, z.shape[1], BLOCK):
        b = z[:, a:a + BLOCK]
        big = b.abs().amax(1, keepdim=True)
        unit = 2.0 ** torch.ceil(torch.log2(big.clamp(min=1e-300) / 448)).clamp(-126, 127)
        v = b / unit
        step = 2.0 ** (torch.floor(torch.log2(v.abs().clamp(min=1e-300))).clamp(min=-6) - 3)
        out[:, a:a + BLOCK] = (torch.round(v / step) * step).clamp(-448, 448) * unit
    return out


def _exact_step(s, c):
    act, E = c["act"], c["E"]
    z = _exact_rows(s, s["x"], s["w1"], s["b1"])
    y = _exact_rows(s, _exact_act(z, act), s["w2"], s["b2"])
    n = c["F"]
    z8 = torch.cat([_exact_e4m3(z[:, a:a + n]) for a in range(0, z.shape[1], n)], 1)
    h, g_z = _exact_act(z8, act, _exact_rows(s, s["g_y"], s["w2"], turned=True))
    out = [y, _exact_rows(s, g_z, s["w1"], turned=True), _exact_weights(s, g_z, s["x"], E),
           _exact_weights(s, s["g_y"], h, E)]
    if s["b1"] is not None:
        out += [_exact_sums(s, g_z, E), _exact_sums(s, s["g_y"], E)]
    return out
