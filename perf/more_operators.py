"""Cases of a mixture-of-experts block around its experts: the norms before and
after it, fused with its gate, residual and residual scale, their gradients, and the
whole expert layer for a few tokens (router product, choice, experts, combine).

``run`` computes a case in its plain form (elementary torch operations in 32
bits, 64 for the router's logits and choice and for sums over many rows) or, with
``own`` set, through this repository's entry points.  ``exact`` computes it from
the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

GATED = ("swiglu", "geglu")
GATES = ("none", "channel", "token", "element")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm(op, T, H, dtype="bfloat16", kind="rms", post=False, pre=True, residual=True,
          gate="none", scale=1.0, bias=False):
    """A norm before a block (pre), after it (post) or both at once."""
    return dict(op=op, T=T, H=H, dtype=dtype, kind=kind, post=post, pre=pre, residual=residual,
                gate=gate, scale=scale, bias=bias)


def _layer(T, E, K, H, F, act="swiglu", score="softmax", bias=False, groups=1, keep=1,
           group_top=1, renorm=True, scale=1.0, router="bfloat16", biases=False):
    return dict(op="layer", T=T, E=E, K=K, H=H, F=F, act=act, score=score, bias=bias,
                groups=groups, keep=keep, group_top=group_top, renorm=renorm, scale=scale,
                router=router, biases=biases)


def listed():
    return [
        # one token of an answer enters a block: the stream takes the attention's result
        # and is normalised; latency alone
        dict(name="norm one token", **_norm("norm", 1, 4096)),
        # a training batch between two blocks: norm after the one with its gate and scale,
        # residual, norm before the next
        dict(name="norm between blocks", **_norm("norm", 16384, 4096, post=True, gate="channel",
                                                 scale=0.5)),
        # layer norm in 16 bits at a width that fills no vector
        dict(name="norm odd", **_norm("norm", 4099, 1009, "float16", "layer", bias=True)),
        # a training batch's gradient at the norm before a block
        dict(name="norm bwd before", **_norm("norm_bwd", 16384, 4096)),
        # the same at both norms, of the widest layer, gated element by element
        dict(name="norm bwd both", **_norm("norm_bwd", 32768, 7168, post=True, gate="element")),
        # layer norms in 32 bits with a gate for each token
        dict(name="norm bwd fp32", **_norm("norm_bwd", 2047, 2050, "float32", "layer", post=True,
                                           gate="token", bias=True)),
        # one token of an answer through a small layer: latency alone
        dict(name="layer small", **_layer(1, 16, 4, 256, 128, score="sigmoid", bias=True,
                                          router="float32")),
        # one token through a large layer: its experts' weights are read for it alone
        dict(name="layer one token", **_layer(1, 128, 8, 4096, 1024)),
        # eight answers at once, choice limited to groups and evened by a bias
        dict(name="layer groups", **_layer(8, 256, 8, 7168, 512, score="sigmoid", bias=True,
                                           groups=8, keep=4, group_top=2, scale=2.5)),
        # widths that fill no tile, with biases
        dict(name="layer odd", **_layer(13, 40, 3, 1001, 333, "gelu", renorm=False,
                                        router="float32", biases=True)),
        # 64 answers at once: every expert has a few rows
        dict(name="layer 64 tokens", **_layer(64, 64, 6, 2048, 1024)),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "layer"])
    if op != "layer":
        T, H = _between(rng, 1, 32768), _between(rng, 32, 8192)
        if rng.random() < 0.7:
            H = (H + 7) // 8 * 8
        dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
        T = max(1, min(T, 32768 * 7168 * 2 // (H * (4 if dtype == "float32" else 2))))
        post = rng.random() < 0.5
        return _norm(op, T, H, dtype, rng.choice(["rms", "rms", "layer"]), post,
                     not post or rng.random() < 0.6, rng.random() < 0.8, rng.choice(GATES),
                     rng.choice([1.0, 0.22]), rng.random() < 0.5)
    groups = rng.choice([1, 1, 4, 8])
    E = groups * _between(rng, 8 // groups, 256 // groups)
    keep = rng.randint((groups + 1) // 2, groups)
    K = rng.randint(1, min(10, keep * (E // groups)))
    T = _between(rng, 1, 64)
    H = _between(rng, 64, 7168)
    act = rng.choice(["swiglu", "swiglu", "geglu", "gelu", "relu", "silu"])
    parts = 3 if act in GATED else 2
    # weights: 5.6 GB of all experts, 1.3 GB of the picked ones at most
    most = min(2.8e9 / E, 0.65e9 / min(T * K, E)) / (parts * H)
    F = _between(rng, 32, max(32, min(4096, int(most))))
    if rng.random() < 0.8:
        H, F = (H + 7) // 8 * 8, max(32, F // 8 * 8)
    return _layer(T, E, K, H, F, act, rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5,
                  groups, keep, rng.choice([1, 2]) if groups > 1 else 1, rng.random() < 0.7,
                  rng.choice([1.0, 2.5]), rng.choice(["bfloat16", "float32"]),
                  rng.random() < 0.3)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

EPS = {"rms": 1e-6, "layer": 1e-5}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(std).to(dtype)

    s = dict(case=case)
    if case["op"] == "layer":
        T, E, H, F = case["T"], case["E"], case["H"], case["F"]
        P = 2 * F if case["act"] in GATED else F
        s["x"] = normal(T, H)
        s["router"] = normal(E, H, std=H ** -0.5, dtype=getattr(torch, case["router"]))
        s["bias"] = normal(E, std=0.02, dtype=torch.float32) if case["bias"] else None
        s["w1"], s["w2"] = normal(E, P, H, std=H ** -0.5), normal(E, H, F, std=F ** -0.5)
        s["b1"] = normal(E, P, std=0.1) if case["biases"] else None
        s["b2"] = normal(E, H, std=0.1) if case["biases"] else None
        if own:
            import unpermute_routing_indices_gb300 as mp
            s["workspace"] = torch.empty(mp.mp_moe_layer_workspace_size(T, E, case["K"], H, F, H),
                                         dtype=torch.uint8, device=dev)
        return s
    T, H, dt = case["T"], case["H"], getattr(torch, case["dtype"])
    # a stream with a few strong channels and means away from zero, as deep layers have
    strong = torch.ones(H, device=dev)
    strong[torch.randperm(H, generator=g, device=dev)[:max(1, H // 256)]] = 12.0
    s["x"] = (normal(T, H, dtype=torch.float32) * strong + 0.2).to(dt)
    s["residual"] = normal(T, H, std=2.0, dtype=dt) if case["residual"] else None
    shape = dict(none=None, channel=(H,), token=(T, 1), element=(T, H))[case["gate"]]
    s["gate"] = None if shape is None else \
        torch.sigmoid(normal(*shape, dtype=torch.float32)).to(dt)
    for name in ("post", "pre"):
        s[name + "_weight"] = (1 + normal(H, std=0.2, dtype=torch.float32)).to(dt) \
            if case[name] else None
        s[name + "_bias"] = normal(H, std=0.1, dtype=dt) if case[name] and case["bias"] else None
    if case["op"] == "norm_bwd":
        # what the pass forward left: the stream, and each row's mean and 1 / deviation
        stream, _, stats = _norm_forward(s, case, torch.float32)
        s["stream"], s["stats"] = stream.to(dt), stats
        s["residual"] = None                       # the stream holds it
        s["g_stream"] = normal(T, H, dtype=dt)
        s["g_out"] = normal(T, H, dtype=dt) if case["pre"] else None
    return s


def work(case):
    """Bytes: each input that the operator needs read once, each output
    written once."""
    if case["op"] == "layer":
        T, E, K, H, F = (case[k] for k in ("T", "E", "K", "H", "F"))
        weights = H * F * (3 if case["act"] in GATED else 2)
        # of E experts, this many are picked by T tokens on average
        busy = E * (1 - (1 - K / E) ** T)
        size = 2 if case["router"] == "bfloat16" else 4
        return dict(bytes=int(2 * busy * weights + size * E * H + 4 * T * H + 8 * T * K),
                    flops=2 * T * K * weights + 2 * T * E * H)
    T, H = case["T"], case["H"]
    size = 4 if case["dtype"] == "float32" else 2
    gate = dict(none=0, channel=H, token=T, element=T * H)[case["gate"]]
    vectors = (case["post"] + case["pre"]) * H * (2 if case["bias"] else 1)
    plain = not (case["residual"] or case["post"] or case["gate"] != "none" or case["scale"] != 1.0)
    if case["op"] == "norm":
        # the stream is an output of its own unless it is x itself
        rows = 1 + case["residual"] + (not plain) + case["pre"]
        return dict(bytes=size * (rows * T * H + gate + vectors) + 16 * T, flops=12 * T * H)
    rows = (case["post"] or case["gate"] != "none") + 2 * case["pre"] + 1   # x; stream, g_out; g_stream
    rows += 1 + (case["post"] or case["gate"] != "none" or case["scale"] != 1.0)   # g_residual; g_x
    return dict(bytes=size * (rows * T * H + 2 * gate + 2 * vectors) + 16 * T, flops=25 * T * H)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    return _there({"layer": _run_layer, "norm": _run_norm, "norm_bwd": _run_norm_bwd}[case["op"]](state, case))


def _there(outputs):
    """Without the outputs that the case does not have."""
    return [t for t in outputs if t is not None]


def _moments(v, kind, eps):
    """Each row's mean (0 for rms) and 1 / sqrt(mean square + eps) around it."""
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    d = v - mean
    return mean, 1 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)


def _norm_forward(s, c, to):
    """(stream, result of the norm before the next block or None, stats), in `to`."""
    u = s["x"].to(to)
    T = u.shape[0]
    stats = torch.zeros(T, 4, dtype=to, device=u.device)
    if c["post"]:
        mean, rstd = _moments(u, c["kind"], EPS[c["kind"]])
        stats[:, 0:1], stats[:, 1:2] = mean, rstd
        u = (u - mean) * rstd * s["post_weight"].to(to)
        if s["post_bias"] is not None:
            u = u + s["post_bias"].to(to)
    if s["gate"] is not None:
        u = u * s["gate"].to(to)
    stream = c["scale"] * u
    if s["residual"] is not None:
        stream = stream + s["residual"].to(to)
    out = None
    if c["pre"]:
        mean, rstd = _moments(stream, c["kind"], EPS[c["kind"]])
        stats[:, 2:3], stats[:, 3:4] = mean, rstd
        out = (stream - mean) * rstd * s["pre_weight"].to(to)
        if s["pre_bias"] is not None:
            out = out + s["pre_bias"].to(to)
    return stream, out, stats


def _run_norm(s, c):
    if own:
        import unpermute_routing_indices_gb300 as mp
        return list(mp.mp_block_norm(
            s["x"], s["residual"], post_weight=s["post_weight"], post_bias=s["post_bias"],
            gate=s["gate"], scale=c["scale"], pre_weight=s["pre_weight"], pre_bias=s["pre_bias"],
            kind=c["kind"], eps=EPS[c["kind"]], with_stats=True))
    stream, out, stats = _norm_forward(s, c, torch.float32)
    dt = s["x"].dtype
    return [stream.to(dt), None if out is None else out.to(dt), stats]


def _run_norm_bwd(s, c):
    """(g_x, g_residual, g_gate, g_post_weight, g_post_bias, g_pre_weight, g_pre_bias)"""
    if own:
        import unpermute_routing_indices_gb300 as mp
        return list(mp.mp_block_norm_bwd(
            s["g_stream"], s["g_out"], s["x"], s["stream"], s["stats"],
            post_weight=s["post_weight"], post_bias=s["post_bias"], gate=s["gate"],
            scale=c["scale"], pre_weight=s["pre_weight"], pre_bias=s["pre_bias"], kind=c["kind"]))
    dt, layer = s["x"].dtype, c["kind"] == "layer"
    mean0, rstd0, mean1, rstd1 = s["stats"].split(1, 1)
    total = s["g_stream"].float()
    g_gate = g_post_w = g_post_b = g_pre_w = g_pre_b = None

    def over_rows(t):
        return t.sum(0, dtype=torch.float64).to(dt)

    if c["pre"]:
        hat, g = (s["stream"].float() - mean1) * rstd1, s["g_out"].float()
        g_pre_w = over_rows(g * hat)
        g_pre_b = over_rows(g) if s["pre_bias"] is not None else None
        d = g * s["pre_weight"].float()
        back = d - hat * (d * hat).mean(1, keepdim=True)
        if layer:
            back = back - d.mean(1, keepdim=True)
        total = total + rstd1 * back
    g_residual = total.to(dt)
    g = c["scale"] * total
    x = s["x"].float()
    hat = (x - mean0) * rstd0 if c["post"] else None
    if s["gate"] is not None:
        u = x
        if c["post"]:
            u = hat * s["post_weight"].float()
            if s["post_bias"] is not None:
                u = u + s["post_bias"].float()
        g_gate = g * u
        g_gate = {"channel": over_rows, "element": lambda t: t.to(dt),
                  "token": lambda t: t.sum(1, keepdim=True).to(dt)}[c["gate"]](g_gate)
        g = g * s["gate"].float()
    if c["post"]:
        g_post_w = over_rows(g * hat)
        g_post_b = over_rows(g) if s["post_bias"] is not None else None
        d = g * s["post_weight"].float()
        back = d - hat * (d * hat).mean(1, keepdim=True)
        if layer:
            back = back - d.mean(1, keepdim=True)
        g = rstd0 * back
    return [g.to(dt), g_residual, g_gate, g_post_w, g_post_b, g_pre_w, g_pre_b]


def _act(z, act):
    """act(z) of 32-bit values; gated forms take the gate's columns, then the others."""
    if act in GATED:
        a, b = z.chunk(2, -1)
        return _act(a, "silu" if act == "swiglu" else "gelu") * b
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return 0.5 * z * (1 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))


def _choose(logits, bias, c):
    """The experts of each token, in 64 bits: two scores may lie next to each other."""
    z = logits.double()
    T, E = z.shape
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-z))
    else:
        e = torch.exp(z - z.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    value = z if bias is None else score + bias.double()   # the scores rise with the logits
    if c["groups"] > 1:
        top = min(c["group_top"], E // c["groups"])
        by = value if bias is not None or top == 1 else score
        best = by.view(T, c["groups"], -1).sort(2, descending=True).values
        worth = best[:, :, 0] if top == 1 else best[:, :, 0] + best[:, :, 1]
        kept = worth.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        mask = torch.zeros_like(worth, dtype=torch.bool).scatter_(1, kept, True)
        value = value.masked_fill(~mask.repeat_interleave(E // c["groups"], 1), -math.inf)
    return value.sort(dim=1, descending=True, stable=True).indices[:, :c["K"]]


def _run_layer(s, c):
    """(y, idx, weights)"""
    if own:
        import unpermute_routing_indices_gb300 as mp
        return list(mp.mp_moe_layer(
            s["x"], s["router"], s["w1"], s["w2"], c["K"], b1=s["b1"], b2=s["b2"], act=c["act"],
            score=c["score"], bias=s["bias"], n_groups=c["groups"], topk_groups=c["keep"],
            group_top=c["group_top"], renorm=c["renorm"], scale=c["scale"],
            workspace=s["workspace"]))
    T, E, K = c["T"], c["E"], c["K"]
    logits = (s["x"].double() @ s["router"].double().T).float()
    at = _choose(logits, s["bias"], c)
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
    else:
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    picked = score.gather(1, at)
    weights = c["scale"] * (picked / picked.sum(1, keepdim=True) if c["renorm"] else picked)
    x = s["x"].float()
    if T * K <= E // 4:
        # few routes: the weights of each
        e = at.flatten()
        rows = x.repeat_interleave(K, 0)
        z = torch.bmm(s["w1"][e].float(), rows[:, :, None])[:, :, 0]
        if s["b1"] is not None:
            z = z + s["b1"][e].float()
        y = torch.bmm(s["w2"][e].float(), _act(z, c["act"])[:, :, None])[:, :, 0]
        if s["b2"] is not None:
            y = y + s["b2"][e].float()
        y = (weights.flatten()[:, None] * y).view(T, K, -1).sum(1)
        return [y.to(torch.bfloat16), at.int(), weights]
    # every token through every expert, a batch of experts at a time
    spread = torch.zeros(T, E, device=x.device).scatter_(1, at, weights)
    y = torch.zeros(T, s["w2"].shape[1], device=x.device)
    step = max(1, int(1e9) // (s["w1"].shape[1] * s["w1"].shape[2]))
    for i in range(0, E, step):
        w1, w2 = s["w1"][i:i + step].float(), s["w2"][i:i + step].float()
        z = torch.matmul(x, w1.transpose(1, 2))
        if s["b1"] is not None:
            z = z + s["b1"][i:i + step].float()[:, None, :]
        out = torch.bmm(_act(z, c["act"]), w2.transpose(1, 2))
        if s["b2"] is not None:
            out = out + s["b2"][i:i + step].float()[:, None, :]
        y = y + (spread[:, i:i + step].T[:, :, None] * out).sum(0)
    return [y.to(torch.bfloat16), at.int(), weights]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return _there({"layer": _exact_layer, "norm": _exact_norm, "norm_bwd": _exact_norm_bwd}[case["op"]](s, case))


def _standard(v, kind, eps):
    """(values off their mean, mean [T], 1 / deviation [T])"""
    m = v.sum(1) / v.shape[1] if kind == "layer" else v.new_zeros(v.shape[0])
    v = v - m[:, None]
    return v, m, (v.square().sum(1) / v.shape[1] + eps).rsqrt()


def _exact_norm(s, c):
    f = {k: v.double() if torch.is_tensor(v) else v for k, v in s.items()}
    kind, eps = c["kind"], EPS[c["kind"]]
    zero = torch.zeros(c["T"], dtype=torch.float64, device=s["x"].device)
    stats, u = [zero] * 4, f["x"]
    if c["post"]:
        d, stats[0], stats[1] = _standard(u, kind, eps)
        u = torch.einsum("th,t,h->th", d, stats[1], f["post_weight"])
        if f["post_bias"] is not None:
            u += f["post_bias"]
    u = u * c["scale"] * (1.0 if f["gate"] is None else f["gate"])
    if f["residual"] is not None:
        u = u + f["residual"]
    out = None
    if c["pre"]:
        d, stats[2], stats[3] = _standard(u, kind, eps)
        out = torch.einsum("th,t,h->th", d, stats[3], f["pre_weight"])
        if f["pre_bias"] is not None:
            out += f["pre_bias"]
    return [u, out, torch.stack(stats, 1)]


def _exact_back(g, v, mean, rstd, w, kind):
    """(gradient of the norm's input, g times the normalised value) at the given statistics."""
    n = v.shape[1]
    hat = (v - mean[:, None]) * rstd[:, None]
    d = g * w
    along = torch.einsum("th,th->t", d, hat) / n
    flat = d.sum(1) / n if kind == "layer" else torch.zeros_like(along)
    return (d - flat[:, None] - hat * along[:, None]) * rstd[:, None], g * hat, hat


def _exact_norm_bwd(s, c):
    f = {k: v.double() if torch.is_tensor(v) else v for k, v in s.items()}
    st, total = f["stats"], f["g_stream"]
    pw = pb = qw = qb = gate = None
    if c["pre"]:
        back, gh, _ = _exact_back(f["g_out"], f["stream"], st[:, 2], st[:, 3], f["pre_weight"], c["kind"])
        qw, total = gh.sum(0), total + back
        if f["pre_bias"] is not None:
            qb = f["g_out"].sum(0)
    g = total * c["scale"]
    u = f["x"]
    if c["post"]:
        u = (u - st[:, 0:1]) * st[:, 1:2] * f["post_weight"]
        if f["post_bias"] is not None:
            u = u + f["post_bias"]
    if f["gate"] is not None:
        gate = g * u
        if c["gate"] == "channel":
            gate = gate.sum(0)
        elif c["gate"] == "token":
            gate = gate.sum(1, keepdim=True)
        g = g * f["gate"]
    if c["post"]:
        if f["post_bias"] is not None:
            pb = g.sum(0)
        g, gh, _ = _exact_back(g, f["x"], st[:, 0], st[:, 1], f["post_weight"], c["kind"])
        pw = gh.sum(0)
    return [g, total, gate, pw, pb, qw, qb]


def _exact_layer(s, c):
    T, E, K, act = c["T"], c["E"], c["K"], c["act"]
    l = torch.einsum("th,eh->te", s["x"].double(), s["router"].double()).float().double()
    score = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    by = l if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        size = E // c["groups"]
        top = min(c["group_top"], size)
        worth = (score if s["bias"] is None and top > 1 else by).view(T, c["groups"], size)
        worth = worth.topk(top, 2).values.sum(2)
        rank = (worth[:, None, :] > worth[:, :, None]).sum(2)
        rank += torch.tril(worth[:, None, :] == worth[:, :, None], -1).sum(2)
        by = torch.where((rank < c["keep"])[:, :, None].expand(-1, -1, size).reshape(T, E), by, -math.inf)
    picks = []
    for _ in range(K):
        first = (by == by.amax(1, keepdim=True)).to(torch.int32).argmax(1, keepdim=True)
        picks.append(first)
        by = by.scatter(1, first, -math.inf)
    at = torch.cat(picks, 1)
    w = score.gather(1, at) * c["scale"]
    if c["renorm"]:
        w = w / score.gather(1, at).sum(1, keepdim=True)
    y = torch.zeros(T, s["w2"].shape[1], dtype=torch.float64, device=l.device)
    for e in at.unique().tolist():
        t, k = (at == e).nonzero(as_tuple=True)
        z = s["x"][t].double() @ s["w1"][e].double().T
        if s["b1"] is not None:
            z = z + s["b1"][e].double()
        a, b = z.chunk(2, 1) if act in GATED else (z, 1.0)
        if act in ("swiglu", "silu"):
            h = a * torch.sigmoid(a) * b
        elif act == "relu":
            h = a.relu()
        else:
            h = a * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)) * b
        out = h @ s["w2"][e].double().T
        if s["b2"] is not None:
            out = out + s["b2"][e].double()
        y.index_add_(0, t, w[t, k][:, None] * out)
    return [y, at, w]
