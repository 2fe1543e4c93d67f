"""The norms of a block and a whole expert layer in 64 bits, with bounds on what fp32
sums, one rounding of each result and the stated roundings inside may be off by."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24          # half a step of fp32, relative


def half(dtype):
    return torch.finfo(dtype).eps / 2


def terms(H):
    """Roundings that a value passes in fp32 at most: a sum of H values adds up runs of at
    most H/32 of them one after another, then by a tree; and the steps around it."""
    return H / 32 + 40


def rows(T, H, dtype, seed, device="cuda", mean=0.3, std=1.0):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return (torch.randn(T, H, generator=g, device=device) * std + mean).to(dtype)


def make(T, H, dtype, *, kind="rms", post=False, pre=True, residual=True, gate="none", scale=1.0,
         bias=False, seed=0, device="cuda"):
    """Arguments of block_norm (tensors or None) by name, and the plain ones."""
    shape = dict(none=None, channel=(1, H), token=(T, 1), element=(T, H))[gate]
    t = dict(x=rows(T, H, dtype, seed, device),
             residual=rows(T, H, dtype, seed + 1, device, -0.1, 2.0) if residual else None,
             gate=None if shape is None else rows(*shape, dtype, seed + 2, device, 0.5, 0.7),
             post_weight=rows(1, H, dtype, seed + 3, device, 1.0, 0.3)[0] if post else None,
             post_bias=rows(1, H, dtype, seed + 4, device, 0.0, 0.2)[0] if post and bias else None,
             pre_weight=rows(1, H, dtype, seed + 5, device, 1.0, 0.3)[0] if pre else None,
             pre_bias=rows(1, H, dtype, seed + 6, device, 0.0, 0.2)[0] if pre and bias else None)
    if gate == "channel":
        t["gate"] = t["gate"][0]
    return t, dict(kind=kind, scale=scale, eps=1e-5)


def _norm(v, w, b, kind, eps, size):
    """(normed, mean, rstd, size of the result's terms); size: of v's own."""
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    d = v - mean
    rstd = 1 / (d.square().mean(1, keepdim=True) + eps).sqrt()
    out = d * rstd * w
    big = (size + (size.mean(1, keepdim=True) if kind == "layer" else 0)) * rstd * w.abs()
    # an error of the deviation moves every value of the row by its share
    big = big + (d * rstd * w).abs() * (1 + size.mean(1, keepdim=True) * rstd)
    if b is not None:
        out, big = out + b, big + b.abs()
    return out, mean, rstd, big


def forward(t, how):
    """s, y, stats and the sizes of their terms, in 64 bits; differentiable."""
    f = {k: None if v is None else v.double() for k, v in t.items()}
    x = f["x"]
    u, size, zero = x, x.detach().abs(), torch.zeros_like(x[:, :1])
    mean0 = rstd0 = mean1 = rstd1 = zero
    if f["post_weight"] is not None:
        u, mean0, rstd0, size = _norm(x, f["post_weight"], f["post_bias"], how["kind"], how["eps"], size)
    if f["gate"] is not None:
        u, size = u * f["gate"], size * f["gate"].abs()
    s, size = how["scale"] * u, abs(how["scale"]) * size
    if f["residual"] is not None:
        s, size = s + f["residual"], size + f["residual"].abs()
    y = big = None
    if f["pre_weight"] is not None:
        y, mean1, rstd1, big = _norm(s, f["pre_weight"], f["pre_bias"], how["kind"], how["eps"], size)
    return s, y, torch.cat([mean0, rstd0, mean1, rstd1], 1), size, big


def check_forward(t, how, s, y, stats):
    T, H = t["x"].shape
    want_s, want_y, want_stats, size, big = forward(t, how)
    n, r = terms(H) * U32, half(t["x"].dtype)
    within(s, want_s, r * want_s.abs() + n * size)
    if want_y is None:
        assert y is None
    else:
        within(y, want_y, r * want_y.abs() + 2 * n * big)
    if stats is not None:
        sizes = torch.cat([t["x"].double().abs().mean(1, keepdim=True)] * 2 +
                          [size.mean(1, keepdim=True)] * 2, 1)
        # a deviation's relative error: that of the sum, and of its values
        rel = torch.ones_like(sizes)
        rel[:, 1] += sizes[:, 1] * want_stats[:, 1]
        rel[:, 3] += sizes[:, 3] * want_stats[:, 3]
        bound = torch.stack([sizes[:, 0], rel[:, 1] * want_stats[:, 1], sizes[:, 2],
                             rel[:, 3] * want_stats[:, 3]], 1)
        within(stats, want_stats, n * bound)


def _back(g, gsize, v, mean, rstd, w, kind):
    hat = (v - mean) * rstd
    d, dsize = g * w, gsize * w.abs()
    hsize = (v.abs() + mean.abs()) * rstd
    out = d - hat * (d * hat).mean(1, keepdim=True)
    big = dsize + hsize * (dsize * hsize).mean(1, keepdim=True)
    if kind == "layer":
        out, big = out - d.mean(1, keepdim=True), big + dsize.mean(1, keepdim=True)
    return rstd * out, rstd * big, hat, hsize


def backward(t, how, g_s, g_y, s, stats):
    """{name: (gradient, size of its terms, rows summed)} at the given s and stats, in 64 bits."""
    f = {k: None if v is None else v.double() for k, v in t.items()}
    kind, scale, T = how["kind"], how["scale"], t["x"].shape[0]
    mean0, rstd0, mean1, rstd1 = stats.double().split(1, 1)
    x, out = f["x"], {}
    total = torch.zeros_like(x) if g_s is None else g_s.double()
    size = total.abs()
    if f["pre_weight"] is not None:
        g = g_y.double()
        back, big, hat, hsize = _back(g, g.abs(), s.double(), mean1, rstd1, f["pre_weight"], kind)
        total, size = total + back, size + big
        out["pre_weight"] = (g * hat).sum(0), (g.abs() * hsize).sum(0), T
        out["pre_bias"] = g.sum(0), g.abs().sum(0), T
    out["residual"] = total, size, 0
    g, gsize = scale * total, abs(scale) * size
    hat, hsize = (x - mean0) * rstd0, (x.abs() + mean0.abs()) * rstd0
    if f["gate"] is not None:
        u, usize = x, x.abs()
        if f["post_weight"] is not None:
            u, usize = hat * f["post_weight"], hsize * f["post_weight"].abs()
            if f["post_bias"] is not None:
                u, usize = u + f["post_bias"], usize + f["post_bias"].abs()
        gg, gg_size = g * u, gsize * usize
        if f["gate"].dim() == 1:
            out["gate"] = gg.sum(0), gg_size.sum(0), T
        elif f["gate"].shape[1] == 1 and x.shape[1] > 1:
            out["gate"] = gg.sum(1, keepdim=True), gg_size.sum(1, keepdim=True), 0
        else:
            out["gate"] = gg, gg_size, 0
        g, gsize = g * f["gate"], gsize * f["gate"].abs()
    if f["post_weight"] is not None:
        out["post_weight"] = (g * hat).sum(0), (gsize * hsize).sum(0), T
        out["post_bias"] = g.sum(0), gsize.sum(0), T
        g, gsize, _, _ = _back(g, gsize, x, mean0, rstd0, f["post_weight"], kind)
    out["x"] = g, gsize, 0
    return out


NAMES = ("x", "residual", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias")


def check_backward(t, how, g_s, g_y, s, stats, got):
    want = backward(t, how, g_s, g_y, s, stats)
    H = t["x"].shape[1]
    for name, g in zip(NAMES, got):
        if t[name] is None and name != "residual":
            assert g is None, name
            continue
        if g is None:
            continue
        w, size, summed = want[name]
        # fp32 sums over the rows: runs of T/152 of them, then 152 in pairs of fp32
        within(g, w, half(g.dtype) * w.abs() + (2 * terms(H) + summed / 64) * U32 * size, name)


def within(got, want, bound, name=""):
    assert got.shape == want.shape, (name, got.shape, want.shape)
    off = (got.double() - want).abs()
    # Below the smallest normal value a type's steps are as wide as they are there: fp16's
    # 2^-24 under 2^-14, where half a step is more than half an eps of the value.
    info = torch.finfo(got.dtype)
    bad = ~(off <= bound + info.smallest_normal * info.eps / 2)
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(bad.sum())} values out, first at {i}: "
                             f"{got[i].item()} for {want[i].item()}, bound {bound[i].item()}")


# ---------------------------------------------------------------------------
# the whole layer
# ---------------------------------------------------------------------------

def _act(z, act):
    """act(z) and a bound on its slope's magnitude."""
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.sigmoid(1.5957691216057308 * (z + 0.044715 * z ** 3))
    if act == "relu":
        return z.clamp(min=0)
    return z


def layer(x, w1, w2, b1, b2, act, idx, weights, kept=2.0 ** -16):
    """y in 64 bits for the given choice and weights, and how far a result may be off: h off by
    `kept` of it (the nearest bf16 value is off by 2^-8 of it at most, and the rest, kept as
    bf16 too, by 2^-8 of that) and, for the activation, 2^-15, y rounded once, sums in fp32."""
    T, H = x.shape
    F, O = w2.shape[2], w2.shape[1]
    inner = dict(swiglu="silu", geglu="gelu").get(act, act)
    y = torch.zeros(T, O, dtype=torch.float64, device=x.device)
    off = torch.zeros_like(y)
    n1, n2 = (H + 8) * U32, (F + 8) * U32
    for e in idx.unique().tolist():
        if e < 0:
            continue
        t, k = (idx == e).nonzero(as_tuple=True)
        xe, a = x[t].double(), w1[e].double()
        z, size = xe @ a.T, xe.abs() @ a.abs().T
        if b1 is not None:
            z, size = z + b1[e].double(), size + b1[e].double().abs()
        if act in ("swiglu", "geglu"):
            (z, u), (size, usize) = z.chunk(2, 1), size.chunk(2, 1)
            v = _act(z, inner)
            h, d = v * u, 1.2 * n1 * size * u.abs() + n1 * usize * (v.abs() + 1.2 * n1 * size)
        else:
            h, d = _act(z, inner), 1.2 * n1 * size
        d = d + (kept + 2.0 ** -15) * (h.abs() + d) + 2.0 ** -60
        b = w2[e].double()
        out, osize = h @ b.T, d @ b.abs().T + n2 * (h.abs() @ b.abs().T)
        if b2 is not None:
            out, osize = out + b2[e].double(), osize + U32 * b2[e].double().abs()
        w = weights[t, k].double()[:, None]
        y.index_add_(0, t, w * out)
        off.index_add_(0, t, w.abs() * (osize + 40 * U32 * out.abs()))
    return y, 2.0 ** -8 * y.abs() + 1.01 * off


def logits(x, router):
    """fp32 logits as the layer makes them: exact products, summed in 64 bits."""
    return (x.double() @ router.double().T).float()


def choice(l, topk, *, score="softmax", bias=None, n_groups=1, topk_groups=1, group_top=1, renorm=True,
           scale=1.0):
    """idx and weights of fp32 logits in 64 bits, ties to the lowest index."""
    z = l.double()
    T, E = z.shape
    s = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)
    by = z if bias is None else s + bias.double()
    if n_groups > 1:
        top = min(group_top, E // n_groups)
        worth = (s if bias is None and top > 1 else by).view(T, n_groups, -1).sort(
            2, descending=True).values[:, :, :top].sum(2)
        kept = worth.sort(dim=1, descending=True, stable=True).indices[:, :topk_groups]
        mask = torch.zeros(T, n_groups, dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        by = by.masked_fill(~mask.repeat_interleave(E // n_groups, 1), -float("inf"))
    idx = by.sort(dim=1, descending=True, stable=True).indices[:, :topk]
    w = s.gather(1, idx)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    return idx.int(), scale * w
