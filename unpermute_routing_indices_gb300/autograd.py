"""Differentiable forms of the dispatch / combine path for a training step.

Each function is a ``torch.autograd.Function`` whose forward and backward are
calls of the C-ABI binding (every value is computed by the library's CUDA
kernels).  The operations and their gradients are those of the pages:
``moe_permute_with_probs`` / ``moe_unpermute_mask`` ("d9d 0.1.0 —
d9d/kernel/moe/permute_with_probs.py"), the batch-invariant ``unpermute`` and
its rank-partial form ("core.transformer.moe.batch_invariant"), the fused
chunk sort + pad and its restore ("[PyTorch] Fuse MoE chunk sorting and
padding"), and the top-K softmax router ("moe-ops 0.1.0", Operators).

    idx, probs = topk_softmax(logits, 8)
    rows, rows_probs, d = permute(x, idx, num_experts, probs)
    ...  expert computation on rows (d.routed_rows() rows are routed)  ...
    y = unpermute(expert_out, d, probs)

Rows of the permuted buffer past the routed count (empty slots, routes
dropped by a capacity) are zero in the forward output and get zero gradient,
so a computation over the whole buffer stays finite.  Rows of a restored
tensor that no chunk names (past the sum of the split sizes) are zero too.

Gradients are of first order: one taken with create_graph may be used, but
differentiating it again raises.
"""
from __future__ import annotations

import functools
from dataclasses import dataclass

import torch

from . import (mp_block_norm, mp_block_norm_bwd, mp_build_map, mp_build_map_capacity,
               mp_expert_mlp, mp_expert_mlp_bwd, mp_permute, mp_permute_bwd, mp_route, mp_route_bwd,
               mp_sort_chunks_pad, mp_sort_chunks_pad_bwd, mp_topk_softmax,
               mp_topk_softmax_bwd, mp_unpad_restore, mp_unpad_restore_bwd, mp_unpermute,
               mp_unpermute_bwd, mp_unpermute_ep, mp_zero_rows_from)

__all__ = ["Dispatch", "block_norm", "topk_softmax", "route", "permute", "expert_mlp", "unpermute",
           "unpermute_ep", "sort_chunks_pad", "unpad_restore"]


@dataclass
class Dispatch:
    """The routing map of one batch.

    row_id_map [T,K]: the permuted row of slot (t,k), -1 if none;
    sorted_to_flat [rows]: the slot t*K+k of each routed row;
    counts [E] / offsets [E+1]: rows per expert and where each expert's rows
    start (offsets[E] = routed rows); idx [T,K]: the experts; num_rows: rows
    of the permuted buffer."""

    row_id_map: torch.Tensor
    sorted_to_flat: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    idx: torch.Tensor
    num_experts: int
    num_rows: int

    def routed_rows(self) -> torch.Tensor:
        """The routed row count, a one-element device tensor."""
        return self.offsets[-1:]


class _Final(torch.autograd.Function):
    """The gradients given, as results of `on` that cannot be differentiated again."""

    @staticmethod
    def forward(ctx, name, count, *tensors):
        ctx.name = name
        return tuple(t.detach() for t in tensors[:count])

    @staticmethod
    def backward(ctx, *g):
        raise RuntimeError(f"{ctx.name}: gradients of gradients are not implemented")


def _first_order(backward):
    """A backward pass whose results cannot be differentiated again.  Where a graph of it
    is asked for (create_graph), they depend on what they are computed from, the
    gradients given and the tensors kept, by a node that refuses: without it their
    second derivatives would be left out of a sum without a word."""
    @functools.wraps(backward)
    def checked(ctx, *grads):
        results = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return results
        on = [t for t in (*grads, *ctx.saved_tensors) if t is not None and t.requires_grad]
        made = [t for t in results if t is not None]
        if not on or not made:
            return results
        final = iter(_Final.apply(backward.__qualname__.split(".")[0].strip("_"), len(made), *made, *on))
        return tuple(None if t is None else next(final) for t in results)
    return checked


class _Permute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, probs, row_id_map, routed, num_rows):
        out, out_probs = mp_permute(x, row_id_map, probs, num_out_rows=num_rows)
        mp_zero_rows_from(out, routed)
        if out_probs is not None:
            mp_zero_rows_from(out_probs, routed)
        ctx.save_for_backward(row_id_map)
        ctx.has_probs = probs is not None
        return out, out_probs

    @staticmethod
    @_first_order
    def backward(ctx, g_out, g_out_probs):
        (row_id_map,) = ctx.saved_tensors
        gp = None
        if ctx.has_probs and ctx.needs_input_grad[1]:
            gp = torch.zeros(g_out.shape[0], dtype=torch.float32, device=g_out.device) \
                if g_out_probs is None else g_out_probs.contiguous()
        g_x, g_probs = mp_permute_bwd(g_out.contiguous(), row_id_map, gp)
        return g_x, g_probs, None, None, None


class _Unpermute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, probs, row_id_map, routed, ep):
        if ep is None:
            y = mp_unpermute(rows, row_id_map, probs)
        else:
            idx, E, ep_size, bf16p, fp64 = ep
            y = mp_unpermute_ep(rows, row_id_map, idx, E, ep_size, probs, bf16_partials=bf16p,
                                fp64_cross_rank=fp64)
        ctx.save_for_backward(rows if probs is not None else None, probs, row_id_map, routed)
        ctx.num_rows = rows.shape[0]
        return y

    @staticmethod
    @_first_order
    def backward(ctx, g_y):
        rows, probs, row_id_map, routed = ctx.saved_tensors
        g_rows, g_probs = mp_unpermute_bwd(g_y.contiguous(), row_id_map, rows, probs,
                                           num_out_rows=ctx.num_rows)
        mp_zero_rows_from(g_rows, routed)
        return g_rows, g_probs, None, None, None


class _TopkSoftmax(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, topk, n_groups, topk_groups):
        idx, probs = mp_topk_softmax(logits, topk, n_groups=n_groups, topk_groups=topk_groups)
        ctx.mark_non_differentiable(idx)
        ctx.save_for_backward(probs, idx)
        ctx.num_experts = logits.shape[1]
        return idx, probs

    @staticmethod
    @_first_order
    def backward(ctx, g_idx, g_probs):
        probs, idx = ctx.saved_tensors
        g = mp_topk_softmax_bwd(g_probs.contiguous(), probs, idx, ctx.num_experts)
        return g, None, None, None


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias, topk, choice, how):
        idx, weights = mp_route(logits, topk, bias=bias, **choice, **how)
        ctx.mark_non_differentiable(idx)
        ctx.save_for_backward(logits, idx)
        ctx.how = how
        return idx, weights

    @staticmethod
    @_first_order
    def backward(ctx, g_idx, g_weights):
        logits, idx = ctx.saved_tensors
        return mp_route_bwd(g_weights.contiguous(), logits, idx, **ctx.how), None, None, None, None


class _ExpertMlp(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, offsets, w1, w2, b1, b2, act, checkpoint, status):
        y, z, z_exp = mp_expert_mlp(rows, w1, w2, offsets, b1, b2, act=act, save=checkpoint,
                                    status=status)
        ctx.save_for_backward(rows, offsets, w1, w2, z, z_exp)
        ctx.act, ctx.status = act, status
        return y

    @staticmethod
    @_first_order
    def backward(ctx, g_y):
        rows, offsets, w1, w2, z, z_exp = ctx.saved_tensors
        need = ctx.needs_input_grad
        g_x, g_w1, g_w2, g_b1, g_b2 = mp_expert_mlp_bwd(
            g_y.contiguous(), rows, w1, w2, offsets, z, z_exp, act=ctx.act,
            need=(need[0], need[2], need[3], need[4], need[5]), status=ctx.status)
        return g_x, None, g_w1, g_w2, g_b1, g_b2, None, None, None


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gate, post_weight, post_bias, pre_weight, pre_bias, kind, eps, scale,
                keep, status):
        s, y, stats = mp_block_norm(x, residual, post_weight=post_weight, post_bias=post_bias,
                                    gate=gate, scale=scale, pre_weight=pre_weight,
                                    pre_bias=pre_bias, kind=kind, eps=eps, with_stats=keep,
                                    status=status)
        ctx.set_materialize_grads(False)
        ctx.has_stream = s is not x
        if keep:
            ctx.save_for_backward(x if post_weight is not None or gate is not None else None,
                                  s if pre_weight is not None else None, stats, gate, post_weight,
                                  post_bias, pre_weight, pre_bias)
            ctx.kind, ctx.scale, ctx.status = kind, scale, status
        return (s if ctx.has_stream else None), y

    @staticmethod
    @_first_order
    def backward(ctx, g_s, g_y):
        x, s, stats, gate, post_weight, post_bias, pre_weight, pre_bias = ctx.saved_tensors
        if g_s is None and g_y is None:
            return (None,) * 12
        if pre_weight is not None and g_y is None:
            g_y = torch.zeros_like(s)
        g = mp_block_norm_bwd(
            None if g_s is None else g_s.contiguous(), None if g_y is None else g_y.contiguous(),
            x, s, stats, post_weight=post_weight, post_bias=post_bias, gate=gate, scale=ctx.scale,
            pre_weight=pre_weight, pre_bias=pre_bias, kind=ctx.kind, need=ctx.needs_input_grad[:7],
            status=ctx.status)
        return *g, None, None, None, None, None


class _SortChunksPad(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, probs, split_sizes, chunk_order, num_groups, align, out_rows,
                padded_sizes):
        out, out_probs, row_map, group_off = mp_sort_chunks_pad(
            x, split_sizes, chunk_order, num_groups, align, out_rows, probs,
            padded_sizes=padded_sizes)
        ctx.mark_non_differentiable(row_map, group_off)
        ctx.save_for_backward(row_map)
        ctx.num_rows = x.shape[0]
        ctx.has_probs = probs is not None
        return out, out_probs, row_map, group_off

    @staticmethod
    @_first_order
    def backward(ctx, g_out, g_out_probs, g_row_map, g_group_off):
        (row_map,) = ctx.saved_tensors
        g_x = torch.zeros((ctx.num_rows, g_out.shape[1]), dtype=g_out.dtype,
                          device=g_out.device)
        gp = g_pr = None
        if ctx.has_probs and ctx.needs_input_grad[1]:
            gp = torch.zeros(g_out.shape[0], dtype=torch.float32, device=g_out.device) \
                if g_out_probs is None else g_out_probs.contiguous()
            g_pr = torch.zeros(ctx.num_rows, dtype=torch.float32, device=g_out.device)
        mp_sort_chunks_pad_bwd(g_out.contiguous(), row_map, ctx.num_rows, gp, g_x=g_x,
                               g_probs=g_pr)
        return g_x, g_pr, None, None, None, None, None, None


class _UnpadRestore(torch.autograd.Function):
    @staticmethod
    def forward(ctx, padded, padded_probs, row_map, num_rows):
        y = torch.zeros((num_rows, padded.shape[1]), dtype=padded.dtype, device=padded.device)
        y_probs = None if padded_probs is None else \
            torch.zeros(num_rows, dtype=torch.float32, device=padded.device)
        mp_unpad_restore(padded, row_map, num_rows, padded_probs, y=y, y_probs=y_probs)
        ctx.save_for_backward(row_map)
        ctx.has_probs = padded_probs is not None
        return y, y_probs

    @staticmethod
    @_first_order
    def backward(ctx, g_y, g_y_probs):
        (row_map,) = ctx.saved_tensors
        gp = None
        if ctx.has_probs and ctx.needs_input_grad[1]:
            gp = torch.zeros(g_y.shape[0], dtype=torch.float32, device=g_y.device) \
                if g_y_probs is None else g_y_probs.contiguous()
        g_padded, g_padded_probs = mp_unpad_restore_bwd(g_y.contiguous(), row_map, gp)
        return g_padded, g_padded_probs, None, None


def topk_softmax(logits: torch.Tensor, topk: int, n_groups: int = 1, topk_groups: int = 1):
    """fp32 logits [T,E] -> (idx int32 [T,K], probs fp32 [T,K]); probs is
    differentiable w.r.t. the logits (softmax over the K picks)."""
    return _TopkSoftmax.apply(logits, int(topk), int(n_groups), int(topk_groups))


def route(logits: torch.Tensor, topk: int, *, score: str = "softmax", bias=None,
          n_groups: int = 1, topk_groups: int = 1, group_top: int = 1, renorm: bool = True,
          scale: float = 1.0):
    """logits [T,E] (fp32, bf16, fp16) -> (idx int32 [T,K], weights fp32 [T,K]);
    the weights are differentiable w.r.t. the logits.  `bias` (fp32 [E], no
    gradient) moves the choice only.  Empty slots are -1 with weight 0."""
    return _Route.apply(logits, bias, int(topk),
                        dict(n_groups=n_groups, topk_groups=topk_groups, group_top=group_top),
                        dict(score=score, renorm=renorm, scale=scale))


def block_norm(x: torch.Tensor, residual=None, *, post_weight=None, post_bias=None, gate=None,
               scale: float = 1.0, pre_weight=None, pre_bias=None, kind: str = "rms",
               eps: float = 1e-6, status=None):
    """The norm after a block and the one before the next, with gate, residual scale and
    residual between them (mp_block_norm): x [T,H] -> (s, y),

        u = norm(x) * post_weight + post_bias  (x without a post_weight)
        s = residual + scale * gate * u
        y = norm(s) * pre_weight + pre_bias    (None without a pre_weight)

    differentiable w.r.t. x, residual, gate ([H], [T,1] or [T,H]), weights and biases.
    For the backward pass x, s and four fp32 values a row are kept.  `status` (int32 [1])
    gets "stalled" where results of either pass are invalid."""
    tensors = (x, residual, gate, post_weight, post_bias, pre_weight, pre_bias)
    keep = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)
    s, y = _BlockNorm.apply(*tensors, kind, float(eps), float(scale), keep, status)
    return (x if s is None else s), y


def expert_mlp(rows: torch.Tensor, offsets, w1: torch.Tensor, w2: torch.Tensor, b1=None,
               b2=None, *, act: str = "swiglu", checkpoint: str = "bf16",
               status=None) -> torch.Tensor:
    """The experts on rows in expert order: act(rows w1[e]^T + b1[e]) w2[e]^T + b2[e].

    rows bf16 [R,H]; `offsets` int32 [E+1], or the Dispatch that permute gave;
    w1 bf16 [E,F,H] ([E,2F,H] for geglu and swiglu, gate first), w2 bf16
    [E,H',F].  For the backward pass the product before the activation is kept
    as bf16, or in 8 bits where the caller asks for it (checkpoint="e4m3", 4
    significant bits and a power of two per 32 columns, 9/16 of the bytes),
    and the activation's result is computed from it again; its gradients are
    those at the kept values.  Rows that no expert has (before offsets[0], from
    offsets[E] on) are zero in the result and in the gradient.
    `status` (int32 [1]) gets the bits of both passes, to be read when the
    caller synchronises: "bad_offsets", and "stalled", which says that results
    are invalid (status_bits)."""
    if act not in ("relu", "gelu", "silu", "geglu", "swiglu"):
        raise ValueError(f"expert_mlp needs an activation, got {act!r}")
    if checkpoint not in ("e4m3", "bf16"):
        raise ValueError(f"checkpoint must be e4m3 or bf16, got {checkpoint!r}")
    if isinstance(offsets, Dispatch):
        offsets = offsets.offsets
    # Nothing is kept where no backward pass can follow.  (Inside forward(), grad mode is
    # off and needs_input_grad says what the inputs require whatever the mode was.)
    if not (torch.is_grad_enabled() and
            any(t is not None and t.requires_grad for t in (rows, w1, w2, b1, b2))):
        checkpoint = "none"
    return _ExpertMlp.apply(rows, offsets, w1, w2, b1, b2, act, checkpoint, status)


def permute(x: torch.Tensor, idx: torch.Tensor, num_experts: int, probs=None, *,
            capacity: int | None = None):
    """bf16 x [T,H], int32 idx [T,K] (-1 = empty slot) -> (rows bf16 [R,H],
    rows_probs fp32 [R] or None, Dispatch).  R = T*K, or min(T*K, E*capacity)
    when each expert keeps at most `capacity` routes (the earliest)."""
    T, K = idx.shape
    if capacity is None:
        rim, s2f, counts, offsets = mp_build_map(idx, num_experts)
        R = T * K
    else:
        rim, s2f, counts, offsets = mp_build_map_capacity(idx, num_experts, capacity)
        R = min(T * K, num_experts * int(capacity))
    d = Dispatch(rim, s2f, counts, offsets, idx, int(num_experts), R)
    rows, rows_probs = _Permute.apply(x, probs, rim, d.routed_rows(), R)
    return rows, rows_probs, d


def unpermute(rows: torch.Tensor, dispatch: Dispatch, probs=None) -> torch.Tensor:
    """bf16 rows [R,H] -> y bf16 [T,H]: slot-order fp32 fused multiply-adds
    (plain adds without probs), one bf16 rounding."""
    return _Unpermute.apply(rows, probs, dispatch.row_id_map, dispatch.routed_rows(), None)


def unpermute_ep(rows: torch.Tensor, dispatch: Dispatch, ep_size: int, probs=None, *,
                 bf16_partials: bool = False, fp64_cross_rank: bool = False) -> torch.Tensor:
    """unpermute as a rank-ordered sum over `ep_size` expert-parallel ranks
    (per-rank partials, optionally bf16; cross-rank sum in fp32 or fp64).  The
    gradient is that of the plain combine: the summation tree changes the
    rounding, not the derivative."""
    ep = (dispatch.idx, dispatch.num_experts, int(ep_size), bool(bf16_partials),
          bool(fp64_cross_rank))
    return _Unpermute.apply(rows, probs, dispatch.row_id_map, dispatch.routed_rows(), ep)


def sort_chunks_pad(x: torch.Tensor, split_sizes: torch.Tensor, chunk_order: torch.Tensor,
                    num_groups: int, align: int, out_rows: int, probs=None, *,
                    padded_sizes=None):
    """Fused chunk sort + zero pad: (out [out_rows,H], out_probs or None,
    row_map int32 [out_rows], group_off int64 [G+1]).  The gradient of a
    padding row is dropped; rows of x that no chunk names get zero gradient."""
    return _SortChunksPad.apply(x, probs, split_sizes, chunk_order, int(num_groups), int(align),
                                int(out_rows), padded_sizes)


def unpad_restore(padded: torch.Tensor, row_map: torch.Tensor, num_rows: int,
                  padded_probs=None):
    """Inverse of sort_chunks_pad: (y [num_rows,H], y_probs or None); rows no
    chunk names are zero; padding rows get zero gradient."""
    return _UnpadRestore.apply(padded, padded_probs, row_map, int(num_rows))
