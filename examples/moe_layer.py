"""A mixture-of-experts layer from this package's operators: router, permute, the
experts' products, combine; a training loop, and single tokens afterwards.

    python examples/moe_layer.py

trains a disturbed copy of a layer back towards it on random tokens, keeping the
experts' activations in 8 bits and the load of the experts even by a bias on the
router's choice, and prints the loss and the load.
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from unpermute_routing_indices_gb300 import autograd as ag  # noqa: E402
from unpermute_routing_indices_gb300 import (mp_build_map, mp_expert_mlp, mp_moe_layer,  # noqa: E402
                                             mp_permute, mp_route, mp_unpermute, status_bits)


@dataclass
class MoeLayer:
    """T tokens of width H through the K best of E experts: sigmoid scores, weights that
    sum to one, swiglu experts of width F."""

    router: torch.Tensor    # fp32 [E,H]
    bias: torch.Tensor      # fp32 [E]: moves the choice only
    w1: torch.Tensor        # bf16 [E,2F,H], the gate's rows first
    w2: torch.Tensor        # bf16 [E,H,F]
    topk: int

    @staticmethod
    def make(H: int, F: int, E: int, topk: int, seed: int, device="cuda") -> "MoeLayer":
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, generator=g, device=device) * std
        return MoeLayer(normal(E, H, std=H ** -0.5), torch.zeros(E, device=device),
                        normal(E, 2 * F, H, std=H ** -0.5).bfloat16(),
                        normal(E, H, F, std=F ** -0.5).bfloat16(), topk)

    def parameters(self):
        return [self.router, self.w1, self.w2]

    def train_step(self, x: torch.Tensor, status=None):
        """x bf16 [T,H] -> (y bf16 [T,H], rows of each expert int32 [E]); y is
        differentiable w.r.t. x and the parameters.  `status` (int32 [1]) collects
        the experts' status bits of both passes."""
        idx, weights = ag.route(x.float() @ self.router.t(), self.topk, score="sigmoid",
                                bias=self.bias)
        rows, _, d = ag.permute(x, idx, self.router.shape[0])
        out = ag.expert_mlp(rows, d, self.w1, self.w2, act="swiglu", checkpoint="e4m3",
                            status=status)
        return ag.unpermute(out, d, weights), d.counts

    @torch.no_grad()
    def answer(self, x: torch.Tensor) -> torch.Tensor:
        """The same without gradients, for prompts and for single tokens."""
        idx, weights = mp_route(x.float() @ self.router.t(), self.topk, score="sigmoid",
                                bias=self.bias)
        row_id_map, _, _, offsets = mp_build_map(idx, self.router.shape[0],
                                                 with_sorted_to_flat=False)
        rows, _ = mp_permute(x, row_id_map)
        out, _, _ = mp_expert_mlp(rows, self.w1, self.w2, offsets, act="swiglu")
        return mp_unpermute(out, row_id_map, weights)

    @torch.no_grad()
    def answer_few(self, x: torch.Tensor) -> torch.Tensor:
        """The same for up to MAX_LAYER_TOKENS tokens, as answers are written: two kernels in
        all, with fewer roundings on the way."""
        return mp_moe_layer(x, self.router, self.w1, self.w2, self.topk, score="sigmoid",
                            bias=self.bias)[0]

    @torch.no_grad()
    def balance(self, counts: torch.Tensor, rate: float) -> None:
        """Raises the bias of experts with fewer rows than the mean, lowers the others'."""
        load = counts.float()
        self.bias += rate * torch.sign(load.mean() - load)


def train(steps: int = 300, T: int = 2048, H: int = 256, F: int = 128, E: int = 16, topk: int = 4,
          rate: float = 2e-3, seed: int = 1, report=None):
    """Trains a disturbed copy of a layer back towards it, by Adam on 32-bit weights;
    returns (layer, teacher, losses, largest load over the mean load, step by step)."""
    teacher, layer = MoeLayer.make(H, F, E, topk, seed), MoeLayer.make(H, F, E, topk, seed + 1)
    masters = [(t.float() + 0.3 * p.float()).requires_grad_()
               for t, p in zip(teacher.parameters(), layer.parameters())]
    optimizer = torch.optim.Adam(masters, lr=rate)
    schedule = torch.optim.lr_scheduler.CosineAnnealingLR(optimizer, steps)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 2)
    losses, loads = [], []
    status = torch.zeros(1, dtype=torch.int32, device="cuda")   # read once, at the end
    for step in range(steps):
        x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
        for p, m in zip(layer.parameters(), masters):
            p.requires_grad_(False).copy_(m.detach())
            p.requires_grad_(True)
        y, counts = layer.train_step(x, status)
        loss = (y.float() - teacher.answer(x).float()).square().mean()
        for m, d in zip(masters, torch.autograd.grad(loss, layer.parameters())):
            m.grad = d.float()
        optimizer.step()
        schedule.step()
        layer.balance(counts, 1e-4)
        losses.append(loss.detach())
        loads.append((counts.max() * E / counts.sum()).detach())
        if report and (step % 50 == 0 or step == steps - 1):
            report(f"step {step:4d}  loss {losses[-1].item():.4f}  "
                   f"largest load {loads[-1].item():.2f} of the mean")
    if int(status):
        raise RuntimeError(f"the experts' products report {sorted(status_bits(int(status)))}")
    for p in layer.parameters():
        p.requires_grad_(False)
    return layer, teacher, torch.stack(losses), torch.stack(loads)


def main() -> None:
    layer, teacher, _, _ = train(report=print)
    x = torch.randn(1, layer.router.shape[1], device="cuda").bfloat16()
    y, want = layer.answer_few(x).float(), teacher.answer_few(x).float()
    print(f"one token: {float((y - want).norm() / want.norm()):.3f} off the teacher's answer")


if __name__ == "__main__":
    main()
