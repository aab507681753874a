"""A mixture-of-experts layer on libblockq: 4-bit expert weights, tokens sorted by expert, two
expert products with a gated activation between them, and the weighted way back.

    python examples/expert_layer.py [--tokens 64] [--experts 16] [--topk 4] [--hidden 1024]
                                    [--inner 512] [--group 64]

Runs the layer for one token, for a batch, and for a batch with dropped choices, compares each
with the same layer in plain torch, and takes the gradients of the
dispatch and of the way back in a training step.  Every buffer is the caller's and is made once.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_wire_amd as bq  # noqa: E402


class Weights4:
    """One 4-bit matrix for each expert, quantized from bf16 (experts, rows, cols)."""

    def __init__(self, w: torch.Tensor, group: int):
        e, n, k = w.shape
        groups = -(-(k // group) // 4) * 4                   # rows of scales are whole fours
        self.group, self.rows, self.cols = group, n, k
        self.codes = torch.empty((e, n, -(-(k // 2) // 16) * 16), dtype=torch.uint8, device=w.device)
        self.scale = torch.zeros((e, n, groups), dtype=w.dtype, device=w.device)
        flat = self.codes.view(e * n, -1), self.scale.view(e * n, -1)
        bq.bq_quant_i4(w.reshape(e * n, k), *flat, group=group)

    def values(self, e: int) -> torch.Tensor:
        """What expert e's codes stand for, exactly, in binary32.  (bq_dequant_i4 rounds the same
        to bf16, for a user who wants bf16 weights.)"""
        c = self.codes[e, :, : self.cols // 2]
        code = torch.stack((c & 15, c >> 4), -1).view(self.rows, -1, self.group).float()
        scale = self.scale[e, :, : self.cols // self.group].float()
        return ((code - 8) * scale[:, :, None]).view(self.rows, self.cols)


class ExpertLayer:
    """x -> sum over choices of weight * down(silu(gate(x)) * up(x)), for up to max_tokens."""

    def __init__(self, gate_up: torch.Tensor, down: torch.Tensor, topk: int, max_tokens: int,
                 group: int):
        dev, dt = gate_up.device, gate_up.dtype
        self.first, self.second = Weights4(gate_up, group), Weights4(down, group)
        self.experts, self.topk, self.inner = gate_up.shape[0], topk, down.shape[2]
        slots = max_tokens * topk
        ints = lambda n: torch.empty(n, dtype=torch.int32, device=dev)  # noqa: E731
        self.off, self.src, self.pos = ints(self.experts + 1), ints(slots), ints(slots)
        self.ws = torch.empty(bq.bq_moe_sort_ws_bytes(max_tokens, topk, self.experts),
                              dtype=torch.uint8, device=dev)
        self.mid = torch.empty((slots, 2 * self.inner), dtype=dt, device=dev)
        self.out = torch.empty((slots, down.shape[1]), dtype=dt, device=dev)

    def __call__(self, x: torch.Tensor, ids: torch.Tensor, weight: torch.Tensor,
                 y: torch.Tensor) -> None:
        slots = x.shape[0] * self.topk
        src, pos = self.src[:slots], self.pos[:slots]
        bq.bq_moe_sort(ids, self.experts, self.off, src, pos, self.ws)
        # the first product takes each sorted row straight from its token
        bq.bq_moe_mm_i4(x, self.off, self.first.codes, self.first.scale, self.mid[:slots],
                        group=self.first.group, src=src, topk=self.topk)
        gate, up = self.mid[:slots, : self.inner], self.mid[:slots, self.inner:]
        act = torch.nn.functional.silu(gate.float()).mul_(up).to(x.dtype)
        bq.bq_moe_mm_i4(act, self.off, self.second.codes, self.second.scale, self.out[:slots],
                        group=self.second.group)
        bq.bq_moe_combine(self.out[:slots], pos, self.off, y, weight=weight, topk=self.topk)

    def plain(self, x, ids, weight):
        """The same layer, choice by choice, in binary32 torch."""
        y = torch.zeros((x.shape[0], self.out.shape[1]), device=x.device)
        for e in range(self.experts):
            t, j = torch.where(ids == e)
            mid = (x[t].float() @ self.first.values(e).t()).to(x.dtype).float()
            act = torch.nn.functional.silu(mid[:, : self.inner]) * mid[:, self.inner:]
            rows = (act.to(x.dtype).float() @ self.second.values(e).t()).to(x.dtype).float()
            y.index_add_(0, t, weight[t, j, None] * rows)
        return y


class Dispatch(torch.autograd.Function):
    """Rows of x to their sorted places; the gradient is the combine without weights."""

    @staticmethod
    def forward(ctx, x, pos, off, topk):
        ctx.save_for_backward(pos, off)
        ctx.topk, ctx.tokens = topk, x.shape[0]
        out = x.new_empty((x.shape[0] * topk, x.shape[1]))
        bq.bq_moe_gather(x, pos, off, out, topk=topk)
        return out

    @staticmethod
    def backward(ctx, grad):
        pos, off = ctx.saved_tensors
        dx = grad.new_empty((ctx.tokens, grad.shape[1]))
        bq.bq_moe_combine_f32(grad.contiguous(), pos, off, dx, topk=ctx.topk)
        return dx, None, None, None


class Combine(torch.autograd.Function):
    """The weighted sum of every token's rows."""

    @staticmethod
    def forward(ctx, rows, weight, pos, off):
        ctx.save_for_backward(rows, weight, pos, off)
        y = rows.new_empty((weight.shape[0], rows.shape[1]))
        bq.bq_moe_combine_f32(rows, pos, off, y, weight=weight, topk=weight.shape[1])
        return y

    @staticmethod
    def backward(ctx, dy):
        rows, weight, pos, off = ctx.saved_tensors
        drows, dweight = torch.empty_like(rows), torch.empty_like(weight)
        bq.bq_moe_combine_bwd_f32(dy.contiguous(), rows, pos, off, weight, drows, dweight)
        return drows, dweight, None, None


def choices(tokens, experts, topk, drop, gen, dev):
    logits = torch.randn((tokens, experts), generator=gen, device=dev)
    top, ids = torch.topk(logits, topk, dim=1)
    ids = ids.to(torch.int32)
    ids[torch.rand(ids.shape, generator=gen, device=dev) < drop] = -1      # no expert here
    return ids.contiguous(), torch.softmax(top, 1).contiguous()


def run(tokens=64, experts=16, topk=4, hidden=1024, inner=512, group=64, seed=0) -> dict:
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    bf16 = lambda *s: (torch.randn(s, generator=gen, device=dev) / s[-1] ** 0.5).bfloat16()  # noqa: E731
    layer = ExpertLayer(bf16(experts, 2 * inner, hidden), bf16(experts, hidden, inner), topk, tokens,
                        group)
    errors = {}
    for name, t, drop in (("one token", 1, 0.0), ("batch", tokens, 0.0), ("dropped", tokens, 0.3)):
        x = torch.randn((t, hidden), generator=gen, device=dev).bfloat16()
        ids, weight = choices(t, experts, topk, drop, gen, dev)
        y = torch.empty((t, hidden), dtype=torch.bfloat16, device=dev)
        layer(x, ids, weight, y)
        want = layer.plain(x, ids, weight)
        errors[name] = float((y.float() - want).norm() / want.norm())

    # a training step of the two movements around experts that are plain scalings
    ids, weight = choices(tokens, experts, topk, 0.2, gen, dev)
    off, src, pos = (torch.empty(n, dtype=torch.int32, device=dev)
                     for n in (experts + 1, tokens * topk, tokens * topk))
    bq.bq_moe_sort(ids, experts, off, src, pos, layer.ws)
    x = torch.randn((tokens, hidden), generator=gen, device=dev, requires_grad=True)
    w = weight.clone().requires_grad_(True)
    row_expert = torch.searchsorted(off[1:].long(), torch.arange(tokens * topk, device=dev), right=True)
    gain = (1.0 + row_expert)[:, None]
    loss = Combine.apply(Dispatch.apply(x, pos, off, topk) * gain, w, pos, off).square().sum()
    loss.backward()
    x2, w2 = x.detach().clone().requires_grad_(True), weight.clone().requires_grad_(True)
    live = ids >= 0
    mix = torch.where(live, w2 * (1.0 + ids), torch.zeros_like(w2)).sum(1, keepdim=True)
    (x2 * mix).square().sum().backward()
    errors["dx"] = float((x.grad - x2.grad).norm() / x2.grad.norm())
    errors["dweight"] = float((w.grad - w2.grad).norm() / w2.grad.norm())
    return errors


def close(errors: dict) -> bool:
    """Whether the distances are those of roundings: less than one bf16 step for the layer, of
    binary32 sums for the training step.  A NaN is not close."""
    return all(errors[k] < 2.0 ** -8 for k in ("one token", "batch", "dropped")) and all(
        errors[k] < 2.0 ** -12 for k in ("dx", "dweight"))


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 64), ("experts", 16), ("topk", 4), ("hidden", 1024),
                          ("inner", 512), ("group", 64)):
        ap.add_argument("--" + name, type=int, default=default)
    for name, err in run(**vars(ap.parse_args())).items():
        print(f"{name:10s} relative distance from plain torch: {err:.2e}")


if __name__ == "__main__":
    main()
