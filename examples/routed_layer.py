"""A mixture-of-experts layer from the library's operators.

The gate's logits (bf16 GEMM) are routed to experts (moe_route), the rows put into expert order
(moe_place), multiplied by every expert's up- and down-projection in one launch each, and added
up per token with the router's weights (moe_combine). The experts' weights are kept in 8-bit
integers with a scale per channel (int8_quant, int8_grouped_gemm, which gathers each row's token
itself) or in FP8 with 128x128 block scales (act_quant, fp8_grouped_gemm): the placement's offsets
serve both. gradient() takes a training step's gradient back through the combination and the
router.

Run it to check the layer against a plain torch one and to time a decode step and a prefill:

    python examples/routed_layer.py
"""
from __future__ import annotations

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_act_quant_amd as fq  # noqa: E402


class RoutedLayer:
    """gate [E, H], up [E, 2 F, H] (the first F channels go through SiLU and multiply the others),
    down [E, H, F], all bfloat16; balance: float32 [E], added to the scores for the selection."""

    def __init__(self, gate, up, down, balance, *, top_k, groups=1, topk_groups=1, scale=1.0, weights="int8"):
        self.gate, self.balance, self.weights = gate, balance, weights
        self.routing = dict(top_k=top_k, bias=balance, groups=groups, topk_groups=topk_groups, scale=scale)
        self.experts = gate.shape[0]
        quantise = fq.int8_quant if weights == "int8" else _blocks_of
        self.up, self.down = quantise(up), quantise(down)

    def __call__(self, x):
        logits = fq.bf16_gemm(x, self.gate, out_dtype=torch.float32)
        w, experts = fq.moe_route(logits, **self.routing)
        offsets, rows, slots = fq.moe_place(experts, self.experts)
        if self.weights == "int8":
            h = fq.int8_grouped_gemm(*fq.int8_quant(x), *self.up, offsets, rows=rows)
            h = fq.int8_grouped_gemm(*fq.int8_quant(_gated(h)), *self.down, offsets)
        else:
            h = fq.fp8_grouped_gemm(*fq.act_quant(x[rows]), *self.up, offsets)
            h = fq.fp8_grouped_gemm(*fq.act_quant(_gated(h)), *self.down, offsets)
        self.saved = logits, experts, slots, w, h
        return fq.moe_combine(h, slots, w)

    def gradient(self, dy):
        """Of the last call: the gradients of the experts' outputs (rows in expert order) and of
        the gate's logits, from the layer's."""
        logits, experts, slots, w, h = self.saved
        dh, dw = fq.moe_combine_backward(dy, h, slots, w)
        return dh, fq.moe_route_backward(dw, logits, experts, scale=self.routing["scale"])


def _gated(h):
    a, b = h.chunk(2, dim=-1)
    return torch.nn.functional.silu(a).mul_(b)


def _blocks_of(w):
    """FP8 codes and block scales of every expert's weight."""
    q, s = zip(*(fq.weight_quant(w[e]) for e in range(w.shape[0])))
    return torch.stack(q), torch.stack(s)


def plain(layer_args, routing, x):
    """The layer in float32 torch, unquantised, expert by expert."""
    gate, up, down, balance = (t.float() for t in layer_args)
    x = x.float()
    score = torch.sigmoid(x @ gate.t())
    choice, G = score + balance, routing.get("groups", 1)
    if G > 1:
        value = choice.view(x.shape[0], G, -1).topk(2, dim=-1).values.sum(-1)
        out = torch.ones_like(value, dtype=torch.bool).scatter_(1, value.topk(routing["topk_groups"]).indices, False)
        choice = choice.masked_fill(out.repeat_interleave(choice.shape[1] // G, dim=1), float("-inf"))
    experts = choice.topk(routing["top_k"]).indices
    w = score.gather(1, experts)
    w = routing.get("scale", 1.0) * w / w.sum(-1, keepdim=True)
    y = torch.zeros_like(x)
    for e in range(gate.shape[0]):
        t, j = (experts == e).nonzero(as_tuple=True)
        if len(t):
            y.index_add_(0, t, w[t, j, None] * (_gated(x[t] @ up[e].t()) @ down[e].t()))
    return y


def example_weights(E, H, F, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)
    return (normal(E, H, std=H ** -0.5), normal(E, 2 * F, H, std=H ** -0.5), normal(E, H, F, std=F ** -0.5),
            0.05 * torch.randn(E, generator=g, device="cuda"))


def main():
    routing = dict(top_k=8, groups=8, topk_groups=4, scale=2.5)
    args = example_weights(32, 512, 256)
    x = torch.randn((200, 512), device="cuda").bfloat16()
    ref = plain(args, routing, x)
    for weights in ("int8", "fp8"):
        y = RoutedLayer(*args, weights=weights, **routing)(x).float()
        print(f"{weights}: relative error {float((y - ref).norm() / ref.norm()):.4f} against unquantised float32")
    E, H, F = 64, 7168, 2048
    args = example_weights(E, H, F)
    for weights in ("int8", "fp8"):
        layer = RoutedLayer(*args, weights=weights, **routing)
        for T in (1, 16, 2048):
            x = torch.randn((T, H), device="cuda").bfloat16()
            for _ in range(5):
                layer(x)
            torch.cuda.synchronize()
            t, n = time.perf_counter(), 20
            for _ in range(n):
                layer(x)
            torch.cuda.synchronize()
            print(f"{weights}: {T} tokens, {E} experts, {H} -> {F}: {(time.perf_counter() - t) / n * 1e6:.0f} us")


if __name__ == "__main__":
    main()
