"""A dense feed-forward block from the library's operators, for training and for serving with adapters.

    n = rms_norm(x, before)                               (of the block before it: residual_norm's z)
    h = act(n Wg^T) * (n Wu^T)                            gated_linear
    y = h Wd^T (+ the row's adapter)                      bf16_gemm, or adapter_linear
    t = scale * x + gate * norm(y, after)                 residual_norm, which gives the next block's
    z = norm(t, next)                                     normed input too

gradient() goes back through all of it: residual_norm_backward, the down-projection's two products,
gated_linear_backward, rms_norm_backward. The down-projection may instead be an FP8 or an 8-bit one, to
whose output adapter_add brings the adapters.

Run it to check the block against a plain torch one and to time a decode step and a prefill:

    python examples/dense_block.py
"""
from __future__ import annotations

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_act_quant_amd as fq  # noqa: E402


class DenseBlock:
    """up [2 F, H] (gate rows, then up rows) and down [H, F] bfloat16; before, after, next and gate float32 [H];
    adapters: (a [L, r, F], b [L, H, r], scales [L]) of the down-projection, or None."""

    def __init__(self, up, down, before, after, next, gate, *, scale=1.0, act="silu", adapters=None, down_weights="bf16"):
        self.up, self.down, self.before, self.after, self.next, self.gate = up, down, before, after, next, gate
        self.scale, self.act, self.adapters, self.down_weights = scale, act, adapters, down_weights
        if down_weights == "fp8":
            self.codes = fq.weight_quant(down)
        elif down_weights == "int8":
            self.codes = fq.int8_quant(down)

    def _project(self, h, ids):
        if self.down_weights == "bf16" and ids is not None:
            a, b, scales = self.adapters
            return fq.adapter_linear(h, self.down, a, b, ids, scales)
        if self.down_weights == "bf16":
            return fq.bf16_gemm(h, self.down)
        y = fq.linear(h, self.codes[0], weight_scale=self.codes[1]) if self.down_weights == "fp8" \
            else fq.int8_linear(h, *self.codes)
        if ids is not None:
            a, b, scales = self.adapters
            fq.adapter_add(y, h, a, b, ids, scales, out=y)
        return y

    def __call__(self, x, ids=None, keep=False):
        """x [T, H] bfloat16, ids int32 [T] (each row's adapter): ``(t, z)``. keep: for gradient()."""
        n = fq.rms_norm(x, self.before)
        h = fq.gated_linear(n, self.up, act=self.act, keep=keep)
        h, gu = h if keep else (h, None)
        y = self._project(h, ids)
        t, z = fq.residual_norm(x, y, self.next, post=self.after, gate=self.gate, scale=self.scale)
        if keep:
            self.saved = x, n, h, gu, y, t
        return t, z

    def gradient(self, dt, dz):
        """Of the last call with keep (without adapters): a dict of gradients, from those of t and z."""
        x, n, h, gu, y, t = self.saved
        dx, dy, dnext, dafter, dgate = fq.residual_norm_backward(dt, dz, t, y, self.next, post=self.after, gate=self.gate,
                                                                 scale=self.scale)
        dh = fq.bf16_gemm(dy, self.down.t().contiguous())
        ddown = dy.float().t() @ h.float()
        dn, dup = fq.gated_linear_backward(dh, n, self.up, gu, act=self.act)
        dx2, dbefore = fq.rms_norm_backward(dn, x, self.before)
        return dict(x=dx + dx2, up=dup, down=ddown, before=dbefore, after=dafter, next=dnext, gate=dgate)


def plain(block, x, ids=None):
    """The block in float64 torch, unquantised."""
    def norm(v, w):
        return w * v / (v.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    up, down, before, after, nxt, gate = (v.double() if v.dtype != torch.float64 else v for v in (
        block.up, block.down, block.before, block.after, block.next, block.gate))
    x = x.double() if x.dtype != torch.float64 else x
    g, u = (norm(x, before) @ up.t()).chunk(2, dim=-1)
    act = torch.nn.functional.silu if block.act == "silu" else torch.nn.functional.gelu
    h = act(g) * u
    y = h @ down.t()
    if ids is not None:
        a, b, scales = (v.double() for v in block.adapters)
        for e in range(a.shape[0]):
            at = (ids == e).nonzero()[:, 0]
            y = y.index_add(0, at, scales[e] * (h[at] @ a[e].t() @ b[e].t()))
    t = block.scale * x + gate * norm(y, after)
    return t, norm(t, nxt)


def example_weights(H, F, adapters=0, rank=16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    def near_one(n):
        return 1 + 0.1 * torch.randn(n, generator=g, device="cuda")
    lora = None
    if adapters:
        lora = (normal(adapters, rank, F, std=F ** -0.5), normal(adapters, H, rank, std=0.2),
                0.5 + torch.rand(adapters, generator=g, device="cuda"))
    return (normal(2 * F, H, std=H ** -0.5), normal(H, F, std=F ** -0.5), near_one(H), near_one(H), near_one(H),
            0.5 * near_one(H)), lora


def main():
    args, lora = example_weights(1024, 512, adapters=8)
    x = torch.randn((200, 1024), device="cuda").bfloat16()
    ids = torch.randint(-1, 8, (200,), device="cuda", dtype=torch.int32)
    for weights in ("bf16", "fp8", "int8"):
        block = DenseBlock(*args, adapters=lora, down_weights=weights)
        t, ref = block(x, ids)[0].double(), plain(block, x, ids)[0]
        print(f"down-projection in {weights}: relative error {float((t - ref).norm() / ref.norm()):.4f} against float64")
    H, F = 7168, 2048
    args, lora = example_weights(H, F, adapters=32)
    block = DenseBlock(*args, adapters=lora)
    for T in (1, 48, 4096):
        x = torch.randn((T, H), device="cuda").bfloat16()
        ids = torch.randint(-1, 32, (T,), device="cuda", dtype=torch.int32) if T < 4096 else \
            torch.arange(T, device="cuda", dtype=torch.int32) // 512
        for _ in range(5):
            block(x, ids)
        torch.cuda.synchronize()
        t, n = time.perf_counter(), 20
        for _ in range(n):
            block(x, ids)
        torch.cuda.synchronize()
        print(f"{T} tokens, {H} -> {F}, 32 adapters: {(time.perf_counter() - t) / n * 1e6:.0f} us")


if __name__ == "__main__":
    main()
