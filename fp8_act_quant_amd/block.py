"""The dense block around the linear layers: norms with the residual and the block's gate, gated
projections, and linear layers with an adapter per token.

``residual_norm`` stands between two blocks (``rms_norm`` before the first), ``gated_linear`` is a
feed-forward block's first half, ``adapter_linear`` a projection of requests that each have a
low-rank adapter of their own (``adapter_add`` beside the output of another projection). What
training needs has its gradient beside it. Every step runs in the kernels behind the C ABI;
arguments are checked by the native binding (TypeError, ValueError), which allocates the outputs
with torch and launches on torch's current stream.
"""
from __future__ import annotations

import torch

from ._binding import native, out_code
from ._lib import FP8Q_ACT_GELU, FP8Q_ACT_SILU, FP8Q_GATED_WIDE

_ACTS = {"silu": FP8Q_ACT_SILU, "gelu": FP8Q_ACT_GELU}


def _act(act: str) -> int:
    code = _ACTS.get(act)
    if code is None:
        raise ValueError('act must be "silu" or "gelu"')
    return code


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6) -> torch.Tensor:
    """x / sqrt(mean(x^2) + eps) * weight over the last dimension. x [..., H] (float32 or bfloat16,
    H from 8 to 16384), weight float32 [H]. In float32, rounded once."""
    return native.norm(x, None, weight, None, None, 1.0, eps)


def rms_norm_backward(dz: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6):
    """Gradients of rms_norm: ``(dx, dweight)``, dx as x, dweight float32 [H]."""
    dx, _, dweight, _, _ = native.norm_backward(None, dz, x, None, weight, None, None, 1.0, eps)
    return dx, dweight


def residual_norm(x: torch.Tensor, y: torch.Tensor, weight: torch.Tensor | None = None, *,
                  post: torch.Tensor | None = None, gate: torch.Tensor | None = None, scale: float = 1.0,
                  eps: float = 1e-6):
    """A block's output y put into the residual stream x, and the stream normed for the next block:
    t = scale * x + gate * n with n = rms_norm(y, post) (or y without post), z = rms_norm(t, weight).

    x, y [..., H] of one dtype (float32 or bfloat16); weight and post float32 [H]; gate float32 [H], or
    of x's shape and dtype, or None for 1. Returns ``(t, z)`` in x's dtype, z None without weight; z is formed
    from t before t's rounding."""
    return native.norm(x, _given(y, "y"), weight, post, gate, scale, eps)


def residual_norm_backward(dt: torch.Tensor | None, dz: torch.Tensor | None, t: torch.Tensor, y: torch.Tensor,
                           weight: torch.Tensor | None = None, *, post: torch.Tensor | None = None,
                           gate: torch.Tensor | None = None, scale: float = 1.0, eps: float = 1e-6):
    """Gradients of residual_norm from dt (of t besides the way through z, or None) and dz (of z;
    with weight, and only then), at t as that call returned it and y; other arguments as in it.

    Returns ``(dx, dy, dweight, dpost, dgate)``: dx, dy as t; dweight, dpost float32 [H]; dgate as gate; None
    for what the call did not have."""
    return native.norm_backward(dt, dz, t, _given(y, "y"), weight, post, gate, scale, eps)


def gated_linear(x: torch.Tensor, w: torch.Tensor, act: str = "silu", keep: bool = False, out_dtype=torch.bfloat16):
    """h = act(x Wg^T) * (x Wu^T): both projections of a gated feed-forward block, the activation
    ("silu", or "gelu" with the normal distribution's integral) and the product in one kernel.

    x bfloat16 [..., K]; w bfloat16 [2 F, K], Wg its first F rows and Wu the others (K and F multiples
    of 8). Returns h [..., F] in out_dtype (bfloat16 or float32), or with keep ``(h, gu)``, gu bfloat16
    [..., 2 F] being both projections, for gated_linear_backward."""
    return native.gated(x, w, _act(act), keep, out_code(out_dtype))


def gated_linear_backward(dh: torch.Tensor, x: torch.Tensor, w: torch.Tensor, gu: torch.Tensor | None = None,
                          act: str = "silu", dx_dtype=torch.bfloat16, dw_dtype=torch.float32, wide: bool = False):
    """Gradients of gated_linear: ``(dx, dw)`` of x's and w's shapes from dh bfloat16 [..., F]. gu as the
    call with keep returned it; without it the projections are computed again. The projections'
    gradient is rounded to bfloat16 on its way into both (also where they are float32), or with
    wide goes into them with 16 bits, as two bfloat16 numbers, which takes 1.3 to 2.7 times as long."""
    return native.gated_backward(dh, x, w, gu, _act(act) | (FP8Q_GATED_WIDE if wide else 0), out_code(dx_dtype),
                                 out_code(dw_dtype))


def adapter_linear(x: torch.Tensor, w: torch.Tensor, a: torch.Tensor, b: torch.Tensor, ids: torch.Tensor,
                   scales: torch.Tensor | None = None, bias: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """y = x w^T (+ bias) + scales[e] * (x a[e]^T) b[e]^T, e the row's adapter ids[...]: a linear layer
    for a batch of requests that have an adapter each, or none (ids outside 0 .. adapters - 1).

    x bfloat16 [..., K], w bfloat16 [N, K] shared by all; a [adapters, rank, K] and b [adapters, N, rank]
    bfloat16 (K a multiple of 8, rank one up to 256, lower ranks padded with zeros); ids int32 [...]
    on the device, in any order; scales float32 [adapters]; bias float32 [N]. Returns [..., N] in
    out_dtype (bfloat16 or float32); out, if given, overlaps no other argument."""
    return native.adapter(x, _given(w, "w"), a, b, ids, scales, bias, None, out_code(out_dtype), out)


def adapter_add(y: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, ids: torch.Tensor,
                scales: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """y + scales[e] * (x a[e]^T) b[e]^T: the adapters beside another projection's output y [..., N] (float32
    or bfloat16; of fp8_gemm, int8_linear, ...), in y's dtype. out may be y itself, and overlaps
    neither a part of it nor b or ids. Other arguments as for adapter_linear."""
    return native.adapter(x, None, a, b, ids, scales, None, y, 0, out)


def _given(t, name: str):
    if t is None:
        raise TypeError(f"{name} must be a torch.Tensor")
    return t
