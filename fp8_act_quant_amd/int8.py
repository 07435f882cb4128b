"""Products in 8-bit integers with one scale per token and one per output channel.

``int8_quant`` quantises rows (an activation's tokens, or a weight's channels), ``int8_gemm``
multiplies, ``int8_linear`` does both for bf16 activations and ``int8_grouped_gemm`` multiplies
every expert's rows by its own weight. The integer sums are exact. Every step runs in the
kernels behind the C ABI; arguments are checked by the native binding (TypeError, ValueError),
which allocates the outputs with torch and launches on torch's current stream.
"""
from __future__ import annotations

import torch

from ._binding import native, out_code


def int8_quant(x: torch.Tensor):
    """One scale per row of a bf16 x [..., K] (K a multiple of 16): the tokens of an
    activation, or the output channels of a weight. Returns ``(q, s)``: q int8 [..., K] in
    -127 .. 127 and s float32 [...], s = max|x| * float32(1 / 127), q = x / s rounded to
    nearest even."""
    return native.quant(x)


def int8_gemm(a: torch.Tensor, a_s: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor,
              bias: torch.Tensor | None = None, out_dtype=torch.bfloat16,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """Y = (a . w^T) * a_s * w_s (+ bias). a int8 [..., K] with scales a_s float32 [...], w int8
    [N, K] with w_s float32 [N] (K a multiple of 16 below 2^17), bias: optional float32 [N],
    added before the output's rounding. Returns [..., N] in out_dtype (bfloat16 or float32)."""
    return native.gemm(a, a_s, w, w_s, bias, out_code(out_dtype), out)


def int8_linear(x: torch.Tensor, weight: torch.Tensor, weight_scale: torch.Tensor,
                bias: torch.Tensor | None = None, out_dtype=torch.bfloat16) -> torch.Tensor:
    """y = x . weight^T (+ bias) for bf16 activations x [..., K] and an 8-bit weight [N, K] with
    one scale per channel [N] (as int8_quant gives them): int8_gemm of int8_quant(x), bit for
    bit, in one call (a few tokens: in one launch)."""
    return native.linear(x, weight, weight_scale, bias, out_code(out_dtype))


def int8_grouped_gemm(a: torch.Tensor, a_s: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor,
                      offsets: torch.Tensor, rows: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                      out: torch.Tensor | None = None) -> torch.Tensor:
    """Routed experts' products in one launch: row r, of the expert e with offsets[e] <= r <
    offsets[e + 1], is a[rows[r]] (or a[r] without rows) times w[e]. a int8 [tokens, K] with
    a_s float32 [tokens]; w int8 [E, N, K] with w_s float32 [E, N]; offsets int64 [E + 1] and
    rows int32 [R] as moe_place returns them, on the device. Returns [R, N] (R = tokens
    without rows) in out_dtype; rows that no expert owns are left as they were in `out`, or
    uninitialised."""
    return native.grouped_gemm(a, a_s, w, w_s, offsets, rows, out_code(out_dtype), out)
