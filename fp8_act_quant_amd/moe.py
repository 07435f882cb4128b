"""Routing of tokens to experts, and rows into expert order and back.

Around a mixture-of-experts layer's grouped products (fp8_grouped_gemm, int8_grouped_gemm):
``moe_route`` gives each token its experts and their weights, ``moe_place`` the grouped
products' offsets and which token each row is, ``moe_combine`` the weighted sum of a token's
rows. Each has its gradient beside it. Every step runs in the kernels behind the C ABI;
arguments are checked by the native binding (TypeError, ValueError), which allocates the
outputs with torch and launches on torch's current stream.
"""
from __future__ import annotations

import torch

from ._binding import native
from ._lib import FP8Q_MOE_GROUP_MAX, FP8Q_MOE_KEEP_SCORES, FP8Q_MOE_SOFTMAX

_SCORES = {"sigmoid": 0, "softmax": FP8Q_MOE_SOFTMAX}
_GROUPS = {"top2": 0, "max": FP8Q_MOE_GROUP_MAX}


def _flags(score: str, renormalize: bool) -> int:
    flags = _SCORES.get(score)
    if flags is None:
        raise ValueError('score must be "sigmoid" or "softmax"')
    return flags if renormalize else flags | FP8Q_MOE_KEEP_SCORES


def moe_route(logits: torch.Tensor, top_k: int, *, score: str = "sigmoid", bias: torch.Tensor | None = None,
              groups: int = 1, topk_groups: int = 1, group_score: str = "top2", renormalize: bool = True,
              scale: float = 1.0):
    """Each token's experts. logits [..., E] (float32 or bfloat16, E at most 1024) are the gate's.

    Scores are sigmoid(x) or softmax(x); bias [E] (float32) is added for the selection only.
    With groups > 1 (at most 64) the experts are that many equal runs, of which the topk_groups
    with the largest value (the sum of a run's two largest choices, or with group_score="max" its
    largest) take part. Returns ``(weights, experts)``, both [..., top_k] (at most 32): float32
    weights (the scores, divided by their sum if renormalize, times scale) and int32 experts, the
    largest choice first, equal ones by index."""
    best = _GROUPS.get(group_score)
    if best is None:
        raise ValueError('group_score must be "top2" or "max"')
    return native.route(logits, top_k, bias, groups, topk_groups, scale, _flags(score, renormalize) | best)


def moe_route_backward(dweights: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, *,
                       score: str = "sigmoid", renormalize: bool = True, scale: float = 1.0) -> torch.Tensor:
    """Gradient of moe_route's weights with respect to the logits (which it has the shape and
    dtype of). dweights [..., k] float32 and experts [..., k] int32 as moe_route returned
    them; score, renormalize and scale as in that call. The selection has no gradient."""
    return native.route_backward(dweights, logits, experts, scale, _flags(score, renormalize))


def moe_place(experts: torch.Tensor, n_experts: int, *, first: int = 0):
    """Rows in expert order. experts [T, k] int32 are each token's; those in
    [first, first + n_experts) get rows (one GPU's experts of an expert-parallel layer).

    Returns ``(offsets, rows, slots)``: offsets int64 [n_experts + 1], the grouped products'
    bounds; rows int32 [T * k], each row's token (ascending within an expert; -1 past the
    last row, offsets[-1]); slots int32 [T, k], each choice's row or -1."""
    return native.place(experts, n_experts, first)


def moe_combine(h: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """y[t] = sum over j of weights[t, j] * h[slots[t, j]], [T, H] in h's dtype (float32 or
    bfloat16), summed in float32. Slots outside h's rows (-1) add nothing. weights float32
    [T, k], or None for all 1: with moe_place's slots that is the gradient of x[rows]."""
    return native.combine(h, slots, weights, out)


def moe_combine_backward(dy: torch.Tensor, h: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor):
    """Gradients of moe_combine: ``(dh, dweights)``, dh[slots[t, j]] = weights[t, j] * dy[t] in
    h's shape and dtype and dweights[t, j] = <dy[t], h[slots[t, j]]> in float32. Rows of dh
    that no slot names are uninitialised (no expert owns them)."""
    return native.combine_backward(dy, h, slots, weights)
