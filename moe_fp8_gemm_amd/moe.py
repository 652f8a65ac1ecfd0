"""Mixture-of-experts operators: routing, expert layout, dispatch, combination.

Each function checks types, devices and shapes, allocates the outputs that are not
passed in, and calls the C ABI of ``include/dgfp8.h`` on torch's current stream (in
``csrc/binding.cpp``: a decoding step's calls are shorter than these checks would
take in Python).

A layer runs

    indices, weights = route_topk(logits, topk, ...)
    layout = expert_layout_contiguous(indices, num_experts)
    a = dispatch_cast_fp8(x, layout.slot_row, rows=layout.rows)
    m_grouped_fp8_gemm_nt_contiguous(a, b, d, layout.m_indices)
    out = combine(d, layout.slot_row, weights)

and nothing in it reads the routing on the host.  The results are plain tensors: autograd records none of the calls,
and a training step calls ``route_topk_grad`` and ``combine_grad`` itself.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import _native, lib


class ExpertLayout(NamedTuple):
    """Rows of the chosen experts (see ``expert_layout_contiguous`` / ``_masked``)."""
    m_indices: Optional[torch.Tensor]   # int32 [rows], expert of the row or -1; None in the masked layout
    row_slot: torch.Tensor              # int32 [rows], token * topk + j of the row's slot, or -1
    slot_row: torch.Tensor              # int32 [tokens, topk], row of the slot, or -1
    counts: torch.Tensor                # int32 [experts]: slots of each expert (masked layout: masked_m)

    @property
    def rows(self) -> int:
        return self.row_slot.shape[0]


def route_topk(logits: torch.Tensor, topk: int, *, score: str = "softmax", bias: Optional[torch.Tensor] = None,
               num_expert_groups: int = 1, topk_groups: int = 1, group_score: str = "max",
               renormalize: bool = True, scale: float = 1.0, indices: Optional[torch.Tensor] = None,
               weights: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The topk experts of each token and their weights: (indices int32, weights fp32), both [tokens, topk].

    logits: float32, bfloat16 or float16 [tokens, experts] (up to 1024 experts, 64 slots).  ``score``: "softmax"
    over a token's logits or "sigmoid" of each.  ``bias`` (fp32 [experts]) is added to the scores for the choice
    only.  ``num_expert_groups`` > 1: only the best ``topk_groups`` of that many equal consecutive groups take part,
    by their largest key (``group_score`` "max") or the sum of their two largest scores ("top2").  Equal keys go to
    the lower number.  Weights are the scores, divided by their sum if ``renormalize``, times ``scale``.  A logit or
    bias of -inf takes an expert out; slots without an expert get index -1 and weight 0.  A NaN makes a token's
    weights NaN.
    """
    return _native.route_topk(logits, topk, score, bias, num_expert_groups, topk_groups, group_score, renormalize,
                              scale, indices, weights)


def route_topk_grad(logits: torch.Tensor, indices: torch.Tensor, dweights: torch.Tensor, *, score: str = "softmax",
                    renormalize: bool = True, scale: float = 1.0,
                    dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of ``route_topk``'s weights: dlogits [tokens, experts] of the logits' type.

    indices int32 and dweights fp32 are [tokens, topk]; the other arguments as they were given to ``route_topk``.
    The choice of experts is held fixed, so a bias or groups do not enter.
    Under plain softmax (not renormalised) a NaN logit makes its token's row NaN; otherwise only the chosen logits enter.
    """
    return _native.route_topk_grad(logits, indices, dweights, score, renormalize, scale, dlogits)


def expert_layout_rows(tokens: int, topk: int, num_experts: int) -> int:
    """Rows that hold every routing of these sizes in the contiguous layout (a multiple of 128)."""
    return int(lib.dg_expert_layout_rows(int(tokens), int(topk), int(num_experts)))


def expert_layout_contiguous(indices: torch.Tensor, num_experts: int, rows: Optional[int] = None) -> ExpertLayout:
    """Rows of the contiguous layout for a routing: experts in order, each from a multiple of 128 rows, an expert's
    slots in order of token and slot.

    indices int32 [tokens, topk]; others than 0..num_experts-1 get no row.  ``rows`` defaults to
    ``expert_layout_rows(...)``, which holds every routing; with fewer, slots beyond them are dropped.
    """
    return ExpertLayout._make(_native.expert_layout_contiguous(indices, num_experts, rows))


def expert_layout_masked(indices: torch.Tensor, num_experts: int, max_m: int) -> ExpertLayout:
    """Rows of the masked layout: expert e's slots get rows e * max_m, e * max_m + 1, ... (a [experts, max_m, ...]
    tensor seen as [experts * max_m, ...]); slots past max_m are dropped.  ``counts`` is the GEMM's masked_m."""
    return ExpertLayout._make(_native.expert_layout_masked(indices, num_experts, max_m))


def dispatch_cast_fp8(x: torch.Tensor, slot_row: torch.Tensor, rows: Optional[int] = None, ue8m0: bool = False,
                      q: Optional[torch.Tensor] = None,
                      sf: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Cast of token rows into their experts' rows: (E4M3 codes [rows, k], fp32 scales [rows, k/128]).

    x bf16 or fp32 [tokens, k]; slot_row int32 [tokens, topk] as a layout holds it (no row twice).  Codes and scales
    are ``per_token_cast_fp8``'s.  Rows without a slot are left untouched (unspecified in tensors allocated here);
    the grouped GEMMs do not use them.  ``sf`` may have any strides; allocated here, a block's scales lie beside one
    another along the rows, as the GEMMs read them best.
    """
    return _native.dispatch_cast_fp8(x, slot_row, rows, ue8m0, q, sf)


def dispatch_cast_int8(x: torch.Tensor, slot_row: torch.Tensor, rows: Optional[int] = None,
                       q: Optional[torch.Tensor] = None,
                       sf: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """As ``dispatch_cast_fp8`` with the int8 cast: (int8 codes [rows, k], fp32 scales [rows])."""
    return _native.dispatch_cast_int8(x, slot_row, rows, q, sf)


def combine(y: torch.Tensor, slot_row: torch.Tensor, weights: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] * y[slot_row[t, j]] over the slots that have a row.

    y bf16 [rows, h]; slot_row int32 and weights fp32 [tokens, topk] (None: all ones, which makes this the gradient of
    dispatching tokens to rows); out bf16 (default) or fp32 [tokens, h].  Sums are fp32, in slot order.
    """
    return _native.combine(y, slot_row, weights, out)


def combine_grad(dout: torch.Tensor, y: torch.Tensor, slot_row: torch.Tensor, row_slot: torch.Tensor,
                 weights: torch.Tensor, dy: Optional[torch.Tensor] = None,
                 dweights: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gradient of ``combine``: (dy bf16 [rows, h], dweights fp32 [tokens, topk]).

    dout bf16 [tokens, h]; y, slot_row and weights as given to ``combine``; row_slot from the same layout.  Rows of dy
    without a slot, and dweights of slots without a row, are zero.
    """
    return _native.combine_grad(dout, y, slot_row, row_slot, weights, dy, dweights)
