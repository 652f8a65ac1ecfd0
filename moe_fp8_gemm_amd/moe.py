"""Mixture-of-experts operators: routing, expert layout, dispatch, combination.

Argument marshalling only, like the rest of the binding: each function checks
types, devices and shapes, allocates the outputs that are not passed in, and
calls the C ABI of ``include/dgfp8.h`` on torch's current stream.

A layer runs

    indices, weights = route_topk(logits, topk, ...)
    layout = expert_layout_contiguous(indices, num_experts)
    a = dispatch_cast_fp8(x, layout.slot_row, rows=layout.rows)
    m_grouped_fp8_gemm_nt_contiguous(a, b, d, layout.m_indices)
    out = combine(d, layout.slot_row, weights)

and nothing in it reads the routing on the host.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import _check, _stream, lib

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_SCORES = {"softmax": 0, "sigmoid": 1}


class ExpertLayout(NamedTuple):
    """Rows of the chosen experts (see ``expert_layout_contiguous`` / ``_masked``)."""
    m_indices: Optional[torch.Tensor]   # int32 [rows], expert of the row or -1; None in the masked layout
    row_slot: torch.Tensor              # int32 [rows], token * topk + j of the row's slot, or -1
    slot_row: torch.Tensor              # int32 [tokens, topk], row of the slot, or -1
    counts: torch.Tensor                # int32 [experts]: slots of each expert (masked layout: masked_m)

    @property
    def rows(self) -> int:
        return self.row_slot.shape[0]


def _refuse(t: torch.Tensor, name: str, dtypes, dim: int) -> None:
    if t.dtype not in dtypes or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor of type {' or '.join(str(d) for d in dtypes)}, "
                        f"got {t.dtype} on {t.device}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")
    if t.numel() > 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")


# The checks run on every call, and a small call costs little more than they do: one
# expression for the usual case, and the reason is worked out on refusal.
def _device(t: torch.Tensor, name: str, dtypes, dim: int) -> torch.Tensor:
    if t.dtype not in dtypes or t.get_device() < 0 or t.dim() != dim or t.stride(-1) != 1:
        _refuse(t, name, dtypes, dim)
    return t


def _ld(t: torch.Tensor, cols: int) -> int:
    """Row stride; a matrix of at most one row may carry any."""
    ld = t.stride(0)
    return ld if ld >= cols or t.shape[0] > 1 else cols


def _same_device(first: torch.Tensor, *others: Optional[torch.Tensor]) -> None:
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"a tensor is on {t.device}, the first on {first.device}")


def _out(t: Optional[torch.Tensor], shape, dtype, like: torch.Tensor, name: str) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _device(t, name, (dtype,), len(shape))
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _codes8(q: Optional[torch.Tensor], rows: int, k: int, like: torch.Tensor) -> torch.Tensor:
    """int8 codes [rows, k]; allocated here, rows begin at 128-byte lines, which the GEMM reads up to a third faster than
    rows that straddle them."""
    if q is not None or k % 128 == 0:
        return _out(q, (rows, k), torch.int8, like, "q")
    return torch.empty((rows, (k + 127) // 128 * 128), dtype=torch.int8, device=like.device)[:, :k]


def _score(score: str) -> int:
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    return _SCORES[score]


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
    _device(logits, "logits", _DTYPES, 2)
    t, e = logits.shape
    if group_score not in ("max", "top2"):
        raise ValueError(f"group_score must be 'max' or 'top2', got {group_score!r}")
    if bias is not None:
        _device(bias, "bias", (torch.float32,), 1)
        if bias.shape[0] != e:
            raise ValueError(f"bias must have {e} elements, got {bias.shape[0]}")
    indices = _out(indices, (t, topk), torch.int32, logits, "indices")
    weights = _out(weights, (t, topk), torch.float32, logits, "weights")
    _same_device(logits, bias, indices, weights)
    _check(lib.dg_route_topk(logits.data_ptr(), _DTYPES[logits.dtype], _ld(logits, e),
                             None if bias is None else bias.data_ptr(), indices.data_ptr(), _ld(indices, topk),
                             weights.data_ptr(), _ld(weights, topk), t, e, topk, num_expert_groups, topk_groups,
                             group_score == "top2", _score(score), bool(renormalize), scale, _stream()),
           "dg_route_topk")
    return indices, weights


def route_topk_grad(logits: torch.Tensor, indices: torch.Tensor, dweights: torch.Tensor, *, score: str = "softmax",
                    renormalize: bool = True, scale: float = 1.0,
                    dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of ``route_topk``'s weights: dlogits [tokens, experts] of the logits' type.

    indices int32 and dweights fp32 are [tokens, topk]; the other arguments as they were given to ``route_topk``.
    The choice of experts is held fixed, so a bias or groups do not enter.
    """
    _device(logits, "logits", _DTYPES, 2)
    _device(indices, "indices", (torch.int32,), 2)
    _device(dweights, "dweights", (torch.float32,), 2)
    t, e = logits.shape
    topk = indices.shape[1]
    if indices.shape[0] != t or indices.shape != dweights.shape:
        raise ValueError(f"indices {tuple(indices.shape)} and dweights {tuple(dweights.shape)} must be [{t}, topk]")
    dlogits = _out(dlogits, (t, e), logits.dtype, logits, "dlogits")
    _same_device(logits, indices, dweights, dlogits)
    _check(lib.dg_route_topk_grad(logits.data_ptr(), _DTYPES[logits.dtype], _ld(logits, e), indices.data_ptr(),
                                  _ld(indices, topk), dweights.data_ptr(), _ld(dweights, topk), dlogits.data_ptr(), _ld(dlogits, e),
                                  t, e, topk, _score(score), bool(renormalize), scale, _stream()),
           "dg_route_topk_grad")
    return dlogits


def expert_layout_rows(tokens: int, topk: int, num_experts: int) -> int:
    """Rows that hold every routing of these sizes in the contiguous layout (a multiple of 128)."""
    return int(lib.dg_expert_layout_rows(int(tokens), int(topk), int(num_experts)))


def _layout_buffers(indices: torch.Tensor, num_experts: int, m_rows: int, rows: int):
    """m_indices, row_slot, slot_row, counts and the workspace (or None), as parts of one allocation."""
    t, k = indices.shape
    sizes = [max(m_rows, 0), max(rows, 0), t * k, max(num_experts, 0)]
    n = lib.dg_expert_layout_workspace_size(t, k, num_experts) // 4
    if n:
        sizes.append(-sum(sizes) % 4)                    # the workspace begins at a 16-byte boundary
        sizes.append(n)
    parts = torch.empty(sum(sizes), dtype=torch.int32, device=indices.device).split(sizes)
    return parts[0], parts[1], parts[2].view(t, k), parts[3], parts[5] if n else None


def expert_layout_contiguous(indices: torch.Tensor, num_experts: int, rows: Optional[int] = None) -> ExpertLayout:
    """Rows of the contiguous layout for a routing: experts in order, each from a multiple of 128 rows, an expert's
    slots in order of token and slot.

    indices int32 [tokens, topk]; others than 0..num_experts-1 get no row.  ``rows`` defaults to
    ``expert_layout_rows(...)``, which holds every routing; with fewer, slots beyond them are dropped.
    """
    _device(indices, "indices", (torch.int32,), 2)
    t, k = indices.shape
    if rows is None:
        rows = expert_layout_rows(t, k, num_experts)
    m_indices, row_slot, slot_row, counts, ws = _layout_buffers(indices, num_experts, rows, rows)
    _check(lib.dg_expert_layout_contiguous(indices.data_ptr(), _ld(indices, k), t, k, num_experts, rows,
                                           m_indices.data_ptr(), row_slot.data_ptr(), slot_row.data_ptr(),
                                           counts.data_ptr(), None if ws is None else ws.data_ptr(),
                                           0 if ws is None else 4 * ws.numel(), _stream()), "dg_expert_layout_contiguous")
    return ExpertLayout(m_indices, row_slot, slot_row, counts)


def expert_layout_masked(indices: torch.Tensor, num_experts: int, max_m: int) -> ExpertLayout:
    """Rows of the masked layout: expert e's slots get rows e * max_m, e * max_m + 1, ... (a [experts, max_m, ...]
    tensor seen as [experts * max_m, ...]); slots past max_m are dropped.  ``counts`` is the GEMM's masked_m."""
    _device(indices, "indices", (torch.int32,), 2)
    t, k = indices.shape
    _, row_slot, slot_row, masked_m, ws = _layout_buffers(indices, num_experts, 0, num_experts * max_m)
    _check(lib.dg_expert_layout_masked(indices.data_ptr(), _ld(indices, k), t, k, num_experts, max_m,
                                       masked_m.data_ptr(), row_slot.data_ptr(), slot_row.data_ptr(),
                                       None if ws is None else ws.data_ptr(), 0 if ws is None else 4 * ws.numel(),
                                       _stream()), "dg_expert_layout_masked")
    return ExpertLayout(None, row_slot, slot_row, masked_m)


def _dispatch_args(x: torch.Tensor, slot_row: torch.Tensor, rows: Optional[int], q: Optional[torch.Tensor]):
    _device(x, "x", (torch.bfloat16, torch.float32), 2)
    _device(slot_row, "slot_row", (torch.int32,), 2)
    if slot_row.shape[0] != x.shape[0]:
        raise ValueError(f"slot_row has {slot_row.shape[0]} tokens, x has {x.shape[0]}")
    if q is not None:
        if rows is not None and rows != q.shape[0]:
            raise ValueError(f"q has {q.shape[0]} rows, expected {rows}")
        rows = q.shape[0]
    if rows is None:
        raise ValueError("rows (or q) must be given")
    return rows


def dispatch_cast_fp8(x: torch.Tensor, slot_row: torch.Tensor, rows: Optional[int] = None, ue8m0: bool = False,
                      q: Optional[torch.Tensor] = None, sf: Optional[torch.Tensor] = None):
    """Cast of token rows into their experts' rows: (E4M3 codes [rows, k], fp32 scales [rows, k/128]).

    x bf16 or fp32 [tokens, k]; slot_row int32 [tokens, topk] as a layout holds it (no row twice).  Codes and scales
    are ``per_token_cast_fp8``'s.  Rows without a slot are left untouched (unspecified in tensors allocated here);
    the grouped GEMMs do not use them.  ``sf`` may have any strides; allocated here, a block's scales lie beside one
    another along the rows, as the GEMMs read them best.
    """
    rows = _dispatch_args(x, slot_row, rows, q)
    (t, k), topk = x.shape, slot_row.shape[1]
    if q is None:
        q = torch.empty((rows, k), dtype=torch.float8_e4m3fn, device=x.device)
    if sf is None:
        sf = torch.empty((k // 128, rows), dtype=torch.float32, device=x.device).t()
    _device(q, "q", (torch.float8_e4m3fn, torch.uint8), 2)
    if sf.dtype != torch.float32 or not sf.is_cuda or tuple(sf.shape) != (rows, k // 128):
        raise ValueError(f"sf must be an fp32 device tensor of shape {(rows, k // 128)}")
    if q.shape[1] != k:
        raise ValueError(f"q must have {k} columns, got {q.shape[1]}")
    _same_device(x, slot_row, q, sf)
    _check(lib.dg_dispatch_cast_fp8(x.data_ptr(), _DTYPES[x.dtype], _ld(x, k), slot_row.data_ptr(), _ld(slot_row, topk),
                                    q.data_ptr(), _ld(q, k), sf.data_ptr(), sf.stride(0), sf.stride(1), t,
                                    topk, rows, k, bool(ue8m0), _stream()), "dg_dispatch_cast_fp8")
    return q, sf


def dispatch_cast_int8(x: torch.Tensor, slot_row: torch.Tensor, rows: Optional[int] = None,
                       q: Optional[torch.Tensor] = None, sf: Optional[torch.Tensor] = None):
    """As ``dispatch_cast_fp8`` with the int8 cast: (int8 codes [rows, k], fp32 scales [rows])."""
    rows = _dispatch_args(x, slot_row, rows, q)
    (t, k), topk = x.shape, slot_row.shape[1]
    q = _codes8(q, rows, k, x)
    if sf is None:
        sf = torch.empty(rows, dtype=torch.float32, device=x.device)
    if sf.dtype != torch.float32 or not sf.is_cuda or tuple(sf.shape) != (rows,):
        raise ValueError(f"sf must be an fp32 device tensor of shape {(rows,)}")
    _same_device(x, slot_row, q, sf)
    _check(lib.dg_dispatch_cast_int8(x.data_ptr(), _DTYPES[x.dtype], _ld(x, k), slot_row.data_ptr(), _ld(slot_row, topk),
                                     q.data_ptr(), _ld(q, k), sf.data_ptr(), sf.stride(0), t, topk, rows,
                                     k, _stream()), "dg_dispatch_cast_int8")
    return q, sf


def combine(y: torch.Tensor, slot_row: torch.Tensor, weights: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] * y[slot_row[t, j]] over the slots that have a row.

    y bf16 [rows, h]; slot_row int32 and weights fp32 [tokens, topk] (None: all ones, which makes this the gradient of
    dispatching tokens to rows); out bf16 (default) or fp32 [tokens, h].  Sums are fp32, in slot order.
    """
    _device(y, "y", (torch.bfloat16,), 2)
    _device(slot_row, "slot_row", (torch.int32,), 2)
    t, k = slot_row.shape
    rows, h = y.shape
    if weights is not None:
        _device(weights, "weights", (torch.float32,), 2)
        if weights.shape != slot_row.shape:
            raise ValueError(f"weights must have shape {(t, k)}, got {tuple(weights.shape)}")
    if out is None:
        out = torch.empty((t, h), dtype=torch.bfloat16, device=y.device)
    _device(out, "out", (torch.bfloat16, torch.float32), 2)
    if out.shape != (t, h):
        raise ValueError(f"out must have shape {(t, h)}, got {tuple(out.shape)}")
    _same_device(y, slot_row, weights, out)
    _check(lib.dg_combine(y.data_ptr(), _ld(y, h), slot_row.data_ptr(), _ld(slot_row, k),
                          None if weights is None else weights.data_ptr(), 0 if weights is None else _ld(weights, k),
                          out.data_ptr(), _DTYPES[out.dtype], _ld(out, h), t, k, rows, h, _stream()), "dg_combine")
    return out


def combine_grad(dout: torch.Tensor, y: torch.Tensor, slot_row: torch.Tensor, row_slot: torch.Tensor,
                 weights: torch.Tensor, dy: Optional[torch.Tensor] = None,
                 dweights: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gradient of ``combine``: (dy bf16 [rows, h], dweights fp32 [tokens, topk]).

    dout bf16 [tokens, h]; y, slot_row and weights as given to ``combine``; row_slot from the same layout.  Rows of dy
    without a slot, and dweights of slots without a row, are zero.
    """
    _device(dout, "dout", (torch.bfloat16,), 2)
    _device(y, "y", (torch.bfloat16,), 2)
    _device(slot_row, "slot_row", (torch.int32,), 2)
    _device(row_slot, "row_slot", (torch.int32,), 1)
    _device(weights, "weights", (torch.float32,), 2)
    t, k = slot_row.shape
    rows, h = y.shape
    if dout.shape != (t, h) or weights.shape != slot_row.shape or row_slot.shape[0] != rows:
        raise ValueError(f"dout must have shape {(t, h)}, weights {(t, k)} and row_slot {(rows,)}, got "
                         f"{tuple(dout.shape)}, {tuple(weights.shape)} and {tuple(row_slot.shape)}")
    dy = _out(dy, (rows, h), torch.bfloat16, y, "dy")
    dweights = _out(dweights, (t, k), torch.float32, y, "dweights")
    _same_device(y, dout, slot_row, row_slot, weights, dy, dweights)
    _check(lib.dg_combine_grad(dout.data_ptr(), _ld(dout, h), y.data_ptr(), _ld(y, h), slot_row.data_ptr(), _ld(slot_row, k),
                               row_slot.data_ptr(), weights.data_ptr(), _ld(weights, k), dy.data_ptr(), _ld(dy, h),
                               dweights.data_ptr(), _ld(dweights, k), t, k, rows, h, _stream()), "dg_combine_grad")
    return dy, dweights
