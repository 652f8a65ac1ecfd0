"""Around a layer's products: norm, gated activation, and weights' gradients.

The norm adds the residual and writes rows or the next product's 8-bit operand; the gated activation
writes the second product's operand and, for training, an 8-bit checkpoint of its input;
the gradients read what the forward pass kept.  A mixture-of-experts layer's training step:

    y, h, rstd = rms_norm(x, w, residual)
    a = dispatch_cast_fp8(y, layout.slot_row, rows=layout.rows)           # kept: the first product's operand
    m_grouped_fp8_gemm_nt_contiguous(a, up, gate_up, layout.m_indices)
    act, kept = swiglu_checkpoint_fp8(gate_up, m_indices=layout.m_indices)  # both kept
    m_grouped_fp8_gemm_nt_contiguous(act, down, rows, layout.m_indices)
    ...
    m_grouped_weight_grad_contiguous(drows, act, d_down, layout.counts)
    dh, g = swiglu_grad_cast_fp8(dact, kept, m_indices=layout.m_indices)
    m_grouped_weight_grad_contiguous(dh, a, d_up, layout.counts)

With ``ue8m0=True`` in the casts whose codes a weight's gradient reads, its products are exact; with the casts' default
scales each value is rounded to bfloat16 first.

Argument marshalling only (in ``csrc/binding.cpp``); the contract is in ``include/dgfp8.h``.  Autograd records none of
the calls.
"""
from __future__ import annotations

from typing import Optional, Tuple, Union

import torch

from . import _native

Pair = Tuple[torch.Tensor, torch.Tensor]
Rows = Union[torch.Tensor, Pair]


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None, *,
             eps: float = 1e-6, y: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
             rstd: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, h, rstd): h = x + residual, rstd = (mean h^2 + eps)^-1/2 of each row, y = h * rstd * weight.

    x float32, bfloat16 or float16 [rows, k] (k a multiple of 8 up to 16384); residual like x, or None: h is x itself;
    weight [k] of x's type or float32, or None: ones.  y and h have x's type, rstd float32 [rows].  The norm is that of
    the rounded h.  y and h may be given x or residual to be written in place, y not x where x is the h that is returned
    (no residual, no h given).  Without columns rstd is NaN: the mean of nothing.
    """
    return _native.rms_norm(x, weight, residual, eps, y, h, rstd)


def rms_norm_cast_fp8(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                      *, eps: float = 1e-6, ue8m0: bool = False, q: Optional[torch.Tensor] = None,
                      sf: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                      h: Optional[torch.Tensor] = None,
                      rstd: Optional[torch.Tensor] = None) -> Tuple[Pair, torch.Tensor, torch.Tensor]:
    """((codes, scales), h, rstd): ``rms_norm`` with the FP8 cast of its fp32 rows: E4M3 [rows, k], fp32 [rows, k/128],
    k a multiple of 128.

    ``y`` given: also the rows themselves, for a router or another layer.  ``sf`` may have any strides; allocated here,
    a block's scales lie beside one another along the rows, as the GEMMs read them best.  A NaN in a block makes its
    scale NaN.
    """
    return _native.rms_norm_cast_fp8(x, weight, residual, eps, ue8m0, q, sf, y, h, rstd)


def rms_norm_cast_int8(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                       *, eps: float = 1e-6, q: Optional[torch.Tensor] = None, sf: Optional[torch.Tensor] = None,
                       y: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                       rstd: Optional[torch.Tensor] = None) -> Tuple[Pair, torch.Tensor, torch.Tensor]:
    """As ``rms_norm_cast_fp8`` with the int8 cast: (int8 codes [rows, k], fp32 scales [rows]), k a multiple of 16.
    Without columns the scales are those of rows of zeros."""
    return _native.rms_norm_cast_int8(x, weight, residual, eps, q, sf, y, h, rstd)


def rms_norm_grad(dy: torch.Tensor, h: torch.Tensor, weight: Optional[torch.Tensor], rstd: torch.Tensor,
                  dh: Optional[torch.Tensor] = None, *, dx: Optional[torch.Tensor] = None,
                  dweight: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(dx, dweight): the gradient of x and of the residual (of dy's type), and of the weight (float32 [k]; None
    without a weight).

    dy, h: [rows, k] of one type; h and rstd as the norm gave them; dh: the gradient that reaches h by another way (the
    residual stream).  dx may be dy, h or dh.
    """
    return _native.rms_norm_grad(dy, h, weight, rstd, dh, dx, dweight)


def swiglu_cast_fp8(h: torch.Tensor, *, m_indices: Optional[torch.Tensor] = None,
                    masked_m: Optional[torch.Tensor] = None, ue8m0: bool = False, q: Optional[torch.Tensor] = None,
                    sf: Optional[torch.Tensor] = None) -> Pair:
    """FP8 cast of silu(h[:, :n]) * h[:, n:]: (E4M3 [rows, n], fp32 [rows, n/128]), n a multiple of 128.

    h float32, bfloat16 or float16 [rows, 2 n].  With ``m_indices`` (int32 [rows]) rows whose entry is negative are left
    untouched; with ``masked_m`` (int32 [groups]) h is the masked layout's [groups * max_m, 2 n], and rows of a group from
    masked_m[g] on are.  (Unspecified in tensors allocated here; the grouped GEMMs do not use them.)
    """
    return _native.swiglu_cast_fp8(h, m_indices, masked_m, ue8m0, q, sf)


def swiglu_checkpoint_fp8(h: torch.Tensor, *, m_indices: Optional[torch.Tensor] = None,
                          masked_m: Optional[torch.Tensor] = None, ue8m0: bool = False,
                          q: Optional[torch.Tensor] = None, sf: Optional[torch.Tensor] = None,
                          hq: Optional[torch.Tensor] = None,
                          hsf: Optional[torch.Tensor] = None) -> Tuple[Pair, Pair]:
    """``swiglu_cast_fp8`` and, from the same pass, the FP8 cast of h itself: the checkpoint that ``swiglu_grad`` takes in
    h's place, (E4M3 [rows, 2 n], fp32 [rows, 2 n / 128])."""
    return _native.swiglu_checkpoint_fp8(h, m_indices, masked_m, ue8m0, q, sf, hq, hsf)


def swiglu_cast_int8(h: torch.Tensor, *, m_indices: Optional[torch.Tensor] = None,
                     masked_m: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                     sf: Optional[torch.Tensor] = None) -> Pair:
    """As ``swiglu_cast_fp8`` with the int8 cast: (int8 codes [rows, n], fp32 scales [rows]), n a multiple of 16 up to
    16384.  Without columns the scales are those of rows of zeros."""
    return _native.swiglu_cast_int8(h, m_indices, masked_m, q, sf)


def _saved(h: Rows):
    return (None,) + tuple(h) if isinstance(h, (tuple, list)) else (h, None, None)


def swiglu_grad(da: torch.Tensor, h: Rows, *, m_indices: Optional[torch.Tensor] = None,
                masked_m: Optional[torch.Tensor] = None, dh: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of silu(h[:, :n]) * h[:, n:]: dh [rows, 2 n] of da's type.

    da [rows, n]; h: the tensor that the activation read (of da's type), or the checkpoint that
    ``swiglu_checkpoint_fp8`` made of it.  Other rows than the layout's are left untouched.  dh may be h.
    """
    return _native.swiglu_grad(da, *_saved(h), m_indices, masked_m, dh)


def swiglu_grad_cast_fp8(da: torch.Tensor, h: Rows, *, m_indices: Optional[torch.Tensor] = None,
                         masked_m: Optional[torch.Tensor] = None, ue8m0: bool = False,
                         dh: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                         sf: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Pair]:
    """(dh, (codes, scales)): ``swiglu_grad`` and the FP8 cast of its fp32 values, for the product that carries the
    gradient on."""
    return _native.swiglu_grad_cast_fp8(da, *_saved(h), m_indices, masked_m, ue8m0, dh, q, sf)


def _operand(x: Rows):
    return tuple(x) if isinstance(x, (tuple, list)) else (x, None)


def weight_grad(dy: torch.Tensor, x: Rows, dw: torch.Tensor, *, accumulate: bool = False) -> torch.Tensor:
    """dw[n, k] = sum over the rows of dy[r, n] * x[r, k] (added to dw with ``accumulate``); returns dw.

    dy bfloat16 [rows, n]; x bfloat16 [rows, k], or the FP8 operand (codes [rows, k], scales [rows, k/128]) that the
    forward product read; dw float32 or bfloat16 [n, k] (float32 with ``accumulate``).  n and k multiples of 8 (codes: k of
    128).  Codes enter exactly where their scales are powers of two, otherwise rounded to bfloat16.
    """
    return _native.weight_grad(dy, *_operand(x), dw, accumulate)


def m_grouped_weight_grad_contiguous(dy: torch.Tensor, x: Rows, dw: torch.Tensor, counts: torch.Tensor, *,
                                     alignment: int = 128, accumulate: bool = False) -> torch.Tensor:
    """``weight_grad`` for each group of rows: dw [groups, n, k], counts int32 [groups] (a layout's ``counts``), read on
    the device.  Groups start at multiples of ``alignment`` rows: 128 as ``expert_layout_contiguous`` places them, 1
    for rows without padding.  Groups without rows get zeros."""
    return _native.weight_grad_contiguous(dy, *_operand(x), dw, counts, alignment, accumulate)


def m_grouped_weight_grad_masked(dy: torch.Tensor, x: Rows, dw: torch.Tensor, masked_m: torch.Tensor, *,
                                 accumulate: bool = False) -> torch.Tensor:
    """``weight_grad`` for each group of the masked layout: dy and x [groups * max_m, ...], dw [groups, n, k], masked_m
    int32 [groups] read on the device."""
    return _native.weight_grad_masked(dy, *_operand(x), dw, masked_m, accumulate)
