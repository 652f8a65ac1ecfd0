"""int8 GEMMs with a scale per token and per channel, and the int8 cast.

Operands are pairs ``(codes, scales)`` as in the FP8 GEMMs: int8 codes, K-major,
and fp32 scales, one for each row of A and of B (any stride).  Outputs are
bfloat16, float16 or float32 of any width and row stride.  Argument marshalling
only (in ``csrc/binding.cpp``); the contract is in ``include/dgfp8.h``.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _AUTO, _native

Pair = Tuple[torch.Tensor, torch.Tensor]


def per_token_cast_int8(x: torch.Tensor, q: Optional[torch.Tensor] = None, sf: Optional[torch.Tensor] = None) -> Pair:
    """x bf16 or fp32 [m, k] -> (int8 codes [m, k], fp32 scales [m]): s = max(amax, 1e-4) / 127, q = round(x / s).

    Rows whose maximum lies below 1e-4 use fewer than 127 steps.

    Codes allocated here have rows that begin at 128-byte lines (a row stride above k where k is no multiple of 128);
    weights laid out once are best kept that way too.
    """
    return _native.per_token_cast_int8(x, q, sf)


def int8_gemm_nt(a: Pair, b: Pair, d: torch.Tensor, workspace=_AUTO) -> torch.Tensor:
    """d[m, n] = sfa[m] * sfb[n] * sum_k a[m, k] * b[n, k], the sums exact.

    a = (codes [m, k], sfa [m]); b = (codes [n, k], sfb [n]); d bf16, fp16 or fp32 [m, n] is overwritten and returned.
    ``workspace`` as for ``fp8_gemm_nt``; it changes the time only, never a bit.
    """
    (qa, sa), (qb, sb) = a, b
    return _native.int8_gemm_nt(qa, sa, qb, sb, d, workspace)


def m_grouped_int8_gemm_nt_contiguous(a: Pair, b: Pair, d: torch.Tensor, m_indices: torch.Tensor,
                                      workspace=_AUTO) -> torch.Tensor:
    """Contiguous layout: a = (codes [m_total, k], sfa [m_total]), b = (codes [G, n, k], sfb [G, n]), d [m_total, n],
    m_indices int32 [m_total]; rows of -1 are left untouched (see ``m_grouped_fp8_gemm_nt_contiguous``)."""
    (qa, sa), (qb, sb) = a, b
    return _native.int8_contiguous(qa, sa, qb, sb, d, m_indices, workspace)


def m_grouped_int8_gemm_nt_masked(a: Pair, b: Pair, d: torch.Tensor, masked_m: torch.Tensor,
                                  expected_m: int) -> torch.Tensor:
    """Masked layout: a = (codes [G, max_m, k], sfa [G, max_m]), b = (codes [G, n, k], sfb [G, n]), d [G, max_m, n],
    masked_m int32 [G] read on the device; rows >= masked_m[g] are left untouched.  ``expected_m``: a hint."""
    (qa, sa), (qb, sb) = a, b
    return _native.int8_masked(qa, sa, qb, sb, d, masked_m, expected_m)
