"""int8 GEMMs with a scale per token and per channel, and the int8 cast.

Operands are pairs ``(codes, scales)`` as in the FP8 GEMMs: int8 codes, K-major,
and fp32 scales, one for each row of A and of B (any stride).  Outputs are
bfloat16, float16 or float32 of any width and row stride.  Argument marshalling
only; the contract is in ``include/dgfp8.h``.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _AUTO, _check, _stream, _workspace_arg, lib
from .moe import _DTYPES, _codes8, _device, _ld, _same_device

Pair = Tuple[torch.Tensor, torch.Tensor]


_CODES = (torch.int8,)


def _scales(s: torch.Tensor, name: str, shape) -> None:
    if s.dtype != torch.float32 or s.get_device() < 0:
        raise TypeError(f"{name} must be a float32 device tensor")
    if s.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(s.shape)}")


def _result(d: torch.Tensor, shape) -> None:
    _device(d, "d", _DTYPES, len(shape))
    if d.shape != shape:
        raise ValueError(f"d must have shape {tuple(shape)}, got {tuple(d.shape)}")


def _rows(t: torch.Tensor, cols: int) -> int:
    """Row stride of a [groups, rows, columns] tensor."""
    ld = t.stride(1)
    return ld if ld >= cols or t.shape[1] > 1 else cols


def per_token_cast_int8(x: torch.Tensor, q: Optional[torch.Tensor] = None, sf: Optional[torch.Tensor] = None) -> Pair:
    """x bf16 or fp32 [m, k] -> (int8 codes [m, k], fp32 scales [m]): s = max(amax, 1e-4) / 127, q = round(x / s).

    Codes allocated here have rows that begin at 128-byte lines (a row stride above k where k is no multiple of 128);
    weights laid out once are best kept that way too."""
    _device(x, "x", (torch.bfloat16, torch.float32), 2)
    m, k = x.shape
    q = _codes8(q, m, k, x)
    if sf is None:
        sf = torch.empty(m, dtype=torch.float32, device=x.device)
    _scales(sf, "sf", (m,))
    _same_device(x, q, sf)
    _check(lib.dg_per_token_cast_int8(x.data_ptr(), _DTYPES[x.dtype], _ld(x, k), q.data_ptr(), _ld(q, k), sf.data_ptr(),
                                      sf.stride(0), m, k, _stream()), "dg_per_token_cast_int8")
    return q, sf


def int8_gemm_nt(a: Pair, b: Pair, d: torch.Tensor, workspace=_AUTO) -> torch.Tensor:
    """d[m, n] = sfa[m] * sfb[n] * sum_k a[m, k] * b[n, k], the sums exact.

    a = (codes [m, k], sfa [m]); b = (codes [n, k], sfb [n]); d bf16, fp16 or fp32 [m, n] is overwritten and returned.
    ``workspace`` as for ``fp8_gemm_nt``; it changes the time only, never a bit.
    """
    (qa, sa), (qb, sb) = a, b
    _device(qa, "a", _CODES, 2)
    _device(qb, "b", _CODES, 2)
    (m, k), (n, kb) = qa.shape, qb.shape
    if kb != k:
        raise ValueError(f"a has {k} columns, b has {kb}")
    _scales(sa, "sfa", (m,))
    _scales(sb, "sfb", (n,))
    _result(d, (m, n))
    _same_device(qa, sa, qb, sb, d)
    ws_ptr, ws_bytes = _workspace_arg(workspace, d.device, lib.dg_int8_gemm_nt_workspace_size(m, n, k))
    _check(lib.dg_int8_gemm_nt(qa.data_ptr(), _ld(qa, k), sa.data_ptr(), sa.stride(0), qb.data_ptr(), _ld(qb, k),
                               sb.data_ptr(), sb.stride(0), d.data_ptr(), _DTYPES[d.dtype], _ld(d, n), m, n, k,
                               ws_ptr or None, ws_bytes, _stream()), "dg_int8_gemm_nt")
    return d


def m_grouped_int8_gemm_nt_contiguous(a: Pair, b: Pair, d: torch.Tensor, m_indices: torch.Tensor,
                                      workspace=_AUTO) -> torch.Tensor:
    """Contiguous layout: a = (codes [m_total, k], sfa [m_total]), b = (codes [G, n, k], sfb [G, n]), d [m_total, n],
    m_indices int32 [m_total]; rows of -1 are left untouched (see ``m_grouped_fp8_gemm_nt_contiguous``)."""
    (qa, sa), (qb, sb) = a, b
    _device(qa, "a", _CODES, 2)
    _device(qb, "b", _CODES, 3)
    (m, k), (g, n, kb) = qa.shape, qb.shape
    if kb != k:
        raise ValueError(f"a has {k} columns, b has {kb}")
    _scales(sa, "sfa", (m,))
    _scales(sb, "sfb", (g, n))
    _result(d, (m, n))
    _device(m_indices, "m_indices", (torch.int32,), 1)
    if m_indices.shape[0] != m:
        raise ValueError(f"m_indices must have {m} elements, got {m_indices.shape[0]}")
    _same_device(qa, sa, qb, sb, d, m_indices)
    need = int(lib.dg_m_grouped_int8_gemm_nt_contiguous_workspace_size(m, n, k, g))
    ws_ptr, ws_bytes = _workspace_arg(workspace, d.device, need)
    _check(lib.dg_m_grouped_int8_gemm_nt_contiguous(
        qa.data_ptr(), _ld(qa, k), sa.data_ptr(), sa.stride(0), qb.data_ptr(), _rows(qb, k), qb.stride(0),
        sb.data_ptr(), sb.stride(1), sb.stride(0), d.data_ptr(), _DTYPES[d.dtype], _ld(d, n), m_indices.data_ptr(),
        m, n, k, g,
        ws_ptr or None, ws_bytes, _stream()), "dg_m_grouped_int8_gemm_nt_contiguous")
    return d


def m_grouped_int8_gemm_nt_masked(a: Pair, b: Pair, d: torch.Tensor, masked_m: torch.Tensor,
                                  expected_m: int) -> torch.Tensor:
    """Masked layout: a = (codes [G, max_m, k], sfa [G, max_m]), b = (codes [G, n, k], sfb [G, n]), d [G, max_m, n],
    masked_m int32 [G] read on the device; rows >= masked_m[g] are left untouched.  ``expected_m``: a hint."""
    (qa, sa), (qb, sb) = a, b
    _device(qa, "a", _CODES, 3)
    _device(qb, "b", _CODES, 3)
    (g, m, k), n = qa.shape, qb.shape[1]
    if qb.shape != (g, n, k):
        raise ValueError(f"b must have shape {(g, n, k)}, got {tuple(qb.shape)}")
    _scales(sa, "sfa", (g, m))
    _scales(sb, "sfb", (g, n))
    _result(d, (g, m, n))
    _device(masked_m, "masked_m", (torch.int32,), 1)
    if masked_m.shape[0] != g:
        raise ValueError(f"masked_m must have {g} elements, got {masked_m.shape[0]}")
    _same_device(qa, sa, qb, sb, d, masked_m)
    _check(lib.dg_m_grouped_int8_gemm_nt_masked(
        qa.data_ptr(), _rows(qa, k), qa.stride(0), sa.data_ptr(), sa.stride(1), sa.stride(0), qb.data_ptr(),
        _rows(qb, k), qb.stride(0), sb.data_ptr(), sb.stride(1), sb.stride(0), d.data_ptr(), _DTYPES[d.dtype],
        _rows(d, n), d.stride(0), masked_m.data_ptr(), g, m, n, k, int(expected_m), _stream()),
        "dg_m_grouped_int8_gemm_nt_masked")
    return d
