"""int8 cast and product with a scale per row of either operand.

Test infrastructure only (see the package header).  The sums are whole numbers in
64 bits; every later step is one IEEE fp32 operation, so the results are the
method's bits.
"""
from __future__ import annotations

import numpy as np

AMAX_FLOOR = np.float32(1e-4)


def cast(x: np.ndarray):
    """x fp32 (or bf16 widened) [M, K], finite -> (int8 codes, fp32 scales [M])."""
    x = np.asarray(x, np.float32)
    s = (np.maximum(np.abs(x).max(axis=1), AMAX_FLOOR) / np.float32(127)).astype(np.float32)
    q = np.rint((x / s[:, None]).astype(np.float32))
    return np.clip(q, -127, 127).astype(np.int8), s


def gemm_nt(qa: np.ndarray, sa: np.ndarray, qb: np.ndarray, sb: np.ndarray) -> np.ndarray:
    """fp32 [M, N]: fp32(sum) * sa * sb, each step rounded to fp32."""
    # products of two codes summed over K <= 131071 stay below 2^31: exact in float64
    acc = qa.astype(np.float64) @ qb.astype(np.float64).T
    with np.errstate(over="ignore", invalid="ignore"):
        return (acc.astype(np.float32) * np.asarray(sa, np.float32)[:, None]) * np.asarray(sb, np.float32)[None, :]

