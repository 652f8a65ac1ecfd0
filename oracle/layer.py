"""Norm, gated activation and weights' gradients in 64 bits.

Test infrastructure only (see the package header).  Written from the definitions; nothing is
shared with the HIP path.
"""
from __future__ import annotations

import numpy as np


def rms_norm(h, weight=None, eps=0.0):
    """(y, rstd) of rows h [rows, k]."""
    h = np.asarray(h, np.float64)
    rstd = 1.0 / np.sqrt(np.sum(h * h, axis=1) / h.shape[1] + eps)
    y = h * rstd[:, None]
    return (y if weight is None else y * np.asarray(weight, np.float64)), rstd


def rms_norm_grad(dy, h, weight, rstd, dh=None):
    """(dx, dweight) of sum(dy * y) + sum(dh * h): d rstd / d h_i = -rstd^3 h_i / k."""
    dy, h, rstd = (np.asarray(v, np.float64) for v in (dy, h, rstd))
    w = np.ones(h.shape[1]) if weight is None else np.asarray(weight, np.float64)
    r = rstd[:, None]
    dx = dy * w * r - r ** 3 * h / h.shape[1] * np.sum(dy * w * h, axis=1, keepdims=True)
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, np.sum(dy * h * r, axis=0)


def sigmoid(g):
    g = np.asarray(g, np.float64)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(h):
    """silu(gate) * up of rows [gate | up]."""
    h = np.asarray(h, np.float64)
    n = h.shape[1] // 2
    return h[:, :n] * sigmoid(h[:, :n]) * h[:, n:]


def swiglu_grad(da, h):
    """[d gate | d up]."""
    da, h = np.asarray(da, np.float64), np.asarray(h, np.float64)
    n = h.shape[1] // 2
    g, u, s = h[:, :n], h[:, n:], sigmoid(h[:, :n])
    return np.concatenate([da * u * (s + g * s * (1 - s)), da * g * s], axis=1)


def segments(counts, rows, alignment=128, max_m=0):
    """[(first row, rows)] of the groups: one after the other from multiples of `alignment`, or max_m rows each."""
    at, out = 0, []
    for g, c in enumerate(counts):
        c = max(0, int(c))
        if max_m:
            out.append((g * max_m, min(c, max_m)))
            continue
        first = min(at, rows)
        out.append((first, min(c, rows - first)))
        at += -(-c // alignment) * alignment
    return out


def weight_grad(dy, x, segs):
    """(dw [groups, n, k], sum of the terms' magnitudes)."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    dw = np.stack([dy[a:a + c].T @ x[a:a + c] for a, c in segs])
    return dw, np.stack([np.abs(dy[a:a + c]).T @ np.abs(x[a:a + c]) for a, c in segs])


def widen_codes(values, scales):
    """Values of codes (their E4M3 values, [rows, k]) times a scale for each 128 columns."""
    return np.asarray(values, np.float64) * np.repeat(np.asarray(scales, np.float64), 128, axis=1)
