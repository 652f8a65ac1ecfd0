"""Mixture-of-experts operators in 64 bits: routing and its gradient, expert
layout, combination and its gradient.

Test infrastructure only (see the package header).  Written from the
definitions, one token, slot or row at a time where that is clearer; nothing is
shared with the HIP path.
"""
from __future__ import annotations

import numpy as np

ALIGN = 128


def scores(x: np.ndarray, score: str) -> np.ndarray:
    """softmax over each row, or the sigmoid of each element; float64.  Elements that are -inf score 0; a NaN (or, under
    softmax, +inf) has no score: it is left out here, and its row is marked by ``route``."""
    x = np.asarray(x, np.float64)
    gone = np.isnan(x) | (x == -np.inf) | ((x == np.inf) & (score == "softmax"))
    s = np.zeros_like(x)
    for t in range(x.shape[0]):
        v = x[t, ~gone[t]]
        if v.size == 0:
            continue
        if score == "softmax":
            e = np.exp(v - v.max())
            s[t, ~gone[t]] = e / e.sum()
        else:
            with np.errstate(over="ignore"):
                s[t, ~gone[t]] = 1.0 / (1.0 + np.exp(-v))
    return s


def route(x, topk, score="softmax", bias=None, groups=1, topk_groups=1, group_score="max", renormalize=True,
          scale=1.0):
    """(indices int32 [T, k], weights float64 [T, k], margin float64 [T]).

    margin: the least gap between keys (or group scores) that the row's choice or order hangs on, as an fp32
    implementation can tell apart; inf where the order is that of the logits themselves or of equal logits."""
    x = np.asarray(x, np.float64)
    t_n, e_n = x.shape
    s = scores(x, score)
    b = np.zeros(e_n) if bias is None else np.asarray(bias, np.float64)
    with np.errstate(invalid="ignore"):
        biased = s + b
    key = x if bias is None else biased
    unscored = np.isnan(x) | ((x == np.inf) & (score == "softmax"))
    out = unscored | (x == -np.inf) | np.isnan(key) | (key == -np.inf)
    idx = np.full((t_n, topk), -1, np.int32)
    w = np.zeros((t_n, topk))
    margin = np.full(t_n, np.inf)
    size = e_n // groups
    for t in range(t_n):
        avail = [e for e in range(e_n) if not out[t, e]]
        if groups > 1:
            gs = []
            for g in range(groups):
                of = key if group_score == "max" else biased
                best = sorted((e for e in avail if e // size == g), key=lambda e: -of[t, e])
                best = best[:1 if group_score == "max" else 2]
                if best:
                    gs.append((sum(of[t, e] for e in best), g, [(x[t, e], b[e]) for e in best]))
            gs.sort(key=lambda p: (-p[0], p[1]))
            kept = {g[1] for g in gs[:topk_groups]}
            if topk_groups < len(gs) and not (group_score == "max" and bias is None):
                last, next_ = gs[topk_groups - 1], gs[topk_groups]
                if last[2] != next_[2]:                     # of the same terms: equal in any arithmetic
                    margin[t] = min(margin[t], last[0] - next_[0])
            avail = [e for e in avail if e // size in kept]
        order = sorted(avail, key=lambda e: (-key[t, e], e))
        if bias is not None:
            for a, c in zip(order[:topk], order[1:topk + 1]):
                if not (x[t, a] == x[t, c] and b[a] == b[c]):
                    margin[t] = min(margin[t], key[t, a] - key[t, c])
        pick = order[:topk]
        idx[t, :len(pick)] = pick
        sel = s[t, pick]
        if renormalize:
            if score == "softmax" and len(pick):       # the same quotient, also where every score underflows
                e = np.exp(x[t, pick] - x[t, pick].max())
                sel = e / e.sum()
            else:
                sel = sel / sel.sum() if sel.sum() > 0 else np.zeros_like(sel)
        bad = unscored[t].any() or (bias is not None and (np.isnan(b) & (x[t] > -np.inf)).any())
        w[t, :len(pick)] = np.nan if bad else scale * sel
    return idx, w, margin


def weights_at(x, idx, score, renormalize, scale):
    """Weights of a fixed choice (indices of -1 unused), float64: what the gradient is the gradient of."""
    s = scores(x, score)
    w = np.zeros(idx.shape)
    for t in range(x.shape[0]):
        on = idx[t] >= 0
        v = s[t, idx[t, on]]
        if renormalize:
            v = v / v.sum() if v.sum() > 0 else np.zeros_like(v)
        w[t, on] = scale * v
    return w


def route_grad(x, idx, g, score="softmax", renormalize=True, scale=1.0):
    """dlogits float64 [T, E], from the matrix of derivatives of the chosen scores by the logits."""
    x = np.asarray(x, np.float64)
    s = scores(x, score)
    dx = np.zeros_like(x)
    for t in range(x.shape[0]):
        on = np.flatnonzero(idx[t] >= 0)
        if on.size == 0:
            continue
        e = idx[t, on]
        gj, sj = scale * np.asarray(g, np.float64)[t, on], s[t, e]
        if renormalize:
            total = sj.sum()
            if total == 0:
                continue
            ds = gj / total - (gj * sj).sum() / total ** 2
        else:
            ds = gj
        if score == "sigmoid":
            for a, c in zip(e, ds * sj * (1 - sj)):
                dx[t, a] += c
        else:
            jac = -np.outer(s[t], sj)                   # d s_e' / d x: s_e' ([e == e'] - s_e)
            jac[e, np.arange(e.size)] += sj
            dx[t] = jac @ ds
    return dx


def layout_contiguous(idx, experts, rows):
    """(m_indices, row_slot, slot_row, counts) as the definition places them, slot by slot."""
    idx = np.asarray(idx)
    counts = np.zeros(experts, np.int32)
    for e in idx.ravel():
        if 0 <= e < experts:
            counts[e] += 1
    start = np.concatenate([[0], np.cumsum(-(-counts // ALIGN) * ALIGN)])
    m_indices = np.full(rows, -1, np.int32)
    row_slot = np.full(rows, -1, np.int32)
    slot_row = np.full(idx.size, -1, np.int32)
    seen = np.zeros(experts, np.int64)
    for s, e in enumerate(idx.ravel()):
        if not 0 <= e < experts:
            continue
        r = start[e] + seen[e]
        seen[e] += 1
        if r < rows:
            m_indices[r], row_slot[r], slot_row[s] = e, s, r
    return m_indices, row_slot, slot_row.reshape(idx.shape), counts


def layout_masked(idx, experts, max_m):
    """(row_slot, slot_row, masked_m)."""
    idx = np.asarray(idx)
    row_slot = np.full(experts * max_m, -1, np.int32)
    slot_row = np.full(idx.size, -1, np.int32)
    masked_m = np.zeros(experts, np.int32)
    for s, e in enumerate(idx.ravel()):
        if 0 <= e < experts and masked_m[e] < max_m:
            r = e * max_m + masked_m[e]
            masked_m[e] += 1
            row_slot[r], slot_row[s] = s, r
    return row_slot, slot_row.reshape(idx.shape), masked_m


def combine(y, slot_row, weights=None):
    """out float64 [T, H]; rows outside y are skipped and never read."""
    y = np.asarray(y, np.float64)
    t_n, k = slot_row.shape
    out = np.zeros((t_n, y.shape[1]))
    for t in range(t_n):
        for j in range(k):
            r = slot_row[t, j]
            if 0 <= r < y.shape[0]:
                out[t] += (1.0 if weights is None else float(weights[t, j])) * y[r]
    return out


def combine_grad(dout, y, slot_row, weights):
    """(dy, dweights) in float64."""
    dout, y = np.asarray(dout, np.float64), np.asarray(y, np.float64)
    dy, dw = np.zeros_like(y), np.zeros(slot_row.shape)
    for t in range(slot_row.shape[0]):
        for j in range(slot_row.shape[1]):
            r = slot_row[t, j]
            if 0 <= r < y.shape[0]:
                dy[r] = float(weights[t, j]) * dout[t]
                dw[t, j] = dout[t] @ y[r]
    return dy, dw
