"""Pins of the mixture-of-experts oracle: worked examples, and its gradients
against central differences of its own forward definitions."""
import numpy as np
import pytest

from oracle import moe


def test_route_worked_example():
    x = np.log([[1.0, 2.0, 3.0, 4.0]])                       # softmax: 0.1 0.2 0.3 0.4
    idx, w, _ = moe.route(x, 2, renormalize=False)
    assert idx.tolist() == [[3, 2]] and np.allclose(w, [[0.4, 0.3]])
    idx, w, _ = moe.route(x, 2, renormalize=True, scale=7.0)
    assert np.allclose(w, [[4.0, 3.0]])
    idx, w, _ = moe.route(x, 2, bias=np.array([0.5, 0.0, 0.0, 0.0]), renormalize=False)
    assert idx.tolist() == [[0, 3]] and np.allclose(w, [[0.1, 0.4]])   # the bias chooses, it does not weigh
    idx, _, _ = moe.route(x, 2, groups=2, topk_groups=1)
    assert idx.tolist() == [[3, 2]]
    # group 0 holds the larger sum, group 1 the larger single score
    s = np.array([[0.45, 0.45, 0.6, 0.1]])
    x = np.log(s / (1 - s))
    assert moe.route(x, 1, score="sigmoid", groups=2, topk_groups=1, group_score="top2")[0].tolist() == [[0]]
    assert moe.route(x, 1, score="sigmoid", groups=2, topk_groups=1, group_score="max")[0].tolist() == [[2]]


def test_route_masks_and_ties():
    inf = np.inf
    idx, w, _ = moe.route(np.array([[0.0, 0.0, 0.0], [-inf, 1.0, -inf], [-inf] * 3, [np.nan, 1.0, 2.0]]), 2)
    assert idx.tolist() == [[0, 1], [1, -1], [-1, -1], [2, 1]]
    assert np.allclose(w[:3], [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0]]) and np.isnan(w[3]).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_grad_against_differences(score, renormalize):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 7))
    x[3, 2] = -np.inf
    idx, _, _ = moe.route(x, 3, score=score)
    idx[1, 2] = -1
    g = rng.standard_normal((4, 3))
    dx = moe.route_grad(x, idx, g, score, renormalize, 1.7)
    h = 1e-6
    for t in range(4):
        for e in range(7):
            if np.isinf(x[t, e]):
                assert dx[t, e] == 0
                continue
            hi, lo = x.copy(), x.copy()
            hi[t, e] += h
            lo[t, e] -= h
            f = [(g * moe.weights_at(v, idx, score, renormalize, 1.7)).sum() for v in (hi, lo)]
            assert abs((f[0] - f[1]) / (2 * h) - dx[t, e]) < 1e-8


def test_layouts_worked_example():
    idx = np.array([[1, 0], [1, -1], [2, 1]])
    m, row_slot, slot_row, counts = moe.layout_contiguous(idx, 3, 512)
    assert counts.tolist() == [1, 3, 1]
    assert slot_row.tolist() == [[128, 0], [129, -1], [256, 130]]
    assert row_slot[[0, 128, 129, 130, 256]].tolist() == [1, 0, 2, 5, 4] and (row_slot >= 0).sum() == 5
    assert m[[0, 1, 128, 130, 131, 256, 384]].tolist() == [0, -1, 1, 1, -1, 2, -1]
    row_slot, slot_row, masked_m = moe.layout_masked(idx, 3, 2)
    assert masked_m.tolist() == [1, 2, 1] and slot_row.tolist() == [[2, 0], [3, -1], [4, -1]]
    assert row_slot.tolist() == [1, -1, 0, 2, 4, -1]


def test_combine_and_its_gradient_against_differences():
    rng = np.random.default_rng(6)
    y, w = rng.standard_normal((5, 3)), rng.standard_normal((2, 3))
    slot_row = np.array([[4, 0, -1], [2, -1, 1]])
    out = moe.combine(y, slot_row, w)
    assert np.allclose(out[0], w[0, 0] * y[4] + w[0, 1] * y[0])
    g = rng.standard_normal(out.shape)
    dy, dw = moe.combine_grad(g, y, slot_row, w)
    h = 1e-6
    for a, grad in ((y, dy), (w, dw)):
        for i in np.ndindex(a.shape):
            old = a[i]
            a[i] = old + h
            hi = (g * moe.combine(y, slot_row, w)).sum()
            a[i] = old - h
            lo = (g * moe.combine(y, slot_row, w)).sum()
            a[i] = old
            assert abs((hi - lo) / (2 * h) - grad[i]) < 1e-7
