"""The 64-bit definitions of the norm, the gated activation and the weights' gradients against worked examples,
central differences and brute force."""
import numpy as np
import pytest

from oracle import layer


def differences(f, x, step=1e-6):
    """Gradient of the scalar f at x by central differences."""
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        at = x.copy()
        at[i] += step
        up = f(at)
        at[i] -= 2 * step
        out[i] = (up - f(at)) / (2 * step)
    return out


def test_norm_worked():
    y, rstd = layer.rms_norm([[3.0, -4.0, 0.0, 0.0]], [1, 2, 3, 4])
    assert rstd[0] == 0.4 and np.allclose(y, [[1.2, -3.2, 0, 0]], rtol=1e-15)
    y, rstd = layer.rms_norm(np.zeros((2, 8)), eps=0.25)
    assert np.all(y == 0) and np.all(rstd == 2)
    y, _ = layer.rms_norm(np.full((1, 16), 7.0))
    assert np.allclose(y, 1, rtol=1e-15)


@pytest.mark.parametrize("through", [False, True])
def test_norm_gradient_is_that_of_differences(through):
    rng = np.random.default_rng(0)
    h, dy, w = rng.normal(size=(3, 8)), rng.normal(size=(3, 8)), rng.normal(size=8)
    dh = rng.normal(size=(3, 8)) if through else None
    dx, dw = layer.rms_norm_grad(dy, h, w, layer.rms_norm(h, w, 0.1)[1], dh)

    def loss(hh, ww):
        return np.sum(dy * layer.rms_norm(hh, ww, 0.1)[0]) + (np.sum(dh * hh) if through else 0)
    # central differences: rounding 1e-16 / 1e-6 against curvature 1e-12
    assert np.allclose(dx, differences(lambda v: loss(v, w), h), atol=1e-8)
    assert np.allclose(dw, differences(lambda v: loss(h, v), w), atol=1e-8)


def test_swiglu_worked_and_its_ends():
    a = layer.swiglu([[0.0, np.log(3.0), 800.0, -800.0, 5.0, 8.0, 2.0, 2.0]])
    assert np.allclose(a, [[0, np.log(3.0) * 0.75 * 8, 1600, 0]], rtol=1e-15)


def test_swiglu_gradient_is_that_of_differences():
    rng = np.random.default_rng(1)
    h, da = rng.normal(size=(3, 12)) * 3, rng.normal(size=(3, 6))
    want = differences(lambda v: np.sum(da * layer.swiglu(v)), h)
    assert np.allclose(layer.swiglu_grad(da, h), want, atol=1e-8)


def test_segments():
    assert layer.segments([3, 0, 130, -4, 1], 1000) == [(0, 3), (128, 0), (128, 130), (384, 0), (384, 1)]
    assert layer.segments([3, 0, 5], 1000, alignment=1) == [(0, 3), (3, 0), (3, 5)]
    assert layer.segments([200, 100], 256) == [(0, 200), (256, 0)]
    assert layer.segments([5, 9, 0], 24, max_m=8) == [(0, 5), (8, 8), (16, 0)]


def test_weight_gradient_by_brute_force():
    rng = np.random.default_rng(2)
    dy, x = rng.integers(-4, 5, (20, 3)), rng.integers(-4, 5, (20, 4))
    segs = [(0, 7), (7, 0), (9, 11)]
    dw, size = layer.weight_grad(dy, x, segs)
    for g, (a, c) in enumerate(segs):
        for n in range(3):
            for k in range(4):
                terms = [int(dy[r, n]) * int(x[r, k]) for r in range(a, a + c)]
                assert dw[g, n, k] == sum(terms) and size[g, n, k] == sum(abs(t) for t in terms)


def test_a_weight_gradient_is_that_of_the_product():
    rng = np.random.default_rng(3)
    x, w, dy = rng.normal(size=(5, 4)), rng.normal(size=(3, 4)), rng.normal(size=(5, 3))
    want = differences(lambda v: np.sum(dy * (x @ v.T)), w)
    assert np.allclose(layer.weight_grad(dy, x, [(0, 5)])[0][0], want, atol=1e-8)


def test_codes_carry_their_block_s_scale():
    v = layer.widen_codes(np.ones((2, 256)), [[2.0, 0.5], [1.0, 4.0]])
    assert np.all(v[0, :128] == 2) and np.all(v[0, 128:] == 0.5) and np.all(v[1, 128:] == 4)
