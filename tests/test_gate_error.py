"""The sigmoid of the gated activation: its error does not grow with the gate as that of a rounded product's power would.

With u = 2^-24, g in [-87, 87] (e^-g and its reciprocal are normal numbers there), w = 1 - s, s = 1 / (1 + e^-g):
* t = fl(-g log2 e).  2^t is the hardware's, within a unit of the last place: 2 u.  What t's rounding left out comes back
  as the factor 1 + c, c = -g - t ln 2 in one rounding.  ln 2 in fp32 is off by 0.05 u of itself, which c takes |g| times:
  |g| u / 16 covers it.  The product and sum e + e c is rounded once: u.  c^2 / 2, what 1 + c leaves of e^c, is below
  (1.3 |g| u)^2, 2^-10 u.  In all e^-g is within (3 + |g| / 16) u, rounded up to (4 + |g| / 16) u.
* d = 1 + e^-g takes the share w of that, and rounds: u.  Its reciprocal, corrected once, rounds: u and a little.
  sigma = (3 + w (4 + |g| / 16)) u bounds the relative error of s.
* With da = up = 1 the gradient shows s itself: du = g s with one more rounding, |g| s (sigma + u).
  dg = fma(g s, 1 - s, s): g s is off by sigma + u of itself, 1 - s by s sigma and u of itself, s by s sigma, the sum by u:
  |g| s w (sigma + 2 u) + |g| s^2 sigma + s sigma + u |dg| = s (|g| + 1) sigma + 2 |g| s w u + u |dg|.
Without the correction e^-g is off by up to |g| u: at |g| = 80 seven times what is allowed here.
"""
import numpy as np
import pytest
import torch

from oracle import layer

U = 2.0 ** -24


def gates():
    """[16, 2048], the smallest magnitudes among them."""
    g = np.linspace(-87, 87, 16 * 2048).astype(np.float32)
    g[::97] = np.float32(2.0) ** np.linspace(-120, 6, g[::97].size).astype(np.float32)
    g[1::97] = -g[::97][:g[1::97].size]
    return np.random.default_rng(0).permutation(g).reshape(16, 2048)


def bounds(g):
    """(dg, du, and how far either may be off) for da = up = 1."""
    g = g.astype(np.float64)
    both = layer.swiglu_grad(np.ones_like(g), np.concatenate([g, np.ones_like(g)], 1))
    dg, du = np.split(both, 2, axis=1)
    s = layer.sigmoid(g)
    w = layer.sigmoid(-g)
    sigma = (3 + w * (4 + np.abs(g) / 16)) * U
    return dg, du, s * (np.abs(g) + 1) * sigma + 2 * np.abs(g) * s * w * U + U * np.abs(dg), np.abs(g) * s * (sigma + U)


def fma(a, b, c):
    return (np.float64(a) * np.float64(b) + np.float64(c)).astype(np.float32)


def in_fp32(g, corrected):
    """The kernel's formula in fp32, with exact powers of two."""
    one = np.float32(1)
    t = g * np.float32(-1.44269504088896341)
    e = np.exp2(t.astype(np.float64)).astype(np.float32)
    d = one + (fma(e, fma(t, np.float32(-0.693147180559945309), -g), e) if corrected else e)
    s = (1 / d.astype(np.float64)).astype(np.float32)
    gs = g * s
    return fma(gs, one - s, s), gs


def test_the_bound_tells_the_corrected_power_from_the_plain_one():
    g = gates()
    dg, du, off_g, off_u = bounds(g)
    a, b = in_fp32(g, True)
    assert np.all(np.abs(a - dg) <= off_g) and np.all(np.abs(b - du) <= off_u)
    a, b = in_fp32(g, False)
    assert np.sum(np.abs(a - dg) > off_g) > 1000 and np.sum(np.abs(b - du) > off_u) > 1000
    near = (np.abs(g) < 16) & (g < 0)                    # not at the far ends only
    assert np.any((np.abs(b - du) > off_u) & near)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
def test_gradient_shows_the_sigmoid():
    import moe_fp8_gemm_amd as dg
    g = gates()
    want_g, want_u, off_g, off_u = bounds(g)
    h = torch.from_numpy(np.concatenate([g, np.ones_like(g)], 1)).cuda()
    da = torch.ones(g.shape, device="cuda")
    for dh in (dg.swiglu_grad(da, h), dg.swiglu_grad_cast_fp8(da, h)[0]):
        got = dh.cpu().double().numpy()
        for name, v, want, off in (("dg", got[:, :2048], want_g, off_g), ("du", got[:, 2048:], want_u, off_u)):
            r = np.abs(v - want) / np.maximum(off, 1e-300)
            assert np.all(np.abs(v - want) <= off), f"{name}: {r.max()} of the bound at {g.reshape(-1)[r.argmax()]}"
