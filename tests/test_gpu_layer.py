"""Norm, gated activation and weights' gradients on the GPU against the 64-bit definitions.

Tolerances, with u = 2^-24 (half a step of fp32) and half(t) = finfo(t).eps / 2 of a result's type t:
* A row's sum of squares has at most 8 * 8 products in one lane, 6 steps across a wave and 16 across waves: 90
  roundings on the longest path of positive terms, so rstd is off by at most 45 u and a mean, a root, a division: 50 u.
  y adds two products: Y = 64 u covers it.  The gradient's mean runs over terms of both signs: 100 u of the mean of
  their magnitudes.
* e^-g comes from a rounded product with log2 e (|g| u) and the hardware's 2^x (2 u), then a sum, a reciprocal (2 u) and
  two products: (|g| + 8) u of the result; where e^-g leaves fp32's normal range, 2^-118 of the other factors.
* A code q with scale s stands for v up to half a step: 2^-4 |v|, at least 2^-10 s (E4M3's subnormal step is
  2^-9), or s / 2 (int8), besides v's own error; a scale's error is its maximum's and two roundings.
* A weight's gradient sums exact products (8 by 8 significant bits): at most `rows` additions, each off by a
  step 2 u of a partial sum, itself at most the sum of the terms' magnitudes.  A code times a scale that is no power of
  two is rounded to bfloat16 first: half(bf16) of each term.
"""
import numpy as np
import pytest
import torch

from oracle import int8 as oint8
from oracle import layer, quant
from gpu_util import codes, device

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_fp8_gemm_amd as dg  # noqa: E402

U = 2.0 ** -24
Y = 64 * U
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
FP8 = torch.float8_e4m3fn


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half a step of a type's subnormals."""
    return torch.finfo(t).tiny * torch.finfo(t).eps / 2


def rows(shape, dtype, seed, spread=2.0):
    rng = np.random.default_rng(seed)
    v = rng.normal(size=shape) * 2.0 ** rng.uniform(-spread, spread, size=shape[:-1] + (1,))
    return torch.from_numpy(v.astype(np.float32)).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def strided(t, pad=64):
    """The same rows on the device, as part of a wider matrix whose other columns are NaN."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=device())
    wide[:, :t.shape[1]] = t.to(device())
    return wide[:, :t.shape[1]]


def near(got, want, bound, what=""):
    got, bound = f64(got) if torch.is_tensor(got) else got, np.broadcast_to(bound, np.shape(want))
    off = np.abs(got - want)
    assert got.shape == np.shape(want) and np.all(off <= bound), \
        f"{what}: {np.sum(~(off <= bound))} of {off.size}, worst {np.nanmax(off / np.maximum(bound, 1e-300))} of the bound"


def near_codes(q, sf, want, err, ue8m0=False, what=""):
    """Codes and scales of blocks of 128 whose exact values are `want`, known to the kernel up to `err`."""
    s = f64(sf)
    amax = np.abs(want).reshape(want.shape[0], -1, 128).max(2)
    e = np.broadcast_to(err, want.shape).reshape(want.shape[0], -1, 128).max(2)
    lo, hi = (np.maximum(amax + d * (e + 2 * U * amax), 1e-4) / 448 for d in (-1, 1))
    if ue8m0:
        lo, hi = 2.0 ** np.ceil(np.log2(lo * (1 - 2 * U))), 2.0 ** np.ceil(np.log2(hi * (1 + 2 * U)))
        assert np.all(np.log2(s) == np.round(np.log2(s))), what
    assert np.all(s >= lo * (1 - 2 * U)) and np.all(s <= hi * (1 + 2 * U)), f"{what}: scales"
    value = layer.widen_codes(f64(q.view(FP8).float()), s)
    sr = np.repeat(s, 128, axis=1)
    # a value whose magnitude exceeds 448 s by its error is clamped: no more than that error
    near(value, want, (np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * sr) + err) * (1 + 2.0 ** -16), what)


# ---------------------------------------------------------------- norm

NORM_SHAPES = [(1, 8), (1, 7168), (2, 128), (5, 512), (3, 520), (7, 1024), (4, 1032), (33, 2048), (9, 2056), (5, 4096),
               (6, 4104), (3, 8192), (2, 8200), (3, 16384), (17, 16376), (1025, 256), (300, 4104), (257, 2056)]


def norm_inputs(m, k, dtype, seed, residual=True):
    x, r = rows((m, k), dtype, seed), rows((m, k), dtype, seed + 1, 0.0) if residual else None
    w = rows((1, k), F32, seed + 2, 0.0)[0]
    h = x if r is None else (x.float() + r.float()).to(dtype)
    return x, r, w, h


@pytest.mark.parametrize("m,k", NORM_SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_norm(m, k, dtype):
    x, r, w, h = norm_inputs(m, k, dtype, m + k)
    wt = w.to(dtype) if k % 16 else w
    y, rstd = layer.rms_norm(f64(h), f64(wt), 1e-5)
    gy, gh, gr = dg.rms_norm(strided(x), wt.to(device()), strided(r), eps=1e-5)
    assert torch.equal(gh.cpu(), h) and gy.dtype == dtype
    near(gr, rstd, 50 * U * rstd, "rstd")
    near(gy, y, np.abs(y) * (Y + half(dtype) * (1 + Y)) + tiny(dtype), "y")
    gy2, gh2, _ = dg.rms_norm(x.to(device()), None, eps=1e-5)
    y, _ = layer.rms_norm(f64(x), None, 1e-5)
    near(gy2, y, np.abs(y) * (Y + half(dtype) * (1 + Y)) + tiny(dtype), "no weight")
    assert torch.equal(gh2.cpu(), x)


def test_signs_of_zeros_and_of_what_rounds_to_them():
    """The casts keep them, as the plain ones do: codes 0x00 and 0x80."""
    x = torch.zeros((2, 256))
    x[0, ::2], x[1, 1::3], x[1, 5], x[1, 200] = -0.0, -1e-30, 2.0, -3.0
    h = torch.cat([x, torch.ones(2, 256)], 1)
    _, (hq, hs) = dg.swiglu_checkpoint_fp8(h.to(device()))
    oq, osf = quant.per_token_cast(h.numpy())
    assert np.array_equal(codes(hq), oq) and np.array_equal(hs.cpu().numpy(), osf) and (oq == 0x80).sum() > 200
    y = torch.empty((2, 256), device=device())
    (q, sf), _, _ = dg.rms_norm_cast_fp8(x.to(device()), y=y, eps=1e-3)
    assert np.array_equal(codes(q), quant.per_token_cast(y.cpu().numpy())[0]) and (codes(q) == 0x80).sum() > 200


def test_norm_in_place_and_outputs_that_are_given():
    x, r, w, h = norm_inputs(37, 2048, BF16, 5)
    want = dg.rms_norm(x.to(device()), w.to(device()), r.to(device()))
    xd, rd, wd = x.to(device()), r.to(device()), w.to(device())
    rstd = torch.empty(37, device=device())
    y, hh, rr = dg.rms_norm(xd, wd, rd, y=xd, h=rd, rstd=rstd)
    assert y is xd and hh is rd and rr is rstd
    for a, b in zip((y, hh, rr), want):
        assert torch.equal(a, b)
    h2 = torch.empty_like(want[1])
    _, got, _ = dg.rms_norm(want[1], wd, h=h2)          # without a residual, h is x
    assert got is h2 and torch.equal(h2, want[1])


@pytest.mark.parametrize("m,k", [(1, 128), (1, 7168), (5, 512), (3, 640), (33, 1024), (4, 1152), (9, 2176), (3, 4096),
                                 (2, 8192), (2, 8320), (3, 16384), (600, 256), (260, 4224), (258, 8320)])
@pytest.mark.parametrize("ue8m0", [False, True])
def test_norm_cast_fp8(m, k, ue8m0):
    """fp32 rows: the codes are those of the cast of the rows that the same call returns, bit for bit; 16-bit rows: within
    the norm's error of the exact values."""
    x, r, w, h = norm_inputs(m, k, F32, 3 * m + k)
    y = torch.empty((m, k), device=device())
    (q, sf), gh, rstd = dg.rms_norm_cast_fp8(x.to(device()), w.to(device()), strided(r), ue8m0=ue8m0, y=y)
    want = dg.rms_norm(x.to(device()), w.to(device()), r.to(device()))
    assert torch.equal(y, want[0]) and torch.equal(gh, want[1]) and torch.equal(rstd, want[2])
    oq, osf = quant.per_token_cast(y.cpu().numpy(), ue8m0)
    assert np.array_equal(codes(q), oq) and np.array_equal(sf.cpu().numpy(), osf)
    for dtype in (BF16, F16):
        x, r, w, h = norm_inputs(m, k, dtype, 5 * m + k)
        sf = torch.empty((m, k // 128), device=device())
        (q, got), _, _ = dg.rms_norm_cast_fp8(strided(x), w.to(device()), r.to(device()), ue8m0=ue8m0, sf=sf)
        assert got is sf
        y64, _ = layer.rms_norm(f64(h), f64(w), 1e-6)
        near_codes(q, sf, y64, np.abs(y64) * Y, ue8m0, "fp8")


@pytest.mark.parametrize("m,k", [(1, 16), (1, 7168), (5, 528), (33, 1024), (4, 1040), (9, 2176), (3, 7152), (2, 8208),
                                 (3, 16384), (257, 4112), (259, 2064)])
def test_norm_cast_int8(m, k):
    x, r, w, h = norm_inputs(m, k, F32, 7 * m + k)
    y = torch.empty((m, k), device=device())
    (q, sf), gh, rstd = dg.rms_norm_cast_int8(x.to(device()), w.to(device()), r.to(device()), y=y)
    oq, osf = oint8.cast(y.cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(sf.cpu().numpy(), osf)
    assert torch.equal(y, dg.rms_norm(x.to(device()), w.to(device()), r.to(device()))[0])
    x, r, w, h = norm_inputs(m, k, BF16, 9 * m + k)
    (q, sf), gh, _ = dg.rms_norm_cast_int8(strided(x), w.to(BF16).to(device()), strided(r))
    y64, _ = layer.rms_norm(f64(h), f64(w.to(BF16)), 1e-6)
    s = np.abs(y64).max(1) / 127
    near(sf, s, s * (Y + 2 * U))
    near(f64(q) * f64(sf)[:, None], y64, s[:, None] / 2 * (1 + Y) + np.abs(y64) * (Y + 2 * U))


def test_norm_of_rows_with_nan_infinity_and_zeros():
    x = rows((6, 512), BF16, 1)
    x[0, 3], x[1, 200], x[2] = float("nan"), float("inf"), 0
    x[3] = 1e30                                          # its square leaves fp32
    y, _, rstd = dg.rms_norm(x.to(device()), eps=1e-6)
    y, rstd = y.cpu().float(), rstd.cpu()
    assert y[0].isnan().all() and rstd[0].isnan()
    assert y[1, 200].isnan() and bool((y[1, :200] == 0).all()) and rstd[1] == 0
    assert bool((y[2] == 0).all()) and bool((y[3] == 0).all()) and bool(y[4:].isfinite().all())
    (q, sf), _, _ = dg.rms_norm_cast_fp8(x.to(device()))
    sf = sf.cpu()
    assert sf[0].isnan().all() and sf[1].isnan().tolist() == [False, True, False, False] and sf[2:].isfinite().all()
    (q, s8), _, _ = dg.rms_norm_cast_int8(x.to(device()))
    assert s8.isnan().tolist() == [True, True, False, False, False, False]
    y, _, _ = dg.rms_norm(x[2:3].to(device()), eps=0.0)
    assert y.isnan().all()
    for f in (dg.rms_norm, dg.rms_norm_cast_fp8, dg.rms_norm_cast_int8):
        out, h, rstd = f(torch.empty((0, 512), dtype=BF16, device=device()))
        assert rstd.shape == (0,)


@pytest.mark.parametrize("m,k", NORM_SHAPES + [(4099, 264), (511, 1032), (1000, 2048), (1030, 4104), (1100, 1048)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_norm_grad(m, k, dtype):
    h, dy, dh = rows((m, k), dtype, m + k), rows((m, k), dtype, m + k + 1, 0.0), rows((m, k), dtype, m + k + 2, 0.0)
    w = rows((1, k), F32, m + k + 3, 0.0)[0]
    rstd = torch.from_numpy(layer.rms_norm(f64(h), None, 1e-6)[1].astype(np.float32))
    r = f64(rstd)[:, None]
    n = f64(h) * r
    for through in (True, False):
        dx, dw = layer.rms_norm_grad(f64(dy), f64(h), f64(w), f64(rstd), f64(dh) if through else None)
        gx, gw = dg.rms_norm_grad(strided(dy), strided(h), w.to(device()), rstd.to(device()),
                                  strided(dh) if through else None)
        wdy = f64(w) * f64(dy)
        size = r * (np.abs(wdy) + np.abs(n) * np.abs(wdy * n).mean(1, keepdims=True))
        if through:
            size = size + np.abs(f64(dh))
        near(gx, dx, 110 * U * size + half(dtype) * (np.abs(dx) + 110 * U * size) + tiny(dtype), "dx")
        terms = np.abs(f64(dy) * n).sum(0)
        # each workgroup adds at most 8 + rows / 1024 of its rows, then 1024 partial sums in 16 chains
        near(gw, dw, (m / 512 + 100) * U * terms, "dw")
    gx, gw = dg.rms_norm_grad(dy.to(device()), h.to(device()), None, rstd.to(device()))
    assert gw is None
    near(gx, layer.rms_norm_grad(f64(dy), f64(h), None, f64(rstd))[0],
         110 * U * r * (np.abs(f64(dy)) + np.abs(n) * np.abs(f64(dy) * n).mean(1, keepdims=True))
         + half(dtype) * (np.abs(layer.rms_norm_grad(f64(dy), f64(h), None, f64(rstd))[0]) * 1.01) + tiny(dtype))


def test_norm_grad_in_place_is_the_same_and_empty_batches_give_zeros():
    h, dy, dh = (rows((70, 1536), BF16, i).to(device()) for i in range(3))
    w = torch.rand(1536, device=device())
    rstd = dg.rms_norm(h)[2]
    want = dg.rms_norm_grad(dy, h, w, rstd, dh)
    for name in ("dy", "h", "dh"):
        t = dict(dy=dy.clone(), h=h.clone(), dh=dh.clone())
        dx, dw = dg.rms_norm_grad(t["dy"], t["h"], w, rstd, t["dh"], dx=t[name])
        assert dx is t[name] and torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    out = torch.full((1536,), 7.0, device=device())
    dx, dw = dg.rms_norm_grad(dy[:0], h[:0], w, rstd[:0], dweight=out)
    assert dw is out and bool((out == 0).all()) and dx.shape == (0, 1536)


def test_norm_gradient_is_that_of_differences():
    """The kernels' gradient against central differences of the kernels' own norm, in fp32: a step of 2^-6 of values
    about 1 leaves curvature of 2^-12 / 6 times third derivatives of at most about 10 |dy|, and rounding 64 u / 2^-6."""
    k = 64
    h, dy = rows((1, k), F32, 3, 0.0), rows((1, k), F32, 4, 0.0)
    w = rows((1, k), F32, 5, 0.0)[0].to(device())
    rstd = dg.rms_norm(h.to(device()), w)[2]
    dx, _ = dg.rms_norm_grad(dy.to(device()), h.to(device()), w, rstd)
    step = 2.0 ** -6
    up = dg.rms_norm((h + step * torch.eye(k)).to(device()), w)[0].cpu().double()
    down = dg.rms_norm((h - step * torch.eye(k)).to(device()), w)[0].cpu().double()
    want = ((up - down) * dy.double()).sum(1) / (2 * step)
    size = float((dy.abs().double() * w.cpu().abs().double()).sum())
    near(dx[0], want.numpy(), step ** 2 / 6 * 10 * size / k + 64 * U / step * size)


# ---------------------------------------------------------------- gated activation

def act_error(h):
    """(a, its error) in fp32 of rows h."""
    h = f64(h)
    n = h.shape[1] // 2
    g, u = np.abs(h[:, :n]), np.abs(h[:, n:])
    a = layer.swiglu(h)
    return a, np.abs(a) * (g + 8) * U + 2.0 ** -118 * g * u


def grad_error(da, h):
    da, h = np.abs(f64(da)), f64(h)
    n = h.shape[1] // 2
    g, u, s = np.abs(h[:, :n]), np.abs(h[:, n:]), layer.sigmoid(h[:, :n])
    rel = (g + 12) * U
    return np.concatenate([da * u * ((s + g * s * (1 - s)) + g * s * s) * rel + 2.0 ** -118 * da * u * (1 + g),
                           da * g * s * rel + 2.0 ** -118 * da * g], 1)


def layout_of(kind, m, seed):
    """(keyword, valid rows) for m rows."""
    rng = np.random.default_rng(seed)
    if kind == "all":
        return {}, np.ones(m, bool)
    if kind == "marked":
        mi = rng.integers(-1, 3, m).astype(np.int32)
        return {"m_indices": torch.from_numpy(mi).to(device())}, mi >= 0
    groups = next(g for g in (4, 3, 2, 1) if m % g == 0)
    per = m // groups
    count = rng.integers(-1, per + 3, groups).astype(np.int32)
    count[0] = 0 if groups > 1 else per
    valid = np.concatenate([np.arange(per) < c for c in count])
    return {"masked_m": torch.from_numpy(count).to(device())}, valid


def raw(t):
    return t.view(torch.uint8) if t.dtype == FP8 else t


def sentinel(shape):
    return torch.full(shape, 0x7D, dtype=torch.uint8, device=device())


ACT_SHAPES = [(1, 128), (4, 2048), (9, 384), (100, 640), (12, 2176), (300, 128), (3, 4096), (64, 1024)]


@pytest.mark.parametrize("m,n", ACT_SHAPES)
@pytest.mark.parametrize("kind", ["all", "marked", "masked"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_swiglu_cast_fp8(m, n, kind, dtype):
    h = rows((m, 2 * n), dtype, m + n)
    where, valid = layout_of(kind, m, m * n)
    a, err = act_error(h)
    for ue8m0 in (False, True):
        q, hq = sentinel((m, n)), sentinel((m, 2 * n))
        sf = torch.full((m, n // 128), -7.0, device=device())
        (gq, gs), (kq, ks) = dg.swiglu_checkpoint_fp8(strided(h), **where, ue8m0=ue8m0, q=q, sf=sf, hq=hq)
        assert gq is q and gs is sf and kq is hq
        near_codes(q[valid], sf[valid], a[valid], err[valid], ue8m0, "activation")
        oq, osf = quant.per_token_cast(h[valid].float().numpy(), ue8m0)
        assert np.array_equal(codes(kq)[valid], oq) and np.array_equal(ks.cpu().numpy()[valid], osf)
        assert (codes(q)[~valid] == 0x7D).all() and (codes(hq)[~valid] == 0x7D).all()
        assert (sf.cpu().numpy()[~valid] == -7).all()
        q2, sf2 = dg.swiglu_cast_fp8(h.to(device()), **where, ue8m0=ue8m0)
        assert np.array_equal(codes(q2)[valid], codes(q)[valid]) and torch.equal(sf2[valid], sf[valid])


@pytest.mark.parametrize("m,n", [(1, 16), (4, 2048), (9, 400), (100, 656), (12, 2064), (3, 4112), (5, 8192), (4, 16384)])
@pytest.mark.parametrize("kind", ["all", "marked", "masked"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_swiglu_cast_int8(m, n, kind, dtype):
    h = rows((m, 2 * n), dtype, m + n)
    where, valid = layout_of(kind, m, m * n)
    a, err = act_error(h)
    q = torch.full((m, n), 77, dtype=torch.int8, device=device())
    sf = torch.full((m,), -7.0, device=device())
    dg.swiglu_cast_int8(strided(h), **where, q=q, sf=sf)
    top = np.maximum(np.abs(a).max(1), 1e-4)
    near(f64(sf)[valid], (top / 127)[valid], ((err.max(1) + 2 * U * top) / 127)[valid])
    near((f64(q) * f64(sf)[:, None])[valid], a[valid], (f64(sf)[:, None] / 2 * (1 + 4 * U) + 2 * err + 2 * U * np.abs(a))[valid])
    assert (q.cpu().numpy()[~valid] == 77).all() and (sf.cpu().numpy()[~valid] == -7).all()


@pytest.mark.parametrize("m,n", ACT_SHAPES + [(5, 8), (7, 1400), (33, 264)])
@pytest.mark.parametrize("kind", ["all", "marked", "masked"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_swiglu_grad(m, n, kind, dtype):
    h, da = rows((m, 2 * n), dtype, m + n), rows((m, n), dtype, m + n + 1)
    where, valid = layout_of(kind, m, m * n)
    forms = [(strided(h), h)]
    if n % 128 == 0:
        kept = dg.swiglu_checkpoint_fp8(h.to(device()))[1]
        forms.append((kept, torch.from_numpy(layer.widen_codes(f64(kept[0].float()), f64(kept[1])))))
        forms.append(((kept[0].view(torch.uint8), kept[1].contiguous()), forms[-1][1]))
    for given, value in forms:
        # a code times its scale is rounded to fp32: u of g and u, which moves the result by at most
        # u |da u| s (1 - s) |g| (2 + |g|) and u, twice the error that is there already
        want, err = layer.swiglu_grad(f64(da), f64(value)), grad_error(da, value) * (3 if isinstance(given, tuple) else 1)
        bound = err + half(dtype) * (np.abs(want) + err) + tiny(dtype)
        out = torch.full((m, 2 * n), 7.0, dtype=dtype, device=device())
        assert dg.swiglu_grad(strided(da), given, **where, dh=out) is out
        near(f64(out)[valid], want[valid], bound[valid], "dh")
        assert bool((out[torch.from_numpy(~valid).to(device())] == 7).all())
        if n % 128 == 0:
            q = sentinel((m, 2 * n))
            dh, (gq, gs) = dg.swiglu_grad_cast_fp8(da.to(device()), given, **where, q=q)
            assert gq is q and torch.equal(dh[valid], out[valid]) and (codes(q)[~valid] == 0x7D).all()
            near_codes(q[valid], gs[valid], want[valid], err[valid], False, "cast")
            if dtype is F32:
                oq, osf = quant.per_token_cast(dh[valid].cpu().numpy())
                assert np.array_equal(codes(q)[valid], oq) and np.array_equal(gs.cpu().numpy()[valid], osf)


@pytest.mark.parametrize("saved", ["rows", "codes"])
def test_swiglu_of_many_rows(saved):
    """2^24 elements and more: threads take two pieces each.  The same rows in batches of 100 give the same bits, and
    those are compared with the formulas above."""
    m, n, part = 8400, 2176, 100
    h, da = (rows((m, w), BF16, 4 + w, 0.0).to(device()) for w in (2 * n, n))
    mi = torch.randint(-1, 3, (m,), dtype=torch.int32, device=device())
    for where in ({}, {"m_indices": mi}, {"masked_m": torch.tensor([0, 5, 1400, 699, 1, 1300], dtype=torch.int32,
                                                                   device=device())}):
        valid = torch.ones(m, dtype=torch.bool, device=device())
        if "m_indices" in where:
            valid = mi >= 0
        if "masked_m" in where:
            valid = (torch.arange(m // 6, device=device())[None] < where["masked_m"][:, None]).reshape(-1)
        q, hq = sentinel((m, n)), sentinel((m, 2 * n))
        (_, sf), (_, hs) = dg.swiglu_checkpoint_fp8(h, **where, q=q, hq=hq)
        dq, given = sentinel((m, 2 * n)), h
        if saved == "codes":
            given = dg.swiglu_checkpoint_fp8(h)[1]
        dh, (_, ds) = dg.swiglu_grad_cast_fp8(da, given, **where, q=dq)
        for i in range(0, m, part):
            s, v = slice(i, i + part), valid[i:i + part]
            (q2, sf2), (hq2, hs2) = dg.swiglu_checkpoint_fp8(h[s])
            piece = tuple(t[s] for t in given) if saved == "codes" else given[s]
            dh2, (dq2, ds2) = dg.swiglu_grad_cast_fp8(da[s], piece)
            for a, b in ((q, q2), (hq, hq2), (dq, dq2), (sf, sf2), (hs, hs2), (ds, ds2), (dh, dh2)):
                assert torch.equal(raw(a[s])[v], raw(b)[v])
            assert bool((q[s][~v] == 0x7D).all()) and bool((hq[s][~v] == 0x7D).all()) and bool((dq[s][~v] == 0x7D).all())


def test_swiglu_grad_in_place():
    h, da = rows((40, 512), BF16, 1).to(device()), rows((40, 256), BF16, 2).to(device())
    want = dg.swiglu_grad(da, h)
    assert dg.swiglu_grad(da, h, dh=h) is h and torch.equal(h, want)


def test_swiglu_at_the_ends():
    """Gates beyond the exponential's range, NaN and infinities: they show in their block (FP8) or row (int8)."""
    h = torch.ones((4, 512), dtype=F32)
    h[0, :6] = torch.tensor([1e30, -1e30, 100.0, -100.0, 88.9, -88.9])
    h[1, 5], h[2, 300], h[3, 256] = float("nan"), float("inf"), float("nan")
    q, sf = dg.swiglu_cast_fp8(h.to(device()))
    sf = sf.cpu()
    assert sf[0, 0] == np.float32(1e30) / np.float32(448) and sf[0, 1].isfinite()
    assert sf.isnan().tolist() == [[False, False], [True, False], [False, False], [True, False]]
    assert sf[2].isinf().tolist() == [True, False]
    _, s8 = dg.swiglu_cast_int8(h.to(device()))
    assert s8.isnan().tolist() == [False, True, False, True] and s8.isinf().tolist() == [False, False, True, False]
    _, (hq, hs) = dg.swiglu_checkpoint_fp8(h.to(device()))
    assert hs.isnan().cpu().tolist() == [[False] * 4, [True] + [False] * 3, [False] * 4, [False, False, True, False]]
    _, (_, hs) = dg.swiglu_checkpoint_fp8(h.to(device()), ue8m0=True)
    assert bool(hs.isnan().any(1).tolist() == [False, True, False, True]) and bool((hs[~hs.isnan()] > 0).all())
    dh = dg.swiglu_grad(torch.ones((4, 256), device=device()), h.to(device())).cpu()
    assert dh[0].isfinite().all()
    assert dh[0, :6].tolist()[:4] == [1, 0, 1, 0] and dh[0, 256].item() == pytest.approx(1e30)


def test_swiglu_without_rows():
    e = torch.empty((0, 512), dtype=BF16, device=device())
    assert dg.swiglu_cast_fp8(e)[0].shape == (0, 256) and dg.swiglu_grad(e[:, :256], e).shape == (0, 512)
    assert dg.swiglu_cast_int8(e, masked_m=torch.zeros(4, dtype=torch.int32, device=device()))[1].shape == (0,)


# ---------------------------------------------------------------- weights' gradients

def kept_rows(x, power):
    """(codes, scales) of rows on the device and the values that they stand for."""
    q, sf = quant.per_token_cast(x.float().numpy(), power)
    value = layer.widen_codes(f64(torch.from_numpy(q).view(FP8).float()), sf)
    sf = torch.from_numpy(sf).to(device())
    return (torch.from_numpy(q).to(device()).view(FP8), sf.t().contiguous().t() if power else sf), value


def check_weight_grad(got, dy, value, segs, out, rounded, start=None):
    want, size = layer.weight_grad(f64(dy), value, segs)
    n = np.array([c for _, c in segs])[:, None, None]
    bound = (n + 40) * 2 * U * size + (half(BF16) * size if rounded else 0)
    if start is not None:
        want = want + start
        bound = bound + 2 * U * np.abs(want)
    bound = bound + half(out) * (np.abs(want) + bound) if out is BF16 else bound
    got = f64(got).reshape(want.shape)
    near(got, want, bound, "dw")
    assert all(np.all(got[g] == (0 if start is None else start[g])) for g, (_, c) in enumerate(segs) if c == 0)


WGRAD_SHAPES = [(1, 8, 8), (1, 128, 128), (63, 64, 256), (64, 256, 256), (65, 264, 136), (200, 8, 1032), (777, 136, 264),
                (1000, 512, 640), (130, 2112, 384), (4097, 128, 128)]


@pytest.mark.parametrize("m,n,k", WGRAD_SHAPES)
@pytest.mark.parametrize("out", [F32, BF16])
def test_weight_grad(m, n, k, out):
    dy, x = rows((m, n), BF16, m + n), rows((m, k), BF16, m + k)
    dw = torch.full((n, k + 8), 7.0, dtype=out, device=device())
    got = dg.weight_grad(strided(dy), strided(x), dw[:, :k])
    check_weight_grad(got, dy, f64(x), [(0, m)], out, False)
    assert bool((dw[:, k:] == 7).all())
    k = (k + 127) // 128 * 128
    x = rows((m, k), BF16, m + k)
    for power in (True, False):
        pair, value = kept_rows(x, power)
        dw = torch.empty((n, k), dtype=out, device=device())
        assert dg.weight_grad(dy.to(device()), pair, dw) is dw
        check_weight_grad(dw, dy, value, [(0, m)], out, not power)
    dw = torch.empty((n, k), dtype=out, device=device())
    wide = sentinel((m, k + 64))
    wide[:, :k] = pair[0].view(torch.uint8)
    dg.weight_grad(strided(dy), (wide[:, :k], pair[1]), dw)
    check_weight_grad(dw, dy, value, [(0, m)], out, True)


GROUPS = [([5], 1, 200, 136), ([0, 3, 0, 130, 1, 64], 128, 64, 256), ([0, 3, 0, 130, 1, 64], 1, 64, 256),
          ([129, 0, 0, 257], 128, 264, 128), ([1] * 40, 1, 128, 128), ([7, 65, 300, 12], 32, 512, 384),
          ([0, 0], 1, 128, 128), ([40, -3, 9], 128, 8, 128), ([64] * 3, 1, 2048, 4096),
          ([0, 1, 33, 70, 0, 200, 32, 64, 31, 0] * 14, 1, 264, 136), ([0] * 300 + [9] + [0] * 20 + [130], 1, 40, 128)]


@pytest.mark.parametrize("i", range(len(GROUPS)))
@pytest.mark.parametrize("fp8", [False, True])
def test_weight_grad_contiguous(i, fp8):
    """Rows between the segments are NaN (codes and scales too) and must not count."""
    count, align, n, k = GROUPS[i]
    k = (k + 127) // 128 * 128 if fp8 else k
    total = sum(-(-max(0, c) // align) * align for c in count) + 3
    segs = layer.segments(count, total, align)
    valid = np.zeros(total, bool)
    for a, c in segs:
        valid[a:a + c] = True
    gone = torch.from_numpy(~valid)
    dy, x = rows((total, n), BF16, n + i), rows((total, k), BF16, k + i)
    counts = torch.tensor(count, dtype=torch.int32, device=device())
    value = f64(x)
    dyd, xd = dy.clone(), x.clone()
    dyd[gone], xd[gone] = float("nan"), float("nan")
    given = xd.to(device())
    if fp8:
        (q, sf), value = kept_rows(x, True)
        q, sf = q.view(torch.uint8).clone(), sf.clone()
        q[gone], sf[gone] = 0x7F, float("nan")
        given = (q.view(FP8), sf)
    for out in (F32, BF16):
        dw = torch.full((len(count), n, k), float("nan"), dtype=out, device=device())
        dg.m_grouped_weight_grad_contiguous(dyd.to(device()), given, dw, counts, alignment=align)
        check_weight_grad(dw, dy, value, segs, out, False)
    start = torch.from_numpy(np.random.default_rng(i).normal(size=(len(count), n, k)).astype(np.float32))
    dw = start.to(device())
    dg.m_grouped_weight_grad_contiguous(dyd.to(device()), given, dw, counts, alignment=align, accumulate=True)
    check_weight_grad(dw, dy, value, segs, F32, False, f64(start))


def test_weight_grad_counts_past_the_rows_are_cut():
    dy, x = rows((100, 64), BF16, 1), rows((100, 128), BF16, 2)
    counts = torch.tensor([60, 90, 7], dtype=torch.int32, device=device())
    dw = torch.empty((3, 64, 128), device=device())
    dg.m_grouped_weight_grad_contiguous(dy.to(device()), x.to(device()), dw, counts, alignment=1)
    check_weight_grad(dw, dy, f64(x), [(0, 60), (60, 40), (100, 0)], F32, False)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("groups,max_m,n,k", [(4, 32, 128, 256), (3, 200, 264, 128), (1, 5, 8, 128), (16, 64, 512, 512)])
def test_weight_grad_masked(groups, max_m, n, k, fp8):
    rng = np.random.default_rng(groups + max_m)
    count = rng.integers(-1, max_m + 4, groups)
    count[-1] = max_m + 3
    segs = layer.segments(count, groups * max_m, max_m=max_m)
    dy, x = rows((groups * max_m, n), BF16, 1), rows((groups * max_m, k), BF16, 2)
    given, value = kept_rows(x, True) if fp8 else (x.to(device()), f64(x))
    dw = torch.empty((groups, n, k), device=device())
    dg.m_grouped_weight_grad_masked(dy.to(device()), given, dw,
                                    torch.from_numpy(count.astype(np.int32)).to(device()))
    check_weight_grad(dw, dy, value, segs, F32, False)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("out", [F32, BF16])
def test_weight_grad_is_the_same_on_few_cus(fp8, out):
    """Fewer workgroups take more tiles each, in the same way."""
    shapes = (([70, 0, 33, 1, 300, 64] * 12, 520, 384), ([700, 12], 264, 256))
    for count, n, k in shapes:
        total = sum(count)
        dy, x = rows((total, n), BF16, n), rows((total, k), BF16, k)
        given, value = kept_rows(x, True) if fp8 else (x.to(device()), f64(x))
        counts = torch.tensor(count, dtype=torch.int32, device=device())
        got = []
        cus = dg.get_num_cus()
        for few in (cus, 8, 24, 1):
            dg.set_num_cus(few)
            try:
                dw = torch.empty((len(count), n, k), dtype=out, device=device())
                dg.m_grouped_weight_grad_contiguous(dy.to(device()), given, dw, counts, alignment=1)
            finally:
                dg.set_num_cus(cus)
            got.append(dw)
        assert all(torch.equal(got[0], g) for g in got[1:])
        check_weight_grad(got[0], dy, value, layer.segments(count, total, 1), out, False)


def test_operands_of_more_than_2_to_the_32_bytes():
    """Rows that lie 2^16 elements apart: offsets pass 32 bits.  What they hold is compared with the same
    rows side by side."""
    m, n, k = 33000, 264, 256
    dy, x = rows((m, n), BF16, 1, 0.0).to(device()), rows((m, k), BF16, 2, 0.0).to(device())
    wide = torch.empty((m, 65536), dtype=BF16, device=device())
    for count in ([m - 200, 0, 77, 123], [1, 2, 0, m - 3] * 9):
        counts = torch.tensor(count, dtype=torch.int32, device=device())
        total = min(m, sum(count))
        wide[:, :k], wide[:, k:k + n] = x, dy
        want, got = (torch.empty((len(count), n, k), device=device()) for _ in range(2))
        dg.m_grouped_weight_grad_contiguous(dy, x, want, counts, alignment=1)
        dg.m_grouped_weight_grad_contiguous(wide[:, k:k + n], wide[:, :k], got, counts, alignment=1)
        assert torch.equal(got, want) and bool(want[0].any())
    w = torch.rand(k, device=device())
    y, h, rstd = dg.rms_norm(x, w)
    wide[:, k:2 * k] = x
    _, gh, gr = dg.rms_norm(wide[:, k:2 * k], w, y=wide[:, :k], h=wide[:, 2 * k:3 * k])
    assert torch.equal(wide[:, :k], y) and torch.equal(gh, h) and torch.equal(gr, rstd)
    dx, dw = dg.rms_norm_grad(y, x, w, rstd, x)
    gx, gw = dg.rms_norm_grad(wide[:, :k], wide[:, k:2 * k], w, rstd, wide[:, 2 * k:3 * k], dx=wide[:, 3 * k:4 * k])
    assert torch.equal(gx, dx) and torch.equal(gw, dw)
    (q, sf), (hq, hs) = dg.swiglu_checkpoint_fp8(x)
    bytes_ = wide.view(torch.uint8)
    at = 65536
    (q2, sf2), (hq2, hs2) = dg.swiglu_checkpoint_fp8(wide[:, k:2 * k], q=bytes_[:, at:at + k // 2], hq=bytes_[:, at + k:at + 2 * k])
    for a, b in ((q, q2), (sf, sf2), (hq, hq2), (hs, hs2)):
        assert torch.equal(raw(a), raw(b))
    da = dy[:, :k // 2]
    assert torch.equal(dg.swiglu_grad(da, x), dg.swiglu_grad(da, wide[:, k:2 * k], dh=wide[:, 4 * k:5 * k]))
    assert torch.equal(dg.swiglu_grad(da, (hq, hs)), dg.swiglu_grad(da, (hq2, hs2), dh=wide[:, 4 * k:5 * k]))


def test_weight_grad_without_rows_or_columns():
    dw = torch.full((2, 64, 128), 7.0, device=device())
    e = torch.empty((0, 64), dtype=BF16, device=device())
    c = torch.tensor([3, 0], dtype=torch.int32, device=device())
    dg.m_grouped_weight_grad_contiguous(e, torch.empty((0, 128), dtype=BF16, device=device()), dw, c)
    assert bool((dw == 0).all())
    dw.fill_(7)
    dg.m_grouped_weight_grad_masked(e, torch.empty((0, 128), dtype=BF16, device=device()), dw, c)
    assert bool((dw == 0).all())
    dg.weight_grad(e, torch.empty((0, 128), dtype=BF16, device=device()), dw[0], accumulate=True)
    assert bool((dw == 0).all())
    dg.weight_grad(torch.ones((4, 0), dtype=BF16, device=device()), torch.ones((4, 128), dtype=BF16, device=device()),
                   torch.empty((0, 128), device=device()))


def test_weight_grad_of_groups_that_lie_apart():
    """dw as a slice of a larger tensor: group and row strides of their own, nothing written beside it."""
    dy, x = rows((64, 72), BF16, 1), rows((64, 136), BF16, 2)
    big = torch.full((3, 80, 160), 7.0, device=device())
    dg.m_grouped_weight_grad_contiguous(dy.to(device()), x.to(device()), big[::2, :72, :136],
                                        torch.tensor([30, 34], dtype=torch.int32, device=device()), alignment=1)
    check_weight_grad(big[::2, :72, :136], dy, f64(x), [(0, 30), (30, 34)], F32, False)
    big[::2, :72, :136] = 7
    assert bool((big == 7).all())


def test_nan_and_infinity_in_counted_rows_show_in_their_rows_and_columns():
    dy, x = torch.ones((70, 64), dtype=BF16), torch.ones((70, 128), dtype=BF16)
    dy[3, 5], x[69, 9] = float("nan"), float("inf")
    dw = torch.empty((64, 128), device=device())
    dg.weight_grad(dy.to(device()), x.to(device()), dw)
    bad = ~dw.cpu().isfinite()
    want = torch.zeros((64, 128), dtype=torch.bool)
    want[5], want[:, 9] = True, True
    assert torch.equal(bad, want)


# ---------------------------------------------------------------- the calls of a program

REFUSED = [
    (TypeError, lambda: dg.rms_norm(torch.ones((4, 64), device=device(), dtype=torch.float64))),
    (ValueError, lambda: dg.rms_norm(torch.ones(64, device=device()))),
    (ValueError, lambda: dg.rms_norm(torch.ones((64, 4), device=device()).t())),
    (ValueError, lambda: dg.rms_norm(torch.ones((4, 64), device=device()), torch.ones(63, device=device()))),
    (TypeError, lambda: dg.rms_norm(torch.ones((4, 64), device=device()), torch.ones(64, device=device(), dtype=BF16))),
    (TypeError, lambda: dg.rms_norm(torch.ones((4, 64), device=device()), None, torch.ones((4, 64), device=device(), dtype=BF16))),
    (ValueError, lambda: dg.rms_norm(torch.ones((4, 64), device=device()), None, torch.ones((3, 64), device=device()))),
    (TypeError, lambda: dg.rms_norm(torch.ones((4, 64), device=device()), eps="x")),
    (dg.DgError, lambda: dg.rms_norm(torch.ones((4, 64), device=device()), eps=-1.0)),
    (dg.DgError, lambda: dg.rms_norm(torch.ones((4, 60), device=device()))),
    (dg.DgError, lambda: dg.rms_norm(torch.ones((4, 16392), device=device()))),
    (dg.DgError, lambda: dg.rms_norm_cast_fp8(torch.ones((4, 64), device=device()))),
    (dg.DgError, lambda: dg.rms_norm_cast_int8(torch.ones((4, 72), device=device()))),
    (ValueError, lambda: dg.rms_norm_cast_fp8(torch.ones((4, 128), device=device()), sf=torch.ones((4, 2), device=device()))),
    (ValueError, lambda: dg.rms_norm_grad(torch.ones((4, 64), device=device()), torch.ones((4, 64), device=device()), None,
                                          torch.ones(3, device=device()))),
    (ValueError, lambda: dg.rms_norm_grad(torch.ones((4, 64), device=device()), torch.ones((4, 64), device=device()), None,
                                          torch.ones(4, device=device()), dweight=torch.ones(64, device=device()))),
    (ValueError, lambda: dg.swiglu_cast_fp8(torch.ones((4, 255), device=device()))),
    (dg.DgError, lambda: dg.swiglu_cast_fp8(torch.ones((4, 192), device=device()))),
    (ValueError, lambda: dg.swiglu_cast_fp8(torch.ones((4, 256), device=device()),
                                            m_indices=torch.zeros(3, dtype=torch.int32, device=device()))),
    (ValueError, lambda: dg.swiglu_cast_fp8(torch.ones((4, 256), device=device()),
                                            masked_m=torch.zeros(3, dtype=torch.int32, device=device()))),
    (ValueError, lambda: dg.swiglu_cast_int8(torch.ones((4, 256), device=device()),
                                             m_indices=torch.zeros(4, dtype=torch.int32, device=device()),
                                             masked_m=torch.zeros(2, dtype=torch.int32, device=device()))),
    (ValueError, lambda: dg.swiglu_grad(torch.ones((4, 64), device=device()), torch.ones((4, 64), device=device()))),
    (TypeError, lambda: dg.swiglu_grad(torch.ones((4, 64), device=device()), torch.ones((4, 128), device=device(), dtype=BF16))),
    (ValueError, lambda: dg.swiglu_grad(torch.ones((4, 128), device=device()),
                                        (sentinel((4, 256)), torch.ones((4, 1), device=device())))),
    (dg.DgError, lambda: dg.swiglu_grad_cast_fp8(torch.ones((4, 64), device=device()), torch.ones((4, 128), device=device()))),
    (TypeError, lambda: dg.weight_grad(torch.ones((4, 64), device=device()), torch.ones((4, 64), device=device(), dtype=BF16),
                                       torch.ones((64, 64), device=device()))),
    (TypeError, lambda: dg.weight_grad(torch.ones((4, 64), device=device(), dtype=BF16), torch.ones((4, 64), device=device()),
                                       torch.ones((64, 64), device=device()))),
    (ValueError, lambda: dg.weight_grad(torch.ones((4, 64), device=device(), dtype=BF16),
                                        torch.ones((3, 64), device=device(), dtype=BF16), torch.ones((64, 64), device=device()))),
    (ValueError, lambda: dg.weight_grad(torch.ones((4, 64), device=device(), dtype=BF16),
                                        torch.ones((4, 64), device=device(), dtype=BF16), torch.ones((64, 72), device=device()))),
    (dg.DgError, lambda: dg.weight_grad(torch.ones((4, 64), device=device(), dtype=BF16),
                                        torch.ones((4, 64), device=device(), dtype=BF16),
                                        torch.ones((64, 64), device=device(), dtype=BF16), accumulate=True)),
    (dg.DgError, lambda: dg.weight_grad(torch.ones((4, 60), device=device(), dtype=BF16),
                                        torch.ones((4, 64), device=device(), dtype=BF16), torch.ones((60, 64), device=device()))),
    (dg.DgError, lambda: dg.m_grouped_weight_grad_contiguous(
        torch.ones((4, 64), device=device(), dtype=BF16), torch.ones((4, 64), device=device(), dtype=BF16),
        torch.ones((2, 64, 64), device=device()), torch.zeros(2, dtype=torch.int32, device=device()), alignment=0)),
    (ValueError, lambda: dg.m_grouped_weight_grad_masked(
        torch.ones((5, 64), device=device(), dtype=BF16), torch.ones((5, 64), device=device(), dtype=BF16),
        torch.ones((2, 64, 64), device=device()), torch.zeros(2, dtype=torch.int32, device=device()))),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_refusals(i):
    error, call = REFUSED[i]
    with pytest.raises(error):
        call()


def test_y_and_h_must_differ():
    x = torch.ones((4, 64), device=device())
    with pytest.raises(ValueError):
        dg.rms_norm(x, None, x, y=x, h=x)


def program(x, res, w, dy, counts, marks, dw_out):
    """The calls of a small layer's forward and backward pass, in order, on the current stream."""
    pair, h, rstd = dg.rms_norm_cast_fp8(x, w, res, ue8m0=True)
    act, kept = dg.swiglu_checkpoint_fp8(h, m_indices=marks, ue8m0=True)
    dh, cast = dg.swiglu_grad_cast_fp8(dy[:, :h.shape[1] // 2], kept, m_indices=marks)
    dg.m_grouped_weight_grad_contiguous(dy, pair, dw_out, counts)
    dx, dw = dg.rms_norm_grad(dh, h, w, rstd, dy)
    return [pair[0].view(torch.uint8), pair[1], h, rstd, dx, dw, dw_out]


def program_inputs(seed):
    m, k = 384, 1024
    x, res, dy = (rows((m, k), BF16, seed + i, 0.0).to(device()) for i in range(3))
    counts = torch.tensor([100, 128, 70], dtype=torch.int32)
    marks = torch.full((m,), -1, dtype=torch.int32)
    for g, c in enumerate(counts.tolist()):
        marks[g * 128:g * 128 + c] = g
    return [x, res, torch.rand(k, device=device()) + 0.5, dy, counts.to(device()), marks.to(device()),
            torch.zeros((3, k, k), device=device())]


def valid_of(out, marks):
    """Outputs with rows that no slot has taken out (they are unspecified)."""
    keep = marks >= 0
    return [t[keep] if t.dim() == 2 and t.shape[0] == marks.shape[0] else t for i, t in enumerate(out) if i != 5]


def test_captured_and_replayed():
    """Two captured graphs in turn, with eager work between them: every replay gives the eager calls' bits."""
    sets = [program_inputs(1), program_inputs(50)]
    eager = [[t.clone() for t in valid_of(program(*s), s[5])] for s in sets]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in sets:
            program(*s)
    torch.cuda.current_stream().wait_stream(side)
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(program(*s))
        graphs.append(g)
    for turn in range(4):
        for i in (0, 1):
            sets[i][6].fill_(float("nan"))
        for i in ((0, 1) if turn % 2 else (1, 0)):
            graphs[i].replay()
        other = program(*program_inputs(99))
        torch.cuda.synchronize()
        for i in (0, 1):
            for a, b in zip(valid_of(outs[i], sets[i][5]), eager[i]):
                assert torch.equal(a, b)
        del other


def test_two_streams_at_once():
    sets = [program_inputs(3), program_inputs(70)]
    want = [[t.clone() for t in valid_of(program(*s), s[5])] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i] = program(*sets[i])
    torch.cuda.synchronize()
    for i in (0, 1):
        for a, b in zip(valid_of(got[i], sets[i][5]), want[i]):
            assert torch.equal(a, b)
