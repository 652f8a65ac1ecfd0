"""Refusals of the norm, gated activation and weights' gradients: every bad argument comes back as a status before
anything is launched, and the binding rejects wrong tensors.  Addresses are fake and never dereferenced."""
import pytest
import torch

import moe_fp8_gemm_amd as dg

lib = dg.lib
P = 0x10000
OK, INVALID, UNSUPPORTED = 0, 1, 2
NAN, INF = float("nan"), float("inf")


def call(fn, defaults, **kw):
    assert not set(kw) - set(defaults), kw
    return fn(*{**defaults, **kw}.values())


NORM = dict(x=P, dtype=1, ldx=256, residual=P, ldr=256, weight=P, weight_dtype=1, eps=1e-6, h=P, ldh=256, y=P, ldy=256,
            rstd=P, rows=4, k=256, stream=None)
NORM_CASES = [
    (dict(rows=0), OK), (dict(k=0), OK), (dict(rows=0, x=None), OK), (dict(rows=-1), INVALID), (dict(k=-8), INVALID),
    (dict(dtype=3), INVALID), (dict(x=None), INVALID), (dict(ldx=255), INVALID), (dict(ldr=255), INVALID),
    (dict(ldh=248), INVALID), (dict(ldy=0), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=NAN), INVALID),
    (dict(eps=INF), INVALID), (dict(weight_dtype=2), INVALID), (dict(weight_dtype=7), INVALID),
    (dict(x=P + 8), UNSUPPORTED), (dict(h=P + 2), UNSUPPORTED), (dict(y=P + 4), UNSUPPORTED),
    (dict(residual=P + 8), UNSUPPORTED), (dict(weight=P + 2), UNSUPPORTED), (dict(rstd=P + 2), UNSUPPORTED),
    (dict(ldx=260), UNSUPPORTED), (dict(ldr=1 << 41), UNSUPPORTED), (dict(k=252), UNSUPPORTED),
    (dict(rows=(1 << 23) + 1), UNSUPPORTED),
    (dict(rows=(1 << 21) + 1, k=8448, ldx=8448, ldr=8448, ldh=8448, ldy=8448), UNSUPPORTED),
    (dict(k=16392, ldx=16392, ldr=16392, ldh=16392, ldy=16392), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", NORM_CASES + [(dict(y=None), INVALID)])
def test_norm(kw, status):
    assert call(lib.dg_rms_norm, NORM, **kw) == status


NORM_FP8 = dict(**{k: v for k, v in NORM.items() if k not in ("rows", "k", "stream")}, q=P, ldq=256, sf=P, sf_sm=2, sf_sk=1,
                rows=4, k=256, ue8m0=0, stream=None)


@pytest.mark.parametrize("kw,status", NORM_CASES + [
    (dict(q=None), INVALID), (dict(sf=None), INVALID), (dict(ldq=255), INVALID), (dict(sf_sm=-1), INVALID),
    (dict(q=P + 8), UNSUPPORTED), (dict(ldq=264), UNSUPPORTED), (dict(sf=P + 2), UNSUPPORTED), (dict(k=192), UNSUPPORTED),
    (dict(sf_sk=1 << 41), UNSUPPORTED)])
def test_norm_fp8(kw, status):
    assert call(lib.dg_rms_norm_cast_fp8, NORM_FP8, **kw) == status


NORM_INT8 = dict(**{k: v for k, v in NORM.items() if k not in ("rows", "k", "stream")}, q=P, ldq=256, sf=P, sf_s=1, rows=4,
                 k=256, stream=None)


@pytest.mark.parametrize("kw,status", NORM_CASES + [
    (dict(q=None), INVALID), (dict(sf=None), INVALID), (dict(sf_s=-1), INVALID), (dict(k=248), UNSUPPORTED),
    (dict(ldq=264), UNSUPPORTED)])
def test_norm_int8(kw, status):
    assert call(lib.dg_rms_norm_cast_int8, NORM_INT8, **kw) == status


NORM_GRAD = dict(dy=P, dtype=0, lddy=256, h=P, ldh=256, weight=P, weight_dtype=0, rstd=P, dh=P, lddh=256, dx=P, lddx=256,
                 dweight=P, rows=4, k=256, ws=P, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=0), OK), (dict(rows=0, dweight=None), OK), (dict(rows=-1), INVALID), (dict(dtype=-1), INVALID),
    (dict(dy=None), INVALID), (dict(h=None), INVALID), (dict(dx=None), INVALID), (dict(rstd=None), INVALID),
    (dict(lddy=255), INVALID), (dict(lddh=255), INVALID), (dict(lddx=255), INVALID), (dict(ws=None), INVALID),
    (dict(ws_bytes=256 * 4 - 1), INVALID), (dict(weight_dtype=1), INVALID), (dict(ws=P + 4), UNSUPPORTED),
    (dict(dweight=P + 2), UNSUPPORTED), (dict(dx=P + 8), UNSUPPORTED), (dict(k=252), UNSUPPORTED),
    (dict(rows=(1 << 23) + 1, ws_bytes=1 << 30), UNSUPPORTED)])
def test_norm_grad(kw, status):
    assert call(lib.dg_rms_norm_grad, NORM_GRAD, **kw) == status


def test_norm_grad_workspace_is_bounded():
    size = lib.dg_rms_norm_grad_workspace_size
    assert size(0, 256) == 0 and size(-1, 256) == 0 and size(4, 12) == 0 and size(4, 1 << 20) == 0
    assert 4 * 256 <= size(1, 256) <= size(4, 256) <= 4 * 4 * 256
    assert size(1 << 23, 16384) <= 1 << 27


SWIGLU = dict(h=P, dtype=1, ldh=512, m_indices=None, masked_m=None, groups=0, q=P, ldq=256, sf=P, sf_sm=2, sf_sk=1, hq=P,
              ldhq=512, hsf=P, hsf_sm=4, hsf_sk=1, rows=8, inner=256, ue8m0=0, stream=None)
SET_CASES = [(dict(m_indices=P, masked_m=P, groups=2), INVALID), (dict(masked_m=P, groups=0), INVALID),
             (dict(masked_m=P, groups=3), INVALID), (dict(m_indices=P + 2), UNSUPPORTED),
             (dict(masked_m=P + 1, groups=2), UNSUPPORTED), (dict(masked_m=P, groups=2048, rows=4096), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", SET_CASES + [
    (dict(rows=0), OK), (dict(inner=0), OK), (dict(rows=-1), INVALID), (dict(inner=-1), INVALID), (dict(dtype=5), INVALID),
    (dict(h=None), INVALID), (dict(q=None), INVALID), (dict(sf=None), INVALID), (dict(hsf=None), INVALID),
    (dict(ldh=511), INVALID), (dict(ldq=255), INVALID), (dict(ldhq=511), INVALID), (dict(hsf_sk=-1), INVALID),
    (dict(h=P + 8), UNSUPPORTED), (dict(hq=P + 8), UNSUPPORTED), (dict(inner=192), UNSUPPORTED),
    (dict(rows=(1 << 23) + 8), UNSUPPORTED)])
def test_swiglu_fp8(kw, status):
    assert call(lib.dg_swiglu_cast_fp8, SWIGLU, **kw) == status


SWIGLU8 = dict(h=P, dtype=1, ldh=512, m_indices=None, masked_m=None, groups=0, q=P, ldq=256, sf=P, sf_s=1, rows=8, inner=256,
               stream=None)


@pytest.mark.parametrize("kw,status", SET_CASES + [
    (dict(rows=0), OK), (dict(h=None), INVALID), (dict(sf=None), INVALID), (dict(sf_s=-1), INVALID),
    (dict(inner=248), UNSUPPORTED), (dict(inner=16400, ldh=32800, ldq=16400), UNSUPPORTED), (dict(ldq=264), UNSUPPORTED)])
def test_swiglu_int8(kw, status):
    assert call(lib.dg_swiglu_cast_int8, SWIGLU8, **kw) == status


SWIGLU_GRAD = dict(da=P, dtype=1, ldda=256, h=P, ldh=512, hq=None, ldhq=0, hsf=None, hsf_sm=0, hsf_sk=0, m_indices=None,
                   masked_m=None, groups=0, dh=P, lddh=512, q=None, ldq=0, sf=None, sf_sm=0, sf_sk=0, rows=8, inner=256,
                   ue8m0=0, stream=None)
KEPT = dict(h=None, hq=P, ldhq=512, hsf=P, hsf_sm=4, hsf_sk=1)
CAST = dict(q=P, ldq=512, sf=P, sf_sm=4, sf_sk=1)


@pytest.mark.parametrize("kw,status", SET_CASES + [
    (dict(rows=0), OK), (dict(inner=0), OK), (dict(da=None), INVALID), (dict(dh=None), INVALID), (dict(h=None), INVALID),
    (dict(KEPT, h=P), INVALID), (dict(KEPT, hsf=None), INVALID), (dict(KEPT, ldhq=256), INVALID), (dict(CAST, sf=None), INVALID),
    (dict(CAST, ldq=256), INVALID), (dict(ldda=255), INVALID), (dict(lddh=256), INVALID), (dict(inner=252), UNSUPPORTED),
    (dict(KEPT, inner=200), UNSUPPORTED), (dict(CAST, inner=200), UNSUPPORTED), (dict(dh=P + 8), UNSUPPORTED),
    (dict(KEPT, hq=P + 8), UNSUPPORTED)])
def test_swiglu_grad(kw, status):
    assert call(lib.dg_swiglu_grad, SWIGLU_GRAD, **kw) == status


WGRAD = dict(dy=P, lddy=64, x=P, ldx=256, sf=None, sf_sm=0, sf_sk=0, dw=P, out=0, lddw=256, accumulate=0, rows=32, n=64,
             k=256, ws=None, ws_bytes=0, stream=None)
SCALED = dict(sf=P, sf_sm=2, sf_sk=1)
WGRAD_CASES = [
    (dict(n=0), OK), (dict(k=0), OK), (dict(n=-8), INVALID), (dict(out=2), INVALID), (dict(dw=None), INVALID),
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(lddy=63), INVALID), (dict(ldx=255), INVALID),
    (dict(lddw=255), INVALID), (dict(SCALED, sf_sm=-1), INVALID), (dict(SCALED, sf=P + 2), UNSUPPORTED),
    (dict(accumulate=1, out=1), UNSUPPORTED), (dict(n=60), UNSUPPORTED), (dict(k=252), UNSUPPORTED),
    (dict(SCALED, k=192), UNSUPPORTED), (dict(SCALED, ldx=264), UNSUPPORTED), (dict(lddy=68), UNSUPPORTED),
    (dict(dy=P + 8), UNSUPPORTED), (dict(x=P + 8), UNSUPPORTED), (dict(dw=P + 8), UNSUPPORTED),
    (dict(lddw=258), UNSUPPORTED), (dict(lddy=1 << 24), UNSUPPORTED), (dict(ldx=1 << 24), UNSUPPORTED),
    (dict(ws=P + 8, ws_bytes=1 << 20), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", WGRAD_CASES + [(dict(rows=-1), INVALID), (dict(rows=1 << 31), UNSUPPORTED)])
def test_weight_grad(kw, status):
    assert call(lib.dg_weight_grad, WGRAD, **kw) == status


WGRAD_CONTIGUOUS = dict(dy=P, lddy=64, x=P, ldx=256, sf=None, sf_sm=0, sf_sk=0, dw=P, out=0, lddw=256, dw_gs=64 * 256,
                        counts=P, groups=4, alignment=128, accumulate=0, rows=512, n=64, k=256, ws=None, ws_bytes=0,
                        stream=None)


@pytest.mark.parametrize("kw,status", WGRAD_CASES + [
    (dict(groups=0), OK), (dict(groups=-1), INVALID), (dict(counts=None), INVALID), (dict(alignment=0), INVALID),
    (dict(alignment=1 << 31), UNSUPPORTED), (dict(groups=1025), UNSUPPORTED), (dict(counts=P + 2), UNSUPPORTED),
    (dict(dw_gs=-1), INVALID), (dict(dw_gs=2), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED)])
def test_weight_grad_contiguous(kw, status):
    assert call(lib.dg_m_grouped_weight_grad_contiguous, WGRAD_CONTIGUOUS, **kw) == status


WGRAD_MASKED = dict(dy=P, lddy=64, x=P, ldx=256, sf=None, sf_sm=0, sf_sk=0, dw=P, out=0, lddw=256, dw_gs=64 * 256, masked_m=P,
                    groups=4, max_m=128, accumulate=0, n=64, k=256, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("kw,status", WGRAD_CASES + [
    (dict(groups=0), OK), (dict(groups=-1), INVALID), (dict(masked_m=None), INVALID), (dict(max_m=-1), INVALID),
    (dict(max_m=1 << 29), UNSUPPORTED), (dict(groups=1025), UNSUPPORTED)])
def test_weight_grad_masked(kw, status):
    assert call(lib.dg_m_grouped_weight_grad_masked, WGRAD_MASKED, **kw) == status


def test_weight_grad_workspace_is_bounded():
    size = lib.dg_weight_grad_workspace_size
    assert size(0, 64, 64, 1) == 0 and size(64, 0, 64, 1) == 0 and size(64, 64, 64, 0) == 0
    assert size(16, 64, 64, 1) == 0                     # too few rows to share
    assert size(32768, 4096, 7168, 8) == 0              # enough tiles
    assert 0 < size(32768, 128, 128, 1) <= 64 * 128 * 128 * 4


def test_binding_rejects_wrong_tensors():
    """Host tensors, before any library call."""
    x, i, b = torch.zeros((4, 256)), torch.zeros(4, dtype=torch.int32), torch.zeros((4, 256), dtype=torch.bfloat16)
    for f in (lambda: dg.rms_norm(x), lambda: dg.rms_norm_cast_fp8(x), lambda: dg.rms_norm_cast_int8(x),
              lambda: dg.rms_norm_grad(x, x, None, x[:, 0]), lambda: dg.swiglu_cast_fp8(x),
              lambda: dg.swiglu_checkpoint_fp8(x), lambda: dg.swiglu_cast_int8(x), lambda: dg.swiglu_grad(x, x),
              lambda: dg.swiglu_grad_cast_fp8(x, (b, x)), lambda: dg.weight_grad(b, b, x),
              lambda: dg.m_grouped_weight_grad_contiguous(b, b, x[None], i),
              lambda: dg.m_grouped_weight_grad_masked(b, b, x[None], i)):
        with pytest.raises(TypeError):
            f()
