"""Refusals of the norm, gated activation and weights' gradients at the bounds of what the header allows, before
anything is launched.  Addresses are fake and never dereferenced."""
import pytest

from test_layer_abi_cpu import (INVALID, OK, SWIGLU8, UNSUPPORTED, WGRAD, WGRAD_CONTIGUOUS, WGRAD_MASKED, call,
                                lib)

P = 0x10000


@pytest.mark.parametrize("kw,status", [
    (dict(sf=None), INVALID), (dict(sf_s=-1), INVALID), (dict(sf=P + 2), UNSUPPORTED), (dict(rows=0, sf=None), OK),
    (dict(rows=(1 << 23) + 8), UNSUPPORTED), (dict(m_indices=P, masked_m=P, groups=2), INVALID)])
def test_int8_scales_of_rows_without_columns(kw, status):
    assert call(lib.dg_swiglu_cast_int8, SWIGLU8, **dict(dict(inner=0, h=None, q=None, ldh=0, ldq=0), **kw)) == status


def wide(n, k):
    return dict(n=n, k=k, lddy=n, ldx=k, lddw=k)


@pytest.mark.parametrize("n,k,groups", [(1 << 18, (1 << 18) + 8, 1), ((1 << 24) - 8, 4104, 1), (8192, 8200, 1024),
                                        (8, (1 << 19) + 8, 1024), (8, (1 << 24) - 8, 33)])
def test_weight_grad_of_too_many_tiles(n, k, groups):
    if groups == 1:
        assert call(lib.dg_weight_grad, WGRAD, **wide(n, k)) == UNSUPPORTED
    kw = dict(wide(n, k), groups=groups, dw_gs=n * k)
    assert call(lib.dg_m_grouped_weight_grad_contiguous, WGRAD_CONTIGUOUS, **kw) == UNSUPPORTED
    assert call(lib.dg_m_grouped_weight_grad_masked, WGRAD_MASKED, **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw,status", [(dict(dw_gs=0), INVALID), (dict(dw_gs=252), INVALID), (dict(dw_gs=-256), INVALID),
                                       (dict(dw_gs=0, out=1, accumulate=0), INVALID), (dict(dw_gs=2), UNSUPPORTED)])
def test_weight_grad_of_groups_in_one_place(kw, status):
    assert call(lib.dg_m_grouped_weight_grad_contiguous, WGRAD_CONTIGUOUS, **kw) == status
    assert call(lib.dg_m_grouped_weight_grad_masked, WGRAD_MASKED, **kw) == status
