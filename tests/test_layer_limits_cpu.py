"""Refusals of the norm, gated activation and weights' gradients at the bounds of what the header allows, before
anything is launched.  Addresses are fake and never dereferenced."""
import pytest

from test_layer_abi_cpu import INVALID, OK, SWIGLU8, UNSUPPORTED, call, lib

P = 0x10000


@pytest.mark.parametrize("kw,status", [
    (dict(sf=None), INVALID), (dict(sf_s=-1), INVALID), (dict(sf=P + 2), UNSUPPORTED), (dict(rows=0, sf=None), OK),
    (dict(rows=(1 << 23) + 8), UNSUPPORTED), (dict(m_indices=P, masked_m=P, groups=2), INVALID)])
def test_int8_scales_of_rows_without_columns(kw, status):
    assert call(lib.dg_swiglu_cast_int8, SWIGLU8, **dict(dict(inner=0, h=None, q=None, ldh=0, ldq=0), **kw)) == status
