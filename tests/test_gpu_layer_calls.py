"""Calls of the norm, the gated activation and the weights' gradients at the edges of what their documentation allows."""
import pytest
import torch

from gpu_util import device

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_fp8_gemm_amd as dg  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("norm", [dg.rms_norm, dg.rms_norm_cast_fp8, dg.rms_norm_cast_int8])
def test_norm_does_not_write_y_over_the_h_that_it_returns(norm):
    """Without a residual the h that is returned is x: a gradient from it would be that of other rows."""
    x = torch.randn((5, 256), device=device())
    kept = x.clone()
    with pytest.raises(ValueError):
        norm(x, y=x)
    assert torch.equal(x, kept)
    want = norm(kept)
    h = torch.empty_like(x)
    out, got, rstd = norm(x, y=x, h=h)          # a copy of x is kept
    assert got is h and torch.equal(h, kept) and torch.equal(rstd, want[2]) and not torch.equal(x, kept)
    x.copy_(kept)
    _, got, _ = norm(x, None, torch.zeros_like(x), y=x)
    assert torch.equal(got, kept)
    y = torch.empty_like(x)
    x.copy_(kept)
    _, got, _ = norm(x, y=y)
    assert got is x and torch.equal(x, kept)
