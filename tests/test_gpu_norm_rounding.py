"""What the norm's rows are before they are stored or cast: h w rstd in one rounding where h and w have 12 significant bits
or fewer, whose product fp32 holds.  Codes are then those of the exact products' casts, bit for bit: a quotient that lies on
a midpoint of two codes, as 16-bit factors often make, is decided by as few roundings as there can be."""
import numpy as np
import pytest
import torch

from gpu_util import codes, device

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_fp8_gemm_amd as dg  # noqa: E402
from oracle import int8 as oint8  # noqa: E402
from oracle import quant  # noqa: E402
from test_gpu_layer import BF16, F16, U, f64, half, near, norm_inputs, strided, tiny  # noqa: E402


def exact(h, w, rstd):
    """h w rstd in 64 bits (12 + 12 + 24 bits: exact), rounded to fp32 once."""
    return (h.double().cpu().numpy() * w.double().cpu().numpy() * rstd.double().cpu().numpy()[:, None]).astype(np.float32)


@pytest.mark.parametrize("m,k", [(1, 7168), (40, 512), (33, 2176), (300, 4224), (3, 8320), (257, 1024)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_one_rounding_before_the_cast(m, k, dtype):
    x, r, w, h = norm_inputs(m, k, dtype, 11 * m + k)
    w = w.to(dtype)
    wd = w.to(device())
    y, _, rstd = dg.rms_norm(h.float().to(device()), w.float().to(device()))
    assert np.array_equal(y.cpu().numpy(), exact(h, w, rstd))
    for ue8m0 in (False, True):
        (q, sf), gh, rstd = dg.rms_norm_cast_fp8(strided(x), wd, strided(r), ue8m0=ue8m0)
        oq, osf = quant.per_token_cast(exact(h, w, rstd), ue8m0)
        assert torch.equal(gh.cpu(), h) and np.array_equal(codes(q), oq) and np.array_equal(sf.cpu().numpy(), osf)
    (q, sf), _, rstd = dg.rms_norm_cast_int8(x.to(device()), wd, r.to(device()))
    oq, osf = oint8.cast(exact(h, w, rstd))
    assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(sf.cpu().numpy(), osf)
    # Stored rows: E = h w rstd is rounded to fp32 (U |E|) and then to the type (half a step of at most (1 + U) |E|), or, where
    # the conversion is part of the product's instruction, to the type at once (half a step of |E|): the bound holds both.
    y, _, rstd = dg.rms_norm(x.to(device()), wd, r.to(device()))
    e = f64(h) * f64(w) * f64(rstd)[:, None]
    near(y, e, (half(dtype) * (1 + U) + U) * np.abs(e) + tiny(dtype))


def test_weights_and_rows_at_the_ends_of_fp32():
    """Rows whose squares fp32 holds, with weights of that size: their product is finite and no subnormal number."""
    x = torch.full((2, 256), 1e18, device=device())
    x[1] = 1e-18
    w = torch.full((256,), 1e19, device=device())
    y, _, rstd = dg.rms_norm(x, w, eps=0.0)
    assert bool(((y / 1e19 - 1).abs() < 64 * 2.0 ** -24).all())
    y, _, _ = dg.rms_norm(x, 1 / w, eps=0.0)
    assert bool(((y * 1e19 - 1).abs() < 64 * 2.0 ** -24).all())
