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


def test_rows_without_columns():
    """What does not depend on columns is written: NaN for the mean of nothing, and the scale that a row of zeros has."""
    e = torch.empty((5, 0), dtype=BF16, device=device())
    zeros = torch.zeros((5, 128), dtype=BF16, device=device())
    floor = dg.per_token_cast_int8(zeros)[1]
    for norm in (dg.rms_norm, dg.rms_norm_cast_fp8, dg.rms_norm_cast_int8):
        for residual in (None, e):
            rstd = torch.full((5,), 7.0, device=device())
            out, h, got = norm(e, None, residual, rstd=rstd)
            assert got is rstd and h.shape == (5, 0) and bool(rstd.isnan().all())
    sf = torch.full((10,), 7.0, device=device())
    dg.rms_norm_cast_int8(e, sf=sf[::2])
    assert torch.equal(sf[::2], floor) and bool((sf[1::2] == 7).all())
    sf = torch.full((5,), 7.0, device=device())
    q, got = dg.swiglu_cast_int8(e, sf=sf)
    assert got is sf and q.shape == (5, 0) and torch.equal(sf, floor)
    sf.fill_(7)
    dg.swiglu_cast_int8(e, m_indices=torch.tensor([0, -1, 2, -1, 0], dtype=torch.int32, device=device()), sf=sf)
    assert torch.equal(sf[::2], floor[::2]) and bool((sf[1::2] == 7).all())
    sf = torch.full((4,), 7.0, device=device())
    dg.swiglu_cast_int8(e[:4], masked_m=torch.tensor([1, 5], dtype=torch.int32, device=device()), sf=sf)
    assert torch.equal(sf[[0, 2, 3]], floor[:3]) and sf[1] == 7
    dx, dw = dg.rms_norm_grad(e, e, torch.empty(0, device=device()), torch.ones(5, device=device()))
    assert dx.shape == (5, 0) and dw.shape == (0,)
    assert dg.swiglu_cast_fp8(e)[1].shape == (5, 0) and dg.swiglu_grad(e, e).shape == (5, 0)


def test_weight_grad_of_as_many_rows_as_there_can_be():
    """2^31 - 1 rows of one group, 34 GB: zeros but for a few rows of whole numbers, whose products are exact."""
    rows, n = 2 ** 31 - 1, 8
    dy = torch.zeros((rows, n), dtype=BF16, device=device())
    at = torch.tensor([0, 31, 2 ** 20 + 3, 2 ** 30, 2 ** 31 - 34, 2 ** 31 - 33, 2 ** 31 - 2], device=device())
    dy[at] = ((torch.arange(7 * n, device=device()).view(7, n) * 5) % 13 - 6).to(BF16)
    few = dy[at].double()
    want = (few.t() @ few).float()
    count = torch.tensor([rows], dtype=torch.int32, device=device())
    assert dg.lib.dg_weight_grad_workspace_size(rows, n, n, 1) > 0
    dw = torch.empty((n, n), device=device())
    assert torch.equal(dg.weight_grad(dy, dy, dw), want)
    for f in (dg.m_grouped_weight_grad_contiguous, dg.m_grouped_weight_grad_masked):
        dw = torch.ones((1, n, n), device=device())
        assert torch.equal(f(dy, dy, dw, count, accumulate=True)[0], want + 1)
    count -= 31                                   # the last rows are behind the last whole stage
    dy[-31:] = float("nan")
    few[-1] = 0
    dw = torch.empty((1, n, n), device=device())
    assert torch.equal(dg.m_grouped_weight_grad_contiguous(dy, dy, dw, count)[0], (few.t() @ few).float())


def test_weight_grad_refuses_groups_in_one_place_and_takes_interleaved_ones():
    """An expanded dw would be written by all groups at once; rows of the groups in turn are as good as any other."""
    dy, x = (torch.randn((64, w), device=device()).to(BF16) for w in (24, 128))
    counts = torch.tensor([30, 0, 34], dtype=torch.int32, device=device())
    masked = torch.tensor([32, 30], dtype=torch.int32, device=device())
    for f, c in ((dg.m_grouped_weight_grad_contiguous, counts), (dg.m_grouped_weight_grad_masked, masked)):
        g = c.shape[0]
        kept = torch.full((1, 24, 128), 7.0, device=device())
        with pytest.raises(dg.DgError):
            f(dy, x, kept.expand(g, -1, -1), c)
        assert bool((kept == 7).all())
        one = dict(alignment=1) if c is counts else {}
        want = f(dy, x, torch.empty((g, 24, 128), device=device()), c, **one)
        turns = torch.empty((24, g, 128), device=device()).transpose(0, 1)
        assert f(dy, x, turns, c, **one) is turns and torch.equal(turns, want)
    one = torch.tensor([64], dtype=torch.int32, device=device())
    dw = torch.empty((24, 128), device=device())
    got = dg.m_grouped_weight_grad_contiguous(dy, x, dw.expand(1, -1, -1), one)        # one group: no other's place
    assert torch.equal(got[0], dg.weight_grad(dy, x, torch.empty_like(dw)))
