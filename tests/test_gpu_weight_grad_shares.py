"""Weights' gradients where several workgroups share a group's rows through the workspace, and a second launch adds their
sums.  Tolerances as in test_gpu_layer: the shares' sums are additions as the others are, and with at most 16 shares they are
among the 40 that are allowed besides the rows.
"""
import numpy as np
import pytest
import torch

from gpu_util import device

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_fp8_gemm_amd as dg  # noqa: E402
from oracle import layer  # noqa: E402
from test_gpu_layer import BF16, F32, check_weight_grad, f64, kept_rows, rows, strided  # noqa: E402

UNEVEN = [8000, 0, 0, 1, 40, 3, 600]     # shares of few rows have none
CASES = [([2000, 0, 37, 1500], 128, 136, 264), ([2000, 0, 37, 1500], 1, 136, 264), (UNEVEN, 128, 8, 136),
         (UNEVEN, 1, 264, 8), ([1024, 1025, -5, 1023], 1, 128, 512), ([513], 128, 128, 128)]


def shares(total, n, k, groups):
    size = dg.lib.dg_weight_grad_workspace_size(total, n, k, groups)
    assert size % (groups * n * k * 4) == 0
    return size // (groups * n * k * 4)


def operands(total, n, k, fp8, seed):
    """(dy, x on the device as given, dy and x's values)."""
    dy, x = rows((total, n), BF16, seed), rows((total, k), BF16, seed + 1)
    given, value = kept_rows(x, True) if fp8 else (x.to(device()), f64(x))
    return strided(dy), given, dy, value


def some(shape, seed):
    return torch.from_numpy(np.random.default_rng(seed).normal(size=shape).astype(np.float32))


@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("fp8", [False, True])
def test_contiguous(i, fp8):
    count, align, n, k = CASES[i]
    k = (k + 127) // 128 * 128 if fp8 else k
    total = sum(-(-max(0, c) // align) * align for c in count) + 3
    assert shares(total, n, k, len(count)) > 1
    dyd, given, dy, value = operands(total, n, k, fp8, i)
    segs = layer.segments(count, total, align)
    counts = torch.tensor(count, dtype=torch.int32, device=device())
    for out in (F32, BF16):
        dw = torch.full((len(count), n, k + 8), float("nan"), dtype=out, device=device())
        dg.m_grouped_weight_grad_contiguous(dyd, given, dw[..., :k], counts, alignment=align)
        check_weight_grad(dw[..., :k], dy, value, segs, out, False)
        assert bool(dw[..., k:].isnan().all())
    start = some((len(count), n, k), i)
    dw = start.to(device())
    dg.m_grouped_weight_grad_contiguous(dyd, given, dw, counts, alignment=align, accumulate=True)
    check_weight_grad(dw, dy, value, segs, F32, False, f64(start))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("groups,max_m,n,k", [(3, 900, 264, 128), (5, 2000, 8, 256), (1, 600, 40, 128)])
def test_masked(groups, max_m, n, k, fp8):
    count = [max_m + 4, 0, 33, -1, max_m // 2][:groups]
    assert shares(groups * max_m, n, k, groups) > 1
    dyd, given, dy, value = operands(groups * max_m, n, k, fp8, groups)
    segs = layer.segments(count, groups * max_m, max_m=max_m)
    counts = torch.tensor(count, dtype=torch.int32, device=device())
    start = some((groups, n, k), 3)
    for accumulate in (False, True):
        dw = start.to(device())
        dg.m_grouped_weight_grad_masked(dyd, given, dw, counts, accumulate=accumulate)
        check_weight_grad(dw, dy, value, segs, F32, False, f64(start) if accumulate else None)


@pytest.mark.parametrize("fp8", [False, True])
def test_dense_is_added_to_what_is_there(fp8):
    m, n, k = 4097, 128, 128
    assert shares(m, n, k, 1) > 8
    dyd, given, dy, value = operands(m, n, k, fp8, 5)
    start = some((n, k), 6)
    dw = start.to(device())
    for turn in (1, 2):
        assert dg.weight_grad(dyd, given, dw, accumulate=True) is dw
        check_weight_grad(dw, dy, value * turn, [(0, m)], F32, False, f64(start)[None])
    plain = torch.empty((n, k), device=device())
    dg.weight_grad(dyd, given, plain)
    check_weight_grad(plain, dy, value, [(0, m)], F32, False)


def test_with_and_without_a_workspace():
    """The C entry without one, or with a smaller one, multiplies a group's rows in one workgroup."""
    count, n, k = [2000, 0, 37, 1500], 136, 256
    total, g = sum(count), 4
    _, x, dy, value = operands(total, n, k, False, 9)
    dyd, counts = dy.to(device()), torch.tensor(count, dtype=torch.int32, device=device())
    need = shares(total, n, k, g) * g * n * k * 4
    ws = torch.full((need // 4,), float("nan"), device=device())
    got = []
    for p, size in ((None, 0), (ws.data_ptr(), need - 1), (ws.data_ptr(), need), (ws.data_ptr(), need)):
        dw = torch.empty((g, n, k), device=device())
        status = dg.lib.dg_m_grouped_weight_grad_contiguous(
            dyd.data_ptr(), n, x.data_ptr(), k, None, 0, 0, dw.data_ptr(), 0, k, n * k, counts.data_ptr(), g, 1, 0, total,
            n, k, p, size, torch.cuda.current_stream().cuda_stream)
        assert status == 0
        check_weight_grad(dw, dy, value, layer.segments(count, total, 1), F32, False)
        got.append(dw)
    assert torch.equal(got[0], got[1]) and torch.equal(got[2], got[3]) and not torch.equal(got[1], got[2])


def test_the_same_on_few_cus():
    count, n, k = UNEVEN, 264, 128
    total = sum(count)
    dyd, x, dy, value = operands(total, n, k, True, 11)
    assert shares(total, n, k, len(count)) > 1
    counts = torch.tensor(count, dtype=torch.int32, device=device())
    cus, got = dg.get_num_cus(), []
    for few in (cus, 8, 24, 1):
        dg.set_num_cus(few)
        try:
            dw = torch.empty((len(count), n, k), device=device())
            dg.m_grouped_weight_grad_contiguous(dyd, x, dw, counts, alignment=1)
        finally:
            dg.set_num_cus(cus)
        got.append(dw)
    assert all(torch.equal(got[0], g) for g in got[1:])
    check_weight_grad(got[0], dy, value, layer.segments(count, total, 1), F32, False)


def set_of(seed):
    count = [1500, 37, 2000]
    total, n, k = sum(count), 136, 256
    assert shares(total, n, k, 3) > 1
    dyd, x, _, _ = operands(total, n, k, bool(seed % 2), seed)
    return dyd, x, torch.tensor(count, dtype=torch.int32, device=device()), torch.zeros((3, n, k), device=device())


def passes(dyd, x, counts, dw):
    """A gradient, one added to it, and a dense one: three workspaces, one after the other."""
    dg.m_grouped_weight_grad_contiguous(dyd, x, dw, counts, alignment=1)
    dg.m_grouped_weight_grad_contiguous(dyd, x, dw, counts, alignment=1, accumulate=True)
    dense = torch.empty(dw.shape[1:], device=device())
    dg.weight_grad(dyd, x, dense)
    return [dw, dense]


def test_captured_and_replayed():
    """Two graphs in turn, with eager calls between them: every replay gives the eager calls' bits."""
    sets = [set_of(1), set_of(50)]
    eager = [[t.clone() for t in passes(*s)] for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in sets:
            passes(*s)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(passes(*s))
        graphs.append(g)
    other = set_of(99)
    for turn in range(4):
        for s in sets:
            s[3].fill_(float("nan"))
        for i in ((0, 1) if turn % 2 else (1, 0)):
            graphs[i].replay()
        passes(*other)
        torch.cuda.synchronize()
        for i in (0, 1):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], eager[i]))


def test_two_streams_at_once():
    sets = [set_of(3), set_of(70)]
    want = [[t.clone() for t in passes(*s)] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i] = passes(*sets[i])
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
