"""Expert layout, dispatch and combination on the GPU against the oracles.

Layouts, routing of rows and codes are equal element for element.  Combination:
each output is an fp32 sum of at most 64 products (error under 64 * 2^-24 of the sum of the terms'
magnitudes); a bf16 output is that sum rounded once, bit for bit.  The gradient's dot products run over
h <= 8192 elements with at most 80 roundings on the longest path: 80 * 2^-24 of the
terms' magnitudes; dy is one fp32 product rounded to bf16, bit for bit.
"""
import numpy as np
import pytest
import torch

from oracle import moe, quant
from gpu_util import codes, device

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_fp8_gemm_amd as dg  # noqa: E402


def routing(t, k, e, seed, drop=0.1, skew=1.0):
    """Distinct experts for each token where there are enough, some dropped."""
    rng = np.random.default_rng(seed)
    p = (np.arange(e) + 1.0) ** -skew
    keys = np.log(p) + rng.gumbel(size=(t, e))
    idx = np.argsort(-keys, axis=1)[:, :k].astype(np.int32)
    idx[rng.random((t, k)) < drop] = -1
    return idx


@pytest.mark.parametrize("t,k,e", [(0, 2, 4), (1, 1, 1), (1, 8, 256), (5, 3, 3), (64, 8, 256), (127, 2, 8), (128, 2, 8),
                                   (511, 8, 60), (512, 8, 256), (513, 8, 256), (700, 7, 256), (3000, 8, 1024),
                                   (4097, 1, 16), (9000, 4, 5), (33, 64, 64)])
def test_layouts(t, k, e):
    idx = routing(t, k, e, seed=t + k)
    if t > 2:
        idx[t // 2] = -1
        idx[t - 1, 0] = e + 3                            # outside: no row
    dev = torch.from_numpy(idx).to(device())
    rows = dg.expert_layout_rows(t, k, e)
    assert rows % 128 == 0
    lay = dg.expert_layout_contiguous(dev, e)
    m, row_slot, slot_row, counts = moe.layout_contiguous(idx, e, rows)
    assert np.array_equal(lay.counts.cpu().numpy(), counts)
    assert np.array_equal(lay.slot_row.cpu().numpy(), slot_row)
    assert np.array_equal(lay.m_indices.cpu().numpy(), m) and np.array_equal(lay.row_slot.cpu().numpy(), row_slot)
    assert (slot_row >= 0).sum() == counts.sum()         # the default holds every slot
    fewer = max(0, rows // 256 * 128)
    lay = dg.expert_layout_contiguous(dev, e, rows=fewer)
    m, row_slot, slot_row, counts = moe.layout_contiguous(idx, e, fewer)
    assert np.array_equal(lay.slot_row.cpu().numpy(), slot_row) and np.array_equal(lay.m_indices.cpu().numpy(), m)
    assert np.array_equal(lay.row_slot.cpu().numpy(), row_slot) and np.array_equal(lay.counts.cpu().numpy(), counts)
    for max_m in (1, 7, 256):
        lay = dg.expert_layout_masked(dev, e, max_m)
        row_slot, slot_row, masked_m = moe.layout_masked(idx, e, max_m)
        assert np.array_equal(lay.counts.cpu().numpy(), masked_m)
        assert np.array_equal(lay.slot_row.cpu().numpy(), slot_row)
        assert np.array_equal(lay.row_slot.cpu().numpy(), row_slot)


@pytest.mark.parametrize("t,k,e", [(129, 8, 256), (256, 8, 256), (257, 8, 700), (1025, 1, 5), (384, 8, 60), (385, 8, 60),
                                   (3073, 1, 1), (1024, 3, 1024)])
def test_layouts_around_the_sizes_of_one_launch(t, k, e):
    test_layouts(t, k, e)


def test_layout_of_one_crowded_expert_and_of_strided_indices():
    idx = np.full((3000, 3), -1, np.int32)
    idx[:, 1] = 5
    dev = torch.full((3000, 8), 2, dtype=torch.int32, device=device())
    dev[:, 3:6] = torch.from_numpy(idx).to(device())
    lay = dg.expert_layout_contiguous(dev[:, 3:6], 9)
    want = moe.layout_contiguous(idx, 9, lay.rows)
    assert np.array_equal(lay.m_indices.cpu().numpy(), want[0]) and np.array_equal(lay.slot_row.cpu().numpy(), want[2])


def test_capacity_bound_is_reached():
    """Every used expert's segment may be padded by 127 rows."""
    idx = np.repeat(np.arange(6), 129)[:, None].astype(np.int32)
    lay = dg.expert_layout_contiguous(torch.from_numpy(idx).to(device()), 6)
    assert int(lay.slot_row.max()) == 5 * 256 + 128 and lay.rows == (6 * 129 + 6 * 127) // 128 * 128


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,k,e,cols", [(1, 1, 1, 128), (3, 8, 16, 640), (40, 2, 8, 7168), (17, 5, 60, 4096),
                                        (9, 3, 7, 4224), (65, 64, 64, 128)])
def test_dispatch_fp8(t, k, e, cols, dtype):
    rng = np.random.default_rng(t)
    x = torch.from_numpy((rng.standard_normal((t, cols)) * np.exp2(rng.uniform(-9, 9, (t, 1)))).astype(np.float32))
    x[0, :128] = 0.0
    x = x.to(dtype)
    idx = routing(t, k, e, seed=t)
    lay = dg.expert_layout_contiguous(torch.from_numpy(idx).to(device()), e)
    slot_row = lay.slot_row.cpu().numpy()
    for ue8m0 in (False, True):
        q = torch.full((lay.rows, cols), 0x55, dtype=torch.uint8, device=device())
        sf = torch.full((cols // 128, lay.rows), -7.0, device=device()).t() if ue8m0 else \
            torch.full((lay.rows, cols // 128), -7.0, device=device())
        dg.dispatch_cast_fp8(x.to(device()), lay.slot_row, ue8m0=ue8m0, q=q, sf=sf)
        oq, os_ = quant.per_token_cast(x.float().numpy(), ue8m0)
        want_q = np.full((lay.rows, cols), 0x55, np.uint8)
        want_s = np.full((lay.rows, cols // 128), -7.0, np.float32)
        for a in range(t):
            for r in slot_row[a][slot_row[a] >= 0]:
                want_q[r], want_s[r] = oq[a], os_[a]
        assert np.array_equal(codes(q), want_q) and np.array_equal(sf.cpu().numpy(), want_s)
    q, sf = dg.dispatch_cast_fp8(x.to(device()), lay.slot_row, rows=lay.rows)
    held = lay.row_slot.cpu().numpy() >= 0
    pq, ps = dg.per_token_cast_fp8(x.to(device()))
    token = lay.row_slot.cpu().numpy()[held] // k
    assert np.array_equal(codes(q)[held], codes(pq)[token])
    assert np.array_equal(sf.cpu().numpy()[held], ps.cpu().numpy()[token])


def test_dispatch_skips_rows_outside():
    x = torch.randn((4, 128), device=device())
    q = torch.full((6, 128), 0x55, dtype=torch.uint8, device=device())
    sf = torch.full((6, 1), -7.0, device=device())
    slot_row = torch.tensor([[0, 6], [-1, 1 << 30], [5, -(1 << 31)], [2, 3]], dtype=torch.int32, device=device())
    dg.dispatch_cast_fp8(x, slot_row, q=q, sf=sf)
    touched = (sf[:, 0] != -7.0).cpu().numpy()
    assert touched.tolist() == [True, False, True, True, False, True]
    assert bool((q[[1, 4]] == 0x55).all())


COMBINE = [(1, 1, 1, 8), (1, 8, 256, 7168), (3, 5, 7, 1000), (64, 2, 8, 2048), (33, 8, 16, 2056), (20, 9, 60, 264),
           (7, 64, 64, 4104)]


@pytest.mark.parametrize("t,k,e,h", COMBINE)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(t, k, e, h, weighted):
    rng = np.random.default_rng(h)
    idx = routing(t, k, e, seed=h)
    if t > 2:
        idx[1] = -1                                      # a token nobody answers
    lay = dg.expert_layout_contiguous(torch.from_numpy(idx).to(device()), e)
    y = torch.from_numpy(rng.standard_normal((lay.rows, h)).astype(np.float32)).to(torch.bfloat16)
    y[lay.row_slot.cpu() < 0] = float("nan")             # what no slot holds is never read
    w = rng.standard_normal((t, k)).astype(np.float32)
    slot_row = lay.slot_row.cpu().numpy()
    wd = w.copy()
    wd[slot_row < 0] = np.nan
    args = (y.to(device()), lay.slot_row) + ((torch.from_numpy(wd).to(device()),) if weighted else ())
    host = np.nan_to_num(y.float().numpy())
    want = moe.combine(host, slot_row, w if weighted else None)
    size = moe.combine(np.abs(host), slot_row, np.abs(w) if weighted else None)
    got32 = dg.combine(*args, out=torch.empty((t, h), device=device()))
    assert np.all(np.abs(got32.cpu().numpy() - want) <= 64 * 2.0 ** -24 * size)
    assert torch.equal(dg.combine(*args), got32.to(torch.bfloat16))


@pytest.mark.parametrize("t,k,e,h", COMBINE)
def test_combine_grad(t, k, e, h):
    rng = np.random.default_rng(h + 1)
    idx = routing(t, k, e, seed=h)
    lay = dg.expert_layout_contiguous(torch.from_numpy(idx).to(device()), e)
    slot_row = lay.slot_row.cpu().numpy()
    y = torch.from_numpy(rng.standard_normal((lay.rows, h)).astype(np.float32)).to(torch.bfloat16)
    dout = torch.from_numpy(rng.standard_normal((t, h)).astype(np.float32)).to(torch.bfloat16)
    y[lay.row_slot.cpu() < 0] = float("nan")
    w = rng.standard_normal((t, k)).astype(np.float32)
    wd = w.copy()
    wd[slot_row < 0] = np.nan
    dy = torch.full((lay.rows, h), float("nan"), dtype=torch.bfloat16, device=device())
    dw = torch.full((t, k), float("nan"), device=device())
    dg.combine_grad(dout.to(device()), y.to(device()), lay.slot_row, lay.row_slot, torch.from_numpy(wd).to(device()),
                    dy=dy, dweights=dw)
    host, g = np.nan_to_num(y.float().numpy()), dout.float().numpy()
    _, want_dw = moe.combine_grad(g, host, slot_row, w)
    _, size = moe.combine_grad(np.abs(g), np.abs(host), slot_row, w)
    assert np.all(np.abs(dw.cpu().numpy() - want_dw) <= 80 * 2.0 ** -24 * size)
    row_slot = lay.row_slot.cpu().long()
    held = row_slot >= 0
    want_dy = torch.zeros((lay.rows, h), dtype=torch.bfloat16)
    slot = row_slot[held]
    want_dy[held] = (dout.float()[slot // k] * torch.from_numpy(w).view(-1, 1)[slot]).to(torch.bfloat16)
    assert torch.equal(dy.cpu(), want_dy)


def test_row_strides_and_masked_layout():
    idx = routing(50, 3, 4, seed=2)
    lay = dg.expert_layout_masked(torch.from_numpy(idx).to(device()), 4, 16)
    y = torch.randn((64, 272), device=device()).to(torch.bfloat16)
    w = torch.rand((50, 5), device=device())
    out = torch.full((50, 280), -7.0, dtype=torch.bfloat16, device=device())
    dg.combine(y[:, 8:264], lay.slot_row, w[:, 1:4], out=out[:, 16:272])
    assert torch.equal(out[:, 16:272], dg.combine(y[:, 8:264].contiguous(), lay.slot_row, w[:, 1:4].contiguous()))
    assert bool((out[:, :16] == -7).all() and (out[:, 272:] == -7).all())
    dout = torch.randn((50, 320), device=device()).to(torch.bfloat16)
    a = dg.combine_grad(dout[:, 64:], y[:, 8:264], lay.slot_row, lay.row_slot, w[:, 1:4])
    b = dg.combine_grad(dout[:, 64:].contiguous(), y[:, 8:264].contiguous(), lay.slot_row, lay.row_slot,
                        w[:, 1:4].contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_offsets_beyond_32_bits():
    """Rows past 4 GiB from the first, written by the dispatch and read by the combination."""
    cols, rows = 7168, 700_000                           # 5.0 GB of codes
    q = torch.zeros((rows, cols), dtype=torch.uint8, device=device())
    sf = torch.zeros((rows, cols // 128), device=device())
    x = torch.randn((2, cols), device=device()).to(torch.bfloat16)
    slot_row = torch.tensor([[rows - 1, 3], [rows - 2, -1]], dtype=torch.int32, device=device())
    dg.dispatch_cast_fp8(x, slot_row, q=q, sf=sf)
    pq, ps = dg.per_token_cast_fp8(x)
    assert torch.equal(q[[rows - 1, 3, rows - 2]], pq.view(torch.uint8)[[0, 0, 1]])
    assert torch.equal(sf[[rows - 1, 3, rows - 2]], ps[[0, 0, 1]])
    del q, sf
    y = torch.zeros((rows // 2, cols), dtype=torch.bfloat16, device=device())
    slot_row = torch.tensor([[rows // 2 - 1, 3]], dtype=torch.int32, device=device())
    y[[rows // 2 - 1, 3]] = x
    out = dg.combine(y, slot_row, torch.tensor([[2.0, 0.5]], device=device()))
    assert torch.equal(out[0], (2 * x[0].float() + 0.5 * x[1].float()).to(torch.bfloat16))


def test_layer_steps_in_a_graph_and_on_another_stream():
    """Routing to combination captured once, replayed on new logits with eager calls between the replays."""
    t, e, k, h = 300, 16, 4, 256
    x = torch.randn((t, h), device=device()).to(torch.bfloat16)
    logits = torch.randn((t, e), device=device())

    def step():
        idx, w = dg.route_topk(logits, k)
        lay = dg.expert_layout_contiguous(idx, e)
        q, sf = dg.dispatch_cast_fp8(x, lay.slot_row, rows=lay.rows)
        y = torch.empty((lay.rows, h), dtype=torch.bfloat16, device=device())
        y.copy_(q.to(torch.bfloat16))
        return dg.combine(y, lay.slot_row, w), lay.slot_row

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, slot_row = step()
    for r in range(3):
        logits.copy_(torch.randn((t, e), device=device(), generator=torch.Generator(device=device()).manual_seed(r)))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), slot_row.clone()
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---------------------------------------------------------------- layouts of many slots

@pytest.mark.parametrize("t,k,e", [(8193, 8, 256), (9001, 8, 1000), (70001, 1, 7), (21846, 3, 64)])
def test_layouts_past_64_workgroups(t, k, e):
    test_layouts(t, k, e)


@pytest.mark.parametrize("t,k,e", [(131073, 3, 256), (49153, 8, 1000), (400_001, 1, 5)])
def test_layouts_whose_counts_are_summed_apart(t, k, e):
    """Past 96 workgroups of 4096 slots."""
    test_layouts(t, k, e)


def test_masked_rows_at_the_end_of_int32():
    """The last expert's slots outnumber its rows, which end just below 2^31: every slot past them is dropped as -1."""
    t, e, max_m = 2_100_000, 1024, 2_097_151
    assert (e - 1) * max_m + t > 1 << 31 > e * max_m
    lay = dg.expert_layout_masked(torch.full((t, 1), e - 1, dtype=torch.int32, device=device()), e, max_m)
    want = torch.arange(t, dtype=torch.int64, device=device()) + (e - 1) * max_m
    want[max_m:] = -1
    assert torch.equal(lay.slot_row[:, 0].long(), want)
    assert lay.counts.tolist() == [0] * (e - 1) + [max_m]
    assert bool((lay.row_slot[:(e - 1) * max_m] == -1).all())
    assert torch.equal(lay.row_slot[(e - 1) * max_m:], torch.arange(max_m, dtype=torch.int32, device=device()))


def test_layout_time_grows_with_the_slots():
    """Four times the slots take about four times as long, not sixteen times."""
    def least(t):
        idx = torch.randint(0, 256, (t, 8), generator=torch.Generator(device=device()).manual_seed(1), device=device(),
                            dtype=torch.int32)
        times = []
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            dg.expert_layout_masked(idx, 256, 1 << 16)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    small, large = least(1 << 21), least(1 << 23)
    assert large < 8 * small, f"{small} ms, then {large} ms"


def test_small_layouts_take_no_workspace():
    """Up to 3072 slots the calls use none and do not ask for one."""
    for t in (128, 129, 384):
        idx = torch.from_numpy(routing(t, 8, 60, seed=t)).to(device())
        rows = dg.expert_layout_rows(t, 8, 60)
        new = lambda *size: torch.full(size, -7, dtype=torch.int32, device=device())  # noqa: E731
        m, row_slot, slot_row, counts = new(rows), new(rows), new(t, 8), new(60)
        stream = torch.cuda.current_stream().cuda_stream
        assert dg.lib.dg_expert_layout_contiguous(idx.data_ptr(), 8, t, 8, 60, rows, m.data_ptr(), row_slot.data_ptr(),
                                                  slot_row.data_ptr(), counts.data_ptr(), None, 0, stream) == 0
        for got, want in zip((m, row_slot, slot_row, counts), moe.layout_contiguous(idx.cpu().numpy(), 60, rows)):
            assert np.array_equal(got.cpu().numpy(), want)
        row_slot = new(60 * 16)
        assert dg.lib.dg_expert_layout_masked(idx.data_ptr(), 8, t, 8, 60, 16, counts.data_ptr(), row_slot.data_ptr(),
                                              slot_row.data_ptr(), None, 0, stream) == 0
        for got, want in zip((row_slot, slot_row, counts), moe.layout_masked(idx.cpu().numpy(), 60, 16)):
            assert np.array_equal(got.cpu().numpy(), want)


def test_combine_grad_without_columns():
    lay = dg.expert_layout_contiguous(torch.from_numpy(routing(5, 2, 3, seed=1)).to(device()), 3)
    none = torch.empty((lay.rows, 0), dtype=torch.bfloat16, device=device())
    dy, dw = dg.combine_grad(none[:5], none, lay.slot_row, lay.row_slot, torch.ones((5, 2), device=device()))
    assert dy.shape == (lay.rows, 0) and bool((dw == 0).all())
