"""int8 cast and GEMMs on the GPU against the oracle, bit for bit: the sums are exact and
every later step is one IEEE operation, so no tolerance is needed anywhere."""
import numpy as np
import pytest
import torch

from oracle import int8
from gpu_util import device, upload

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_fp8_gemm_amd as dg  # noqa: E402

OUT = [torch.bfloat16, torch.float16, torch.float32]
FILL = -7.0


def operands(m, n, k, seed):
    rng = np.random.default_rng(seed)
    return (rng.integers(-128, 128, (m, k)).astype(np.int8), (rng.random(m) * 0.02 + 1e-4).astype(np.float32),
            rng.integers(-128, 128, (n, k)).astype(np.int8), (rng.random(n) * 0.02 + 1e-4).astype(np.float32))


def expected(dtype, *ops):
    return torch.from_numpy(int8.gemm_nt(*ops)).to(dtype)


def same(got, want):
    return torch.equal(got.cpu().nan_to_num(123.0), want.nan_to_num(123.0))


def run(ops, dtype=torch.bfloat16, **kw):
    qa, sa, qb, sb = (upload(x) for x in ops)
    d = torch.full((qa.shape[0], qb.shape[0]), FILL, dtype=dtype, device=device())
    return dg.int8_gemm_nt((qa, sa), (qb, sb), d, **kw)


# ---------------------------------------------------------------- cast

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k", [(1, 16), (3, 48), (70, 1040), (5, 7168), (4, 8192), (3, 8208), (2, 24576)])
def test_cast(m, k, dtype):
    rng = np.random.default_rng(k)
    x = (rng.standard_normal((m, k)) * np.exp2(rng.uniform(-20, 20, (m, 1)))).astype(np.float32)
    x[0, :] = 0.0
    if m > 2:
        x[1] = np.float32(127.0) * (np.arange(k) % 2)
        x[1, 2:] = (np.arange(k - 2) % 255 - 127) / 2    # codes and ties at scale 1
        x[2, -1] = 3.0e38
    t = torch.from_numpy(x).to(dtype)
    q, s = dg.per_token_cast_int8(t.to(device()))
    oq, os_ = int8.cast(t.float().numpy())
    assert np.array_equal(s.cpu().numpy().view(np.uint32), os_.view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), oq)


@pytest.mark.parametrize("m,k", [(3, 2048), (3, 2064), (2, 4096), (5, 4112), (2, 16384), (2, 16400)])
def test_cast_rows_around_what_registers_hold(m, k):
    test_cast(m, k, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_cast_ties_and_ends(dtype):
    """A maximum of 127 makes the scale 1: halves go to the even code, and the ends stay at +-127."""
    x = torch.tensor([127.0, -127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5, -126.5, 63.5, -64.5, 0.0, -0.0, 0.4375, 126.0])
    q, s = dg.per_token_cast_int8(x.to(dtype).view(1, 16).to(device()))
    assert float(s) == 1.0
    assert q.cpu().view(-1).tolist() == [127, -127, 0, 2, 2, 0, -2, -2, 126, -126, 64, -64, 0, 0, 0, 126]


def test_cast_strides_and_bad_rows():
    x = torch.randn((6, 160), device=device())
    x[2, 9], x[4, 3] = float("nan"), float("inf")
    q = torch.full((6, 192), 99, dtype=torch.int8, device=device())
    sf = torch.full((6, 3), FILL, device=device())
    dg.per_token_cast_int8(x[:, 16:144], q=q[:, 32:160], sf=sf[:, 1])
    want = dg.per_token_cast_int8(x[:, 16:144].contiguous())
    good = [0, 1, 3, 4, 5]
    assert torch.equal(q[good, 32:160], want[0][good]) and torch.equal(sf[good, 1], want[1][good])
    assert bool((q[:, :32] == 99).all() and (q[:, 160:] == 99).all() and (sf[:, ::2] == FILL).all())
    x[4, 50] = float("inf")
    _, s = dg.per_token_cast_int8(x[:, :144])
    assert bool(torch.isnan(s[2])) and bool(torch.isinf(s[4])) and bool(torch.isfinite(s[[0, 1, 3, 5]]).all())


@pytest.mark.parametrize("t,k,e,cols", [(1, 1, 1, 16), (9, 3, 7, 1040), (40, 8, 16, 8208)])
def test_dispatch(t, k, e, cols):
    rng = np.random.default_rng(t)
    idx = np.argsort(rng.random((t, e)), axis=1)[:, :k].astype(np.int32)
    idx[rng.random((t, k)) < 0.1] = -1
    lay = dg.expert_layout_contiguous(upload(idx), e)
    x = torch.randn((t, cols), device=device()).to(torch.bfloat16)
    q = torch.full((lay.rows, cols), 99, dtype=torch.int8, device=device())
    sf = torch.full((lay.rows,), FILL, device=device())
    dg.dispatch_cast_int8(x, lay.slot_row, q=q, sf=sf)
    pq, ps = dg.per_token_cast_int8(x)
    held = lay.row_slot >= 0
    token = lay.row_slot[held].long() // k
    assert torch.equal(q[held], pq[token]) and torch.equal(sf[held], ps[token])
    assert bool((q[~held] == 99).all()) and bool((sf[~held] == FILL).all())


# ---------------------------------------------------------------- dense

@pytest.mark.parametrize("dtype", OUT)
@pytest.mark.parametrize("m,n,k", [(1, 8, 16), (1, 1, 128), (3, 7, 48), (16, 64, 112), (17, 129, 144), (64, 256, 512),
                                   (65, 100, 640), (127, 264, 1040), (128, 128, 128), (129, 257, 272),
                                   (256, 2112, 1536), (300, 520, 7152), (777, 1000, 400), (1, 4096, 7168)])
def test_dense(m, n, k, dtype):
    ops = operands(m, n, k, seed=m + n + k)
    want = expected(dtype, *ops)
    assert same(run(ops, dtype), want)
    assert same(run(ops, dtype, workspace=None), want)


@pytest.mark.parametrize("inst,splits", [(0, 1), (0, 3), (1, 1), (1, 2), (2, 1), (3, 1), (3, 5), (4, 1), (4, 7), (6, 1)])
@pytest.mark.parametrize("m,n,k", [(130, 330, 96), (64, 200, 128), (300, 777, 1424), (513, 1032, 1408)])
def test_forced_plans_give_the_same_bits(inst, splits, m, n, k):
    ops = operands(m, n, k, seed=inst)
    want = expected(torch.float32, *ops)
    dg.set_dense_plan(inst, splits)
    try:
        ws = torch.zeros(64 << 20, dtype=torch.uint8, device=device())
        assert same(run(ops, torch.float32, workspace=ws), want)
        assert same(run(ops, torch.float32, workspace=ws), want)     # the counters come back zero
    finally:
        dg.set_dense_plan(-1)


def test_grid_width_does_not_change_the_bits():
    ops = operands(700, 900, 656, seed=5)
    want = expected(torch.bfloat16, *ops)
    try:
        for cus in (1, 3, 8, 20):
            dg.set_num_cus(cus)
            assert same(run(ops), want)
    finally:
        dg.set_num_cus(0)


def test_extreme_codes_over_the_longest_sum():
    k = 131056
    qa = np.full((5, k), -128, np.int8)
    qb = np.full((6, k), -128, np.int8)
    qa[1], qb[2] = 127, 127
    s = np.ones(6, np.float32)
    ops = (qa, s[:5], qb, s)
    assert same(run(ops, torch.float32), expected(torch.float32, *ops))
    assert same(run(ops, torch.float32, workspace=None), expected(torch.float32, *ops))


def test_scales_of_every_kind_stay_in_their_row_and_column():
    ops = operands(70, 90, 320, seed=9)
    ops[1][3], ops[1][5], ops[1][7], ops[1][9] = np.nan, np.inf, 0.0, -2.0
    ops[3][2], ops[3][4] = np.nan, 0.0
    want = expected(torch.float32, *ops)
    assert same(run(ops, torch.float32), want) and same(run(ops), want.to(torch.bfloat16))


@pytest.mark.parametrize("dtype", OUT)
def test_strides(dtype):
    ops = operands(150, 203, 416, seed=4)
    want = expected(dtype, *ops)
    a = torch.zeros((150, 512), dtype=torch.int8, device=device())
    b = torch.zeros((203, 432), dtype=torch.int8, device=device())
    a[:, 64:480], b[:, 16:] = upload(ops[0]), upload(ops[2])
    sa, sb = torch.zeros((150, 3), device=device()), torch.zeros((203, 2), device=device())
    sa[:, 1], sb[:, 1] = upload(ops[1]), upload(ops[3])
    for left, width in ((0, 203), (8, 216), (3, 210), (1, 209)):     # rows at 16-byte boundaries, or only at elements
        d = torch.full((150, width), FILL, dtype=dtype, device=device())
        if left + 203 > width:
            continue
        dg.int8_gemm_nt((a[:, 64:480], sa[:, 1]), (b[:, 16:], sb[:, 1]), d[:, left:left + 203])
        assert same(d[:, left:left + 203], want)
        assert bool((d[:, :left] == FILL).all() and (d[:, left + 203:] == FILL).all())


def test_empty():
    for m, n in ((0, 64), (64, 0)):
        assert run(operands(m, n, 64, 0)).shape == (m, n)


# ---------------------------------------------------------------- grouped

def contiguous_case(counts, n, k, seed):
    rng = np.random.default_rng(seed)
    m_idx = np.concatenate([np.where(np.arange(-(-c // 128) * 128) < c, g, -1) for g, c in enumerate(counts)]
                           or [np.zeros(0)]).astype(np.int32)
    m, g = m_idx.size, len(counts)
    return (m_idx, rng.integers(-128, 128, (m, k)).astype(np.int8), (rng.random(m) * 0.02 + 1e-4).astype(np.float32),
            rng.integers(-128, 128, (g, n, k)).astype(np.int8), (rng.random((g, n)) * 0.02 + 1e-4).astype(np.float32))


@pytest.mark.parametrize("dtype", OUT)
@pytest.mark.parametrize("counts,n,k", [([1], 8, 16), ([0, 5, 0, 130, 0], 72, 208), ([128, 127, 129, 1], 264, 640),
                                        ([700, 900, 30], 520, 528), ([300] * 8, 100, 1024)])
def test_contiguous(counts, n, k, dtype):
    m_idx, qa, sa, qb, sb = contiguous_case(counts, n, k, seed=n)
    m_idx = np.concatenate([m_idx, np.full(256, -1, np.int32)])      # blocks of padding at the end
    qa = np.concatenate([qa, np.zeros((256, k), np.int8)])
    sa = np.concatenate([sa, np.full(256, np.nan, np.float32)])
    want = torch.full((m_idx.size, n), FILL, dtype=dtype)
    for g in range(len(counts)):
        rows = torch.from_numpy(m_idx == g)
        want[rows] = expected(dtype, qa[m_idx == g], sa[m_idx == g], qb[g], sb[g])
    try:
        for plan in (0, 1, 2):
            dg.set_contiguous_plan(plan)
            for ws in ("auto", None):
                d = torch.full((m_idx.size, n), FILL, dtype=dtype, device=device())
                dg.m_grouped_int8_gemm_nt_contiguous((upload(qa), upload(sa)), (upload(qb), upload(sb)), d,
                                                     upload(m_idx), workspace=ws)
                assert same(d, want), (plan, ws)
    finally:
        dg.set_contiguous_plan(0)


@pytest.mark.parametrize("counts,pad,n,k", [([1], 0, 8, 2560), ([0, 0], 2, 72, 2576), ([5, 0, 200], 1, 200, 2688 + 48),
                                            ([130, 127, 1, 90], 3, 264, 7168), ([129], 70, 128, 4096 + 16)])
def test_contiguous_split(counts, pad, n, k):
    """Few blocks and a long K: one launch that splits K over the blocks that are no padding; the workspace serves
    call after call, the second on other data."""
    for seed in (1, 2):
        m_idx, qa, sa, qb, sb = contiguous_case(counts, n, k, seed)
        m_idx = np.concatenate([np.full(128 * (pad // 2), -1), m_idx, np.full(128 * (pad - pad // 2), -1)]).astype(np.int32)
        lo = 128 * (pad // 2)
        qa = np.concatenate([np.zeros((lo, k), np.int8), qa, np.zeros((m_idx.size - lo - len(qa), k), np.int8)])
        sa = np.concatenate([np.full(lo, np.nan), sa, np.full(m_idx.size - lo - len(sa), np.nan)]).astype(np.float32)
        want = torch.full((m_idx.size, n), FILL, dtype=torch.bfloat16)
        for g in range(len(counts)):
            if counts[g]:
                rows = torch.from_numpy(m_idx == g)
                want[rows] = expected(torch.bfloat16, qa[m_idx == g], sa[m_idx == g], qb[g], sb[g])
        for ws in ("auto", None):
            d = torch.full((m_idx.size, n), FILL, dtype=torch.bfloat16, device=device())
            if m_idx.size:
                dg.m_grouped_int8_gemm_nt_contiguous((upload(qa), upload(sa)), (upload(qb), upload(sb)), d,
                                                     upload(m_idx), workspace=ws)
            assert same(d, want), ws


@pytest.mark.parametrize("dtype", OUT)
@pytest.mark.parametrize("g,max_m,n,k", [(1, 1, 8, 16), (5, 64, 100, 208), (3, 200, 264, 656), (16, 256, 72, 1040)])
@pytest.mark.parametrize("expected_m", [1, 100])
def test_masked(g, max_m, n, k, expected_m, dtype):
    rng = np.random.default_rng(g)
    masked_m = rng.integers(0, max_m + 1, g).astype(np.int32)
    masked_m[0] = max_m + 5                              # clamped
    if g > 2:
        masked_m[1], masked_m[2] = 0, -3
    qa = rng.integers(-128, 128, (g, max_m, k)).astype(np.int8)
    sa = (rng.random((g, max_m)) * 0.02 + 1e-4).astype(np.float32)
    qb = rng.integers(-128, 128, (g, n, k)).astype(np.int8)
    sb = (rng.random((g, n)) * 0.02 + 1e-4).astype(np.float32)
    want = torch.full((g, max_m, n), FILL, dtype=dtype)
    for i in range(g):
        c = int(np.clip(masked_m[i], 0, max_m))
        if c:
            want[i, :c] = expected(dtype, qa[i, :c], sa[i, :c], qb[i], sb[i])
    d = torch.full((g, max_m, n), FILL, dtype=dtype, device=device())
    dg.m_grouped_int8_gemm_nt_masked((upload(qa), upload(sa)), (upload(qb), upload(sb)), d, upload(masked_m),
                                     expected_m)
    assert same(d, want)


@pytest.mark.parametrize("cus", [0, 3, 20])
@pytest.mark.parametrize("expected_m", [0, 1, 16, 17, 40, 90])
def test_masked_plans_agree(expected_m, cus):
    """The hint and the grid width pick the kernel (few rows, 64 to 256 row tiles), never a bit of the result; groups
    hold none to all of the rows whatever the hint says, and K ends inside a block."""
    g, max_m, n, k = 5, 150, 328, 1552
    rng = np.random.default_rng(7)
    masked_m = np.array([0, 1, 17, 150, 65], np.int32)
    qa = rng.integers(-128, 128, (g, max_m, k)).astype(np.int8)
    sa = (rng.random((g, max_m)) * 0.02 + 1e-4).astype(np.float32)
    qb = rng.integers(-128, 128, (g, n, k)).astype(np.int8)
    sb = (rng.random((g, n)) * 0.02 + 1e-4).astype(np.float32)
    dtype = torch.bfloat16
    want = torch.full((g, max_m, n), FILL, dtype=dtype)
    for i, c in enumerate(masked_m):
        if c:
            want[i, :c] = expected(dtype, qa[i, :c], sa[i, :c], qb[i], sb[i])
    d = torch.full((g, max_m, n), FILL, dtype=dtype, device=device())
    try:
        dg.set_num_cus(cus)
        dg.m_grouped_int8_gemm_nt_masked((upload(qa), upload(sa)), (upload(qb), upload(sb)), d, upload(masked_m),
                                         expected_m)
    finally:
        dg.set_num_cus(0)
    assert same(d, want)


def test_graph_replays():
    """Dense with a K split, contiguous and masked in one graph; eager calls on the same workspace between replays."""
    ops = operands(64, 512, 2064, seed=3)
    m_idx, qa, sa, qb, sb = contiguous_case([200, 60], 136, 400, seed=4)
    dense = [upload(x) for x in ops]
    cont = [upload(x) for x in (qa, sa, qb, sb)]
    mi = upload(m_idx)
    mm = torch.tensor([3, 100], dtype=torch.int32, device=device())
    d1 = torch.zeros((64, 512), dtype=torch.bfloat16, device=device())
    d2 = torch.zeros((m_idx.size, 136), dtype=torch.bfloat16, device=device())
    d3 = torch.zeros((2, 128, 136), dtype=torch.bfloat16, device=device())

    def step():
        dg.int8_gemm_nt(tuple(dense[:2]), tuple(dense[2:]), d1)
        dg.m_grouped_int8_gemm_nt_contiguous(tuple(cont[:2]), tuple(cont[2:]), d2, mi)
        dg.m_grouped_int8_gemm_nt_masked((cont[0][:256].view(2, 128, 400), cont[1][:256].view(2, 128)), tuple(cont[2:]),
                                         d3, mm, 16)
    step()
    torch.cuda.synchronize()
    want = [x.clone() for x in (d1, d2, d3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(3):
        for x in (d1, d2, d3):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d1, want[0]) and torch.equal(d2, want[1]) and torch.equal(d3, want[2])
        step()
        torch.cuda.synchronize()


def test_operands_near_the_32_bit_offset_limit():
    """Rows just under 4 GiB from the first are read; one row more is refused."""
    k, ld = 272, 1 << 20
    rows = (1 << 32) // ld - 1
    qa = torch.zeros((rows, ld), dtype=torch.int8, device=device())
    ops = operands(4, 40, k, seed=1)
    qa[-4:, :k] = upload(ops[0])
    sa = torch.zeros(rows, device=device())
    sa[-4:] = upload(ops[1])
    d = torch.full((rows, 40), FILL, device=device())
    dg.int8_gemm_nt((qa[:, :k], sa), (upload(ops[2]), upload(ops[3])), d)
    assert same(d[-4:], expected(torch.float32, *ops))
    st = dg.lib.dg_int8_gemm_nt(qa.data_ptr(), ld, sa.data_ptr(), 1, qa.data_ptr(), ld, sa.data_ptr(), 1, d.data_ptr(), 0,
                                1 << 20, rows + 1, 40, k, None, 0, None)
    assert st == dg.DG_ERROR_NOT_SUPPORTED


# ---------------------------------------------------------------- NaN and infinities

def exactly(got, want):
    """NaN in the same places, everything else equal, infinities among it."""
    got = got.cpu()
    return torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~got.isnan()], want[~want.isnan()])


@pytest.mark.parametrize("dtype", OUT)
@pytest.mark.parametrize("m,n,k", [(3, 40, 256), (8, 520, 1040), (64, 129, 272), (130, 264, 512), (300, 2112, 1424)])
def test_infinite_and_nan_scales_exactly(m, n, k, dtype):
    qa, sa, qb, sb = operands(m, n, k, seed=m)
    sa[0], sa[1], sa[2] = np.inf, np.nan, 0.0
    sb[1], sb[2], sb[3], sb[4] = -np.inf, np.nan, 0.0, 3e38
    qa[:, 0], qb[:, 0] = 127, 127                        # fp16 leaves its range in places
    sb[5:9] = 1e3
    want = expected(dtype, qa, sa, qb, sb)
    assert bool(want.isnan().any() and want.isinf().any())
    assert exactly(run((qa, sa, qb, sb), dtype), want)
    ua, us, ub, ut = (upload(x) for x in (qa, sa, qb, sb))
    for expected_m in (1, m):
        d = torch.full((2, m, n), FILL, dtype=dtype, device=device())
        dg.m_grouped_int8_gemm_nt_masked((ua.expand(2, m, k).contiguous(), us.expand(2, m).contiguous()),
                                         (ub.expand(2, n, k).contiguous(), ut.expand(2, n).contiguous()), d,
                                         torch.tensor([m, m - 1], dtype=torch.int32, device=device()), expected_m)
        assert exactly(d[0], want) and exactly(d[1, :m - 1], want[:m - 1]) and bool((d[1, m - 1] == FILL).all())
    rows = (m + 127) // 128 * 128
    pa, ps = torch.zeros((rows, k), dtype=torch.int8, device=device()), torch.zeros(rows, device=device())
    pa[:m], ps[:m] = ua, us
    idx = torch.full((rows,), -1, dtype=torch.int32, device=device())
    idx[:m] = 0
    d = torch.full((rows, n), FILL, dtype=dtype, device=device())
    dg.m_grouped_int8_gemm_nt_contiguous((pa, ps), (ub[None], ut[None]), d, idx)
    assert exactly(d[:m], want) and bool((d[m:] == FILL).all())
