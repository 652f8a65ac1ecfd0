"""Routing and its gradient on the GPU against the 64-bit oracle.

Tolerances, from the arithmetic: a score is exp of a difference d of logits
(relative error |d| 2^-24 from the subtraction, two ulp from exp), over a sum with
at most 24 roundings on its longest path, with two divisions and a multiplication: under
(64 + 24 + 16) 2^-24 < 1e-5 for |d| up to 32 on either side; weights are held to 1e-5 relative.
A gradient's terms are products of such scores with g, none larger than scale * max |g|, of which
at most two cancel: 2e-5 * scale * max |g| on fp32 logits; on 16-bit logits the gradient equals, bit for bit,
the one on the same logits widened, rounded once.
Indices are equal, except (with a bias, or group sums) in rows whose choice hangs
on keys closer than 4e-6, which an fp32 key cannot tell apart; at most 1 row in 20.
"""
import numpy as np
import pytest
import torch

from oracle import moe
from gpu_util import device

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_fp8_gemm_amd as dg  # noqa: E402

W_TOL = 1e-5
G_TOL = 2e-5
CLOSE = 4e-6
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def check(x, topk, what, bias=None, grad=True, least_clear=0.95, **kw):
    """x: device logits.  Compares choice, weights and gradient with the oracle's."""
    host = x.float().cpu().numpy().astype(np.float64)
    gkw = {k: v for k, v in kw.items() if k in ("score", "renormalize", "scale")}
    okw = dict(kw)
    if "num_expert_groups" in okw:
        okw["groups"] = okw.pop("num_expert_groups")
    idx, w = dg.route_topk(x, topk, bias=bias, **kw)
    want_idx, want_w, margin = moe.route(host, topk, bias=None if bias is None else bias.cpu().numpy(), **okw)
    got_idx, got_w = idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    clear = margin > CLOSE
    assert clear.mean() >= least_clear or x.shape[0] < 20, f"{what}: {clear.mean()} of the rows are clear"
    assert np.array_equal(got_idx[clear], want_idx[clear]), f"{what}: indices differ"
    assert np.array_equal(np.isnan(got_w[clear]), np.isnan(want_w[clear])), what
    ok = np.isclose(got_w, want_w, rtol=W_TOL, atol=1e-37, equal_nan=True) | ~clear[:, None]
    assert ok.all(), f"{what}: weights differ at {np.argwhere(~ok)[:4].tolist()}"
    if not grad:
        return
    rng = np.random.default_rng(1)
    g = torch.from_numpy(rng.standard_normal(got_idx.shape).astype(np.float32)).to(device())
    dx32 = dg.route_topk_grad(x.float(), idx, g, **gkw)
    if x.dtype != torch.float32:
        got = dg.route_topk_grad(x, idx, g, **gkw)
        assert bool((got == dx32.to(x.dtype)).logical_or(torch.isnan(got) & torch.isnan(dx32)).all()), what
    dx = dx32.cpu().numpy().astype(np.float64)
    want = moe.route_grad(host, got_idx, g.cpu().numpy(), **gkw)
    bound = G_TOL * np.abs(g.cpu().numpy()).max(1, keepdims=True) * gkw.get("scale", 1.0)
    sane = np.isfinite(host).all(1) | (host == -np.inf).any(1) & ~np.isnan(host).any(1)
    bad = ~(np.abs(dx - want) <= bound) & sane[:, None]
    assert not bad.any(), f"{what}: gradient off at {np.argwhere(bad)[:4].tolist()}"


def draw(t, e, dtype, seed):
    g = torch.Generator(device=device()).manual_seed(seed)
    return (torch.randn((t, e), generator=g, device=device()) * 2).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (3, 2, 2), (16, 8, 2), (17, 60, 7), (33, 64, 64), (40, 72, 6),
                                   (50, 128, 17), (31, 160, 8), (64, 255, 1), (1, 256, 8), (65, 256, 33),
                                   (20, 257, 8), (9, 384, 64), (21, 1000, 5), (30, 1024, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sizes(t, e, k, dtype, score):
    for renormalize in (False, True):
        check(draw(t, e, dtype, 7 * e + k), k, f"{t}x{e} top {k}", score=score, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("e,groups,topk_groups,k", [(8, 8, 3, 2), (64, 4, 1, 6), (72, 6, 5, 8), (160, 8, 3, 6),
                                                    (256, 8, 4, 8), (256, 32, 7, 8), (256, 64, 64, 3),
                                                    (640, 20, 3, 8), (1024, 64, 33, 4)])
def test_groups_and_bias(score, group_score, e, groups, topk_groups, k):
    g = torch.Generator(device=device()).manual_seed(e + groups)
    bias = torch.randn(e, generator=g, device=device()) * 0.05
    for b in (None, bias):
        check(draw(100, e, torch.float32, e), k, f"{e} in {groups} bias {b is not None}", bias=b, score=score,
              num_expert_groups=groups, topk_groups=topk_groups, group_score=group_score, scale=1.5)


@pytest.mark.parametrize("e", [16, 256, 300])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_number(e, score):
    x = torch.randint(0, 3, (40, e), generator=torch.Generator().manual_seed(3)).float().to(device())
    x[0] = 0.0
    x[1] = torch.where(torch.arange(e, device=device()) % 2 == 0, -0.0, 0.0)   # equal keys
    check(x, min(e, 12), f"ties {e}", score=score)
    check(x.to(torch.bfloat16), min(e, 12), f"ties {e}, equal biases", bias=torch.full((e,), 0.25, device=device()),
          score=score)


@pytest.mark.parametrize("e,groups", [(24, 1), (24, 4), (256, 1), (256, 8), (512, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_and_extreme_logits(e, groups, score):
    inf, low = float("inf"), torch.finfo(torch.float32).min
    x = draw(24, e, torch.float32, 5)
    x[0] = -inf                                          # nothing left
    x[1, 1:] = -inf                                      # one expert left
    x[2, 3:] = -inf                                      # fewer than topk
    x[3, ::2] = -inf
    x[4] = low                                           # the type's lowest value everywhere: all equal, not masked
    x[5, 5:] = low
    x[6, 0], x[6, 1] = 3e38, -3e38
    x[7] = 200.0
    x[8] = torch.linspace(-100, 100, e)
    x[9, :e // 2] = -inf
    kw = dict(score=score, num_expert_groups=groups, topk_groups=max(1, groups // 2))
    for renormalize in (False, True):
        for group_score in ("max", "top2"):
            # (scores of the extreme rows underflow, so that fp32 group sums of theirs may come out equal)
            check(x, 8, "masks", least_clear=0.8, renormalize=renormalize, group_score=group_score, **kw)
    bias = torch.zeros(e, device=device())
    bias[::3] = -inf                                     # experts switched off
    bias[1] = 0.5
    check(x[:4], 8, "masks and a bias", bias=bias, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [30, 256, 700])
def test_nan_marks_the_token_and_no_other(score, e):
    x = draw(20, e, torch.float32, 6)
    x[3, 7] = float("nan")
    x[5, e - 1] = float("nan")
    x[8, 2] = float("inf")
    bias = torch.zeros(e, device=device())
    check(x, 6, "NaN", grad=False, score=score)
    check(x, 6, "NaN, bias", bias=bias, grad=False, score=score)
    bias[4] = float("nan")
    idx, w = dg.route_topk(x, 6, bias=bias, score=score)
    assert bool(torch.isnan(w).all()) and not bool((idx == 4).any())


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_outputs(dtype):
    wide = draw(50, 300, dtype, 8)
    for cols in (slice(0, 64), slice(3, 259), slice(1, 290)):
        x = wide[:, cols]                                # rows at element boundaries only
        check(x, 5, f"columns {cols}")
        idx = torch.full((50, 9), -7, dtype=torch.int32, device=device())
        w = torch.full((50, 9), -7.0, device=device())
        dg.route_topk(x, 5, indices=idx[:, 2:7], weights=w[:, 1:6])
        want = dg.route_topk(x.contiguous(), 5)
        assert torch.equal(idx[:, 2:7], want[0]) and torch.equal(w[:, 1:6], want[1])
        assert bool((idx[:, :2] == -7).all() and (idx[:, 7:] == -7).all() and (w[:, 6:] == -7).all())
        dx = torch.full((50, 301), -7.0, dtype=dtype, device=device())
        g = torch.ones((50, 5), device=device())
        dg.route_topk_grad(x, idx[:, 2:7], g, dlogits=dx[:, 1:1 + x.shape[1]], renormalize=False)
        assert torch.equal(dx[:, 1:1 + x.shape[1]], dg.route_topk_grad(x, want[0], g, renormalize=False))
        assert bool((dx[:, 0] == -7).all() and (dx[:, 1 + x.shape[1]:] == -7).all())


def test_no_tokens_and_repeatability():
    x = draw(0, 64, torch.float32, 1)
    idx, w = dg.route_topk(x, 4)
    assert idx.shape == w.shape == (0, 4) and dg.route_topk_grad(x, idx, w).shape == (0, 64)
    x = draw(5000, 256, torch.bfloat16, 2)
    first = dg.route_topk(x, 8, renormalize=False)
    for _ in range(3):
        again = dg.route_topk(x, 8, renormalize=False)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_gradient_of_unused_slots():
    x = draw(10, 40, torch.float32, 4)
    idx, _ = dg.route_topk(x, 4)
    idx[2] = -1
    idx[3, 1] = -1
    idx[4, 0] = 40                                       # outside: unused as well
    g = torch.randn((10, 4), device=device())
    g[idx < 0] = float("nan")                            # what belongs to no expert is not read into the sums
    g[4, 0] = float("nan")
    host_idx = idx.cpu().numpy().copy()
    host_idx[host_idx >= 40] = -1
    for score in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            dx = dg.route_topk_grad(x, idx, g, score=score, renormalize=renormalize).cpu().numpy()
            want = moe.route_grad(x.cpu().numpy(), host_idx, np.nan_to_num(g.cpu().numpy()), score, renormalize)
            assert np.abs(dx - want).max() <= G_TOL * 4 and np.all(dx[2] == 0)


# ---------------------------------------------------------------- many tokens
# Over 64 experts few tokens take a wave each; these run the same rows among many, four to a wave,
# where neighbours differ in what they need, against the same oracle and bounds.

MANY = 8200


def check_among_many(x, topk, what, bias=None, grad=True, least_clear=0.95, **kw):
    """check() of x's rows repeated to more tokens than a wave each is used for."""
    n, reps = x.shape[0], -(-MANY // x.shape[0])
    host = x.float().cpu().numpy().astype(np.float64)
    gkw = {k: v for k, v in kw.items() if k in ("score", "renormalize", "scale")}
    okw = dict(kw)
    if "num_expert_groups" in okw:
        okw["groups"] = okw.pop("num_expert_groups")
    many = x.repeat(reps, 1)
    idx, w = dg.route_topk(many, topk, bias=bias, **kw)
    want_idx, want_w, margin = moe.route(host, topk, bias=None if bias is None else bias.cpu().numpy(), **okw)
    clear = margin > CLOSE
    assert clear.mean() >= least_clear or n < 20, f"{what}: {clear.mean()} of the rows are clear"
    got_idx = idx.cpu().numpy().reshape(reps, n, topk)[:, clear]
    got_w = w.cpu().numpy().astype(np.float64).reshape(reps, n, topk)[:, clear]
    assert (got_idx == want_idx[clear]).all(), f"{what}: indices differ"
    ok = np.isclose(got_w, np.broadcast_to(want_w[clear], got_w.shape), rtol=W_TOL, atol=1e-37, equal_nan=True)
    assert ok.all(), f"{what}: weights differ at {np.argwhere(~ok)[:4].tolist()}"
    if not grad:
        return
    g = torch.from_numpy(np.random.default_rng(1).standard_normal((n, topk)).astype(np.float32)).to(device())
    dx = dg.route_topk_grad(many, idx, g.repeat(reps, 1), **gkw).float().cpu().numpy().astype(np.float64)
    want = moe.route_grad(host, want_idx, g.cpu().numpy(), **gkw)
    bound = G_TOL * np.abs(g.cpu().numpy()).max(1, keepdims=True) * gkw.get("scale", 1.0)
    if x.dtype != torch.float32:    # and one rounding to the type: half its spacing, or of its smallest numbers
        info = torch.finfo(x.dtype)
        bound = bound + np.abs(want) * info.eps / 2 + info.smallest_normal * info.eps
    sane = np.isfinite(host).all(1) | (host == -np.inf).any(1) & ~np.isnan(host).any(1)
    rows = sane & clear
    bad = ~(np.abs(dx.reshape(reps, n, -1)[:, rows] - want[rows]) <= bound[rows])
    assert not bad.any(), f"{what}: gradient off at {np.argwhere(bad)[:4].tolist()}"


@pytest.fixture
def among_many(monkeypatch):
    monkeypatch.setitem(globals(), "check", check_among_many)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,e,k", [(37, 65, 7), (40, 72, 6), (51, 128, 16), (31, 160, 8), (64, 255, 1), (65, 256, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sizes_among_many(among_many, t, e, k, dtype, score):
    test_sizes(t, e, k, dtype, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("e,groups,topk_groups,k", [(72, 6, 5, 8), (128, 8, 1, 4), (160, 8, 3, 6), (256, 8, 4, 8),
                                                    (256, 32, 7, 8), (256, 64, 64, 3)])
def test_groups_and_bias_among_many(among_many, score, group_score, e, groups, topk_groups, k):
    test_groups_and_bias(score, group_score, e, groups, topk_groups, k)


@pytest.mark.parametrize("e", [100, 256])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_among_many(among_many, e, score):
    test_ties_go_to_the_lowest_number(e, score)


@pytest.mark.parametrize("e,groups", [(120, 4), (256, 1), (256, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masks_among_many(among_many, e, groups, score):
    test_masked_and_extreme_logits(e, groups, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [90, 256])
def test_nan_among_many(among_many, score, e):
    test_nan_marks_the_token_and_no_other(score, e)


# ---------------------------------------------------------------- gradients at the ends of fp32

@pytest.mark.parametrize("t", [6, 3000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_of_renormalised_scores_near_underflow(score, t):
    """Sigmoids of logits below -87.4 are subnormal: they are no divisors for a gradient, their shares are.  A
    subnormal score of 3e-39 or more is right to 2.4e-7 of itself, within what G_TOL allows for a score."""
    x = draw(t, 128, torch.float32, 9) / 100
    x[0::6] -= 88.4
    x[1::6] -= 87.5
    x[2::6] -= 80.0
    x[3::6, ::2] -= 88.4                                 # ordinary logits beside them
    x[4::6, 1:] -= 88.4
    check(x, 6, "scores near underflow", score=score, renormalize=True, scale=16.0)


@pytest.mark.parametrize("t", [6, 5000])
@pytest.mark.parametrize("score,renormalize", [("softmax", False), ("softmax", True), ("sigmoid", False),
                                               ("sigmoid", True)])
def test_gradient_of_a_logit_without_a_score(score, renormalize, t):
    """Plain softmax: every score of the token depends on the logit, so its whole row is NaN.  The other forms depend
    on the chosen logits alone, and a logit without a score is never chosen."""
    x = draw(t, 160, torch.float32, 10)
    x[0, 7] = float("nan")
    x[1, 159] = -float("nan")
    if score == "softmax":
        x[3, 2] = float("inf")
    idx, w = dg.route_topk(x, 6, score=score, renormalize=renormalize)
    lost = torch.isnan(w).all(1).cpu().numpy()
    assert lost.tolist() == [True, True, False, score == "softmax"] + [False] * (t - 4)
    g = torch.randn((t, 6), generator=torch.Generator().manual_seed(1)).to(device())
    dx = dg.route_topk_grad(x, idx, g, score=score, renormalize=renormalize, scale=2.5).cpu().numpy()
    want = moe.route_grad(x.cpu().numpy(), idx.cpu().numpy(), g.cpu().numpy(), score, renormalize, 2.5)
    if score == "softmax" and not renormalize:
        want[lost] = np.nan
    assert np.array_equal(np.isnan(dx), np.isnan(want))
    ok = np.isnan(want).any(1)
    bound = G_TOL * 2.5 * np.abs(g.cpu().numpy()).max(1, keepdims=True)
    assert np.all(np.abs(dx - want)[~ok] <= np.broadcast_to(bound, dx.shape)[~ok])


# ---------------------------------------------------------------- biases at the ends of fp32

@pytest.mark.parametrize("t", [3, 9000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups", [(24, 4), (160, 8), (256, 8), (640, 20)])
def test_group_sums_of_the_largest_biases(e, groups, score, t):
    """The sum of two scores plus biases leaves fp32's range where both biases are the type's lowest or largest
    number; the groups are still there, in the order of their sums.  (A score beside such a bias rounds away.)"""
    size, low, high = e // groups, torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    x = draw(t, e, torch.float32, 12)
    first = torch.arange(size + 2, device=device(), dtype=torch.int32)
    kw = dict(score=score, num_expert_groups=groups, group_score="top2")

    bias = torch.full((e,), low, device=device())        # every expert at the lowest value: all keys equal
    idx, w = dg.route_topk(x, size + 2, bias=bias, topk_groups=2, **kw)
    assert bool((idx == first).all()) and bool((w > 0).all())
    assert np.allclose(w.sum(1).cpu().numpy(), 1.0, atol=1e-5)

    bias[2 * size:3 * size] = 0.0                        # one group free: its experts, then the lowest of group 0
    idx, _ = dg.route_topk(x, size + 2, bias=bias, topk_groups=2, **kw)
    assert bool((idx[:, size:] == first[:2]).all())
    assert bool((idx[:, :size].sort(1).values == first[:size] + 2 * size).all())

    bias = torch.full((e,), 0.9 * high, device=device())
    bias[size:2 * size] = high
    idx, _ = dg.route_topk(x, size, bias=bias, topk_groups=1, **kw)
    assert bool((idx == first[:size] + size).all())
