"""Refusals of the mixture-of-experts and int8 entry points: every bad argument comes back
as a status before anything is launched, and the binding rejects wrong tensors.
Addresses are fake and never dereferenced."""
import ctypes

import pytest
import torch

import moe_fp8_gemm_amd as dg

lib = dg.lib
P = 0x10000
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3


def call(fn, defaults, **kw):
    assert not set(kw) - set(defaults), kw
    return fn(*{**defaults, **kw}.values())


ROUTE = dict(logits=P, dtype=0, ld=64, bias=None, indices=P, ldi=8, weights=P, ldw=8, tokens=5, experts=64, topk=8,
             groups=1, topk_groups=1, top2=0, score=0, renorm=1, scale=1.0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0), OK), (dict(tokens=0, logits=None, indices=None, weights=None), OK),
    (dict(logits=None), INVALID), (dict(indices=None), INVALID), (dict(weights=None), INVALID),
    (dict(dtype=3), INVALID), (dict(score=2), INVALID), (dict(tokens=-1), INVALID), (dict(experts=0), INVALID),
    (dict(topk=0), INVALID), (dict(topk=65, ldi=65, ldw=65), INVALID), (dict(ld=63), INVALID), (dict(ldi=7), INVALID),
    (dict(ldw=7), INVALID), (dict(groups=0), INVALID), (dict(groups=3), INVALID), (dict(groups=4, topk_groups=5), INVALID),
    (dict(groups=4, topk_groups=0), INVALID), (dict(experts=1025, ld=1025), UNSUPPORTED),
    (dict(experts=128, ld=128, topk=65, ldi=65, ldw=65), UNSUPPORTED),
    (dict(experts=130, ld=130, groups=65), UNSUPPORTED), (dict(tokens=(1 << 23) + 1), UNSUPPORTED),
    (dict(ld=(1 << 40) + 1), UNSUPPORTED), (dict(logits=P + 2), UNSUPPORTED), (dict(dtype=1, logits=P + 1), UNSUPPORTED),
    (dict(bias=P + 1), UNSUPPORTED), (dict(indices=P + 2), UNSUPPORTED), (dict(weights=P + 2), UNSUPPORTED)])
def test_route(kw, status):
    assert call(lib.dg_route_topk, ROUTE, **kw) == status


ROUTE_GRAD = dict(logits=P, dtype=1, ld=64, indices=P, ldi=8, dweights=P, ldw=8, dlogits=P, ldd=64, tokens=5,
                  experts=64, topk=8, score=1, renorm=0, scale=1.0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0), OK), (dict(logits=None), INVALID), (dict(indices=None), INVALID), (dict(dweights=None), INVALID),
    (dict(dlogits=None), INVALID), (dict(ldd=63), INVALID), (dict(topk=65, ldi=65, ldw=65), INVALID),
    (dict(dlogits=P + 1), UNSUPPORTED), (dict(ldd=1 << 41), UNSUPPORTED), (dict(experts=2000, ld=2000, ldd=2000),
                                                                           UNSUPPORTED)])
def test_route_grad(kw, status):
    assert call(lib.dg_route_topk_grad, ROUTE_GRAD, **kw) == status


CONTIGUOUS = dict(indices=P, ldi=8, tokens=100, topk=8, experts=64, rows=1024, m_indices=P, row_slot=P, slot_row=P,
                  counts=P, ws=None, ws_bytes=0, stream=None)
BIG = dict(tokens=1000)   # 8000 slots: needs a workspace


@pytest.mark.parametrize("kw,status", [
    (dict(indices=None), INVALID), (dict(slot_row=None), INVALID), (dict(m_indices=None), INVALID),
    (dict(row_slot=None), INVALID), (dict(counts=None), INVALID), (dict(ldi=7), INVALID), (dict(tokens=-1), INVALID),
    (dict(topk=0), INVALID), (dict(experts=0), INVALID), (dict(rows=-128), INVALID), (dict(rows=1000), MISALIGNED),
    (dict(experts=1025), UNSUPPORTED), (dict(topk=65, ldi=65), UNSUPPORTED), (dict(tokens=1 << 28), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(indices=P + 1), UNSUPPORTED), (dict(counts=P + 2), UNSUPPORTED),
    (BIG, INVALID), (dict(BIG, ws=P, ws_bytes=8 * 64 * 4 - 1), INVALID), (dict(BIG, ws=P + 4, ws_bytes=4096), UNSUPPORTED)])
def test_layout_contiguous(kw, status):
    assert call(lib.dg_expert_layout_contiguous, CONTIGUOUS, **kw) == status


MASKED = dict(indices=P, ldi=8, tokens=100, topk=8, experts=64, max_m=32, masked_m=P, row_slot=P, slot_row=P, ws=None,
              ws_bytes=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(max_m=0), INVALID), (dict(masked_m=None), INVALID), (dict(row_slot=None), INVALID), (BIG, INVALID),
    (dict(max_m=1 << 25), UNSUPPORTED), (dict(max_m=1 << 60), UNSUPPORTED)])
def test_layout_masked(kw, status):
    assert call(lib.dg_expert_layout_masked, MASKED, **kw) == status


def test_layout_sizes():
    assert dg.expert_layout_rows(1, 8, 256) == 8 * 128 and dg.expert_layout_rows(0, 8, 256) == 0
    assert dg.expert_layout_rows(4096, 8, 1) == 32768 // 128 * 128
    assert dg.expert_layout_rows(-1, 8, 256) == 0 and dg.expert_layout_rows(1, 65, 256) == 0
    assert lib.dg_expert_layout_workspace_size(128, 8, 256) == 0
    assert lib.dg_expert_layout_workspace_size(129, 8, 256) == 2 * 256 * 4
    assert lib.dg_expert_layout_workspace_size(513, 8, 256) == 5 * 256 * 4
    assert lib.dg_expert_layout_workspace_size(8193, 8, 256) == 17 * 256 * 4


DISPATCH = dict(x=P, dtype=1, ldx=256, slot_row=P, lds=2, q=P, ldq=256, sf=P, sf_sm=2, sf_sk=1, tokens=4, topk=2, rows=8,
                k=256, ue8m0=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0), OK), (dict(rows=0), OK), (dict(k=0), OK), (dict(dtype=2), INVALID), (dict(x=None), INVALID),
    (dict(slot_row=None), INVALID), (dict(q=None), INVALID), (dict(sf=None), INVALID), (dict(lds=1), INVALID),
    (dict(ldx=255), INVALID), (dict(ldq=255), INVALID), (dict(sf_sk=-1), INVALID), (dict(topk=0), INVALID),
    (dict(k=192), UNSUPPORTED), (dict(ldx=260), UNSUPPORTED), (dict(x=P + 8), UNSUPPORTED), (dict(q=P + 8), UNSUPPORTED),
    (dict(ldq=264), UNSUPPORTED), (dict(slot_row=P + 2), UNSUPPORTED), (dict(tokens=1 << 24), UNSUPPORTED),
    (dict(topk=65, lds=65), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED)])
def test_dispatch_fp8(kw, status):
    assert call(lib.dg_dispatch_cast_fp8, DISPATCH, **kw) == status


DISPATCH8 = dict(x=P, dtype=1, ldx=256, slot_row=P, lds=2, q=P, ldq=256, sf=P, sf_s=1, tokens=4, topk=2, rows=8, k=256,
                 stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0), OK), (dict(dtype=2), INVALID), (dict(sf=None), INVALID), (dict(sf_s=-1), INVALID),
    (dict(k=200), UNSUPPORTED), (dict(ldq=264), UNSUPPORTED)])
def test_dispatch_int8(kw, status):
    assert call(lib.dg_dispatch_cast_int8, DISPATCH8, **kw) == status


COMBINE = dict(y=P, ldy=256, slot_row=P, lds=2, weights=P, ldw=2, out=P, out_dtype=1, ldo=256, tokens=4, topk=2, rows=8,
               h=256, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0), OK), (dict(h=0), OK), (dict(out_dtype=2), INVALID), (dict(y=None), INVALID), (dict(out=None), INVALID),
    (dict(slot_row=None), INVALID), (dict(ldw=1), INVALID), (dict(ldy=255), INVALID), (dict(ldo=255), INVALID),
    (dict(h=252), UNSUPPORTED), (dict(ldy=260), UNSUPPORTED), (dict(ldo=260), UNSUPPORTED), (dict(out=P + 8), UNSUPPORTED),
    (dict(weights=P + 1), UNSUPPORTED)])
def test_combine(kw, status):
    assert call(lib.dg_combine, COMBINE, **kw) == status


COMBINE_GRAD = dict(dout=P, ldo=256, y=P, ldy=256, slot_row=P, lds=2, row_slot=P, weights=P, ldw=2, dy=P, lddy=256,
                    dweights=P, lddw=2, tokens=4, topk=2, rows=8, h=256, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0, rows=0), OK), (dict(dout=None), INVALID), (dict(y=None), INVALID), (dict(dy=None), INVALID),
    (dict(row_slot=None), INVALID), (dict(weights=None), INVALID), (dict(dweights=None), INVALID),
    (dict(lddw=1), INVALID), (dict(lddy=255), INVALID), (dict(h=252), UNSUPPORTED), (dict(lddy=260), UNSUPPORTED),
    (dict(tokens=1 << 23, rows=(1 << 31) - 1), UNSUPPORTED)])
def test_combine_grad(kw, status):
    assert call(lib.dg_combine_grad, COMBINE_GRAD, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(row_slot=None), INVALID), (dict(row_slot=P + 2), UNSUPPORTED), (dict(row_slot=None, tokens=0), OK)])
def test_combine_grad_without_columns(kw, status):
    """h == 0: the weights' gradients are still written, so the map is checked with the rest."""
    assert call(lib.dg_combine_grad, dict(COMBINE_GRAD, h=0), **kw) == status


CAST8 = dict(x=P, dtype=1, ldx=256, q=P, ldq=256, sf=P, sf_s=1, m=4, k=256, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=0), OK), (dict(k=0), OK), (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(sf=None), INVALID),
    (dict(m=-1), INVALID), (dict(dtype=2), INVALID), (dict(ldx=255), INVALID), (dict(k=8, ldx=8), UNSUPPORTED),
    (dict(q=P + 8), UNSUPPORTED), (dict(m=(1 << 23) + 1), UNSUPPORTED)])
def test_cast_int8(kw, status):
    assert call(lib.dg_per_token_cast_int8, CAST8, **kw) == status


GEMM8 = dict(a=P, lda=256, sfa=P, sfa_s=1, b=P, ldb=256, sfb=P, sfb_s=1, d=P, out=1, ldd=64, m=32, n=64, k=256, ws=None,
             ws_bytes=0, stream=None)
GEMM8_CASES = [
    (dict(n=0), OK), (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(d=None), INVALID), (dict(sfa=None), INVALID),
    (dict(sfb=None), INVALID), (dict(out=3), INVALID), (dict(lda=255), INVALID), (dict(ldb=128), INVALID),
    (dict(ldd=63), INVALID), (dict(sfa_s=-1), INVALID), (dict(k=-1), INVALID), (dict(k=0), UNSUPPORTED),
    (dict(k=200), UNSUPPORTED), (dict(k=131072, lda=131072, ldb=131072), UNSUPPORTED), (dict(lda=264), UNSUPPORTED),
    (dict(a=P + 8), UNSUPPORTED), (dict(b=P + 4), UNSUPPORTED), (dict(d=P + 1), UNSUPPORTED), (dict(sfa=P + 2), UNSUPPORTED),
    (dict(lda=1 << 41), UNSUPPORTED), (dict(lda=1 << 28), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", GEMM8_CASES + [(dict(m=0), OK), (dict(m=-1), INVALID),
                                                     (dict(ws=P + 8, ws_bytes=1 << 20), UNSUPPORTED)])
def test_int8_dense(kw, status):
    assert call(lib.dg_int8_gemm_nt, GEMM8, **kw) == status


GEMM8_CONTIGUOUS = dict(a=P, lda=256, sfa=P, sfa_s=1, b=P, ldb=256, b_gs=256 * 64, sfb=P, sfb_s=1, sfb_gs=64, d=P, out=1,
                        ldd=64, m_indices=P, m=256, n=64, k=256, groups=2, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("kw,status", GEMM8_CASES + [
    (dict(m=0), OK), (dict(m=200), MISALIGNED), (dict(groups=0), INVALID), (dict(m_indices=None), INVALID),
    (dict(b_gs=-16), INVALID), (dict(b_gs=8), UNSUPPORTED), (dict(m_indices=P + 2), UNSUPPORTED)])
def test_int8_contiguous(kw, status):
    assert call(lib.dg_m_grouped_int8_gemm_nt_contiguous, GEMM8_CONTIGUOUS, **kw) == status


GEMM8_MASKED = dict(a=P, lda=256, a_gs=256 * 32, sfa=P, sfa_s=1, sfa_gs=32, b=P, ldb=256, b_gs=256 * 64, sfb=P, sfb_s=1,
                    sfb_gs=64, d=P, out=1, ldd=64, d_gs=64 * 32, masked_m=P, groups=2, m=32, n=64, k=256, hint=16,
                    stream=None)


@pytest.mark.parametrize("kw,status", GEMM8_CASES + [
    (dict(m=0), OK), (dict(groups=0), INVALID), (dict(masked_m=None), INVALID), (dict(d_gs=-1), INVALID),
    (dict(groups=1025), UNSUPPORTED), (dict(a_gs=8), UNSUPPORTED), (dict(d_gs=1 << 41), UNSUPPORTED)])
def test_int8_masked(kw, status):
    assert call(lib.dg_m_grouped_int8_gemm_nt_masked, GEMM8_MASKED, **kw) == status


def test_binding_rejects_wrong_tensors():
    """Host tensors, and types, before any library call."""
    x, i = torch.zeros((4, 256)), torch.zeros((4, 2), dtype=torch.int32)
    for f in (lambda: dg.route_topk(x, 2), lambda: dg.route_topk_grad(x, i, x), lambda: dg.combine(x, i),
              lambda: dg.expert_layout_contiguous(i, 8), lambda: dg.expert_layout_masked(i, 8, 4),
              lambda: dg.dispatch_cast_fp8(x, i, rows=8), lambda: dg.dispatch_cast_int8(x, i, rows=8),
              lambda: dg.combine_grad(x, x, i, i, x), lambda: dg.per_token_cast_int8(x),
              lambda: dg.int8_gemm_nt((i, x), (i, x), x)):
        with pytest.raises(TypeError):
            f()


def test_status_is_raised():
    assert ctypes.c_int(lib.dg_route_topk(*{**ROUTE, "topk": 0}.values())).value == INVALID
    with pytest.raises(dg.DgError):
        dg._check(INVALID, "dg_route_topk")
