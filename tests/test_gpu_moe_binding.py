"""The compiled marshalling on device tensors: every refusal leaves the process as it was, outputs passed in
are the ones returned, and calls follow torch's current stream."""
import pytest
import torch

from gpu_util import device

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_fp8_gemm_amd as dg  # noqa: E402


def f32(*shape):
    return torch.rand(shape, device=device())


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device=device())


def i8(*shape):
    return torch.ones(shape, dtype=torch.int8, device=device())


def bf16(*shape):
    return torch.ones(shape, dtype=torch.bfloat16, device=device())


REFUSED = [
    (TypeError, lambda: dg.route_topk(3, 2)),
    (TypeError, lambda: dg.route_topk(f32(4, 8).double(), 2)),
    (TypeError, lambda: dg.route_topk(f32(4, 8), "2")),
    (TypeError, lambda: dg.route_topk(f32(4, 8), 2, scale="x")),
    (TypeError, lambda: dg.route_topk(f32(4, 8), 2, score=1)),
    (ValueError, lambda: dg.route_topk(f32(4, 8), 2, score="relu")),
    (ValueError, lambda: dg.route_topk(f32(4, 8), 2, group_score="mean")),
    (ValueError, lambda: dg.route_topk(f32(8), 2)),
    (ValueError, lambda: dg.route_topk(f32(8, 4).t(), 2)),
    (ValueError, lambda: dg.route_topk(f32(4, 8), 2, bias=f32(7))),
    (ValueError, lambda: dg.route_topk(f32(4, 8), 2, indices=i32(4, 3))),
    (ValueError, lambda: dg.route_topk(f32(4, 8), -1)),
    (ValueError, lambda: dg.route_topk(f32(4, 8), 1 << 40)),
    (dg.DgError, lambda: dg.route_topk(f32(4, 8), 9)),
    (dg.DgError, lambda: dg.route_topk(f32(4, 8), 2, num_expert_groups=3)),
    (dg.DgError, lambda: dg.route_topk(f32(4, 1025), 2)),
    (ValueError, lambda: dg.route_topk_grad(f32(4, 8), i32(4, 2), f32(4, 3))),
    (ValueError, lambda: dg.route_topk_grad(f32(4, 8), i32(3, 2), f32(3, 2))),
    (TypeError, lambda: dg.expert_layout_contiguous(f32(4, 2), 8)),
    (dg.DgError, lambda: dg.expert_layout_contiguous(i32(4, 2), 8, rows=100)),
    (dg.DgError, lambda: dg.expert_layout_contiguous(i32(4, 2), -1)),
    (dg.DgError, lambda: dg.expert_layout_masked(i32(4, 2), 8, 0)),
    (dg.DgError, lambda: dg.expert_layout_masked(i32(4, 2), 8, 1 << 40)),
    (ValueError, lambda: dg.dispatch_cast_fp8(f32(4, 128), i32(4, 2))),
    (ValueError, lambda: dg.dispatch_cast_fp8(f32(4, 128), i32(3, 2), rows=8)),
    (ValueError, lambda: dg.dispatch_cast_fp8(f32(4, 128), i32(4, 2), rows=8, sf=f32(8, 2))),
    (ValueError, lambda: dg.dispatch_cast_int8(f32(4, 128), i32(4, 2), rows=7, q=i8(8, 128))),
    (dg.DgError, lambda: dg.dispatch_cast_fp8(f32(4, 192), i32(4, 2), rows=8)),
    (TypeError, lambda: dg.combine(f32(8, 64), i32(4, 2))),
    (ValueError, lambda: dg.combine(bf16(8, 64), i32(4, 2), f32(4, 3))),
    (ValueError, lambda: dg.combine(bf16(8, 64), i32(4, 2), out=bf16(4, 65))),
    (dg.DgError, lambda: dg.combine(bf16(8, 60), i32(4, 2))),
    (ValueError, lambda: dg.combine_grad(bf16(4, 64), bf16(8, 64), i32(4, 2), i32(7), f32(4, 2))),
    (ValueError, lambda: dg.combine_grad(bf16(3, 64), bf16(8, 64), i32(4, 2), i32(8), f32(4, 2))),
    (TypeError, lambda: dg.per_token_cast_int8(i8(4, 64))),
    (dg.DgError, lambda: dg.per_token_cast_int8(f32(4, 72))),
    (ValueError, lambda: dg.int8_gemm_nt((i8(4, 64), f32(4)), (i8(8, 32), f32(8)), bf16(4, 8))),
    (ValueError, lambda: dg.int8_gemm_nt((i8(4, 64), f32(5)), (i8(8, 64), f32(8)), bf16(4, 8))),
    (ValueError, lambda: dg.int8_gemm_nt((i8(4, 64), f32(4)), (i8(8, 64), f32(8)), bf16(4, 9))),
    (TypeError, lambda: dg.int8_gemm_nt((i8(4, 64), f32(4)), (i8(8, 64), bf16(8)), bf16(4, 8))),
    (ValueError, lambda: dg.int8_gemm_nt((i8(4, 64), f32(4)), (i8(8, 64), f32(8)), bf16(4, 8), workspace="big")),
    (TypeError, lambda: dg.int8_gemm_nt((i8(4, 64), f32(4)), (i8(8, 64), f32(8)), bf16(4, 8), workspace=7)),
    (dg.DgError, lambda: dg.int8_gemm_nt((i8(4, 40), f32(4)), (i8(8, 40), f32(8)), bf16(4, 8))),
    (dg.DgError, lambda: dg.m_grouped_int8_gemm_nt_contiguous((i8(4, 64), f32(4)), (i8(2, 8, 64), f32(2, 8)),
                                                              bf16(4, 8), i32(4))),
    (ValueError, lambda: dg.m_grouped_int8_gemm_nt_masked((i8(2, 4, 64), f32(2, 4)), (i8(2, 8, 64), f32(2, 8)),
                                                          bf16(2, 4, 8), i32(3), 4)),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_refusals(i):
    error, call = REFUSED[i]
    with pytest.raises(error):
        call()


def test_status_of_an_error():
    with pytest.raises(dg.DgError) as e:
        dg.expert_layout_contiguous(i32(4, 2), 8, rows=100)
    assert e.value.status == dg.DG_ERROR_MISALIGNED_LAYOUT and "dg_expert_layout_contiguous" in str(e.value)


def test_outputs_are_the_ones_passed_in():
    x, idx, w, d, g = f32(4, 8), i32(4, 2), f32(4, 2), bf16(4, 8), f32(4, 8)
    got = dg.route_topk(x, 2, indices=idx, weights=w)
    assert got[0] is idx and got[1] is w
    assert dg.int8_gemm_nt((i8(4, 64), f32(4)), (i8(8, 64), f32(8)), d) is d
    assert dg.route_topk_grad(x, idx, w, dlogits=g) is g


def test_current_stream_is_followed():
    """Work queued on a side stream stays in its order there: the call reads what the stream writes before it."""
    side = torch.cuda.Stream()
    x = torch.zeros((4096, 64), device=device())
    big = torch.rand((2048, 2048), device=device())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            big = big @ big * 1e-3
        x[:, 5] = 1.0
        idx, _ = dg.route_topk(x, 1)
    side.synchronize()
    assert bool((idx == 5).all())


def test_new_outputs_are_ordinary_tensors():
    """Outputs that the binding allocates belong to torch's allocator: device, autograd, views, streams, reuse."""
    before = torch.cuda.memory_allocated()
    idx, w = dg.route_topk(f32(64, 32), 4)
    q, sf = dg.per_token_cast_int8(f32(5, 80))
    assert idx.device == w.device == q.device == device() and not idx.requires_grad
    assert q.shape == (5, 80) and q.stride() == (128, 1) and sf.shape == (5,)
    assert torch.cuda.memory_allocated() > before
    w2 = w.clone().requires_grad_()
    (w2 * 2).sum().backward()
    assert torch.equal(w2.grad, torch.full_like(w, 2))
    w.requires_grad_()
    assert (w * 3).sum().requires_grad
    side = torch.cuda.Stream()
    idx.record_stream(side)
    assert idx.view(-1).sort().values.numel() == 256 and idx.t().contiguous().shape == (4, 64)
    del idx, w, w2, q, sf
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() <= before
