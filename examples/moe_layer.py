"""A mixture-of-experts layer on the library's operators, against the same layer in plain torch.

    python examples/moe_layer.py [--int8] [--decode] [--train] [--tokens T] [--experts E] [--hidden H] [--inner I]

Router logits -> route_topk -> expert layout -> dispatch with the cast -> grouped product (gate and up) -> SiLU ->
cast -> grouped product (down) -> combine.  Nothing in the layer reads the routing on the host.

* prefill (default): contiguous layout, experts' rows padded to 128;
* --decode: masked layout, a fixed number of rows for each expert, for few tokens;
* --int8: experts in 8-bit integers with scales per token and channel, instead of FP8 with block scales;
* --train: also the gradient that reaches the router's logits, through combine_grad and route_topk_grad.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_fp8_gemm_amd as dg  # noqa: E402

ROUTE = dict(score="sigmoid", num_expert_groups=4, topk_groups=2, group_score="top2", scale=2.5)


class Experts:
    """Weights of all experts, laid out once: [E, 2 * inner, hidden] and [E, hidden, inner] in 8 bits."""

    def __init__(self, up: torch.Tensor, down: torch.Tensor, int8: bool):
        self.int8 = int8
        self.up, self.down = self._cast(up), self._cast(down)

    def _cast(self, w: torch.Tensor):
        pairs = [dg.per_token_cast_int8(x) if self.int8 else dg.per_block_cast_fp8(x) for x in w]
        return torch.stack([q for q, _ in pairs]), torch.stack([s for _, s in pairs])

    def cast(self, x: torch.Tensor):
        return dg.per_token_cast_int8(x) if self.int8 else dg.per_token_cast_fp8(x)

    def dispatch(self, x: torch.Tensor, layout: dg.ExpertLayout):
        f = dg.dispatch_cast_int8 if self.int8 else dg.dispatch_cast_fp8
        return f(x, layout.slot_row, rows=layout.rows)

    def product(self, a, w, layout: dg.ExpertLayout, max_m: int) -> torch.Tensor:
        """[rows, n]; rows that hold no token are unspecified."""
        g, n, _ = w[0].shape
        d = torch.empty((layout.rows, n), dtype=torch.bfloat16, device=a[0].device)
        if max_m:
            f = dg.m_grouped_int8_gemm_nt_masked if self.int8 else dg.m_grouped_fp8_gemm_nt_masked
            f(tuple(t.unflatten(0, (g, max_m)) for t in a), w, d.view(g, max_m, n), layout.counts, max_m // 2)
        else:
            f = dg.m_grouped_int8_gemm_nt_contiguous if self.int8 else dg.m_grouped_fp8_gemm_nt_contiguous
            f(a, w, d, layout.m_indices)
        return d


def moe_layer(x, logits, bias, experts: Experts, topk: int, max_m: int = 0):
    """out [tokens, hidden], and what the backward pass needs.  max_m > 0: masked layout of that many rows per expert."""
    indices, weights = dg.route_topk(logits, topk, bias=bias, **ROUTE)
    num_experts = logits.shape[1]
    layout = (dg.expert_layout_masked(indices, num_experts, max_m) if max_m
              else dg.expert_layout_contiguous(indices, num_experts))
    h = experts.product(experts.dispatch(x, layout), experts.up, layout, max_m)
    gate, up = h.chunk(2, dim=1)
    y = experts.product(experts.cast(torch.nn.functional.silu(gate) * up), experts.down, layout, max_m)
    return dg.combine(y, layout.slot_row, weights), (indices, weights, layout, y)


def router_grad(dout, logits, saved):
    """Gradient of the loss with respect to the router's logits, the experts' outputs held fixed."""
    indices, weights, layout, y = saved
    _, dweights = dg.combine_grad(dout, y, layout.slot_row, layout.row_slot, weights)
    return dg.route_topk_grad(logits, indices, dweights, score=ROUTE["score"], scale=ROUTE["scale"])


def plain_layer(x, logits, indices, up, down):
    """The layer in fp32 for a given choice of experts, differentiable in the logits: (out, experts' rows per slot)."""
    s = torch.sigmoid(logits).gather(1, indices.long())
    w = ROUTE["scale"] * s / s.sum(1, keepdim=True)
    rows = torch.zeros(indices.shape + (x.shape[1],), device=x.device)
    for e in range(up.shape[0]):
        t, j = (indices == e).nonzero(as_tuple=True)
        if len(t):
            gate, u = (x[t].float() @ up[e].t()).chunk(2, dim=1)
            rows[t, j] = (torch.nn.functional.silu(gate) * u) @ down[e].t()
    return (w[..., None] * rows).sum(1), rows


def main(argv=None) -> dict:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--int8", action="store_true")
    p.add_argument("--decode", action="store_true")
    p.add_argument("--train", action="store_true")
    p.add_argument("--tokens", type=int, default=None)
    p.add_argument("--experts", type=int, default=16)
    p.add_argument("--topk", type=int, default=4)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--inner", type=int, default=1024)
    a = p.parse_args(argv)
    tokens = a.tokens or (32 if a.decode else 4096)
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((tokens, a.hidden), generator=g, device="cuda").to(torch.bfloat16)
    router = torch.randn((a.experts, a.hidden), generator=g, device="cuda") * a.hidden ** -0.5
    bias = torch.randn(a.experts, generator=g, device="cuda") * 0.05
    up = torch.randn((a.experts, 2 * a.inner, a.hidden), generator=g, device="cuda") * a.hidden ** -0.5
    down = torch.randn((a.experts, a.hidden, a.inner), generator=g, device="cuda") * a.inner ** -0.5
    experts = Experts(up, down, a.int8)
    max_m = min(256, -(-tokens // 8) * 8) if a.decode else 0
    logits = x.float() @ router.t()

    out, saved = moe_layer(x, logits, bias, experts, a.topk, max_m)
    want, rows = plain_layer(x, logits, saved[0], up, down)
    found = {"out": float((out.float() - want).norm() / want.norm())}
    if a.train:
        dout = torch.randn(out.shape, generator=g, device="cuda").to(torch.bfloat16)
        leaf = logits.clone().requires_grad_()
        s = torch.sigmoid(leaf).gather(1, saved[0].long())
        w = ROUTE["scale"] * s / s.sum(1, keepdim=True)
        ((w[..., None] * rows).sum(1) * dout.float()).sum().backward()
        got = router_grad(dout, logits, saved)
        found["dlogits"] = float((got - leaf.grad).norm() / leaf.grad.norm())

    torch.cuda.synchronize()
    begun, passes = time.perf_counter(), 20
    for _ in range(passes):
        moe_layer(x, logits, bias, experts, a.topk, max_m)
    torch.cuda.synchronize()
    found["us"] = (time.perf_counter() - begun) / passes * 1e6
    print(f"{'int8' if a.int8 else 'fp8'} {'masked' if a.decode else 'contiguous'}, {tokens} tokens, top {a.topk} of "
          f"{a.experts} experts: " + ", ".join(f"{k} {v:.3g}" for k, v in found.items())
          + "  (relative errors against fp32, time of a pass)", flush=True)
    return found


if __name__ == "__main__":
    main()
