"""Timed cases of the mixture-of-experts operators and of the 8-bit integer product.

Five operators, each in a plain form (elementary torch operations in 32 bits)
and as a user calls it from the package:

* ``route``    -- scores, choice and weights of a token's experts, and the
  gradient of the weights with respect to the logits;
* ``dispatch`` -- the layout of the chosen experts' rows, and the FP8 cast of
  the tokens into it;
* ``combine``  -- the weighted sum of the experts' rows for each token, or its
  gradient;
* ``linear``   -- a layer in 8-bit integers: cast of the activations and the
  product with scales for each token and channel;
* ``experts``  -- the same product over expert groups, contiguous or masked.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
ALIGN = 128       # expert segments start at multiples of this many rows
AMAX_FLOOR = 1e-4  # the casts' least row or block maximum


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a decoding request: biased sigmoid scores, 4 of 8 groups, 8 of 256 experts
        dict(name="route-1", op="route", tokens=1, experts=256, topk=8, score="sigmoid", bias=True, groups=8,
             topk_groups=4, group_score="top2", renormalize=True, scale=2.5, dtype="float32", grad=False),
        # a prefill batch: softmax scores from bfloat16 logits, the tokens of the 256-expert workload
        dict(name="route-32768", op="route", tokens=32768, experts=256, topk=8, score="softmax", bias=False, groups=1,
             topk_groups=1, group_score="max", renormalize=True, scale=1.0, dtype="bfloat16", grad=False),
        # a training step's router, forward and backward, odd sizes: 160 experts in 8 groups of 20, plain softmax weights
        dict(name="route-train-4099", op="route", tokens=4099, experts=160, topk=6, score="softmax", bias=False,
             groups=8, topk_groups=3, group_score="max", renormalize=False, scale=16.0, dtype="float32", grad=True),
        # decoding 64 sequences: few rows scattered over many experts
        dict(name="dispatch-64", op="dispatch", tokens=64, experts=256, topk=8, k=7168, drop=0.0),
        # prefill: 32768 rows over 256 experts of uneven popularity, some assignments dropped
        dict(name="dispatch-4096", op="dispatch", tokens=4096, experts=256, topk=8, k=7168, drop=0.02),
        # the rows of that prefill on their way back
        dict(name="combine-4096", op="combine", tokens=4096, experts=256, topk=8, h=7168, drop=0.02, grad=False),
        # training: the gradient to the experts' rows and to the router's weights
        dict(name="combine-grad-8192", op="combine", tokens=8192, experts=16, topk=4, h=7168, drop=0.02, grad=True),
        # a layer for one token: streaming the weights is all there is
        dict(name="linear-1", op="linear", m=1, n=4096, k=7168),
        # a ragged batch, a narrow output and a depth that is no multiple of 128
        dict(name="linear-777", op="linear", m=777, n=2112, k=7152),
        # prefill, the largest dense layer of the repository's workloads
        dict(name="linear-4096", op="linear", m=4096, n=7168, k=16384),
        # experts' products of a prefill: the 8-expert contiguous workload
        dict(name="experts-8192", op="experts", layout="contiguous", groups=8, rows=8192, most=0, n=4096, k=7168),
        # experts' products of a decoding step: 0..32 rows in each of 16 groups, masked layout
        dict(name="experts-decode", op="experts", layout="masked", groups=16, rows=256, most=32, n=4096, k=7168),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "linear", "experts"])
    if op == "route":
        experts, groups = rng.choice([(8, 1), (16, 4), (60, 1), (64, 8), (72, 6), (128, 1), (160, 8), (256, 1), (256, 8)])
        topk_groups = rng.randint(1, max(1, groups - 1))
        grad = rng.random() < 0.4
        return dict(op=op, tokens=_log(rng, 1, 20000 if grad else 32768), experts=experts,
                    topk=rng.randint(1, min(8, topk_groups * (experts // groups))),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    topk_groups=topk_groups, group_score=rng.choice(["max", "top2"]),
                    renormalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5, 16.0]),
                    dtype=rng.choice(["float32", "bfloat16", "float16"]), grad=grad)
    if op in ("dispatch", "combine"):
        experts = rng.choice([8, 16, 60, 64, 256])
        topk = rng.randint(1, 8)
        drop = rng.choice([0.0, 0.02, 0.3])
        if op == "dispatch":
            return dict(op=op, tokens=_log(rng, 1, 4096), experts=experts, topk=topk, k=_log(rng, 512, 7168, 128),
                        drop=drop)
        grad = rng.random() < 0.5
        return dict(op=op, tokens=_log(rng, 1, 8192 if topk <= 4 else 4096), experts=experts if not grad else 16,
                    topk=topk, h=_log(rng, 512, 7168, 8), drop=drop, grad=grad)
    if op == "linear":
        n, k = _log(rng, 256, 16384, 8), _log(rng, 512, 7168, 16)
        return dict(op=op, m=_log(rng, 1, 4096), n=n, k=k)
    layout = rng.choice(["contiguous", "masked"])
    n, k = _log(rng, 256, 4096, 8), _log(rng, 512, 7168, 16)
    groups = rng.choice([2, 5, 8, 16])
    if layout == "contiguous":
        return dict(op=op, layout=layout, groups=groups, rows=_log(rng, 16, 8192), most=0, n=n, k=k)
    rows = rng.choice([64, 128, 256])
    return dict(op=op, layout=layout, groups=groups, rows=rows, most=_log(rng, 1, rows), n=n, k=k)


# ---------------------------------------------------------------- inputs

def _gen(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1_000_003 + stream) % (1 << 62))
    return g


def _activation(seed, stream, rows, k):
    """Rows of normal values, each row with a factor of its own in [1/16, 16]."""
    x = torch.randn((rows, k), generator=_gen(seed, stream), device="cuda")
    u = torch.rand((rows, 1), generator=_gen(seed, stream + 1), device="cuda") * 8 - 4
    return (x * torch.exp2(u)).to(torch.bfloat16)


def _logits(case, seed, stream):
    """Router logits of standard deviation 2, rounded to the logits' type."""
    x = torch.randn((case["tokens"], case["experts"]), generator=_gen(seed, stream), device="cuda") * 2
    return x.to(DTYPES[case["dtype"]])


def _keys64(case, x, b):
    """Scores, expert keys and group scores in 64 bits."""
    x = x.double()
    s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, -1)
    biased = s if b is None else s + b.double()
    key = x if b is None else biased
    by_group = (key if case["group_score"] == "max" else biased).view(x.shape[0], case["groups"], -1)
    top = by_group.sort(dim=-1, descending=True).values
    gs = top[..., 0] if case["group_score"] == "max" else top[..., :2].sum(-1)
    return s, key, gs


def _chosen64(case, x, b):
    """(indices, scores, whether no choice of the row hangs on less than 32 bits tell apart)."""
    s, key, gs = _keys64(case, x, b)
    t, e, g = x.shape[0], case["experts"], case["groups"]
    clear = torch.ones(t, dtype=torch.bool, device=x.device)
    if g > 1:
        v, order = gs.sort(dim=-1, descending=True, stable=True)
        at = case["topk_groups"]
        if at < g and not (case["group_score"] == "max" and b is None):
            clear &= (v[:, at - 1] - v[:, at]) > 2e-6
        keep = torch.zeros((t, g), dtype=torch.bool, device=x.device).scatter_(1, order[:, :at], True)
        key = key.masked_fill(~keep.repeat_interleave(e // g, 1), -math.inf)
    v, order = key.sort(dim=-1, descending=True, stable=True)
    if b is not None:
        k = min(case["topk"], e - 1)
        gap = v[:, :k] - v[:, 1:k + 1]
        clear &= (gap > 2e-6).all(1)
    idx = order[:, :case["topk"]]
    return idx, s.gather(1, idx), clear


def _route_inputs(case, seed):
    x = _logits(case, seed, 1)
    b = (torch.randn(case["experts"], generator=_gen(seed, 2), device="cuda") * 0.05) if case["bias"] else None
    # The indices are compared whole: rows whose choice hangs on less than 32 bits can tell apart are drawn again.
    for again in range(1, 50):
        clear = _chosen64(case, x, b)[2]
        if bool(clear.all()):
            break
        x = torch.where(clear[:, None], x, _logits(case, seed, 100 + again))
    g = torch.randn((case["tokens"], case["topk"]), generator=_gen(seed, 3), device="cuda") if case["grad"] else None
    return {"x": x, "b": b, "g": g}


def _indices(case, seed):
    """Distinct experts for each token, by a popularity that falls with the expert's number; some dropped (-1)."""
    t, e, k = case["tokens"], case["experts"], case["topk"]
    u = torch.rand((t, e), generator=_gen(seed, 11), device="cuda").clamp_min(1e-12)
    pop = -0.7 * torch.log(torch.arange(1, e + 1, device="cuda", dtype=torch.float32))
    idx = (pop - torch.log(-torch.log(u))).sort(dim=-1, descending=True, stable=True).indices[:, :k].to(torch.int32)
    gone = torch.rand((t, k), generator=_gen(seed, 12), device="cuda") < case["drop"]
    return idx.masked_fill(gone, -1).contiguous()


def _rows(case):
    """Rows that hold the contiguous layout whatever the routing."""
    n = case["tokens"] * case["topk"]
    return (n + min(case["experts"], n) * (ALIGN - 1)) // ALIGN * ALIGN


def _layout(idx, experts, rows):
    """m_indices, row_slot, slot_row, counts of the contiguous layout: experts in order, each from a multiple of ALIGN,
    and within an expert by token and slot."""
    flat = idx.reshape(-1).long()
    n = flat.numel()
    key = torch.where(flat < 0, torch.full_like(flat, experts), flat)
    sorted_e, order = key.sort(dim=0, stable=True)
    counts = (key[:, None] == torch.arange(experts, device=idx.device)).sum(0) if n * experts <= 1 << 26 else \
        torch.zeros(experts + 1, dtype=torch.int64, device=idx.device).index_add_(0, key, torch.ones_like(key))[:experts]
    padded = (counts + ALIGN - 1) // ALIGN * ALIGN
    start = padded.cumsum(0) - padded
    first = counts.cumsum(0) - counts
    none = torch.zeros(1, dtype=torch.int64, device=idx.device)
    row = torch.arange(n, device=idx.device) - torch.cat([first, none])[sorted_e] + torch.cat([start, none])[sorted_e]
    row = torch.where(sorted_e < experts, row, torch.full_like(row, -1))
    slot_row = torch.empty_like(row).index_copy_(0, order, row)
    # one row past the end takes what has no row
    to = torch.where(row < 0, torch.full_like(row, rows), row)
    m_indices = torch.full((rows + 1,), -1, dtype=torch.int32, device=idx.device)
    row_slot = torch.full((rows + 1,), -1, dtype=torch.int32, device=idx.device)
    m_indices[to] = sorted_e.to(torch.int32)
    row_slot[to] = order.to(torch.int32)
    return (m_indices[:rows], row_slot[:rows], slot_row.view(idx.shape).to(torch.int32), counts.to(torch.int32))


def _weights8(seed, stream, lead, n, k):
    """Codes and channel scales of a weight quantized once."""
    q = torch.empty(lead + (n, k), dtype=torch.int8, device="cuda")
    s = torch.empty(lead + (n,), dtype=torch.float32, device="cuda")
    for g in range(lead[0] if lead else 1):
        w = torch.randn((n, k), generator=_gen(seed, stream + g), device="cuda")
        sc = w.abs().amax(1) / 127
        (q[g] if lead else q).copy_(torch.round(w / sc[:, None]))
        (s[g] if lead else s).copy_(sc)
    return q, s


def _counts(case, seed):
    g = torch.Generator().manual_seed(int(seed) * 7 + 3)
    if case["layout"] == "masked":
        return torch.randint(0, case["most"] + 1, (case["groups"],), generator=g).tolist()
    cuts = sorted(torch.randint(0, case["rows"] + 1, (case["groups"] - 1,), generator=g).tolist())
    return [b - a for a, b in zip([0] + cuts, cuts + [case["rows"]])]


def prepare(case, seed):
    op = case["op"]
    s = {"case": case}
    if op == "route":
        s.update(_route_inputs(case, seed))
    elif op == "dispatch":
        rows, k = _rows(case), case["k"]
        # one row past the end takes the dropped assignments of the plain form; scales of one block lie beside each
        # other, as the grouped product reads them best
        q = torch.zeros((rows + 1, k), dtype=torch.uint8, device="cuda")
        sf = torch.zeros((k // 128, rows + 1), device="cuda").t()
        s.update(idx=_indices(case, seed), x=_activation(seed, 21, case["tokens"], k), rows=rows, q_all=q, sf_all=sf,
                 q=q[:rows].view(FP8), sf=sf[:rows])
    elif op == "combine":
        rows, h = _rows(case), case["h"]
        idx = _indices(case, seed)
        _, row_slot, slot_row, _ = _layout(idx, case["experts"], rows)
        w = torch.rand((case["tokens"], case["topk"]), generator=_gen(seed, 32), device="cuda") + 0.05
        s.update(row_slot=row_slot.contiguous(), slot_row=slot_row.contiguous(), w=w / w.sum(1, keepdim=True),
                 y=torch.randn((rows, h), generator=_gen(seed, 33), device="cuda", dtype=torch.bfloat16))
        if case["grad"]:
            s["dout"] = torch.randn((case["tokens"], h), generator=_gen(seed, 34), device="cuda", dtype=torch.bfloat16)
    elif op == "linear":
        qb, sb = _weights8(seed, 41, (), case["n"], case["k"])
        s.update(x=_activation(seed, 51, case["m"], case["k"]), qb=qb, sb=sb)
    else:
        counts = _counts(case, seed)
        qb, sb = _weights8(seed, 61, (case["groups"],), case["n"], case["k"])
        s.update(qb=qb, sb=sb, counts=counts)
        if case["layout"] == "masked":
            rows = case["groups"] * case["rows"]
            lead = (case["groups"], case["rows"])
            s["masked_m"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
            s["expected"] = max(1, (case["most"] + 1) // 2)
        else:
            padded = [-(-c // ALIGN) * ALIGN for c in counts]
            rows = (case["rows"] + case["groups"] * (ALIGN - 1)) // ALIGN * ALIGN  # enough whatever the counts
            lead = (rows,)
            m = torch.full((rows,), -1, dtype=torch.int32)
            at = 0
            for g, (c, p) in enumerate(zip(counts, padded)):
                m[at:at + c] = g
                at += p
            s["m_indices"] = m.cuda()
        s["qa"] = torch.randint(-127, 128, lead + (case["k"],), generator=_gen(seed, 71), device="cuda",
                                dtype=torch.int8)
        s["sa"] = torch.rand(lead, generator=_gen(seed, 72), device="cuda") * 0.05 + 1e-3
        s["d"] = torch.zeros(lead + (case["n"],), dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import moe_fp8_gemm_amd as dg
    case = s["case"]
    op = case["op"]
    if op == "route":
        idx, w = dg.route_topk(s["x"], case["topk"], score=case["score"], bias=s["b"],
                               num_expert_groups=case["groups"], topk_groups=case["topk_groups"],
                               group_score=case["group_score"], renormalize=case["renormalize"], scale=case["scale"])
        if not case["grad"]:
            return {"indices": idx, "weights": w}
        dx = dg.route_topk_grad(s["x"], idx, s["g"], score=case["score"], renormalize=case["renormalize"],
                                scale=case["scale"])
        return {"indices": idx, "weights": w, "dlogits": dx}
    if op == "dispatch":
        lay = dg.expert_layout_contiguous(s["idx"], case["experts"])
        q, sf = dg.dispatch_cast_fp8(s["x"], lay.slot_row, q=s["q"], sf=s["sf"])
        return {"q": q, "sf": sf, "m_indices": lay.m_indices, "row_slot": lay.row_slot, "slot_row": lay.slot_row,
                "counts": lay.counts}
    if op == "combine":
        if not case["grad"]:
            return dg.combine(s["y"], s["slot_row"], s["w"])
        dy, dw = dg.combine_grad(s["dout"], s["y"], s["slot_row"], s["row_slot"], s["w"])
        return {"dy": dy, "dw": dw}
    if op == "linear":
        a = dg.per_token_cast_int8(s["x"])
        d = torch.empty((case["m"], case["n"]), dtype=torch.bfloat16, device="cuda")
        return dg.int8_gemm_nt(a, (s["qb"], s["sb"]), d)
    if case["layout"] == "masked":
        return dg.m_grouped_int8_gemm_nt_masked((s["qa"], s["sa"]), (s["qb"], s["sb"]), s["d"], s["masked_m"],
                                                s["expected"])
    return dg.m_grouped_int8_gemm_nt_contiguous((s["qa"], s["sa"]), (s["qb"], s["sb"]), s["d"], s["m_indices"])


def _plain_route(s):
    case, b = s["case"], s["b"]
    x = s["x"].float()
    t, e, g = x.shape[0], case["experts"], case["groups"]
    if case["score"] == "sigmoid":
        sc = 1 / (1 + torch.exp(-x))
    else:
        ex = torch.exp(x - x.amax(1, keepdim=True))
        sc = ex / ex.sum(1, keepdim=True)
    biased = sc if b is None else sc + b
    key = x if b is None else biased
    if g > 1:
        if case["group_score"] == "max":
            gs = key.view(t, g, -1).amax(-1)
        else:
            gs = biased.view(t, g, -1).sort(dim=-1, descending=True).values[..., :2].sum(-1)
        best = gs.sort(dim=-1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        keep = torch.zeros((t, g), dtype=torch.bool, device=x.device).scatter_(1, best, True)
        key = torch.where(keep.repeat_interleave(e // g, 1), key, -math.inf)
    idx = key.sort(dim=-1, descending=True, stable=True).indices[:, :case["topk"]]
    si = sc.gather(1, idx)
    total = si.sum(1, keepdim=True)
    w = (si / total if case["renormalize"] else si) * case["scale"]
    out = {"indices": idx.to(torch.int32), "weights": w}
    if case["grad"]:
        ds = s["g"] * case["scale"]
        if case["renormalize"]:
            ds = (ds - (ds * si).sum(1, keepdim=True) / total) / total
        if case["score"] == "sigmoid":
            dx = torch.zeros_like(x).scatter_(1, idx, ds * si * (1 - si))
        else:
            dx = torch.zeros_like(x).scatter_(1, idx, ds * si) - sc * (ds * si).sum(1, keepdim=True)
        out["dlogits"] = dx.to(s["x"].dtype)
    return out


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "route":
        return _plain_route(s)
    if op == "dispatch":
        m_indices, row_slot, slot_row, counts = _layout(s["idx"], case["experts"], s["rows"])
        t, k = s["x"].shape
        x = s["x"].float().view(t, k // 128, 128)
        sc = x.abs().amax(2).clamp_min(AMAX_FLOOR) / 448
        q = (x / sc[..., None]).clamp(-448, 448).to(FP8).view(torch.uint8).view(t, k)
        to = slot_row.reshape(-1).long()
        to = torch.where(to < 0, torch.full_like(to, s["rows"]), to)
        token = torch.arange(to.numel(), device=to.device) // case["topk"]
        s["q_all"][to] = q[token]
        s["sf_all"][to] = sc[token]
        return {"q": s["q"], "sf": s["sf"], "m_indices": m_indices, "row_slot": row_slot, "slot_row": slot_row,
                "counts": counts}
    if op == "combine":
        slot = s["slot_row"].long()
        yi = s["y"][slot.clamp_min(0)].float()
        w = torch.where(slot >= 0, s["w"], 0.0)
        if not case["grad"]:
            return (yi * w[..., None]).sum(1).to(torch.bfloat16)
        dout = s["dout"].float()
        dw = (yi * dout[:, None, :]).sum(2)
        row_slot = s["row_slot"].long()
        wr = torch.where(row_slot >= 0, s["w"].reshape(-1)[row_slot.clamp_min(0)], 0.0)
        dy = dout[row_slot.clamp_min(0) // case["topk"]] * wr[:, None]
        return {"dy": dy.to(torch.bfloat16), "dw": torch.where(slot >= 0, dw, 0.0)}
    if op == "linear":
        x = s["x"].float()
        sa = x.abs().amax(1, keepdim=True).clamp_min(AMAX_FLOOR) / 127
        return ((torch.round(x / sa) @ s["qb"].float().t()) * sa * s["sb"]).to(torch.bfloat16)
    if case["layout"] == "masked":
        acc = torch.bmm(s["qb"].float(), s["qa"].float().transpose(1, 2).contiguous()).transpose(1, 2)
        d = (acc * s["sa"][..., None] * s["sb"][:, None, :]).to(torch.bfloat16)
        row = torch.arange(case["rows"], device=d.device)
        s["d"].copy_(torch.where((row < s["masked_m"][:, None])[..., None], d, s["d"]))
        return s["d"]
    at = 0
    for g, c in enumerate(s["counts"]):  # a group's rows lie together
        acc = s["qa"][at:at + c].float() @ s["qb"][g].float().t()
        s["d"][at:at + c] = (acc * s["sa"][at:at + c, None] * s["sb"][g]).to(torch.bfloat16)
        at += -(-c // ALIGN) * ALIGN
    return s["d"]


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        idx, si, _ = _chosen64(case, s["x"], s["b"])
        total = si.sum(1, keepdim=True)
        w = case["scale"] * (si / total if case["renormalize"] else si)
        out = {"indices": idx, "weights": w}
        if case["grad"]:
            # d weights / d scores, then d scores / d logits, as full matrices of the definition's terms
            g = s["g"].double() * case["scale"]
            ds = g / total - (g * si).sum(1, keepdim=True) / total ** 2 if case["renormalize"] else g
            full, _, _ = _keys64(case, s["x"], s["b"])
            up = torch.zeros_like(full).scatter_(1, idx, ds)
            out["dlogits"] = up * full * (1 - full) if case["score"] == "sigmoid" else \
                full * up - full * (full * up).sum(1, keepdim=True)
        return out
    if op == "dispatch":
        k = case["k"]
        x = s["x"].double().view(case["tokens"], k // 128, 128)
        sc = x.abs().amax(2).clamp_min(AMAX_FLOOR) / 448
        sf = torch.zeros((s["rows"], k // 128), dtype=torch.float64, device="cuda")
        _, row_slot, _, _ = _layout(s["idx"], case["experts"], s["rows"])
        there = row_slot >= 0
        sf[there] = sc[row_slot[there].long() // case["topk"]]
        return {"q": None, "sf": sf, "m_indices": None, "row_slot": None, "slot_row": None, "counts": None}
    if op == "combine":
        slot, w = s["slot_row"].long(), s["w"].double()
        if not case["grad"]:
            out = torch.zeros((case["tokens"], case["h"]), dtype=torch.float64, device="cuda")
            for j in range(case["topk"]):
                there = slot[:, j] >= 0
                out[there] += w[there, j, None] * s["y"][slot[there, j]].double()
            return out
        dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(w.shape, dtype=torch.float64, device="cuda")
        for j in range(case["topk"]):
            there = slot[:, j] >= 0
            dout = s["dout"][there].double()
            dy[slot[there, j]] = w[there, j, None] * dout
            dw[there, j] = (dout * s["y"][slot[there, j]].double()).sum(1)
        return {"dy": dy, "dw": dw}
    if op == "linear":
        x = s["x"].double()
        sa = x.abs().amax(1).clamp_min(AMAX_FLOOR) / 127
        q = torch.round(x / sa[:, None])
        return torch.mm(q, s["qb"].double().t()) * torch.outer(sa, s["sb"].double())
    d = torch.zeros(s["d"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for g, c in enumerate(s["counts"]):
        if case["layout"] == "masked":
            qa, sa, to = s["qa"][g, :c], s["sa"][g, :c], d[g, :c]
        else:
            qa, sa, to = s["qa"][at:at + c], s["sa"][at:at + c], d[at:at + c]
            at += -(-c // ALIGN) * ALIGN
        to.copy_(torch.mm(qa.double(), s["qb"][g].double().t()) * torch.outer(sa.double(), s["sb"][g].double()))
    return d


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        el = 4 if case["dtype"] == "float32" else 2
        b = t * e * el + t * k * 8 + (4 * e if case["bias"] else 0)
        if case["grad"]:
            b += t * k * 4 + t * e * el
        return {"bytes": b, "flops": t * e * (10 if case["grad"] else 6)}
    if op == "dispatch":
        t, k, n = case["tokens"], case["k"], case["tokens"] * case["topk"]
        there = n * (1 - case["drop"])
        return {"bytes": t * k * 2 + there * (k + k // 128 * 4) + n * 8 + _rows(case) * 8 + case["experts"] * 4,
                "flops": t * k * 4}
    if op == "combine":
        t, h, n = case["tokens"], case["h"], case["tokens"] * case["topk"]
        there = n * (1 - case["drop"])
        if not case["grad"]:
            return {"bytes": there * h * 2 + t * h * 2 + n * 8, "flops": 2 * there * h}
        return {"bytes": t * h * 2 + there * h * 2 + _rows(case) * (h * 2 + 4) + n * 12, "flops": 3 * there * h}
    n, k = case["n"], case["k"]
    if op == "linear":
        m = case["m"]
        return {"bytes": m * k * 2 + n * k + 4 * n + 2 * m * n, "flops": 2 * m * n * k}
    g = case["groups"]
    rows = g * case["most"] / 2 if case["layout"] == "masked" else case["rows"]
    return {"bytes": rows * (k + 4 + 2 * n) + g * n * (k + 4), "flops": 2 * rows * n * k}
