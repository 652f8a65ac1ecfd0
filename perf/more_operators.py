"""Timed cases of the operators around the products of a layer: norms, the gated activation and weights' gradients.

Five operators, each in a plain form (elementary torch operations in 32 bits)
and as a user calls it from the package:

* ``norm``      -- residual addition and root-mean-square norm of rows, as rows of
  the input's type or quantized for the next product (FP8 blocks, int8 rows);
* ``norm_grad`` -- its gradient: rows and the norm's weight;
* ``gate``      -- SiLU gate times up and the cast for the next product, for the
  valid rows of a layout, with or without an 8-bit checkpoint of the input;
* ``gate_grad`` -- its gradient, from the 8-bit checkpoint or from 16-bit rows,
  with or without a cast for the product that follows;
* ``wgrad``     -- weights' gradients, a sum over the rows of each expert, the
  activations as 16-bit rows or as the FP8 codes that the forward product read.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
ALIGN = 128        # the contiguous layout's segments start at multiples of this many rows
AMAX_FLOOR = 1e-4  # the casts' least row or block maximum
EPS = 1e-6


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a decoding request, before a dense FP8 layer
        dict(name="norm-1", op="norm", rows=1, k=7168, residual=True, out="fp8", dtype="bfloat16"),
        # a ragged decoding batch before an int8 layer; a width that is no multiple of 128
        dict(name="norm-77-int8", op="norm", rows=77, k=2112, residual=True, out="int8", dtype="bfloat16"),
        # prefill: the rows of the largest cast of the repository's workloads, residual and cast in one pass
        dict(name="norm-32768", op="norm", rows=32768, k=7168, residual=True, out="fp8", dtype="bfloat16"),
        # a training step's norm on its way back, rows of odd number, the residual's own gradient added
        dict(name="norm-grad-4099", op="norm_grad", rows=4099, k=2048, through=True, dtype="bfloat16"),
        # the same at the largest width and batch
        dict(name="norm-grad-16384", op="norm_grad", rows=16384, k=7168, through=True, dtype="bfloat16"),
        # decoding: 0..32 rows in each of 16 experts of the masked layout
        dict(name="gate-decode", op="gate", layout="masked", groups=16, rows=256, most=32, inner=2048, out="fp8",
             checkpoint=False, dtype="bfloat16"),
        # a training step's forward pass: 32768 rows over 256 experts, the input kept in 8 bits
        dict(name="gate-32768", op="gate", layout="contiguous", groups=256, rows=32768, most=0, inner=2048, out="fp8",
             checkpoint=True, dtype="bfloat16"),
        # a small dense layer on its way back from 16-bit rows, odd sizes
        dict(name="gate-grad-333", op="gate_grad", layout="dense", groups=1, rows=333, most=0, inner=1408, saved="rows",
             cast=False, dtype="bfloat16"),
        # the way back of that training step, from the checkpoint, with the cast for the product that follows
        dict(name="gate-grad-32768", op="gate_grad", layout="contiguous", groups=256, rows=32768, most=0, inner=2048,
             saved="fp8", cast=True, dtype="bfloat16"),
        # a dense layer of few outputs over a ragged batch: a long sum for a small matrix
        dict(name="wgrad-8191", op="wgrad", layout="dense", groups=1, rows=8191, most=0, n=512, k=2112, saved="rows",
             out="float32", scales="float"),
        # the 8-expert contiguous workload, its activations as the FP8 codes that the forward pass read
        dict(name="wgrad-8x8192", op="wgrad", layout="contiguous", groups=8, rows=8192, most=0, n=4096, k=7168,
             saved="fp8", out="float32", scales="power"),
        # many experts of uneven popularity, rows that lie together without padding, 16-bit gradients
        dict(name="wgrad-64x16384", op="wgrad", layout="ragged", groups=64, rows=16384, most=0, n=2048, k=1408,
             saved="fp8", out="bfloat16", scales="float"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "gate", "gate_grad", "wgrad"])
    if op == "norm":
        out = rng.choice(["rows", "fp8", "int8"])
        step = {"rows": 8, "fp8": 128, "int8": 16}[out]
        dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
        k = _log(rng, 512, 7168, step)
        return dict(op=op, rows=_log(rng, 1, 32768 if dtype != "float32" else 16384), k=k, residual=rng.random() < 0.7,
                    out=out, dtype=dtype)
    if op == "norm_grad":
        dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
        return dict(op=op, rows=_log(rng, 1, 16384 if dtype != "float32" else 8192), k=_log(rng, 512, 7168, 8),
                    through=rng.random() < 0.7, dtype=dtype)
    layout = rng.choice(["dense", "contiguous", "masked"])
    if op in ("gate", "gate_grad"):
        groups = {"dense": 1, "contiguous": rng.choice([8, 16, 60, 256]), "masked": rng.choice([5, 16, 64])}[layout]
        rows = rng.choice([32, 256]) if layout == "masked" else _log(rng, 1, 32768)
        c = dict(op=op, layout=layout, groups=groups, rows=rows, most=_log(rng, 1, rows) if layout == "masked" else 0)
        if op == "gate":
            out = rng.choice(["fp8", "fp8", "int8"])
            return dict(c, inner=_log(rng, 256, 2048, 128 if out == "fp8" else 16), out=out,
                        checkpoint=out == "fp8" and rng.random() < 0.6, dtype=rng.choice(["bfloat16", "bfloat16", "float16"]))
        saved, cast = rng.choice(["fp8", "rows"]), rng.random() < 0.5
        step = 128 if saved == "fp8" or cast else 8
        return dict(c, inner=_log(rng, 256, 2048, step), saved=saved, cast=cast, dtype="bfloat16")
    layout = rng.choice(["dense", "contiguous", "ragged", "masked"])
    groups = 1 if layout == "dense" else rng.choice([3, 8, 16, 64])
    saved = rng.choice(["fp8", "rows"])
    # the outputs of all groups together stay below the largest listed ones
    side = min(7168, int(math.sqrt(8 * 4096 * 7168 / groups)))
    n, k = _log(rng, 256, min(4096, side), 8), _log(rng, 256, side, 128 if saved == "fp8" else 8)
    rows = rng.choice([64, 256]) if layout == "masked" else _log(rng, 16, 8192)
    scales = rng.choice(["power", "float"]) if saved == "fp8" else "float"
    # codes whose scales are no powers of two are rounded to 16 bits once: their gradients are 16-bit ones here
    out = "bfloat16" if saved == "fp8" and scales == "float" else rng.choice(["float32", "bfloat16"])
    return dict(op=op, layout=layout, groups=groups, rows=rows, most=_log(rng, 1, rows) if layout == "masked" else 0,
                n=n, k=k, saved=saved, out=out, scales=scales)


# ---------------------------------------------------------------- inputs

def _gen(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1_000_003 + stream) % (1 << 62))
    return g


def _normal(seed, stream, shape, dtype, spread=0):
    """Normal values; with a spread, each row with a factor of its own in [2^-spread, 2^spread]."""
    x = torch.randn(shape, generator=_gen(seed, stream), device="cuda")
    if spread:
        u = torch.rand(shape[:-1] + (1,), generator=_gen(seed, stream + 1), device="cuda") * 2 - 1
        x = x * torch.exp2(u * spread)
    return x.to(dtype)


def _codes(x, power):
    """Codes and scales of an activation kept in 8 bits, scales of one block beside each other along the rows."""
    r, k = x.shape
    v = x.double().view(r, k // 128, 128)
    s = v.abs().amax(2).clamp_min(AMAX_FLOOR) / 448
    if power:
        m, e = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    s = s.float()
    q = (v / s.double()[..., None]).clamp(-448, 448).float().to(FP8).view(r, k)
    return q, s.t().contiguous().t()


def _counts(case, seed):
    """Rows of each group, on the host: 0..most (masked), or a split of all rows by uneven popularity."""
    g = torch.Generator().manual_seed(int(seed) * 7 + 3)
    if case["layout"] == "dense":
        return [case["rows"]]
    if case["layout"] == "masked":
        return torch.randint(0, case["most"] + 1, (case["groups"],), generator=g).tolist()
    p = 1.0 / torch.arange(1, case["groups"] + 1).double() ** 0.5
    p = p[torch.randperm(case["groups"], generator=g)]
    expert = torch.multinomial(p, case["rows"], replacement=True, generator=g)
    return torch.bincount(expert, minlength=case["groups"]).tolist()


def _segments(case, counts):
    """([(first row, rows)] of the groups, rows in all)."""
    if case["layout"] == "masked":
        return [(i * case["rows"], c) for i, c in enumerate(counts)], case["groups"] * case["rows"]
    step = ALIGN if case["layout"] == "contiguous" else 1
    at, seg = 0, []
    for c in counts:
        seg.append((at, c))
        at += -(-c // step) * step
    return seg, (case["rows"] + case["groups"] * (ALIGN - 1)) // ALIGN * ALIGN if step > 1 else at


def _layout(case, seed):
    """What a layout holds: host segments, rows in all, the valid rows' numbers, m_indices or masked_m, counts."""
    counts = _counts(case, seed)
    seg, rows = _segments(case, counts)
    m = torch.full((rows,), -1, dtype=torch.int32)
    for i, (at, c) in enumerate(seg):
        m[at:at + c] = i
    m = m.cuda()
    return {"seg": seg, "rows": rows, "valid": slice(None) if case["layout"] == "dense" else (m >= 0).nonzero()[:, 0],
            "m_indices": m if case["layout"] == "contiguous" else None,
            "counts": torch.tensor(counts, dtype=torch.int32, device="cuda")}


def _fp8_out(rows, k):
    """Codes and scales to be written: zeros, so that rows without a token compare equal."""
    return (torch.zeros((rows, k), dtype=torch.uint8, device="cuda").view(FP8),
            torch.zeros((k // 128, rows), device="cuda").t())


def prepare(case, seed):
    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_grad"):
        dtype, shape = DTYPES[case["dtype"]], (case["rows"], case["k"])
        s["w"] = (1 + 0.1 * torch.randn(case["k"], generator=_gen(seed, 1), device="cuda")).to(dtype)
        if op == "norm":
            s["x"] = _normal(seed, 2, shape, dtype, spread=2)
            s["r"] = _normal(seed, 4, shape, dtype) if case["residual"] else None
        else:
            s["h"] = _normal(seed, 2, shape, dtype, spread=2)
            s["dy"] = _normal(seed, 4, shape, dtype)
            s["dh"] = _normal(seed, 6, shape, dtype) if case["through"] else None
            s["rstd"] = (1 / (s["h"].double().square().mean(1) + EPS).sqrt()).float()
        return s
    s.update(_layout(case, seed))
    rows = s["rows"]
    if op in ("gate", "gate_grad"):
        inner, dtype = case["inner"], DTYPES[case["dtype"]]
        h = _normal(seed, 11, (rows, 2 * inner), dtype, spread=1)
        if op == "gate":
            s["h"] = h
            if case["out"] == "fp8":
                s["q"], s["sf"] = _fp8_out(rows, inner)
            else:
                s["q"] = torch.zeros((rows, inner), dtype=torch.int8, device="cuda")
                s["sf"] = torch.zeros(rows, device="cuda")
            if case["checkpoint"]:
                s["hq"], s["hsf"] = _fp8_out(rows, 2 * inner)
        else:
            s["h"] = _codes(h, False) if case["saved"] == "fp8" else h
            s["da"] = _normal(seed, 13, (rows, inner), dtype)
            s["out"] = torch.zeros((rows, 2 * inner), dtype=dtype, device="cuda")
            if case["cast"]:
                s["q"], s["sf"] = _fp8_out(rows, 2 * inner)
        return s
    # what lies between the groups' rows is there in memory too and must not count
    s["dy"] = _normal(seed, 21, (rows, case["n"]), torch.bfloat16)
    x = _normal(seed, 23, (rows, case["k"]), torch.bfloat16, spread=1)
    s["x"] = _codes(x, case["scales"] == "power") if case["saved"] == "fp8" else x
    lead = () if case["layout"] == "dense" else (case["groups"],)
    s["dw"] = torch.empty(lead + (case["n"], case["k"]), dtype=DTYPES[case["out"]], device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import moe_fp8_gemm_amd as dg
    case = s["case"]
    op = case["op"]
    if op == "norm":
        if case["out"] == "rows":
            y, h, rstd = dg.rms_norm(s["x"], s["w"], s["r"], eps=EPS)
            return {"y": y, "h": h, "rstd": rstd}
        if case["out"] == "fp8":
            (q, sf), h, rstd = dg.rms_norm_cast_fp8(s["x"], s["w"], s["r"], eps=EPS)
            return {"q": q, "sf": sf, "h": h, "rstd": rstd}
        (q, sf), h, rstd = dg.rms_norm_cast_int8(s["x"], s["w"], s["r"], eps=EPS)
        return {"y": _values(q, sf), "sf": sf, "h": h, "rstd": rstd}
    if op == "norm_grad":
        dx, dw = dg.rms_norm_grad(s["dy"], s["h"], s["w"], s["rstd"], s["dh"])
        return {"dx": dx, "dw": dw}
    where = {}
    if case["layout"] == "masked":
        where = {"masked_m": s["counts"]}
    elif case["layout"] == "contiguous":
        where = {"m_indices": s["m_indices"]}
    if op == "gate":
        if case["out"] == "int8":
            q, sf = dg.swiglu_cast_int8(s["h"], **where, q=s["q"], sf=s["sf"])
            return {"a": _values(q, sf), "sf": sf}
        if case["checkpoint"]:
            (q, sf), (hq, hsf) = dg.swiglu_checkpoint_fp8(s["h"], **where, q=s["q"], sf=s["sf"], hq=s["hq"],
                                                          hsf=s["hsf"])
            return {"q": q, "sf": sf, "hq": hq, "hsf": hsf}
        q, sf = dg.swiglu_cast_fp8(s["h"], **where, q=s["q"], sf=s["sf"])
        return {"q": q, "sf": sf}
    if op == "gate_grad":
        if case["cast"]:
            dh, (q, sf) = dg.swiglu_grad_cast_fp8(s["da"], s["h"], **where, dh=s["out"], q=s["q"], sf=s["sf"])
            return {"dh": dh, "q": q, "sf": sf}
        return dg.swiglu_grad(s["da"], s["h"], **where, dh=s["out"])
    if case["layout"] == "dense":
        return dg.weight_grad(s["dy"], s["x"], s["dw"])
    if case["layout"] == "masked":
        return dg.m_grouped_weight_grad_masked(s["dy"], s["x"], s["dw"], s["counts"])
    return dg.m_grouped_weight_grad_contiguous(s["dy"], s["x"], s["dw"], s["counts"],
                                               alignment=ALIGN if case["layout"] == "contiguous" else 1)


def _values(q, sf):
    """The values that int8 codes stand for, as 16-bit rows."""
    return (q * sf[:, None]).to(torch.bfloat16)


def _quantized(v):
    """(codes, scales) of fp32 rows in blocks of 128."""
    r, k = v.shape
    v = v.view(r, k // 128, 128)
    sf = v.abs().amax(2).clamp_min(AMAX_FLOOR) / 448
    return (v / sf[..., None]).clamp(-448, 448).to(FP8).view(r, k), sf


def _float(x):
    """fp32 rows of 16-bit ones, or of codes and their scales."""
    if isinstance(x, tuple):
        q, sf = x
        r, k = q.shape
        return (q.float().view(r, k // 128, 128) * sf[..., None]).view(r, k)
    return x.float()


def _put(s, name, valid, value):
    """Writes the valid rows of one of the state's buffers."""
    to = s[name].view(torch.uint8) if s[name].dtype == FP8 else s[name]
    to[valid] = value.view(torch.uint8) if s[name].dtype == FP8 else value
    return s[name]


def _rows_of(x, valid):
    """Valid rows of 16-bit rows, or of codes and scales."""
    if isinstance(x, tuple):
        return x[0].view(torch.uint8)[valid].view(FP8), x[1][valid]
    return x[valid]


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        x = s["x"].float()
        h = (x + s["r"].float()).to(s["x"].dtype) if case["residual"] else s["x"]
        hf = h.float()
        rstd = 1 / torch.sqrt((hf * hf).mean(1) + EPS)
        y = hf * rstd[:, None] * s["w"].float()
        if case["out"] == "rows":
            return {"y": y.to(h.dtype), "h": h, "rstd": rstd}
        if case["out"] == "fp8":
            q, sf = _quantized(y)
            return {"q": q, "sf": sf, "h": h, "rstd": rstd}
        sf = y.abs().amax(1).clamp_min(AMAX_FLOOR) / 127
        return {"y": _values(torch.round(y / sf[:, None]), sf), "sf": sf, "h": h, "rstd": rstd}
    if op == "norm_grad":
        hh = s["h"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        g = dy * s["w"].float()
        dx = s["rstd"][:, None] * (g - hh * (g * hh).mean(1, keepdim=True))
        if case["through"]:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(s["h"].dtype), "dw": (dy * hh).sum(0)}
    if op in ("gate", "gate_grad"):
        v, inner = s["valid"], case["inner"]
        h = _float(_rows_of(s["h"], v))
        g, u = h[:, :inner], h[:, inner:]
        sig = 1 / (1 + torch.exp(-g))
        if op == "gate":
            a = g * sig * u
            if case["out"] == "int8":
                sf = a.abs().amax(1).clamp_min(AMAX_FLOOR) / 127
                _put(s, "q", v, torch.round(a / sf[:, None]).to(torch.int8))
                _put(s, "sf", v, sf)
                return {"a": _values(s["q"], s["sf"]), "sf": s["sf"]}
            q, sf = _quantized(a)
            out = {"q": _put(s, "q", v, q), "sf": _put(s, "sf", v, sf)}
            if case["checkpoint"]:
                q, sf = _quantized(h)
                out.update(hq=_put(s, "hq", v, q), hsf=_put(s, "hsf", v, sf))
            return out
        da = s["da"][v].float()
        dh = torch.cat([da * u * sig * (1 + g * (1 - sig)), da * g * sig], 1)
        out = _put(s, "out", v, dh.to(s["out"].dtype))
        if not case["cast"]:
            return out
        q, sf = _quantized(dh)
        return {"dh": out, "q": _put(s, "q", v, q), "sf": _put(s, "sf", v, sf)}
    dw = s["dw"] if s["dw"].dim() == 3 else s["dw"][None]
    for i, (at, c) in enumerate(s["seg"]):  # a group's rows lie together
        x = tuple(t[at:at + c] for t in s["x"]) if isinstance(s["x"], tuple) else s["x"][at:at + c]
        dw[i] = s["dy"][at:at + c].float().t() @ _float(x)
    return s["dw"]


# ---------------------------------------------------------------- the definition in 64 bits

def _codes64(v):
    """(values of the codes, scales) of 64-bit rows in blocks of 128."""
    blocks = v.unflatten(1, (-1, 128))
    sf = blocks.abs().amax(2).clamp_min(AMAX_FLOOR) / 448
    return (blocks / sf[..., None]).clamp(-448, 448).float().to(FP8).double().flatten(1), sf


def _spread(s, value):
    """Valid rows in their places among zeros."""
    if isinstance(s["valid"], slice):
        return value
    out = torch.zeros((s["rows"],) + value.shape[1:], dtype=torch.float64, device="cuda")
    return out.index_copy_(0, s["valid"], value)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double() + s["r"].double() if case["residual"] else s["x"].double()
        # the norm is that of the rows as they are stored
        h = h.to(s["x"].dtype).double()
        rstd = (h.square().sum(1) / case["k"] + EPS) ** -0.5
        y = torch.einsum("rk,r,k->rk", h, rstd, s["w"].double())
        if case["out"] == "rows":
            return {"y": y, "h": h, "rstd": rstd}
        if case["out"] == "fp8":
            q, sf = _codes64(y)
            return {"q": q, "sf": sf, "h": h, "rstd": rstd}
        sf = y.abs().amax(1).clamp_min(AMAX_FLOOR) / 127
        return {"y": torch.round(y / sf[:, None]) * sf[:, None], "sf": sf, "h": h, "rstd": rstd}
    if op == "norm_grad":
        # y_j = w_j h_j rho, d rho / d h_i = -rho^3 h_i / k
        h, dy, rho = s["h"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        w = s["w"].double()
        dx = dy * w * rho - rho ** 3 / case["k"] * h * (dy * w * h).sum(1, keepdim=True)
        return {"dx": dx + s["dh"].double() if case["through"] else dx, "dw": (dy * h * rho).sum(0)}
    if op in ("gate", "gate_grad"):
        inner = case["inner"]
        if isinstance(s["h"], tuple):
            q, sf = s["h"]
            h = q.double() * sf.double().repeat_interleave(128, 1)
        else:
            h = s["h"].double()
        h = h[s["valid"]]
        g, u = h[:, :inner], h[:, inner:]
        if op == "gate":
            a = torch.sigmoid(g) * g * u
            if case["out"] == "int8":
                sf = a.abs().amax(1).clamp_min(AMAX_FLOOR) / 127
                return {"a": _spread(s, torch.round(a / sf[:, None]) * sf[:, None]), "sf": _spread(s, sf)}
            q, sf = _codes64(a)
            out = {"q": _spread(s, q), "sf": _spread(s, sf)}
            if case["checkpoint"]:
                q, sf = _codes64(h)
                out.update(hq=_spread(s, q), hsf=_spread(s, sf))
            return out
        da, sg = s["da"][s["valid"]].double(), torch.sigmoid(g)
        dh = torch.cat([da * u * (sg + g * sg * torch.sigmoid(-g)), da * g * sg], 1)
        if not case["cast"]:
            return _spread(s, dh)
        q, sf = _codes64(dh)
        return {"dh": _spread(s, dh), "q": _spread(s, q), "sf": _spread(s, sf)}
    dw = torch.zeros((case["groups"], case["n"], case["k"]), dtype=torch.float64, device="cuda")
    for i, (at, c) in enumerate(s["seg"]):
        if isinstance(s["x"], tuple):
            x = s["x"][0][at:at + c].double() * s["x"][1][at:at + c].double().repeat_interleave(128, 1)
        else:
            x = s["x"][at:at + c].double()
        torch.mm(s["dy"][at:at + c].double().t().contiguous(), x, out=dw[i])
    return dw[0] if case["layout"] == "dense" else dw


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        r, k, el = case["rows"], case["k"], 4 if case["dtype"] == "float32" else 2
        n = r * k
        if op == "norm":
            b = n * el * (3 if case["residual"] else 1) + k * el + 4 * r
            b += {"rows": n * el, "fp8": n + n // 128 * 4, "int8": n + 4 * r}[case["out"]]
            return {"bytes": b, "flops": 6 * n}
        return {"bytes": n * el * (4 if case["through"] else 3) + k * (el + 4) + 4 * r, "flops": 10 * n}
    rows = case["groups"] * case["most"] / 2 if case["layout"] == "masked" else case["rows"]
    marks = 4 * case["groups"] if case["layout"] == "masked" else 4 * rows if case["layout"] == "contiguous" else 0
    if op == "gate":
        n = rows * case["inner"]
        b = n * 4 + n + (n / 32 if case["out"] == "fp8" else 4 * rows)
        if case["checkpoint"]:
            b += 2 * n * (1 + 1 / 32)
        return {"bytes": b + marks, "flops": 8 * n}
    if op == "gate_grad":
        n = rows * case["inner"]
        b = n * 2 + (2 * n * (1 + 1 / 32) if case["saved"] == "fp8" else 4 * n) + 4 * n
        if case["cast"]:
            b += 2 * n * (1 + 1 / 32)
        return {"bytes": b + marks, "flops": 14 * n}
    n, k = case["n"], case["k"]
    b = rows * n * 2 + rows * (k * (1 + 1 / 32) if case["saved"] == "fp8" else 2 * k)
    b += case["groups"] * (n * k * (4 if case["out"] == "float32" else 2) + 4)
    return {"bytes": b, "flops": 2 * rows * n * k}
