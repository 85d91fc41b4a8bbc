"""Measured cases of the block-scaled linear layers and of the experts' layers.

Five operators, each in a plain form (elementary torch operations, `own` false) and as the calls a
user makes of the package (`own` true):

* quant    `quantize_block128`: bf16 -> E4M3 codes with one fp32 scale per 128 elements of a row
           (activations), per 128 elements of a column (gradients, for weight gradients) or per
           128 x 128 block (weights)
* gemm     `gemm_scaled(fmt="e4m3_block128")`: the product of such operands, forward with its fused
           epilogues, and the two backward products from K-major operands
* grouped  `gemm_grouped`: one such product per expert over rows grouped by expert
* route    `expert_route` and `expert_route_backward`: scores, group-limited top-k, weights, the
           rows in expert order, and the gradient of the logits
* combine  `expert_combine` and `expert_combine_backward`: the weighted sum of the experts' rows

Sizes are those of this repository's workloads (5120-wide hidden states with 17408-wide gated
layers, 2048-wide hidden states, 16 / 1000-odd / 4096 tokens) and generic expert counts.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128


def _div_up(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a decode step's activations before a linear layer: launch latency
        {"name": "quant_rows_t16", "op": "quant", "tiling": "row", "batch": 1, "rows": 16, "cols": 5120},
        # preparing the gate/up weight of a dense layer: a stream over 0.5 GB
        {"name": "quant_blocks_34816", "op": "quant", "tiling": "block", "batch": 1, "rows": 34816, "cols": 5120},
        # down projection with the residual add, one decode step of 16 sequences
        {"name": "gemm_add_t16", "op": "gemm", "kind": "add", "m": 16, "n": 5120, "k": 17408},
        # gate/up projection with SwiGLU over a 4096-token prefill chunk
        {"name": "gemm_swiglu_t4096", "op": "gemm", "kind": "swiglu", "m": 4096, "n": 34816, "k": 5120},
        # fused attention input projection of a ragged chunk
        {"name": "gemm_store_t1111", "op": "gemm", "kind": "store", "m": 1111, "n": 7168, "k": 5120},
        # weight gradient of a 2048 -> 4096 projection over 4000 tokens: dY^T X, both K-major
        {"name": "gemm_dw_t4000", "op": "gemm", "kind": "dw", "m": 4096, "n": 2048, "k": 4000},
        # experts' gate/up projection in a decode step: a stream over the touched experts' weights
        {"name": "grouped_swiglu_t16", "op": "grouped", "epi": "swiglu", "t": 16, "e": 64, "top": 8, "n": 2048,
         "k": 2048},
        # the same over a 4096-token prefill chunk: about 512 rows an expert, none equal
        {"name": "grouped_swiglu_t4096", "op": "grouped", "epi": "swiglu", "t": 4096, "e": 64, "top": 8, "n": 2048,
         "k": 2048},
        # routing of a decode step: sigmoid scores, balance bias, 4 of 8 groups, fp32 logits
        {"name": "route_t16", "op": "route", "t": 16, "e": 256, "top": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "renorm": True, "dtype": "fp32", "grad": False},
        # routing of a training step: softmax scores, bf16 logits, forward and backward
        {"name": "route_t8192", "op": "route", "t": 8192, "e": 128, "top": 8, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "renorm": True, "dtype": "bf16", "grad": True},
        # the experts' outputs of a decode step summed into the residual stream
        {"name": "combine_t16", "op": "combine", "t": 16, "top": 8, "h": 2048, "grad": False},
        # a training chunk: the sum and its gradients
        {"name": "combine_t4096", "op": "combine", "t": 4096, "top": 8, "h": 2048, "grad": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "grouped", "grouped", "route", "combine"])
    if op == "quant":
        return {"op": op, "tiling": rng.choice(["row", "row", "column", "block"]), "batch": rng.choice([1, 1, 3]),
                "rows": _log(rng, 1, 8192), "cols": 16 * _log(rng, 2, 512)}
    if op == "gemm":
        kind = rng.choice(["store", "add", "swiglu", "dx", "dw"])
        n = _log(rng, 96, 16384)
        if kind == "swiglu":
            n = max(256, n // 256 * 256)          # gate and up halves of whole 128-row blocks
        elif kind in ("dx", "dw"):
            n = max(16, n // 16 * 16)             # K-major rows are 16-byte aligned
        m = _log(rng, 1, 4096)
        if kind == "dw":
            m = max(16, m // 16 * 16)
        return {"op": op, "kind": kind, "m": m, "n": n, "k": 16 * _log(rng, 4, 512)}
    if op == "grouped":
        e = rng.choice([8, 16, 60, 64, 128])
        epi = rng.choice(["store", "swiglu"])
        n = 256 * rng.randint(1, 8) if epi == "swiglu" else _log(rng, 64, 2048)
        return {"op": op, "epi": epi, "t": _log(rng, 1, 4096), "e": e, "top": rng.randint(1, 8), "n": n,
                "k": 16 * _log(rng, 8, 128)}
    if op == "route":
        e, groups = rng.choice([(8, 1), (60, 1), (64, 1), (96, 4), (128, 1), (160, 8), (256, 8), (512, 1)])
        return {"op": op, "t": _log(rng, 1, 16384), "e": e, "top": rng.randint(1, 8),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "top_groups": max(1, groups // 2), "renorm": rng.random() < 0.7,
                "dtype": rng.choice(["fp32", "bf16"]), "grad": rng.random() < 0.5}
    return {"op": op, "t": _log(rng, 1, 8192), "top": rng.randint(1, 8), "h": _log(rng, 64, 8192),
            "grad": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _quantize(x, tiling):
    """Codes (uint8) and scales of x [.., R, C] (any float type) by the operator's formula."""
    *lead, R, C = x.shape
    br = 1 if tiling == "row" else BLOCK
    bc = 1 if tiling == "column" else BLOCK
    pr, pc = _div_up(R, br) * br - R, _div_up(C, bc) * bc - C
    p = torch.nn.functional.pad(x.float(), (0, pc, 0, pr))
    p = p.reshape(*lead, (R + pr) // br, br, (C + pc) // bc, bc)
    s = p.abs().amax(dim=(-3, -1), keepdim=True)
    s = s / torch.full_like(s, 448.0)      # a division: by a number, torch multiplies with its reciprocal
    q = (p / torch.where(s == 0, torch.ones_like(s), s)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).reshape(*lead, R + pr, C + pc)[..., :R, :C].contiguous()
    s = s.squeeze(-1).squeeze(-2)
    return q, (s.transpose(-1, -2) if tiling == "row" else s).contiguous()     # row scales: [groups, rows]


def _values(q, s, tiling):
    """The fp32 values that codes q and scales s stand for."""
    R, C = q.shape[-2:]
    if tiling == "row":
        s = s.transpose(-1, -2).repeat_interleave(BLOCK, -1)[..., :C]
    elif tiling == "column":
        s = s.repeat_interleave(BLOCK, -2)[..., :R, :]
    else:
        s = s.repeat_interleave(BLOCK, -2)[..., :R, :].repeat_interleave(BLOCK, -1)[..., :C]
    return q.view(torch.float8_e4m3fn).float() * s


def _experts_of(case, gen, dev):
    """Experts [t, top] of a random router, and the rows in expert order."""
    t, e, top = case["t"], case["e"], case["top"]
    # a popularity per expert makes the groups uneven, as trained routers do
    logits = torch.randn(t, e, generator=gen, device=dev) + 0.5 * torch.randn(e, generator=gen, device=dev)
    return torch.topk(logits, top, dim=1).indices


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op = case["op"]

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    if op == "quant":
        shape = (case["rows"], case["cols"])
        shape = (case["batch"],) + shape if case["batch"] > 1 else shape
        return {"op": op, "tiling": case["tiling"], "x": normal(*shape)}
    if op == "gemm":
        m, n, k, kind = case["m"], case["n"], case["k"], case["kind"]
        if kind == "dw":        # dY [tokens, m] in columns of 128 tokens, X [tokens, n] in blocks
            A, sa = _quantize(normal(k, m, std=0.01), "column")
            W, sw = _quantize(normal(k, n), "block")
        elif kind == "dx":      # dY [m, k] in row groups, the forward weight [k, n] as stored
            A, sa = _quantize(normal(m, k, std=0.01), "row")
            W, sw = _quantize(normal(k, n, std=0.02), "block")
        else:
            A, sa = _quantize(normal(m, k), "row")
            W, sw = _quantize(normal(n, k, std=0.02), "block")
        return {"op": op, "kind": kind, "A": A, "sa": sa, "W": W, "sw": sw,
                "res": normal(m, n) if kind == "add" else None}
    if op == "grouped":
        t, e, top, n, k = case["t"], case["e"], case["top"], case["n"], case["k"]
        experts = _experts_of(case, gen, dev).reshape(-1)
        order = torch.sort(experts, stable=True).indices
        counts = torch.bincount(experts, minlength=e)
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        W, sw = _quantize(normal(e, n, k, std=0.02), "block")
        rows = None
        if case["epi"] == "swiglu":    # first product: the tokens' rows, gathered by the router's order
            A, sa = _quantize(normal(t, k), "row")
            rows = (order // top).to(torch.int32)
        else:                          # second product: rows that stand in expert order already
            A, sa = _quantize(normal(t * top, k), "row")
        return {"op": op, "epi": case["epi"], "A": A, "sa": sa, "W": W, "sw": sw, "offsets": offsets, "rows": rows,
                "most": int(counts.max())}
    if op == "route":
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        t, e = case["t"], case["e"]
        return {"op": op, "top": case["top"], "score": case["score"], "groups": case["groups"],
                "top_groups": case["top_groups"], "renorm": case["renorm"], "scale": 2.5,
                "logits": normal(t, e, std=1.5, dtype=dtype),
                "bias": normal(e, std=0.1, dtype=torch.float32) if case["bias"] else None,
                "grad": normal(t, case["top"], dtype=torch.float32) if case["grad"] else None}
    t, top, h = case["t"], case["top"], case["h"]
    slots = torch.randperm(t * top, generator=gen, device=dev).to(torch.int32).reshape(t, top)
    w = torch.rand(t, top, generator=gen, device=dev) + 0.1
    return {"op": op, "y": normal(t * top, h), "w": w / w.sum(1, keepdim=True), "slots": slots, "res": normal(t, h),
            "grad": normal(t, h, std=0.01) if case["grad"] else None}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _plain_gemm(s):
    kind = s["kind"]
    if kind == "dw":
        y = _values(s["A"], s["sa"], "column").t() @ _values(s["W"], s["sw"], "block")
    elif kind == "dx":
        y = _values(s["A"], s["sa"], "row") @ _values(s["W"], s["sw"], "block")
    else:
        y = _values(s["A"], s["sa"], "row") @ _values(s["W"], s["sw"], "block").t()
    if kind == "add":
        y = y + s["res"].float()
    elif kind == "swiglu":
        g, u = y.chunk(2, dim=1)
        y = g / (1 + torch.exp(-g)) * u
    return y.to(torch.bfloat16)


def _plain_grouped(s):
    off = s["offsets"].long()
    a = _values(s["A"], s["sa"], "row")
    if s["rows"] is not None:
        a = a[s["rows"].long()]
    pos = (off[:-1, None] + torch.arange(s["most"], device=off.device)).clamp(max=a.shape[0] - 1)
    y = torch.bmm(a[pos], _values(s["W"], s["sw"], "block").transpose(1, 2).contiguous())
    r = torch.arange(a.shape[0], device=off.device)
    expert = torch.searchsorted(off[1:].contiguous(), r, right=True)
    y = y[expert, r - off[expert]]
    if s["epi"] == "swiglu":
        g, u = y.chunk(2, dim=1)
        y = g / (1 + torch.exp(-g)) * u
    return y.to(torch.bfloat16)


def _plain_route(s):
    # scores and choices in 64 bits: experts next to the border of the top-k must not swap
    x, top = s["logits"].double(), s["top"]
    T, E = x.shape
    if s["score"] == "softmax":
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-x))
    c = p if s["bias"] is None else p + s["bias"].double()
    if s["groups"] > 1:
        by = c.reshape(T, s["groups"], -1)
        g = torch.sort(by, dim=2, descending=True).values[:, :, :2].sum(2)
        best = torch.sort(g, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        kept = torch.zeros_like(g).scatter(1, best, 1.0)
        c = torch.where(kept[:, :, None] > 0, by, torch.full_like(by, -math.inf)).reshape(T, E)
    experts = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :top]
    chosen = p.gather(1, experts)
    total = chosen.sum(1, keepdim=True)
    w = s["scale"] * (chosen / total if s["renorm"] else chosen)
    flat = experts.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    ends = torch.searchsorted(flat[order].contiguous(), torch.arange(E, device=x.device), right=True)
    offsets = torch.cat([ends.new_zeros(1), ends])
    slots = torch.empty_like(order).scatter(0, order, torch.arange(order.numel(), device=x.device)).reshape(T, top)
    out = {"weights": w.float(), "experts": experts.to(torch.int32), "offsets": offsets.to(torch.int32),
           "rows": (order // top).to(torch.int32), "slots": slots.to(torch.int32)}
    if s["grad"] is not None:
        g = s["scale"] * s["grad"].double()
        if s["renorm"]:
            g = (g - (g * chosen).sum(1, keepdim=True) / total) / total
        if s["score"] == "softmax":
            d = torch.zeros_like(p).scatter(1, experts, g * chosen) - p * (g * chosen).sum(1, keepdim=True)
        else:
            d = torch.zeros_like(p).scatter(1, experts, g * chosen * (1 - chosen))
        out["grad_logits"] = d.to(s["logits"].dtype)
    return out


def _plain_combine(s):
    y = s["y"].float()[s["slots"].long()]                        # [t, top, h]
    out = {"out": ((s["w"][:, :, None] * y).sum(1) + s["res"].float()).to(torch.bfloat16)}
    if s["grad"] is not None:
        g = s["grad"].float()
        out["grad_weights"] = (g[:, None, :] * y).sum(2)
        dy = (s["w"][:, :, None] * g[:, None, :]).reshape(-1, g.shape[1]).to(torch.bfloat16)
        out["grad_y"] = torch.empty_like(s["y"]).index_copy(0, s["slots"].reshape(-1).long(), dy)
    return out


def _own(s):
    import scaled_precision_gemm_amd as spg

    op = s["op"]
    if op == "quant":
        q, scale = spg.quantize_block128(s["x"], s["tiling"])
        return {"values": q.view(torch.float8_e4m3fn), "scale": scale}
    if op == "gemm":
        kind = s["kind"]
        return spg.gemm_scaled(s["A"], s["sa"], s["W"], s["sw"], kind if kind in ("add", "swiglu") else "store",
                               residual=s["res"], fmt="e4m3_block128", a_kmajor=kind == "dw",
                               w_kmajor=kind in ("dx", "dw"))
    if op == "grouped":
        return spg.gemm_grouped(s["A"], s["sa"], s["W"], s["sw"], s["offsets"], s["epi"], rows=s["rows"])
    if op == "route":
        how = {"score": s["score"], "renormalize": s["renorm"], "scale": s["scale"]}
        r = spg.expert_route(s["logits"], s["top"], bias=s["bias"], groups=s["groups"], top_groups=s["top_groups"],
                             **how)
        out = {"weights": r.weights, "experts": r.experts, "offsets": r.offsets, "rows": r.rows, "slots": r.slots}
        if s["grad"] is not None:
            out["grad_logits"] = spg.expert_route_backward(s["grad"], s["logits"], r.experts, **how)
        return out
    out = {"out": spg.expert_combine(s["y"], s["w"], s["slots"], residual=s["res"])}
    if s["grad"] is not None:
        out["grad_y"], out["grad_weights"] = spg.expert_combine_backward(s["grad"], s["y"], s["w"], s["slots"])
    return out


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "quant":
        q, scale = _quantize(state["x"], state["tiling"])
        return {"values": q.view(torch.float8_e4m3fn), "scale": scale}
    if op == "gemm":
        return _plain_gemm(state)
    if op == "grouped":
        return _plain_grouped(state)
    if op == "route":
        return _plain_route(state)
    return _plain_combine(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "quant":
        n = case["batch"] * case["rows"] * case["cols"]
        per = BLOCK * BLOCK if case["tiling"] == "block" else BLOCK
        return {"bytes": 3 * n + 4 * n / per, "flops": 2 * n}
    if op == "gemm":
        m, n, k, kind = case["m"], case["n"], case["k"], case["kind"]
        g = _div_up(k, BLOCK)
        read = m * k + n * k + 4 * g * m + 4 * g * _div_up(n, BLOCK) + (2 * m * n if kind == "add" else 0)
        return {"bytes": read + 2 * m * (n // 2 if kind == "swiglu" else n), "flops": 2 * m * n * k}
    if op == "grouped":
        t, e, top, n, k = case["t"], case["e"], case["top"], case["n"], case["k"]
        touched = e * (1 - (1 - min(1.0, top / e)) ** t)       # experts with a row, expected
        rows = t * top
        a = (t if case["epi"] == "swiglu" else rows) * (k + 4 * _div_up(k, BLOCK))
        w = touched * (n * k + 4 * _div_up(n, BLOCK) * _div_up(k, BLOCK))
        return {"bytes": a + w + 2 * rows * (n // 2 if case["epi"] == "swiglu" else n), "flops": 2 * rows * n * k}
    if op == "route":
        t, e, top = case["t"], case["e"], case["top"]
        size = 2 if case["dtype"] == "bf16" else 4
        grad = t * (2 * e * size + 8 * top) if case["grad"] else 0
        return {"bytes": t * (e * size + 16 * top) + 4 * e + grad, "flops": 20 * t * e * (2 if case["grad"] else 1)}
    t, top, h = case["t"], case["top"], case["h"]
    grad = t * (2 * h + 4 * top * h + 8 * top + 4 * top) if case["grad"] else 0
    return {"bytes": t * (2 * top * h + 4 * h + 8 * top) + grad, "flops": t * top * h * (6 if case["grad"] else 2)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _table():
    """The 256 E4M3 values: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    mag = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    mag[(c & 127) == 127] = np.nan
    return np.where(c & 128, -mag, mag)


def _exact_values(q, s, axis_rows, axis_cols):
    """codes * scale in 64 bits; scale index = (row // axis_rows, col // axis_cols)."""
    v = torch.from_numpy(_table()).to(q.device)[q.long()]
    r = torch.arange(q.shape[-2], device=q.device) // axis_rows
    c = torch.arange(q.shape[-1], device=q.device) // axis_cols
    v *= s.double()[..., r[:, None], c[None, :]]
    return v


def _exact_silu_mul(y):
    n = y.shape[-1] // 2
    return y[..., :n] / (1 + torch.exp(-y[..., :n])) * y[..., n:]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quant":
        x = s["x"].double()
        R, C = x.shape[-2:]
        br = 1 if s["tiling"] == "row" else BLOCK
        bc = 1 if s["tiling"] == "column" else BLOCK
        gr, gc = _div_up(R, br), _div_up(C, bc)
        amax = torch.zeros(*x.shape[:-2], gr * br, gc * bc, dtype=torch.float64, device=x.device)
        amax[..., :R, :C] = x.abs()
        amax = amax.unflatten(-1, (gc, bc)).amax(-1).unflatten(-2, (gr, br)).amax(-2)
        scale = (amax / 448).float().double()                      # the scale is a binary32 number
        r = torch.arange(R, device=x.device) // br
        c = torch.arange(C, device=x.device) // bc
        d = scale[..., r[:, None], c[None, :]]
        v = torch.where(d > 0, x / d, torch.zeros_like(x)).float().double()   # so is the quotient
        step = torch.exp2(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent.double() - 4)
        v = (torch.round(v / step) * step).clamp(-448, 448)
        return {"values": v, "scale": scale.transpose(-1, -2).contiguous() if br == 1 else scale}
    if op == "gemm":
        kind = s["kind"]
        if kind == "dw":
            a = _exact_values(s["A"], s["sa"], BLOCK, 1).t()
        else:
            a = _exact_values(s["A"], s["sa"].t(), 1, BLOCK)
        w = _exact_values(s["W"], s["sw"], BLOCK, BLOCK)
        y = torch.matmul(a, w if kind in ("dx", "dw") else w.t())
        return y + s["res"].double() if kind == "add" else _exact_silu_mul(y) if kind == "swiglu" else y
    if op == "grouped":
        a = _exact_values(s["A"], s["sa"].t(), 1, BLOCK)
        off = s["offsets"].tolist()
        n = case["n"]
        y = torch.zeros(off[-1], n, dtype=torch.float64, device=a.device)
        for e in range(len(off) - 1):
            if off[e + 1] > off[e]:
                rows = torch.arange(off[e], off[e + 1], device=a.device)
                rows = rows if s["rows"] is None else s["rows"].long()[rows]
                y[off[e]:off[e + 1]] = a[rows] @ _exact_values(s["W"][e], s["sw"][e], BLOCK, BLOCK).t()
        return _exact_silu_mul(y) if s["epi"] == "swiglu" else y
    if op == "route":
        x = s["logits"].double().cpu().numpy()
        T, E = x.shape
        top, tg, ng = s["top"], s["top_groups"], s["groups"]
        if s["score"] == "softmax":
            p = np.exp(x - x.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
        else:
            p = 1.0 / (1.0 + np.exp(-x))
        c = p + (0.0 if s["bias"] is None else s["bias"].double().cpu().numpy())
        if ng > 1:
            part = c.reshape(T, ng, E // ng)
            g = np.sort(part, axis=2)[:, :, -2:].sum(2)
            keep = np.zeros((T, ng), dtype=bool)
            np.put_along_axis(keep, np.argsort(-g, axis=1, kind="stable")[:, :tg], True, axis=1)
            c = np.where(np.repeat(keep, E // ng, axis=1), c, -np.inf)
        ids = np.argsort(-c, axis=1, kind="stable")[:, :top]
        pc = np.take_along_axis(p, ids, 1)
        z = pc.sum(1, keepdims=True) if s["renorm"] else np.ones((T, 1))
        w = s["scale"] * pc / z
        order = np.argsort(ids.reshape(-1), kind="stable")
        slots = np.empty(T * top, dtype=np.int64)
        slots[order] = np.arange(T * top)
        offsets = np.concatenate([[0], np.cumsum(np.bincount(ids.reshape(-1), minlength=E))])
        out = {"weights": w, "experts": ids, "offsets": offsets, "rows": order // top, "slots": slots.reshape(T, top)}
        if s["grad"] is not None:
            g = s["grad"].double().cpu().numpy()
            if s["renorm"]:                     # dw_i/dp_j = scale (delta_ij - p_i / z) / z
                gp = s["scale"] * (g - (g * pc / z).sum(1, keepdims=True)) / z
            else:
                gp = s["scale"] * g
            gx = np.zeros_like(p)
            if s["score"] == "softmax":
                np.put_along_axis(gx, ids, gp, 1)
                gx = p * (gx - (gp * pc).sum(1, keepdims=True))
            else:
                np.put_along_axis(gx, ids, gp * pc * (1 - pc), 1)
            out["grad_logits"] = gx
        return out
    y, w, idx = s["y"].double(), s["w"].double(), s["slots"].long()
    acc = s["res"].double()
    for j in range(idx.shape[1]):
        acc = acc + w[:, j:j + 1] * y[idx[:, j]]
    out = {"out": acc}
    if s["grad"] is not None:
        g = s["grad"].double()
        dy = torch.zeros_like(y)
        dw = torch.zeros_like(w)
        for j in range(idx.shape[1]):
            dw[:, j] = (g * y[idx[:, j]]).sum(1)
            dy[idx[:, j]] = w[:, j:j + 1] * g
        out["grad_weights"], out["grad_y"] = dw, dy
    return out
