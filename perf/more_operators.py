"""Measured cases of the norms before the products, of the experts' weight gradients and of gradient clipping.

Three operators, each in a plain form (elementary torch operations, `own` false) and as the calls a
user makes of the package (`own` true):

* norm     `rms_norm` and `rms_norm_backward`: h = x + residual, y = h / rms(h) * weight, leaving as
           bf16 or as E4M3 codes with fp32 scales (per row, or per 128 elements of a row) for the
           product that follows; and the gradients of both
* dw       `gemm_grouped_dw`: the weight gradient of every expert's product, dY^T X over the rows
           of that expert, from bf16 operands in the rows' order of the router
* clip     `clip_gradients`: the norm over all gradients of a step, and the gradients scaled to at
           most a given norm

Sizes are those of this repository's workloads (5120- and 2048-wide hidden states, heads of 128,
17408-wide gated layers, 16 / 1111 / 4000 / 4096 tokens) and generic expert counts.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
EPS = 1e-6


def _div_up(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the norm before a single sequence's next linear layer: launch latency
        {"name": "norm_t1", "op": "norm", "rows": 1, "cols": 5120, "out": "e4m3_row", "residual": True, "w": "bf16",
         "offset": 0.0, "normed": False, "grad": False},
        # the norm before the experts of a decode step of 16 sequences, 128-element scales
        {"name": "norm_t16", "op": "norm", "rows": 16, "cols": 2048, "out": "e4m3_block128", "residual": True,
         "w": "bf16", "offset": 0.0, "normed": False, "grad": False},
        # the norm before a dense layer's projection over a 4096-token prefill chunk
        {"name": "norm_t4096", "op": "norm", "rows": 4096, "cols": 5120, "out": "e4m3_row", "residual": True,
         "w": "bf16", "offset": 0.0, "normed": False, "grad": False},
        # query heads of a ragged chunk of 1111 tokens, 40 heads of 128 each: many short rows
        {"name": "norm_heads_t1111", "op": "norm", "rows": 44440, "cols": 128, "out": "bf16", "residual": False,
         "w": "bf16", "offset": 0.0, "normed": False, "grad": False},
        # a training chunk before an experts' layer: 8 bits for the products, bf16 for the router and the weight
        # gradients, and the gradients with the residual stream's
        {"name": "norm_train_t4096", "op": "norm", "rows": 4096, "cols": 2048, "out": "e4m3_block128",
         "residual": True, "w": "fp32", "offset": 0.0, "normed": True, "grad": True},
        # the weight gradients of a few small experts over 64 tokens: launch latency
        {"name": "dw_t64", "op": "dw", "t": 64, "e": 8, "top": 2, "n": 512, "k": 256, "gather": True, "out": "bf16",
         "add": False, "drop": False},
        # the experts' gate/up weight gradients over a 4096-token chunk: about 512 rows an expert, none equal,
        # tokens gathered by the router's order
        {"name": "dw_gate_up_t4096", "op": "dw", "t": 4096, "e": 64, "top": 8, "n": 2048, "k": 2048, "gather": True,
         "out": "bf16", "add": False, "drop": False},
        # the down projections' gradients of the same chunk, added to those of earlier chunks in fp32; a tenth of
        # the places have no expert
        {"name": "dw_down_add_t4096", "op": "dw", "t": 4096, "e": 64, "top": 8, "n": 2048, "k": 1024,
         "gather": False, "out": "fp32", "add": True, "drop": True},
        # the weight gradient of a dense 2048 -> 4096 projection over 4000 tokens (one expert with every row)
        {"name": "dw_dense_t4000", "op": "dw", "t": 4000, "e": 1, "top": 1, "n": 4096, "k": 2048, "gather": False,
         "out": "fp32", "add": False, "drop": False},
        # the gradients of 200 norm weights and biases of a deep model: many tensors, little data
        {"name": "clip_small", "op": "clip", "count": 200, "least": 128, "most": 17408, "out": "fp32"},
        # the bf16 gradients of a dense gated layer (2 x 17408 x 5120 and 5120 x 17408) and of what is around it
        {"name": "clip_layer", "op": "clip", "count": 9, "least": 2048, "most": 178257920, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "dw", "dw", "clip"])
    if op == "norm":
        out = rng.choice(["bf16", "e4m3_row", "e4m3_block128"])
        cols = _log(rng, 64, 16384) if out == "bf16" else 16 * _log(rng, 4, 1024)
        rows = min(_log(rng, 1, 65536), 4096 * 5120 // cols)
        grad = rng.random() < 0.4 and rows * cols <= 4096 * 2048
        return {"op": op, "rows": rows, "cols": cols, "out": out, "residual": rng.random() < 0.6,
                "w": rng.choice(["bf16", "fp32"]), "offset": rng.choice([0.0, 0.0, 1.0]),
                "normed": out != "bf16" and rng.random() < 0.4, "grad": grad}
    if op == "dw":
        e = rng.choice([1, 3, 8, 60, 64, 128])
        top = 1 if e == 1 else rng.randint(1, min(e, 8))
        n, k = 8 * _log(rng, 4, 256), 8 * _log(rng, 4, 256)
        if e > 64:
            n = max(32, n // 16 * 8)
        return {"op": op, "t": _log(rng, 1, 4096), "e": e, "top": top, "n": n, "k": k, "gather": rng.random() < 0.5,
                "out": rng.choice(["bf16", "fp32"]), "add": rng.random() < 0.4, "drop": rng.random() < 0.3}
    count = _log(rng, 1, 400)
    most = _log(rng, 16, 1 << 26)
    return {"op": op, "count": count, "least": max(1, most // _log(rng, 1, 4096)),
            "most": max(1, min(most, (1 << 28) // count)), "out": rng.choice(["bf16", "fp32"])}


def _sizes(case):
    """Elements of the tensors of a clip case: spread evenly over their logarithm, none round but the ends."""
    n, lo, hi = case["count"], math.log(min(case["least"], case["most"])), math.log(case["most"])
    sizes = [int(round(math.exp(lo + (hi - lo) * (i / max(1, n - 1))))) for i in range(n)]
    if case["least"] == 2048 and case["most"] == 34816 * 5120:      # the dense gated layer
        sizes = [34816 * 5120, 17408 * 5120, 7168 * 5120, 6144 * 5120, 5120, 5120, 7168, 2048, 2048]
    return sizes


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op = case["op"]

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    if op == "norm":
        r, c = case["rows"], case["cols"]
        # a hidden state: channels of unequal size, a few of them far larger, as residual streams have
        channel = torch.exp(0.5 * torch.randn(c, generator=gen, device=dev))
        channel[:: max(1, c // 3)] *= 20.0
        x = (torch.randn(r, c, generator=gen, device=dev) * channel).to(torch.bfloat16)
        wt = torch.float32 if case["w"] == "fp32" else torch.bfloat16
        weight = normal(c, std=0.2, dtype=torch.float32) + (0.0 if case["offset"] else 1.0)
        return {"op": op, "out": case["out"], "x": x, "residual": normal(r, c) if case["residual"] else None,
                "weight": weight.to(wt), "offset": case["offset"], "normed": case["normed"],
                "dy": normal(r, c, std=0.01) if case["grad"] else None,
                "dres": normal(r, c, std=0.01) if case["grad"] and case["residual"] else None}
    if op == "dw":
        t, e, top, n, k = case["t"], case["e"], case["top"], case["n"], case["k"]
        # a popularity per expert makes the groups uneven, as trained routers do
        logits = torch.randn(t, e, generator=gen, device=dev) + 0.5 * torch.randn(e, generator=gen, device=dev)
        flat = torch.topk(logits, top, dim=1).indices.reshape(-1)
        if case["drop"]:         # places without an expert come behind the last expert's rows
            flat = torch.where(torch.rand(t * top, generator=gen, device=dev) < 0.1, torch.full_like(flat, e), flat)
        order = torch.sort(flat, stable=True).indices
        counts = torch.bincount(flat, minlength=e + 1)[:e]
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        rows = None
        if case["gather"]:
            rows = (order // top).to(torch.int32)
            rows[int(offsets[-1]):] = -1
        dt = torch.float32 if case["out"] == "fp32" else torch.bfloat16
        return {"op": op, "dy": normal(t * top, n, std=0.01), "x": normal(t if case["gather"] else t * top, k),
                "offsets": offsets, "rows": rows, "most": max(1, int(counts.max())), "dtype": dt,
                "add": normal(e, n, k, std=0.1, dtype=dt) if case["add"] else None}
    sizes = _sizes(case)
    at, end = [], 0
    for s in sizes:              # tensors of one flat buffer, each on a line of its own
        at.append(end)
        end += _div_up(s, 128) * 128
    dt = torch.float32 if case["out"] == "fp32" else torch.bfloat16
    flat = torch.randn(end, generator=gen, device=dev).mul_(0.01).to(dt)
    to = torch.zeros(end, dtype=dt, device=dev)
    # gradients a half over the limit, as in the steps that clipping is for
    limit = 0.01 * math.sqrt(sum(sizes)) / 1.5
    return {"op": op, "grads": [flat[a:a + s] for a, s in zip(at, sizes)], "max_norm": limit, "to": to,
            "outs": [to[a:a + s] for a, s in zip(at, sizes)]}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _plain_quantize(y, how):
    R, C = y.shape
    size = C if how == "e4m3_row" else BLOCK
    p = torch.nn.functional.pad(y, (0, _div_up(C, size) * size - C)).reshape(R, -1, size)
    s = p.abs().amax(dim=2, keepdim=True)
    s = s / torch.full_like(s, 448.0)      # a division: by a number, torch multiplies with its reciprocal
    q = (p / torch.where(s == 0, torch.ones_like(s), s)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).reshape(R, -1)[:, :C].contiguous().view(torch.float8_e4m3fn)
    s = s.squeeze(2)
    return q, (s.reshape(-1) if how == "e4m3_row" else s.t().contiguous())


def _plain_norm(s):
    x = s["x"]
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(torch.bfloat16)
    hf, w = h.float(), s["weight"].float() + s["offset"]
    rstd = 1 / torch.sqrt((hf * hf).mean(1) + EPS)
    y = hf * rstd[:, None] * w
    out = {}
    if s["residual"] is not None:
        out["h"] = h
    if s["out"] == "bf16":
        out["y"] = y.to(torch.bfloat16)
    else:
        out["values"], out["scale"] = _plain_quantize(y, s["out"])
        if s["normed"]:
            out["normed"] = y.to(torch.bfloat16)
    if s["dy"] is not None:
        xh, dy = hf * rstd[:, None], s["dy"].float()
        g = dy * w
        dx = rstd[:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        out["grad_x"], out["grad_weight"] = dx.to(torch.bfloat16), (dy * xh).sum(0)
    return out


def _plain_dw(s):
    off, R = s["offsets"].long(), s["dy"].shape[0]
    pos = off[:-1, None] + torch.arange(s["most"], device=off.device)
    there = (pos < off[1:, None])[:, :, None]
    pos = pos.clamp(max=R - 1)
    src = pos if s["rows"] is None else s["rows"].long()[pos].clamp(min=0)
    a = torch.where(there, s["dy"][pos].float(), 0.0).transpose(1, 2).contiguous()
    y = torch.bmm(a, torch.where(there, s["x"][src].float(), 0.0))
    if s["add"] is not None:
        y = y + s["add"].float()
    return y.to(s["dtype"])


def _plain_clip(s):
    # 64-bit sums: 10^8 squares added in 32 bits lose the last ones
    n = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
    c = torch.where(n > s["max_norm"], s["max_norm"] / n, torch.ones_like(n)).float()
    [o.copy_(g.float() * c) for o, g in zip(s["outs"], s["grads"])]
    return {"norm": n.float().reshape(1), "grads": s["to"]}


def _own(s):
    import scaled_precision_gemm_amd as spg

    op = s["op"]
    if op == "norm":
        grad = s["dy"] is not None
        r = spg.rms_norm(s["x"], s["weight"], residual=s["residual"], output=s["out"], eps=EPS,
                         weight_offset=s["offset"], normed=s["normed"], rstd=grad)
        out = {}
        if s["residual"] is not None:
            out["h"] = r.h
        if s["out"] == "bf16":
            out["y"] = r.out
        else:
            out["values"], out["scale"] = r.out.view(torch.float8_e4m3fn), r.scale
            if s["normed"]:
                out["normed"] = r.normed
        if grad:
            h = s["x"] if s["residual"] is None else r.h
            out["grad_x"], out["grad_weight"] = spg.rms_norm_backward(s["dy"], h, s["weight"], r.rstd,
                                                                      grad_residual=s["dres"], weight_offset=s["offset"])
        return out
    if op == "dw":
        return spg.gemm_grouped_dw(s["dy"], s["x"], s["offsets"], rows=s["rows"], add=s["add"], dtype=s["dtype"])
    return {"norm": spg.clip_gradients(s["grads"], s["max_norm"], out=s["outs"]), "grads": s["to"]}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    return _plain_norm(state) if op == "norm" else _plain_dw(state) if op == "dw" else _plain_clip(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        r, c = case["rows"], case["cols"]
        scales = {"bf16": 0, "e4m3_row": 4 * r, "e4m3_block128": 4 * r * _div_up(c, BLOCK)}[case["out"]]
        size = 4 if case["w"] == "fp32" else 2
        b = r * c * (2 + (4 if case["residual"] else 0) + (2 if case["out"] == "bf16" else 1) + (2 if case["normed"] else 0))
        b += scales + size * c
        if case["grad"]:
            b += r * c * (6 + (2 if case["residual"] else 0)) + (size + 4) * c + 8 * r
        return {"bytes": b, "flops": r * c * (8 + (12 if case["grad"] else 0))}
    if op == "dw":
        t, e, top, n, k = case["t"], case["e"], case["top"], case["n"], case["k"]
        rows = t * top * (0.9 if case["drop"] else 1.0)
        size = 4 if case["out"] == "fp32" else 2
        read = 2 * rows * n + 2 * (t if case["gather"] else rows) * k + 4 * (e + 1) + (4 * rows if case["gather"] else 0)
        return {"bytes": read + e * n * k * size * (2 if case["add"] else 1), "flops": 2 * rows * n * k}
    n = sum(_sizes(case))
    return {"bytes": 2 * n * (4 if case["out"] == "fp32" else 2), "flops": 3 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "norm":
        h = s["x"].double()
        out = {}
        if s["residual"] is not None:
            # the residual stream is a bf16 tensor: the norm is of what it holds
            h = torch.add(h, s["residual"].double())
            e = torch.frexp(h).exponent.double() - 8
            h = torch.round(h * torch.exp2(-e)) * torch.exp2(e)
            out["h"] = h
        C = h.shape[1]
        w = s["weight"].double() + s["offset"]
        inv = torch.rsqrt(h.square().sum(1, keepdim=True) / C + EPS)
        y = h * inv * w
        if s["out"] == "bf16":
            out["y"] = y
        else:
            size = C if s["out"] == "e4m3_row" else BLOCK
            groups = _div_up(C, size)
            amax = torch.stack([y[:, g * size:(g + 1) * size].abs().amax(1) for g in range(groups)], 1) / 448
            out["scale"] = amax[:, 0].contiguous() if s["out"] == "e4m3_row" else amax.t().contiguous()
            v = y / torch.where(amax > 0, amax, torch.ones_like(amax)).repeat_interleave(size, 1)[:, :C]
            step = torch.exp2(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent.double() - 4)
            out["values"] = (torch.round(v / step) * step).clamp(-448, 448)
            if s["normed"]:
                out["normed"] = y
        if s["dy"] is not None:
            d = s["dy"].double()
            # y_i = h_i inv w_i and d inv / d h_j = -inv^3 h_j / C
            dot = (d * w * h).sum(1, keepdim=True)
            gx = d * w * inv - h * dot * inv ** 3 / C
            out["grad_x"] = gx if s["dres"] is None else gx + s["dres"].double()
            out["grad_weight"] = torch.mv((h * inv * d).t(), torch.ones(h.shape[0], dtype=h.dtype, device=h.device))
        return out
    if op == "dw":
        off = s["offsets"].tolist()
        E, n, k = len(off) - 1, s["dy"].shape[1], s["x"].shape[1]
        y = torch.zeros(E, n, k, dtype=torch.float64, device=s["dy"].device)
        for e in range(E):
            if off[e + 1] > off[e]:
                at = torch.arange(off[e], off[e + 1], device=y.device)
                src = at if s["rows"] is None else s["rows"].long()[at]
                y[e] = torch.matmul(s["dy"][at].double().t(), s["x"][src].double())
            if s["add"] is not None:
                y[e] += s["add"][e].double()
        return y
    total = math.sqrt(math.fsum(float(torch.dot(g.double(), g.double())) for g in s["grads"]))
    factor = min(1.0, s["max_norm"] / total)
    to = torch.zeros(s["to"].numel(), dtype=torch.float64, device=s["to"].device)
    for g, o in zip(s["grads"], s["outs"]):
        a = o.storage_offset()
        to[a:a + g.numel()] = g.double() * factor
    return {"norm": np.array([total]), "grads": to}
