"""The norm, the experts' weight gradients and the clipping as a training step
uses them: a pre-norm experts' layer forward and backward, from the calls of
the package and the plain activation between its products.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF = 2.0 ** -24


@pytest.fixture(scope="module")
def spg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import scaled_precision_gemm_amd as m
    return m


def rand(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def weights(spg, E, H, I):
    wn = (1 + rand((H,), 1, 0.1, F32)).to(BF)
    gu, dn = rand((E, 2 * I, H), 2, 0.05), rand((E, H, I), 3, 0.05)
    q = [spg.quantize_block128(w, "block") for w in (gu, dn)]
    # the codes of the same blocks, transposed, for the gradients of the inputs
    t = [(c.transpose(1, 2).contiguous(), s.transpose(1, 2).contiguous()) for c, s in q]
    return {"norm": wn, "router": rand((E, H), 4, 0.3, F32), "gate_up": q[0], "down": q[1], "gate_up_t": t[0], "down_t": t[1]}


def swiglu(z):
    g, u = z.float().chunk(2, dim=1)
    return (g * torch.sigmoid(g) * u).to(BF)


def swiglu_backward(dh, z):
    (g, u), d = z.float().chunk(2, dim=1), dh.float()
    s = torch.sigmoid(g)
    return torch.cat([d * u * (s + g * s * (1 - s)), d * g * s], 1).to(BF)


def step(spg, W, x, res, dout, top, limit):
    T = x.shape[0]
    f = spg.rms_norm(x, W["norm"], residual=res, output="e4m3_block128", normed=True, rstd=True)
    logits = (f.normed.float()[:, None, :] * W["router"]).sum(2)
    r = spg.expert_route(logits, top)
    z = spg.gemm_grouped(f.out, f.scale, *W["gate_up"], r.offsets, rows=r.rows)
    h = swiglu(z)
    y = spg.gemm_grouped(*spg.quantize_block128(h), *W["down"], r.offsets)
    out = spg.expert_combine(y, r.weights, r.slots, residual=f.h)

    dy, dweights = spg.expert_combine_backward(dout, y, r.weights, r.slots)
    ddown = spg.gemm_grouped_dw(dy, h, r.offsets)
    dh = spg.gemm_grouped(*spg.quantize_block128(dy), *W["down_t"], r.offsets)
    dz = swiglu_backward(dh, z)
    dgate_up = spg.gemm_grouped_dw(dz, f.normed, r.offsets, rows=r.rows, dtype=F32)
    drows = spg.gemm_grouped(*spg.quantize_block128(dz), *W["gate_up_t"], r.offsets)
    dn = spg.expert_combine(drows, torch.ones_like(r.weights), r.slots)
    dlogits = spg.expert_route_backward(dweights, logits, r.experts)
    drouter = (dlogits[:, :, None] * f.normed.float()[:, None, :]).sum(0)
    dn = (dn.float() + (dlogits[:, :, None] * W["router"]).sum(1)).to(BF)
    dx, dnorm = spg.rms_norm_backward(dn, f.h, W["norm"], f.rstd, grad_residual=dout)
    grads = [ddown, dgate_up, drouter.contiguous(), dnorm]
    before = [g.clone() for g in grads]
    total = spg.clip_gradients(grads, limit)
    return {"f": f, "r": r, "z": z, "h": h, "y": y, "out": out, "dy": dy, "dz": dz, "dn": dn, "dx": dx, "before": before,
            "grads": grads, "total": total}


@pytest.mark.parametrize("T,E,top,H,I", [(1, 4, 2, 256, 128), (150, 8, 2, 272, 128), (700, 16, 4, 512, 256)])
def test_step(spg, T, E, top, H, I):
    W = weights(spg, E, H, I)
    x, res, dout = rand((T, H), 10), rand((T, H), 11), rand((T, H), 12, 0.1)
    s = step(spg, W, x, res, dout, top, 1e-3)
    f, r = s["f"], s["r"]

    # the norm, of what the stream holds, in bf16 for the router and the weight gradients
    h = (x.float() + res.float()).to(BF)
    assert torch.equal(f.h, h)
    hd = h.double()
    rstd = 1 / torch.sqrt(hd.square().mean(1) + 1e-6)
    y = hd * rstd[:, None] * W["norm"].double()
    assert bool(((f.normed.double() - y).abs() <= (2.0 ** -8 + 5 * HALF) * y.abs() + 2.0 ** -134).all())

    # the weight gradients, from the step's own operands: fp32 sums of exact products, one rounding
    off, rows = r.offsets.tolist(), r.rows.long()
    for dw, dY, X in ((s["before"][0], s["dy"], s["h"]), (s["before"][1], s["dz"], f.normed[rows])):
        for e in range(E):
            a, b = dY[off[e]:off[e + 1]].double(), X[off[e]:off[e + 1]].double()
            want, S = torch.matmul(a.t(), b), torch.matmul(a.abs().t(), b.abs())
            half = 2.0 ** -8 if dw.dtype == BF else HALF
            n = off[e + 1] - off[e] + 2
            assert bool(((dw[e].double() - want).abs() <= half * want.abs() + n * 2.0 ** -23 * S + 2.0 ** -134).all())

    # the gradient of the stream, with what reaches it past the norm
    d, n = s["dn"].double(), hd * f.rstd.double()[:, None]
    g = d * W["norm"].double()
    want = f.rstd.double()[:, None] * (g - n * (g * n).mean(1, keepdim=True)) + dout.double()
    S = f.rstd.double()[:, None] * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True)) + dout.double().abs()
    assert bool(((s["dx"].double() - want).abs() <= 2.0 ** -8 * want.abs() + 64 * HALF * S + 2.0 ** -134).all())
    want, S = (d * n).sum(0), (d * n).abs().sum(0)
    assert bool(((s["before"][3].double() - want).abs() <= 97 * HALF * S).all())

    # one norm over all of them, and every gradient scaled by it
    total = math.sqrt(math.fsum(float(t.double().square().sum()) for t in s["before"]))
    assert abs(float(s["total"]) - total) <= 1.01 * HALF * total
    for got, was in zip(s["grads"], s["before"]):
        want = was.double() * min(1.0, 1e-3 / total)
        half = 2.0 ** -8 if got.dtype == BF else 0.0
        assert bool(((got.double() - want).abs() <= (half + 2.01 * HALF) * want.abs() + 2.0 ** -133).all())


def flat(s):
    return [s["out"], s["dx"], s["total"], *s["grads"], *s["before"]]


def test_step_captured_and_on_two_streams(spg):
    T, E, top, H, I = 150, 8, 2, 256, 128
    W = weights(spg, E, H, I)
    x, res, dout = rand((T, H), 10), rand((T, H), 11), rand((T, H), 12, 0.1)
    run = lambda: flat(step(spg, W, x, res, dout, top, 0.5))  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = run()
    for i in range(3):
        x.copy_(rand((T, H), 20 + i))
        dout.copy_(rand((T, H), 30 + i, 0.1))
        want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for p, q in zip(kept, want):
            assert torch.equal(p, q)
    # two steps at once, each on a stream of its own
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for _ in range(2):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run())
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(p, q) for p, q in zip(out, want))
