"""GPU tests of rms_norm and rms_norm_backward against plain implementations
in 64 bits.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = 2.0 ** -24                        # half a step of fp32, relative


@pytest.fixture(scope="module")
def spg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import scaled_precision_gemm_amd as m
    return m


def rand(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def ref_forward(x, weight, residual=None, eps=1e-6, w0=0.0):
    """h as it is stored, rstd and y in fp64."""
    h = x if residual is None else (x.float() + residual.float()).to(BF)
    hd = h.double()
    rstd = 1 / torch.sqrt(hd.square().mean(1) + eps)
    return h, rstd, hd * rstd[:, None] * (weight.double() + w0)


def check_bf16(got, y):
    # y: four roundings to fp32 (rstd, h rstd, weight + w0, the product), then half a step of bf16; its
    # smallest step is 2^-133
    off = (got.double() - y).abs()
    assert bool((off <= (2.0 ** -8 + 5 * HALF) * y.abs() + 2.0 ** -134).all()), float((off / y.abs()).max())


def check_codes(spg, q, scale, y, how):
    R, H = y.shape
    size = H if how == "e4m3_row" else 128
    pad = torch.nn.functional.pad(y, (0, -H % size)).reshape(R, -(-H // size), size)
    want = pad.abs().amax(2) / 448
    s = (scale[:, None] if how == "e4m3_row" else scale.t()).double()
    assert s.shape == want.shape
    # y's four roundings and the division's; scales below fp32's normal range by half their step 2^-149
    assert bool(((s - want).abs() <= 6 * HALF * want + 2.0 ** -149).all())
    # a code is the nearest to y / s but for an error of that quotient: five roundings, and two of its own
    sd = s.repeat_interleave(size, 1)[:, :H]
    v = torch.where(sd > 0, y / torch.where(sd > 0, sd, 1.0), 0.0)
    step = torch.exp2(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent.double() - 4)
    c = q.view(torch.float8_e4m3fn).double()
    assert bool(((c - v).abs() <= step / 2 + 8 * HALF * v.abs()).all())
    assert bool((c.signbit() == y.signbit()).all())


def run(spg, R, H, output, residual=True, wt=BF, w0=0.0, normed=False, seed=0, eps=1e-6, std=1.0, **how):
    x = rand((R, H), seed, std)
    r = rand((R, H), seed + 1, std) if residual else None
    w = (rand((H,), seed + 2, 0.3, F32) + (1.0 - w0)).to(wt)
    got = spg.rms_norm(x, w, residual=r, output=output, eps=eps, weight_offset=w0, normed=normed, rstd=True, **how)
    h, rstd, y = ref_forward(x, w, r, eps, w0)
    if residual:
        assert torch.equal(got.h, h)
    else:
        assert got.h is None
    # the sum in 64 bits, one rounding
    assert bool(((got.rstd.double() - rstd).abs() <= 1.001 * HALF * rstd).all())
    if output == "bf16":
        assert got.scale is None and got.normed is got.out
        check_bf16(got.out, y)
    else:
        check_codes(spg, got.out, got.scale, y, output)
        if normed:
            check_bf16(got.normed, y)
            assert torch.equal(got.normed, spg.rms_norm(x, w, residual=r, eps=eps, weight_offset=w0).out)
        else:
            assert got.normed is None
    return got, x, r, w


# every team and number of vectors, both sides of each border; few rows and many
SIZES = [16, 64, 80, 128, 144, 256, 272, 512, 528, 1024, 1040, 2048, 2064, 4096, 4112, 5120, 6144, 6160, 8192, 8208, 16384, 16400,
         32768]


@pytest.mark.parametrize("output", ["bf16", "e4m3_row", "e4m3_block128"])
@pytest.mark.parametrize("H", SIZES)
def test_sizes(spg, H, output):
    for R in (1, 3, 67):
        run(spg, R, H, output, residual=R != 3, wt=BF if R == 1 else F32, w0=1.0 if R == 67 else 0.0, seed=H + R)
    if H in (2048, 5120, 8192):
        run(spg, 300, H, output, seed=H)


@pytest.mark.parametrize("H", [1, 2, 7, 8, 9, 63, 64, 65, 127, 129, 255, 513, 1023, 1025, 2047, 4099, 8191, 8193, 20001, 32767])
def test_odd_sizes(spg, H):
    for R in (1, 5, 66):
        run(spg, R, H, "bf16", residual=R == 5, wt=F32 if R == 66 else BF, seed=H + R)


@pytest.mark.parametrize("output", ["e4m3_row", "e4m3_block128"])
def test_both_outputs(spg, output):
    run(spg, 19, 1040, output, normed=True)
    run(spg, 300, 5120, output, normed=True, residual=False)


@pytest.mark.parametrize("R", [0, 1, 63, 64, 65, 1000, 44440])
def test_row_counts_of_heads(spg, R):
    run(spg, R, 128, "bf16", residual=False)
    run(spg, R, 96, "e4m3_block128", residual=True)


def test_one_rounding_of_the_stream(spg):
    # the norm is of what h holds: the same call on the stored stream gives the same bits
    for output in ("bf16", "e4m3_row", "e4m3_block128"):
        got, x, r, w = run(spg, 33, 2048, output)
        again = spg.rms_norm(got.h, w, output=output, rstd=True)
        assert torch.equal(got.out, again.out) and torch.equal(got.rstd, again.rstd)
        assert got.scale is None or torch.equal(got.scale, again.scale)
    # one group is one row
    x, w = rand((40, 128), 1), rand((128,), 2)
    a, b = spg.rms_norm(x, w, output="e4m3_row"), spg.rms_norm(x, w, output="e4m3_block128")
    assert torch.equal(a.out, b.out) and torch.equal(a.scale, b.scale[0])


@pytest.mark.parametrize("std", [1e-38, 1e-30, 1e-10, 1e10, 1e19, 1e30, 5e37])
@pytest.mark.parametrize("output", ["bf16", "e4m3_row", "e4m3_block128"])
def test_range(spg, std, output):
    # squares past fp32's range at both ends; with and without the eps that then decides
    run(spg, 9, 1040, output, std=std, residual=False, eps=1e-6)
    if std >= 1e-30:
        run(spg, 9, 1040, output, std=std, residual=False, eps=0.0)


def test_zero_rows_and_eps(spg):
    x = torch.zeros((4, 256), dtype=BF, device="cuda")
    x[1] = rand((256,), 1)
    x[2, 128:] = -0.0
    w = torch.ones(256, dtype=BF, device="cuda")
    for output in ("e4m3_row", "e4m3_block128"):
        g = spg.rms_norm(x, w, output=output, rstd=True)
        h, rstd, y = ref_forward(x, w)
        check_codes(spg, g.out, g.scale, y, output)
        assert bool((g.rstd[[0, 2, 3]] == 1000.0).all())
    g = spg.rms_norm(x, w, eps=0.0, rstd=True)         # 1 / sqrt(0): 0 * inf
    assert bool(torch.isinf(g.rstd[[0, 2, 3]]).all()) and bool(torch.isnan(g.out[[0, 2, 3]]).all())
    check_bf16(g.out[1:2], ref_forward(x[1:2], w, eps=0.0)[2])


@pytest.mark.parametrize("H", [256, 1040, 5120, 16384])
def test_nan_and_infinity_stay_in_their_row(spg, H):
    x, w = rand((70, H), 3), rand((H,), 4)
    y = ref_forward(x, w)[2]
    bad = [5, 40]
    x[5, H // 2] = float("nan")
    x[40, H - 1] = float("inf")
    keep = [i for i in range(70) if i not in bad]
    g = spg.rms_norm(x, w)
    check_bf16(g.out[keep], y[keep])
    assert bool(torch.isnan(g.out[5]).all()) and bool(torch.isnan(g.out[40, H - 1]))
    g = spg.rms_norm(x, w, output="e4m3_row")
    check_codes(spg, g.out[keep], g.scale[keep], y[keep], "e4m3_row")
    assert not bool(torch.isfinite(g.scale[bad]).any())
    g = spg.rms_norm(x, w, output="e4m3_block128")
    check_codes(spg, g.out[keep], g.scale[:, keep].contiguous(), y[keep], "e4m3_block128")
    assert not bool(torch.isfinite(g.scale[:, 5]).any()) and not bool(torch.isfinite(g.scale[-1, 40]))


@pytest.mark.parametrize("w0", [0.0, 1.0])
@pytest.mark.parametrize("output", ["e4m3_row", "e4m3_block128"])
def test_codes_of_fp32_weights(spg, output, w0):
    # products that 32 bits do not hold: zero rows, both ends of the range, weights that overflow y
    for std in (1e-38, 1e-10, 1e19, 5e37):
        run(spg, 9, 1040, output, wt=F32, w0=w0, std=std, residual=False, normed=True)
    for R, H in ((5, 16), (9, 208), (300, 400), (7, 1040), (1100, 2048), (9, 4096), (5, 9216), (3, 20000)):
        run(spg, R, H, output, wt=F32, w0=w0, normed=True, seed=H)
    x, w = rand((6, 2048), 1), rand((2048,), 2, dtype=F32)
    x[2] = 0.0
    x[3, 128:] = -0.0
    y = ref_forward(x, w, None, 1e-6, w0)[2]
    g = spg.rms_norm(x, w, output=output, weight_offset=w0)
    check_codes(spg, g.out, g.scale, y, output)
    big = torch.full((2048,), 3e38, device="cuda")
    g = spg.rms_norm(x, big, output=output, weight_offset=w0)     # some |h rstd| of every other row are over 1.2
    rows = g.scale if output == "e4m3_row" else g.scale.amax(0)
    assert bool(torch.isinf(rows[[0, 1, 4, 5]]).all()) and float(rows[2]) == 0.0


@pytest.mark.parametrize("w0", [0.0, 1.0])
@pytest.mark.parametrize("H", [256, 1040, 2048, 5120, 16384])
def test_nan_and_infinity_with_fp32_weights(spg, H, w0):
    x, w = rand((70, H), 3), rand((H,), 4, dtype=F32)
    y = ref_forward(x, w, None, 1e-6, w0)[2]
    bad = [5, 40]
    x[5, H // 2] = float("nan")
    x[40, H - 1] = float("inf")
    keep = [i for i in range(70) if i not in bad]
    g = spg.rms_norm(x, w, output="e4m3_row", weight_offset=w0)
    check_codes(spg, g.out[keep], g.scale[keep], y[keep], "e4m3_row")
    assert not bool(torch.isfinite(g.scale[bad]).any())
    g = spg.rms_norm(x, w, output="e4m3_block128", weight_offset=w0)
    check_codes(spg, g.out[keep], g.scale[:, keep].contiguous(), y[keep], "e4m3_block128")
    assert not bool(torch.isfinite(g.scale[:, 5]).any()) and not bool(torch.isfinite(g.scale[-1, 40]))
    # a weight that is no number: its group alone
    w[H - 1] = float("nan")
    x = rand((3, H), 5)
    g = spg.rms_norm(x, w, output="e4m3_block128", weight_offset=w0)
    assert not bool(torch.isfinite(g.scale[-1]).any()) and bool(torch.isfinite(g.scale[:-1]).all())


@pytest.mark.parametrize("output", ["bf16", "e4m3_row", "e4m3_block128"])
@pytest.mark.parametrize("R,H", [(3, 1040), (300, 2048), (70, 128)])
def test_strides_and_guards(spg, R, H, output):
    # every tensor inside a larger one at an odd place; nothing around the outputs is written
    coded = output != "bf16"

    def inside(dtype, pad, at, fill):
        big = torch.full((R + 2, H + pad), fill, dtype=dtype, device="cuda")
        return big, big[1:R + 1, at:at + H]

    xs, x = inside(BF, 13, 5, 0.0)
    rs, r = inside(BF, 7, 3, 0.0)
    hs, h = inside(BF, 9, 1, 7.0)
    ns, n = inside(BF, 11, 11, 7.0)
    qs, q = inside(torch.uint8, 32, 16, 77)
    x.copy_(rand((R, H), 1))
    r.copy_(rand((R, H), 2))
    w = rand((H + 1,), 3, dtype=F32)[1:]
    before = [t.clone() for t in (xs, rs)]
    kw = dict(out=q, normed=n) if coded else dict(out=n)
    g = spg.rms_norm(x, w, residual=r, output=output, h=h, **kw)
    want, _, y = ref_forward(x, w, r)
    assert torch.equal(h, want) and g.h is h and torch.equal(xs, before[0]) and torch.equal(rs, before[1])
    check_bf16(n, y)
    if coded:
        check_codes(spg, q, g.scale, y, output)
    for big, inner, fill in ((hs, h, 7.0), (ns, n, 7.0), (qs, q, 77)):
        if big is not qs or coded:
            inner.fill_(fill)
            assert bool((big == fill).all())


@pytest.mark.parametrize("H", [128, 1040, 5120, 20000])
def test_in_place(spg, H):
    x, r, w = rand((30, H), 1), rand((30, H), 2), rand((H,), 3)
    want = spg.rms_norm(x, w, residual=r)
    for over in (0, 1):
        a, b = x.clone(), r.clone()
        g = spg.rms_norm(a, w, residual=b, h=(a, b)[over], out=(b, a)[over])
        assert torch.equal(g.h, want.h) and torch.equal(g.out, want.out) and g.h is (a, b)[over]
    a = x.clone()
    assert torch.equal(spg.rms_norm(a, w, out=a).out, spg.rms_norm(x, w).out)


# ---- gradients ---------------------------------------------------------------------

def ref_backward(dy, h, w, rstd, dres=None, w0=0.0):
    d, hd = dy.double(), h.double()
    n = hd * rstd[:, None]
    g = d * (w.double() + w0)
    dx = rstd[:, None] * (g - n * (g * n).mean(1, keepdim=True))
    S = rstd[:, None] * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
        S = S + dres.double().abs()
    return dx, S, (d * n).sum(0), (d * n).abs().sum(0)


def check_grads(gx, gw, ref, R):
    dx, S, dw, A = ref
    # fp32: a row's sum of at most 32 terms a lane and 22 joins, and eight roundings: 64 in all, each half a
    # step of the terms' sum; then half a step of bf16
    off = (gx.double() - dx).abs()
    assert bool((off <= 2.0 ** -8 * dx.abs() + 64 * HALF * S + 2.0 ** -134).all()), float((off / S).max())
    if gw is not None:
        # rows of a workgroup one after another (at least 512 of them side by side), 16 teams, 64 + 8 partial
        # sums, three roundings of the terms
        n = 96 + -(-R // 512)
        off = (gw.double() - dw).abs()
        assert bool((off <= n * HALF * A + 2.0 ** -149).all()), float((off / A).max())


def run_backward(spg, R, H, dres=True, wt=BF, w0=0.0, seed=0):
    x, dy = rand((R, H), seed), rand((R, H), seed + 1, 0.01)
    dr = rand((R, H), seed + 2, 0.01) if dres else None
    w = (rand((H,), seed + 3, 0.3, F32) + (1.0 - w0)).to(wt)
    rstd = spg.rms_norm(x, w, weight_offset=w0, rstd=True).rstd
    gx, gw = spg.rms_norm_backward(dy, x, w, rstd, grad_residual=dr, weight_offset=w0)
    assert gx.dtype == BF and gw.dtype == F32
    check_grads(gx, gw, ref_backward(dy, x, w, rstd.double(), dr, w0), R)
    again = spg.rms_norm_backward(dy, x, w, rstd, grad_residual=dr, weight_offset=w0)
    assert torch.equal(again[0], gx) and torch.equal(again[1], gw)
    only, none = spg.rms_norm_backward(dy, x, w, rstd, grad_residual=dr, weight_offset=w0, grad_weight=False)
    assert none is None and torch.equal(only, gx)
    return gx, gw


@pytest.mark.parametrize("H", [1, 7, 64, 65, 128, 130, 256, 511, 512, 1000, 1024, 2048, 4096, 5120, 6151, 8192, 16384, 32768])
def test_backward_sizes(spg, H):
    for R in (1, 2, 67) if H < 4096 else (1, 2, 7, 9, 67):
        run_backward(spg, R, H, dres=R != 2, wt=F32 if R == 2 else BF, w0=1.0 if R == 67 else 0.0, seed=H + R)


@pytest.mark.parametrize("R,H", [(511, 5120), (512, 4096), (513, 5120), (2049, 2048), (5000, 640), (20000, 128), (50000, 64), (300, 7)])
def test_backward_many_rows(spg, R, H):
    run_backward(spg, R, H)


def test_backward_no_rows(spg):
    z = torch.zeros((0, 96), dtype=BF, device="cuda")
    gx, gw = spg.rms_norm_backward(z, z, rand((96,), 1), torch.zeros(0, device="cuda"))
    assert gx.shape == (0, 96) and bool((gw == 0).all())


def test_backward_strides_guards_and_in_place(spg):
    R, H = 77, 1043
    outer = [torch.full((R + 2, H + p), 3.0, dtype=BF, device="cuda") for p in (5, 7, 9, 11)]
    dy, x, dr, gx = (o[1:R + 1, 3:3 + H] for o in outer)
    for i, t in enumerate((dy, x, dr)):
        t.copy_(rand((R, H), i))
    w = rand((H + 1,), 5, dtype=F32)[1:]
    rstd = spg.rms_norm(x, w, rstd=True).rstd
    ref = ref_backward(dy, x, w, rstd.double(), dr)
    got, gw = spg.rms_norm_backward(dy, x, w, rstd, grad_residual=dr, grad_x=gx)
    assert got is gx
    check_grads(gx, gw, ref, R)
    want = gx.clone()
    for over in (dy, x, dr):
        a, b, c = (t.clone() for t in (dy, x, dr))
        to = {id(dy): a, id(x): b, id(dr): c}[id(over)]
        got = spg.rms_norm_backward(a, b, w, rstd, grad_residual=c, grad_x=to)
        assert torch.equal(got[0], want) and torch.equal(got[1], gw)
    gx.fill_(3.0)
    assert bool((outer[3] == 3.0).all())


def test_gradients_against_differences(spg):
    # the derivative along a direction, by central differences of the 64-bit forward: loss = sum(dy y) +
    # sum(dres h)
    R, H = 6, 272
    x, w, dy, dr = rand((R, H), 1), rand((H,), 2, dtype=F32), rand((R, H), 3), rand((R, H), 4)
    rstd = spg.rms_norm(x, w, rstd=True).rstd
    gx, gw = spg.rms_norm_backward(dy, x, w, rstd, grad_residual=dr)

    def loss(h, weight):
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * weight
        return (dy.double() * y).sum() + (dr.double() * h).sum()

    h, wd, e = x.double(), w.double(), 1e-5
    for seed in range(4):
        v, u = rand((R, H), 10 + seed, dtype=F64), rand((H,), 20 + seed, dtype=F64)
        d = (loss(h + e * v, wd) - loss(h - e * v, wd)) / (2 * e)
        # half a step of bf16 in every element, fp32 sums; the differences' own error e^2 and 2^-53 / e
        S = ref_backward(dy, x, w, rstd.double(), dr)[1]
        assert abs(d - (gx.double() * v).sum()) <= ((2.0 ** -8 + 64 * HALF) * S * v.abs()).sum() + 1e-6
        d = (loss(h, wd + e * u) - loss(h, wd - e * u)) / (2 * e)
        A = ref_backward(dy, x, w, rstd.double(), dr)[3]
        assert abs(d - (gw.double() * u).sum()) <= (128 * HALF * A * u.abs()).sum() + 1e-6


def test_past_32_bits(spg):
    # rows past 2^32 bytes and 2^31 elements in every tensor
    R, H = 280000, 8192
    x, w = torch.zeros((R, H), dtype=BF, device="cuda"), rand((H,), 1)
    some = [0, 1, 131071, 131072, 262143, 262144, R - 1]
    x[some] = rand((len(some), H), 2)
    h, rstd, y = ref_forward(x[some], w, x[some])
    g = spg.rms_norm(x, w, residual=x, output="e4m3_block128", normed=True, rstd=True)
    assert torch.equal(g.h[some], h)
    check_bf16(g.normed[some], y)
    check_codes(spg, g.out[some], g.scale[:, some].contiguous(), y, "e4m3_block128")
    gx, gw = spg.rms_norm_backward(x, g.h, w, g.rstd)
    rd = g.rstd[some].double()
    check_grads(gx[some], None, ref_backward(x[some], h, w, rd), R)
    want, A = ref_backward(x[some], h, w, rd)[2:]
    assert bool(((gw.double() - want).abs() <= 96 * HALF * A).all())


# ---- streams, graphs -----------------------------------------------------------------

def test_captured_and_replayed(spg):
    R, H = 600, 2048
    x, r, dy, w = rand((R, H), 1), rand((R, H), 2), rand((R, H), 3), rand((H,), 4)

    def step():
        f = spg.rms_norm(x, w, residual=r, output="e4m3_block128", normed=True, rstd=True)
        return (*f, *spg.rms_norm_backward(dy, f.h, w, f.rstd, grad_residual=dy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = step()
    for i in range(4):
        x.copy_(rand((R, H), 10 + i))
        dy.copy_(rand((R, H), 20 + i, 0.01))
        want = step()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(kept, want))


def test_two_streams(spg):
    # the same call on two streams at once, each with its own inputs
    streams = [torch.cuda.Stream() for _ in range(2)]
    args = [(rand((500, 5120), i), rand((5120,), 5 + i), rand((500, 5120), 8 + i)) for i in range(2)]
    want = []
    for x, w, dy in args:
        f = spg.rms_norm(x, w, output="e4m3_row", rstd=True)
        want.append((*f[:2], *spg.rms_norm_backward(dy, x, w, f.rstd)))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i, (x, w, dy) in enumerate(args):
            with torch.cuda.stream(streams[i]):
                f = spg.rms_norm(x, w, output="e4m3_row", rstd=True)
                got[i].append((*f[:2], *spg.rms_norm_backward(dy, x, w, f.rstd)))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(out, want[i]))


def test_options_are_read_alike_whatever_call_came_before(spg):
    # two calls with tensors of the same shapes, that differ in one option alone
    def both(refused, call, a, b):
        for i, pair in enumerate(((a, b), (b, a))):
            for option in pair:
                if option in refused and any(type(option) is type(r) for r in refused):
                    with pytest.raises(ValueError):
                        call(i, option)
                else:
                    call(i, option)

    w = rand((64,), 1)
    xs = iter([[rand((n + i, 64), n + i) for i in range(2)] for n in range(1, 40, 2)])
    for a, b in ((False, None), (False, 0)):                      # no bf16 beside a bf16 output
        x = next(xs)
        both([], lambda i, o: spg.rms_norm(x[i], w, normed=o), a, b)
        x = next(xs)
        both([], lambda i, o: spg.rms_norm(x[i], w, output="e4m3_row", normed=o), a, b)
    for a, b in ((False, True), (False, 1)):
        x = next(xs)
        both([b], lambda i, o: spg.rms_norm(x[i], w, normed=o), a, b)
    for b in (np.float32(0.5), Fraction(1, 2), 0.5 + 0j):         # equal to a plain number, and none
        x = next(xs)
        both([b], lambda i, o: spg.rms_norm(x[i], w, eps=o), 0.5, b)
        both([b], lambda i, o: spg.rms_norm(x[i], w, weight_offset=o), 0.5, b)
        both([b], lambda i, o: spg.rms_norm_backward(x[i], x[i], w, torch.ones(len(x[i]), device="cuda"), weight_offset=o), 0.5, b)
    for a, b in ((True, 1), (False, 0)):
        x = next(xs)
        both([b], lambda i, o: spg.rms_norm_backward(x[i], x[i], w, torch.ones(len(x[i]), device="cuda"), grad_weight=o), a, b)
