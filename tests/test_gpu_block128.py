"""GPU parity of the block-scaled FP8 format: quantize_block128 and
gemm_scaled(fmt="e4m3_block128").

Codes and scales must equal the oracle's bit for bit: a group of 128 (or a
128 x 128 block) is quantized as the oracle quantizes a row of those values.
Products must satisfy |gpu - y| <= 2^-8 |y| + 2^-12 S + 2^-134 per element, y
the fp64 result on the same codes and S the scaled sum of |products|: the
rounding to bf16 takes 2^-9 |y| (half a step), and fp32 sums of 128 products
per group and one multiply-add per group err by less than (128 + 3 groups)
2^-24 S, below 2^-14 S for the lengths here.
"""
import numpy as np
import pytest
import torch

import oracle
from synthetic import bf16_normal

pytestmark = pytest.mark.gpu
B = 128


@pytest.fixture(scope="module")
def spg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import scaled_precision_gemm_amd as m
    return m


def dev(x16):
    return torch.from_numpy(np.ascontiguousarray(x16).view(np.int16)).view(torch.bfloat16).cuda()


def host(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def tiles(tiling):
    return (1 if tiling == "row" else B), (1 if tiling == "column" else B)


def quantize_ref(x16, tiling):
    """Oracle codes and scales of one matrix [R, K] of bf16 bits."""
    br, bc = tiles(tiling)
    R, K = x16.shape
    gr, gk = -(-R // br), -(-K // bc)
    p = np.zeros((gr * br, gk * bc), np.uint16)
    p[:R, :K] = x16
    g = p.reshape(gr, br, gk, bc).transpose(0, 2, 1, 3).reshape(gr * gk, br * bc)
    q, s = oracle.quantize_rowwise(g)
    q = q.reshape(gr, gk, br, bc).transpose(0, 2, 1, 3).reshape(gr * br, gk * bc)[:R, :K]
    s = s.reshape(gr, gk)
    return np.ascontiguousarray(q), np.ascontiguousarray(s.T if tiling == "row" else s)


def values(q, s, tiling):
    """fp64 values of the codes with their scales."""
    br, bc = tiles(tiling)
    s = np.asarray(s, np.float64)
    s = s.T if tiling == "row" else s
    return oracle.E4M3_TABLE[q] * s.repeat(br, 0)[:q.shape[0]].repeat(bc, 1)[:, :q.shape[1]]


def check(out, y, S, what):
    ok, excess = oracle.within_tolerance(host(out).reshape(y.shape), y, S)
    bad = np.argwhere(~ok)
    assert ok.all(), f"{what}: {len(bad)} of {ok.size} outside the bound, worst {excess.max():.3g} at {bad[:5].tolist()}"


# ---- quantizer -----------------------------------------------------------------
SHAPES = [(1, 16), (3, 128), (16, 512), (17, 48), (128, 128), (129, 144), (300, 1040), (33, 5120), (1000, 272)]


@pytest.mark.parametrize("tiling", ["row", "column", "block"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_quantize_bitexact(spg, tiling, shape):
    x = bf16_normal(shape, 1.0, 40 + shape[1])
    q, s = spg.quantize_block128(dev(x), tiling)
    qo, so = quantize_ref(x, tiling)
    assert tuple(s.shape) == so.shape == spg.block128_scale_shape(*shape, tiling)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), so.view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), qo)


@pytest.mark.parametrize("tiling", ["row", "column", "block"])
def test_quantize_extreme_groups(spg, tiling):
    # groups of zeros (both signs), of subnormals, of the largest values and
    # groups that mix magnitudes, next to ordinary ones
    x = bf16_normal((300, 656), 1.0, 7)
    x[:130, :140] = 0
    x[1, 5] = 0x8000
    x[140:150, 200:400] = np.random.default_rng(1).integers(1, 0x80, (10, 200)).astype(np.uint16)
    x[200:260, 130:300] = 0x7F7F
    x[260:290, 130:300] |= np.uint16(0x8000)
    x[::7, 500:520] = 0x0001
    x[100:200, 400:420] = 0x7E00
    q, s = spg.quantize_block128(dev(x), tiling)
    qo, so = quantize_ref(x, tiling)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), so.view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), qo)


@pytest.mark.parametrize("tiling", ["row", "column", "block"])
def test_quantize_batch_strides_and_given_outputs(spg, tiling):
    x = bf16_normal((3, 150, 400), 1.0, 9)
    big = dev(bf16_normal((3, 160, 512), 1.0, 10))
    view = big[:, 3:153, 64:464]
    view.copy_(dev(x))
    out = torch.full((3, 150, 432), 0xA5, dtype=torch.uint8, device="cuda")
    scale = torch.empty((3,) + spg.block128_scale_shape(150, 400, tiling), dtype=torch.float32, device="cuda")
    q, s = spg.quantize_block128(view, tiling, out=out[:, :, :400], scale=scale)
    assert s is scale and bool((out[:, :, 400:] == 0xA5).all())
    for b in range(3):
        qo, so = quantize_ref(x[b], tiling)
        assert np.array_equal(q[b].cpu().numpy(), qo)
        assert np.array_equal(s[b].cpu().numpy().view(np.uint32), so.view(np.uint32))


def test_quantize_no_rows(spg):
    q, s = spg.quantize_block128(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 256) and s.shape == (2, 0)


# ---- product -------------------------------------------------------------------
def operands(spg, M, N, K, seed, a_std=1.0, w_std=0.02):
    A, W = bf16_normal((M, K), a_std, seed), bf16_normal((N, K), w_std, seed + 1)
    return spg.quantize_block128(dev(A), "row") + spg.quantize_block128(dev(W), "block")


def sums(qa, sa, qw, sw, ta="row"):
    """fp64 (sum, sum of magnitudes) of A W^T from device codes and scales."""
    a = values(qa.cpu().numpy(), sa.cpu().numpy(), ta)
    w = values(qw.cpu().numpy(), sw.cpu().numpy(), "block")
    return a @ w.T, np.abs(a) @ np.abs(w).T


# (M, N, K): decode widths, half and full tiles, K tails, one column, one
# group, more groups than ring slots, K split with and without a tail
PRODUCTS = [(1, 512, 16), (5, 640, 144), (16, 1000, 1040), (17, 516, 272), (32, 2048, 512), (2, 20, 128),
            (33, 256, 128), (64, 300, 2064), (127, 129, 384), (128, 256, 4096), (129, 520, 1040), (300, 1, 256),
            (257, 300, 144), (512, 768, 640), (700, 512, 2320), (1111, 264, 272), (96, 512, 8208)]


@pytest.mark.parametrize("epi", ["store", "add", "swiglu"])
@pytest.mark.parametrize("shape", PRODUCTS, ids=lambda s: "x".join(map(str, s)))
def test_gemm_parity(spg, shape, epi):
    M, N, K = shape
    if epi == "swiglu":
        N = max(256, N // 256 * 256)
    qa, sa, qw, sw = operands(spg, M, N, K, 100 + M)
    D, S = sums(qa, sa, qw, sw)
    n_out = N // 2 if epi == "swiglu" else N
    res = bf16_normal((M, n_out), 1.0, 5) if epi == "add" else None
    y, S, _ = oracle.epilogue(epi, D, S, 1.0, 1.0, res)
    out = spg.gemm_scaled(qa, sa, qw, sw, epi, residual=None if res is None else dev(res), fmt="e4m3_block128")
    check(out, y, S, f"{epi} {shape}")
    again = spg.gemm_scaled(qa, sa, qw, sw, epi, residual=None if res is None else dev(res), fmt="e4m3_block128")
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_plans_cover_every_kernel(spg):
    plan = lambda *a, **k: spg.gemm_plan(*a, fmt="e4m3_block128", **k)   # noqa: E731
    assert plan(16, 1000, 1040)["kernel"] == 6 and plan(17, 516, 272)["bm"] == 32
    assert plan(64, 300, 2064)["split_k"] > 1 and plan(96, 512, 8208)["split_k"] > 1
    assert plan(4096, 34816, 5120, epilogue="swiglu")["kernel"] == 4
    assert plan(128, 34816, 5120)["kernel"] == 5 and plan(512, 2048, 512)["kernel"] == 5


@pytest.mark.parametrize("M,N,K,tail", [(3000, 8200, 400, False), (3000, 6400, 1040, True), (2600, 12800, 400, True)])
def test_large_tiles(spg, M, N, K, tail):
    # enough tiles for the 256-row kernel, ragged in M, N and K, with and
    # without a last round of 128-row halves; every row of sampled columns
    # and every column of sampled rows
    plan = spg.gemm_plan(M, N, K, fmt="e4m3_block128")
    assert plan["kernel"] == 4 and (plan["tail_tiles"] > 0) == tail
    qa, sa, qw, sw = operands(spg, M, N, K, 300)
    out = spg.gemm_scaled(qa, sa, qw, sw, fmt="e4m3_block128")
    rows = np.r_[0:3, 126:130, 254:258, 1500:1503, M - 6:M]
    cols = np.r_[0:3, 127:130, 255:258, 4000:4003, N - 10:N]
    a = values(qa.cpu().numpy(), sa.cpu().numpy(), "row")
    w = values(qw.cpu().numpy(), sw.cpu().numpy(), "block")
    ar, wc = a[rows], w[cols]
    check(out[torch.from_numpy(rows).cuda()], ar @ w.T, np.abs(ar) @ np.abs(w).T, "rows")
    check(out[:, torch.from_numpy(cols).cuda()], a @ wc.T, np.abs(a) @ np.abs(wc).T, "columns")


@pytest.mark.parametrize("M,N,K", [(16, 512, 384), (200, 528, 400), (2064, 4112, 272)])
def test_input_gradient(spg, M, N, K):
    # dX = dY W: W stored [out = K, in = N] with the forward's blocks
    dy, w = bf16_normal((M, K), 0.01, 1), bf16_normal((K, N), 0.02, 2)
    qy, sy = spg.quantize_block128(dev(dy), "row")
    qw, sw = spg.quantize_block128(dev(w), "block")
    out = spg.gemm_scaled(qy, sy, qw, sw, fmt="e4m3_block128", w_kmajor=True)
    a = values(qy.cpu().numpy(), sy.cpu().numpy(), "row")
    b = values(qw.cpu().numpy(), sw.cpu().numpy(), "block")
    check(out, a @ b, np.abs(a) @ np.abs(b), "dX")


@pytest.mark.parametrize("M,N,T", [(32, 512, 48), (144, 272, 400), (256, 512, 4000)])
def test_weight_gradient(spg, M, N, T):
    # dW = dY^T X over T tokens: both operands K-major
    dy, x = bf16_normal((T, M), 0.01, 1), bf16_normal((T, N), 1.0, 2)
    qy, sy = spg.quantize_block128(dev(dy), "column")
    qx, sx = spg.quantize_block128(dev(x), "block")
    out = spg.gemm_scaled(qy, sy, qx, sx, fmt="e4m3_block128", a_kmajor=True, w_kmajor=True)
    a = values(qy.cpu().numpy(), sy.cpu().numpy(), "column")
    b = values(qx.cpu().numpy(), sx.cpu().numpy(), "block")
    check(out, a.T @ b, np.abs(a).T @ np.abs(b), "dW")


@pytest.mark.parametrize("M,share", [(16, None), (160, None), (160, "w")])
def test_batched_k_major(spg, M, share):
    # both gradients of a batch of products: stored operands with batch
    # strides, scales as stored
    N, T, nb = 272, 400, 3
    dy = bf16_normal((nb, T, M), 0.01, 1)
    x = bf16_normal((T, N), 1.0, 2) if share == "w" else bf16_normal((nb, T, N), 1.0, 2)
    qy, sy = spg.quantize_block128(dev(dy), "column")
    qx, sx = spg.quantize_block128(dev(x), "block")
    dw = spg.gemm_scaled(qy, sy, qx, sx, fmt="e4m3_block128", a_kmajor=True, w_kmajor=True)
    for b in range(nb):
        a = values(qy[b].cpu().numpy(), sy[b].cpu().numpy(), "column")
        w = values((qx if share else qx[b]).cpu().numpy(), (sx if share else sx[b]).cpu().numpy(), "block")
        check(dw[b], a.T @ w, np.abs(a).T @ np.abs(w), f"dW {b}")


@pytest.mark.parametrize("M", [8, 150])
@pytest.mark.parametrize("share", ["none", "a", "w"])
def test_batch(spg, M, share):
    N, K, nb = 520, 400, 3
    A = bf16_normal((nb, M, K), 1.0, 21) if share != "a" else bf16_normal((M, K), 1.0, 21)
    W = bf16_normal((nb, N, K), 0.02, 22) if share != "w" else bf16_normal((N, K), 0.02, 22)
    qa, sa = spg.quantize_block128(dev(A), "row")
    qw, sw = spg.quantize_block128(dev(W), "block")
    R = bf16_normal((nb, M, N), 1.0, 23)
    out = spg.gemm_scaled(qa, sa, qw, sw, "add", residual=dev(R), fmt="e4m3_block128")
    for b in range(nb):
        i, j = (None if share == "a" else b), (None if share == "w" else b)
        D, S = sums(qa if i is None else qa[i], sa if i is None else sa[i], qw if j is None else qw[j],
                    sw if j is None else sw[j])
        y, S, _ = oracle.epilogue("add", D, S, 1.0, 1.0, R[b])
        check(out[b], y, S, f"batch {b}")


@pytest.mark.parametrize("M,K", [(8, 400), (150, 400), (40, 8208)])
@pytest.mark.parametrize("share", ["a", "w", "both"])
@pytest.mark.parametrize("kmajor", [False, True])
def test_one_matrix_and_scales_of_each_entry(spg, M, K, share, kmajor):
    # an operand expanded over the batch (batch stride 0) with a scale plane
    # for each entry: 16-row, 128-row and K-split kernels
    N, nb = 272, 3
    rng = np.random.default_rng(M)

    def operand(rows, std, tiling, seed, shared):
        x = bf16_normal((rows, K) if shared else (nb, rows, K), std, seed)
        q, s = spg.quantize_block128(dev(x), tiling)
        if shared:
            f = rng.uniform(0.25, 4.0, (nb, *s.shape)).astype(np.float32)
            q, s = q[None].expand(nb, *q.shape), s[None] * torch.from_numpy(f).cuda()
        return q, s
    qa, sa = operand(M, 1.0, "row", 31, share != "w")
    qw, sw = operand(N, 0.02, "block", 32, share != "a")
    w, s = qw, sw
    if kmajor:                               # the same values with W stored [K, N]
        w = qw[0].t().contiguous()[None].expand(nb, K, N) if share != "a" else qw.transpose(1, 2).contiguous()
        s = sw.transpose(1, 2).contiguous()
    out = spg.gemm_scaled(qa, sa, w, s, fmt="e4m3_block128", w_kmajor=kmajor)
    for b in range(nb):
        D, S = sums(qa[b], sa[b], qw[b], sw[b])
        y, S, _ = oracle.epilogue("store", D, S, 1.0, 1.0)
        check(out[b], y, S, f"batch {b}")


@pytest.mark.parametrize("M", [9, 64, 300])
def test_bias_rows_splits_and_strides(spg, M):
    N, K = 520, 2064
    qa, sa, qw, sw = operands(spg, M, N, K, 70)
    D, S0 = sums(qa, sa, qw, sw)
    bias = bf16_normal((N,), 1.0, 71)
    y, S, _ = oracle.epilogue("add", D, S0, 1.0, 1.0, bias=oracle.bf16_to_f64(bias))
    check(spg.gemm_scaled(qa, sa, qw, sw, "add", residual=dev(bias), fmt="e4m3_block128"), y, S, "bias row")
    qb, sb = spg.quantize_tensor(dev(bias[None, :512]).contiguous())
    codes = torch.cat([qb[0], qb[0][:8]])
    y, S, _ = oracle.epilogue("add", D, S0, 1.0, 1.0, bias=oracle.bias_e4m3(codes.cpu().numpy(), sb.cpu().numpy()[0]))
    check(spg.gemm_scaled(qa, sa, qw, sw, "add", residual=codes, bias_scale=sb, fmt="e4m3_block128"), y, S, "codes")
    y, S, _ = oracle.epilogue("store", D, S0, 1.0, 1.0)
    parts = spg.gemm_scaled(qa, sa, qw, sw, fmt="e4m3_block128", out_split=[64, 320, 136])
    check(torch.cat(parts, 1), y, S, "split output")
    # an output (and operands) inside larger tensors: the rest stays as it was
    big = torch.full((M + 2, N + 9), 7.0, dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros((M, K + 48), dtype=torch.uint8, device="cuda")
    wide[:, 16:16 + K] = qa
    spg.gemm_scaled(wide[:, 16:16 + K], sa, qw, sw, fmt="e4m3_block128", out=big[1:M + 1, 3:N + 3])
    check(big[1:M + 1, 3:N + 3], y, S, "strided output")
    big[1:M + 1, 3:N + 3] = 7.0
    assert bool((big == 7.0).all())
    # the residual in place
    R = bf16_normal((M, N), 1.0, 72)
    buf = dev(R)
    spg.gemm_scaled(qa, sa, qw, sw, "add", residual=buf, out=buf, fmt="e4m3_block128")
    y, S, _ = oracle.epilogue("add", D, S0, 1.0, 1.0, R)
    check(buf, y, S, "in place")


@pytest.mark.parametrize("M", [7, 140])
def test_scales_over_the_fp32_range(spg, M):
    # rows of A from 2^-60 to 2^60 and weight blocks from 2^-20 to 2^20: the
    # factors sa sw stay normal (|exponent| < 100) and so does each product
    N, K = 512, 512
    rng = np.random.default_rng(3)
    qa, sa, qw, sw = operands(spg, M, N, K, 80)
    sa = sa * torch.from_numpy(np.exp2(rng.integers(-60, 61, (1, M))).astype(np.float32)).cuda()
    sw = sw * torch.from_numpy(np.exp2(rng.integers(-20, 21, tuple(sw.shape))).astype(np.float32)).cuda()
    D, S = sums(qa, sa, qw, sw)
    y, S, _ = oracle.epilogue("store", D, S, 1.0, 1.0)
    check(spg.gemm_scaled(qa, sa, qw, sw, fmt="e4m3_block128"), y, S, "wide scales")


def test_empty_extents(spg):
    z = torch.zeros
    f32, u8 = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.uint8, device="cuda")
    out = spg.gemm_scaled(z((0, 256), **u8), z((2, 0), **f32), z((64, 256), **u8), z((1, 2), **f32), fmt="e4m3_block128")
    assert out.shape == (0, 64)
    out = spg.gemm_scaled(z((40, 256), **u8), z((2, 40), **f32), z((0, 256), **u8), z((0, 2), **f32), fmt="e4m3_block128")
    assert out.shape == (40, 0)


@pytest.mark.parametrize("M,N,K,epi", [(16, 2048, 1040, "swiglu"), (96, 512, 8208, "add"), (600, 768, 400, "store")])
def test_captured_step_replays_like_eager(spg, M, N, K, epi):
    # quantize + product, replayed on new inputs with eager work in between
    A = dev(bf16_normal((M, K), 1.0, 1))
    qw, sw = spg.quantize_block128(dev(bf16_normal((N, K), 0.02, 2)), "block")
    R = dev(bf16_normal((M, N), 1.0, 3)) if epi == "add" else None
    ws = spg.gemm_workspace(torch.empty((M, K), dtype=torch.uint8, device="cuda"), qw, "e4m3_block128", epi, residual=R)

    def step():
        qa, sa = spg.quantize_block128(A, "row")
        return spg.gemm_scaled(qa, sa, qw, sw, epi, residual=R, fmt="e4m3_block128", workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for r in range(3):
        A.copy_(dev(bf16_normal((M, K), 1.0 + r, 50 + r)))
        want = host(step())
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(out), want), f"replay {r}"


def test_workspace_of_another_device_is_refused(spg):
    M, N, K = 96, 512, 8208                  # split along K: partial tiles in the workspace
    ops = operands(spg, M, N, K, 5)
    ws = spg.gemm_workspace(ops[0], ops[2], "e4m3_block128")
    for fmt, o in (("e4m3_block128", ops), ("e4m3_row", (ops[0], ops[1][0].contiguous(), ops[2], torch.ones(N, device="cuda")))):
        with pytest.raises(ValueError, match="workspace"):
            spg.gemm_scaled(*o, fmt=fmt, workspace=torch.empty(ws.numel(), dtype=torch.uint8))
        with pytest.raises(ValueError, match="workspace"):
            spg.gemm_scaled(*o, fmt=fmt, workspace=torch.empty(16, dtype=torch.uint8))


def test_two_streams_at_once(spg):
    ops = [operands(spg, *s, 400 + i) for i, s in enumerate([(96, 512, 8208), (16, 4096, 2048), (600, 768, 400)])]
    want = [host(spg.gemm_scaled(*o, fmt="e4m3_block128")) for o in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for rep in range(3):
        got = [None] * len(ops)
        for i, o in enumerate(ops):
            with torch.cuda.stream(streams[(i + rep) % 2]):
                got[i] = spg.gemm_scaled(*o, fmt="e4m3_block128")
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert np.array_equal(host(g), w)
