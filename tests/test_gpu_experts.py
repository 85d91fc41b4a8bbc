"""GPU tests of the experts' layer: gemm_grouped, expert_route (and its
gradient), expert_sort, expert_combine (and its gradients), each against a
plain implementation in 64 bits, and the whole layer together.
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


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def row_values(q, s):
    s = s.cpu().numpy().astype(np.float64).T.repeat(B, 1)[:, :q.shape[1]]
    return oracle.E4M3_TABLE[q.cpu().numpy()] * s


def block_values(q, s):
    s = s.cpu().numpy().astype(np.float64).repeat(B, 0)[:q.shape[0]].repeat(B, 1)[:, :q.shape[1]]
    return oracle.E4M3_TABLE[q.cpu().numpy()] * s


def check(out, y, S, what):
    ok, excess = oracle.within_tolerance(host(out).reshape(y.shape), y, S)
    bad = np.argwhere(~ok)
    assert ok.all(), f"{what}: {len(bad)} of {ok.size} outside the bound, worst {excess.max():.3g} at {bad[:5].tolist()}"


# ---- experts' products: the bound of test_gpu_block128 -----------------------------

def grouped_ref(qa, sa, qw, sw, offsets, rows, epi):
    """{expert: (first, last, y, S)} in fp64."""
    a = row_values(qa, sa)
    got = {}
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        if hi <= lo:
            continue
        idx = np.arange(lo, hi) if rows is None else np.asarray(rows)[lo:hi]
        ae = np.where(((idx >= 0) & (idx < a.shape[0]))[:, None], a[np.clip(idx, 0, a.shape[0] - 1)], 0.0)
        w = block_values(qw[e], sw[e])
        y, S, _ = oracle.epilogue(epi, ae @ w.T, np.abs(ae) @ np.abs(w).T, 1.0, 1.0)
        got[e] = (lo, hi, y, S)
    return got


def run_grouped(spg, counts, N, K, epi, gather, tail=0, head=0, seed=0, tokens=None):
    E, R = len(counts), head + int(np.sum(counts)) + tail
    offsets = head + np.concatenate([[0], np.cumsum(counts)])
    rng = np.random.default_rng(seed)
    T = tokens or (max(1, R // 3) if gather else R)
    rows = rng.integers(0, T, R) if gather else None
    qa, sa = spg.quantize_block128(dev(bf16_normal((T, K), 1.0, seed + 1)), "row")
    qw, sw = spg.quantize_block128(dev(bf16_normal((E, N, K), 0.02, seed + 2)), "block")
    n_out = N // 2 if epi == "swiglu" else N
    out = torch.full((R, n_out), 3.0, dtype=torch.bfloat16, device="cuda")
    spg.gemm_grouped(qa, sa, qw, sw, i32(offsets), epi, rows=None if rows is None else i32(rows), out=out)
    for e, (lo, hi, y, S) in grouped_ref(qa, sa, qw, sw, offsets, rows, epi).items():
        check(out[lo:hi], y, S, f"expert {e}")
    assert bool((out[:head] == 3.0).all()) and bool((out[R - tail:] == 3.0).all() if tail else True)
    return out


# rows per expert: single tokens, empty experts at both ends and between, one
# expert with everything, tiles that end inside, each tile height
COUNTS = {
    "one_token": [0, 1, 0], "singles": [1] * 9, "decode": [3, 0, 16, 17, 1, 0, 0, 12], "all_in_one": [0, 0, 40, 0],
    "tile128_small": [20, 33, 5, 40], "tile128": [129, 0, 127, 1, 255, 64], "tile128_large": [300, 0, 511, 1, 256],
}


@pytest.mark.parametrize("epi", ["store", "swiglu"])
@pytest.mark.parametrize("gather", [False, True], ids=["in_order", "gathered"])
@pytest.mark.parametrize("counts", COUNTS.values(), ids=COUNTS.keys())
def test_grouped_parity(spg, counts, gather, epi):
    run_grouped(spg, counts, 512 if epi == "swiglu" else 300, 400, epi, gather, tail=5, head=2, seed=len(counts))


@pytest.mark.parametrize("N,K", [(1, 16), (33, 128), (129, 144), (640, 1552)])
@pytest.mark.parametrize("rows", [2, 25, 300])
def test_grouped_odd_sizes(spg, N, K, rows):
    assert spg.grouped_tile_rows(3 * rows, 3, N, K) == {2: 16, 25: 128, 300: 128}[rows]
    run_grouped(spg, [rows, rows - 1, rows + 1], N, K, "store", True, seed=N)


@pytest.mark.parametrize("gather", [False, True], ids=["in_order", "gathered"])
@pytest.mark.parametrize("E,N,K,epi", [(256, 33, 16, "store"), (130, 300, 144, "store"), (130, 512, 400, "swiglu"),
                                       (70, 1100, 144, "store"), (90, 768, 272, "swiglu")])
def test_grouped_256_row_tiles(spg, E, N, K, epi, gather):
    # experts that end on, before and behind a tile's and its strips' last row
    counts = np.resize([256, 0, 1, 500, 63, 255, 257, 0, 192, 300, 64], E)
    assert spg.grouped_tile_rows(int(counts.sum()), E, N, K, epi) == 256
    run_grouped(spg, counts, N, K, epi, gather, tail=3, head=1, seed=E, tokens=None if not gather else 500)


@pytest.mark.parametrize("E", [1, 63, 64, 65, 200])
def test_grouped_many_experts(spg, E):
    rng = np.random.default_rng(E)
    run_grouped(spg, rng.integers(0, 6, E), 256, 144, "swiglu", True, seed=E)


@pytest.mark.parametrize("E,rows,N,K,epi", [(65, 40, 2048, 400, "swiglu"), (40, 500, 1100, 528, "store"),
                                            (512, 12, 300, 400, "store"), (70, 20, 1100, 256, "store")])
def test_grouped_more_tiles_than_compute_units(spg, E, rows, N, K, epi):
    # several rounds of tiles, experts in runs of 64 and not, empty ones in a row
    rng = np.random.default_rng(E)
    counts = rng.integers(0, 2 * rows + 1, E)
    counts[E // 3:E // 3 + 3] = 0
    run_grouped(spg, counts, N, K, epi, True, seed=E, tokens=200)


def test_grouped_offsets_and_indices_out_of_range(spg):
    # device data that the call cannot check: clamped offsets, decreasing
    # pairs (no rows), indices outside A (rows of zeros)
    N, K, R, T = 256, 256, 64, 20
    qa, sa = spg.quantize_block128(dev(bf16_normal((T, K), 1.0, 1)), "row")
    qw, sw = spg.quantize_block128(dev(bf16_normal((4, N, K), 0.02, 2)), "block")
    rows = np.random.default_rng(0).integers(0, T, R)
    rows[[3, 20, 40]] = [-1, T, 2 ** 31 - 1]
    out = torch.full((R, N), 3.0, dtype=torch.bfloat16, device="cuda")
    spg.gemm_grouped(qa, sa, qw, sw, i32([-7, 10, 5, 30, 2 ** 31 - 1]), rows=i32(rows), out=out)
    # expert 0: [0, 10), 1: none, 2: [5, 30), 3: [30, 64); rows 5 .. 9 are either's
    want = grouped_ref(qa, sa, qw, sw, [0, 10, 10, 30, R], rows, "store")
    lo, hi, y, S = want[0]
    check(out[0:5], y[:5], S[:5], "expert 0")
    check(out[10:30], want[2][2], want[2][3], "expert 2")
    check(out[30:], want[3][2], want[3][3], "expert 3")
    assert bool((out[[3, 20, 40]] == 0).all())


@pytest.mark.parametrize("E", [3, 130])
@pytest.mark.parametrize("R", [60, 2000])
def test_grouped_overlapping_offsets_stay_inside(spg, E, R):
    # more tiles than the grid has workgroups: nothing outside the output rows
    # is touched, and every row holds one expert's values or what it held
    N, K = 256, 384
    qa, sa = spg.quantize_block128(dev(bf16_normal((R, K), 1.0, 1)), "row")
    qw, sw = spg.quantize_block128(dev(bf16_normal((1, N, K), 0.02, 2)), "block")
    frame = torch.full((R + 600, N), 3.0, dtype=torch.bfloat16, device="cuda")
    offsets = i32([0 if e % 2 == 0 else R for e in range(E + 1)])
    spg.gemm_grouped(qa, sa, qw.expand(E, N, K), sw.repeat(E, 1, 1), offsets, out=frame[300:300 + R])
    assert bool((frame[:300] == 3.0).all()) and bool((frame[300 + R:] == 3.0).all())
    a, w = row_values(qa, sa), block_values(qw[0], sw[0])
    got = frame[300:300 + R]
    ok, _ = oracle.within_tolerance(host(got), a @ w.T, np.abs(a) @ np.abs(w).T)
    assert bool((torch.from_numpy(ok).cuda() | (got == 3.0)).all()) and ok.any()


def test_grouped_no_rows_and_strides(spg):
    u8, f32 = dict(dtype=torch.uint8, device="cuda"), dict(dtype=torch.float32, device="cuda")
    out = spg.gemm_grouped(torch.zeros((0, 256), **u8), torch.zeros((2, 0), **f32), torch.zeros((3, 64, 256), **u8),
                           torch.zeros((3, 1, 2), **f32), i32([0, 0, 0, 0]))
    assert out.shape == (0, 64)
    # operands and output inside larger tensors, one weight for all experts
    T, N, K = 150, 136, 272
    qa, sa = spg.quantize_block128(dev(bf16_normal((T, K), 1.0, 1)), "row")
    qw, sw = spg.quantize_block128(dev(bf16_normal((N, K), 0.02, 2)), "block")
    wide = torch.zeros((T, K + 32), **u8)
    wide[:, 16:16 + K] = qa
    big = torch.full((T, N + 7), 3.0, dtype=torch.bfloat16, device="cuda")
    offsets = [0, 70, 150]
    two = qw[None].expand(2, N, K)
    sw2 = sw[None].repeat(2, 1, 1)
    spg.gemm_grouped(wide[:, 16:16 + K], sa, two, sw2, i32(offsets), out=big[:, 5:5 + N])
    for lo, hi, y, S in grouped_ref(qa, sa, two, sw2, offsets, None, "store").values():
        check(big[lo:hi, 5:5 + N], y, S, "strided")
    big[:, 5:5 + N] = 3.0
    assert bool((big == 3.0).all())


@pytest.mark.parametrize("epi", ["store", "swiglu"])
@pytest.mark.parametrize("counts,bm", [([3, 0, 2, 4], 16), ([60, 0, 70, 33], 128), ([110] * 256, 256)])
def test_grouped_one_weight_and_scales_of_each_expert(spg, counts, bm, epi):
    # codes that all experts share (expert stride 0), a scale plane for each
    E, R, K, N = len(counts), sum(counts), 272, 256
    assert spg.grouped_tile_rows(R, E, N, K, epi) == bm
    qa, sa = spg.quantize_block128(dev(bf16_normal((R, K), 1.0, 1)), "row")
    qw, sw = spg.quantize_block128(dev(bf16_normal((N, K), 0.02, 2)), "block")
    sw = sw[None] * torch.from_numpy(np.random.default_rng(3).uniform(0.25, 4.0, (E, *sw.shape)).astype(np.float32)).cuda()
    offsets = np.concatenate([[0], np.cumsum(counts)])
    out = spg.gemm_grouped(qa, sa, qw[None].expand(E, N, K), sw, i32(offsets), epi)
    for e, (lo, hi, y, S) in grouped_ref(qa, sa, qw[None].expand(E, N, K), sw, offsets, None, epi).items():
        check(out[lo:hi], y, S, f"expert {e}")


@pytest.mark.parametrize("counts", [[3, 0, 5], [70, 0, 150, 33]])
def test_grouped_input_gradient(spg, counts):
    # dX of an expert's product: the same call with the codes and the scale
    # blocks of its weight transposed
    E, R, N, K = len(counts), sum(counts), 384, 272
    qw, sw = spg.quantize_block128(dev(bf16_normal((E, N, K), 0.02, 2)), "block")
    qy, sy = spg.quantize_block128(dev(bf16_normal((R, N), 0.01, 1)), "row")
    offsets = np.concatenate([[0], np.cumsum(counts)])
    dx = spg.gemm_grouped(qy, sy, qw.transpose(1, 2).contiguous(), sw.transpose(1, 2).contiguous(), i32(offsets))
    y = row_values(qy, sy)
    for e in range(E):
        w, g = block_values(qw[e], sw[e]), y[offsets[e]:offsets[e + 1]]
        if len(g):
            check(dx[offsets[e]:offsets[e + 1]], g @ w, np.abs(g) @ np.abs(w), f"expert {e}")


# ---- routing -----------------------------------------------------------------------

def route_ref(x, top, score="softmax", bias=None, groups=1, top_groups=1, renorm=True, scale=1.0):
    """weights, experts and chosen scores in fp64, one token at a time."""
    T, E = x.shape
    W, X = np.zeros((T, top)), np.full((T, top), -1)
    P = np.zeros((T, E))
    for t in range(T):
        l = x[t].astype(np.float64)
        ok = l > -np.inf
        if score == "softmax":
            m = l[ok].max() if ok.any() else 0.0
            with np.errstate(invalid="ignore"):
                p = np.where(ok, np.where(l == m, 1.0, np.exp(np.where(ok & (l != m), l - m, 0.0))), 0.0)
            z = p.sum()
            p = p / z if z > 0 else p
        else:
            with np.errstate(over="ignore"):
                p = np.where(ok, 1 / (1 + np.exp(np.where(ok, -l, 0.0))), 0.0)
        P[t] = p
        # without bias and groups the logits themselves are compared
        c = l.copy() if bias is None and groups == 1 else p + (0 if bias is None else bias.astype(np.float64))
        c = np.where(ok & (c > -np.inf), c, -np.inf)
        if groups > 1:
            part = c.reshape(groups, -1)
            s = []
            for g in part:
                v = np.sort(g[g > -np.inf])[::-1][:2]
                s.append(v.sum() if len(v) else -np.inf)
            kept = [g for g in sorted(range(groups), key=lambda g: (-s[g], g))[:top_groups] if s[g] > -np.inf]
            keep = np.zeros(groups, bool)
            keep[kept] = True
            c = np.where(keep.repeat(E // groups), c, -np.inf)
        order = [e for e in sorted(range(E), key=lambda e: (-c[e], e)) if c[e] > -np.inf][:top]
        X[t, :len(order)] = order
        pc = p[order]
        total = pc.sum() if renorm else 1.0
        W[t, :len(order)] = scale * pc / total if total > 0 else 0.0
        if np.isnan(l).any():
            W[t] = np.nan
    return W, X, P


def check_order(experts, E, offsets, rows, slots):
    T, top = experts.shape
    flat = experts.reshape(-1)
    there = (flat >= 0) & (flat < E)
    order = np.flatnonzero(there)[np.argsort(flat[there], kind="stable")]
    want = np.concatenate([[0], np.cumsum(np.bincount(flat[there], minlength=E))])
    assert np.array_equal(offsets.cpu().numpy(), want)
    r = rows.cpu().numpy()
    assert np.array_equal(r[:len(order)], order // top) and (r[len(order):] == -1).all()
    s = np.full(T * top, -1)
    s[order] = np.arange(len(order))
    assert np.array_equal(slots.cpu().numpy().reshape(-1), s)


def check_route(spg, x, top, **how):
    """x: fp32 values [T, E], exact in bf16 too; both logit types."""
    bias = how.get("bias")
    # of many tokens, the first and the last ones
    some = np.arange(len(x)) if len(x) <= 300 else np.r_[0:60, len(x) - 60:len(x)]
    W, X, _ = route_ref(x[some], top, how.get("score", "softmax"), bias, how.get("groups", 1), how.get("top_groups", 1),
                        how.get("renormalize", True), how.get("scale", 1.0))
    if bias is not None:
        how = dict(how, bias=torch.from_numpy(bias).cuda())
    for dt in (torch.float32, torch.bfloat16):
        r = spg.expert_route(torch.from_numpy(x).cuda().to(dt), top, **how)
        ids = r.experts.cpu().numpy()
        got = ids[some]
        assert np.array_equal(got, X), f"experts differ at {np.argwhere(got != X)[:5].tolist()}"
        w = r.weights.cpu().numpy()[some]
        assert np.array_equal(np.isnan(w), np.isnan(W))
        # fp64 scores (a few 2^-52) and one rounding to fp32, half a step 2^-24
        np.testing.assert_allclose(w, W, rtol=1.01 * 2.0 ** -24, atol=2.0 ** -140)
        check_order(ids, x.shape[1], r.offsets, r.rows, r.slots)


def logits(T, E, seed, std=1.5):
    return oracle.bf16_to_f64(bf16_normal((T, E), std, seed)).astype(np.float32)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,top", [(1, 1), (2, 2), (7, 3), (60, 4), (64, 8), (65, 6), (128, 8), (160, 16), (256, 17),
                                   (257, 8), (512, 10), (1000, 32), (1024, 2)])
@pytest.mark.parametrize("T", [3, 130, 4100])
def test_route_sizes(spg, score, E, top, T):
    check_route(spg, logits(T, E, E), top, score=score)
    check_route(spg, logits(T, E, E + 1), top, score=score, renormalize=False, scale=2.5,
                bias=(0.3 * np.random.default_rng(E).standard_normal(E)).astype(np.float32))


@pytest.mark.parametrize("T", [0, 1, 16, 129, 1000, 2048, 2049, 4500, 16500])
def test_route_token_counts(spg, T):
    # 64 lanes a token up to 4096 and 16 beyond; the row order counted by
    # itself up to 16384 entries (2048 tokens), from counts of chunks
    # beyond, of more than 32 tokens past 8192
    x = logits(T, 64, T)
    if T > 2000:
        r = spg.expert_route(torch.from_numpy(x).cuda(), 8)
        order = np.argsort(-x, axis=1, kind="stable")[:, :8]
        assert np.array_equal(r.experts.cpu().numpy(), order)
        check_order(order, 64, r.offsets, r.rows, r.slots)
    else:
        check_route(spg, x, 8)
        check_route(spg, x, 8, score="sigmoid", bias=np.linspace(-1, 1, 64, dtype=np.float32))


def test_route_most_tokens(spg):
    # the largest token count: choice, order and gradient, against torch on the GPU
    T, E, top = 2 ** 25 - 1, 4, 2
    x = torch.randn(T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    r = spg.expert_route(x, top)
    best = torch.sort(x.float(), dim=1, descending=True, stable=True)
    assert torch.equal(r.experts, best.indices[:, :top].to(torch.int32))
    w = torch.softmax(best.values[:, :top].double(), 1).float()
    assert bool(((r.weights - w).abs() <= 2.0 ** -23 * w).all())     # two fp64 forms rounded to fp32: one step
    flat = r.experts.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(r.rows, (order // top).to(torch.int32))
    assert torch.equal(r.slots.reshape(-1)[order], torch.arange(T * top, dtype=torch.int32, device="cuda"))
    assert torch.equal(r.offsets[1:].long(), torch.bincount(flat.long(), minlength=E).cumsum(0))
    g = spg.expert_route_backward(torch.ones_like(r.weights), x, r.experts)
    # equal weights' gradients: the shares' derivatives cancel up to fp32 rounding
    assert g.shape == (T, E) and bool((g.float().abs() <= 2.0 ** -21).all())


@pytest.mark.parametrize("E,groups,top_groups,top", [(256, 8, 4, 8), (160, 8, 3, 6), (60, 4, 1, 4), (64, 64, 9, 9),
                                                     (512, 16, 5, 20), (96, 3, 3, 8), (8, 2, 1, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [5, 70, 4200])
def test_route_groups(spg, E, groups, top_groups, top, score, T):
    bias = (0.2 * np.random.default_rng(E).standard_normal(E)).astype(np.float32)
    for b in (None, bias):
        check_route(spg, logits(T, E, groups), top, score=score, groups=groups, top_groups=top_groups, bias=b, scale=2.5)


@pytest.mark.parametrize("E,groups,top_groups,top", [(256, 64, 20, 8), (1024, 64, 9, 32), (1000, 8, 3, 10)])
@pytest.mark.parametrize("T", [5, 4200])
def test_route_groups_of_many_experts(spg, E, groups, top_groups, top, T):
    # the most scores and choices that a workgroup holds in LDS (82 and 70 KiB)
    check_route(spg, logits(T, E, groups), top, score="sigmoid", groups=groups, top_groups=top_groups, scale=2.5)


def test_route_and_sort_captured_with_chunk_counts(spg):
    # more entries than one launch counts: the counts of chunks in a workspace,
    # the call's own or one that two graphs share, replayed one after the other
    T, E, top = 5000, 64, 8
    x = torch.from_numpy(logits(T, E, 1)).cuda()
    ws = spg.expert_workspace(T, top, E)

    def step(w):
        r = spg.expert_route(x, top, score="sigmoid", workspace=w)
        return (*r, *spg.expert_sort(r.experts, E, workspace=w))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(ws)
        step(None)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for w in (ws, ws, None):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(w)
        graphs.append((graph, got))
    for k in range(3):
        x.copy_(torch.from_numpy(logits(T, E, 50 + k)).cuda())
        want = [t.clone() for t in step(None)]
        torch.cuda.synchronize()
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, got in graphs:
            assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {k}"
        check_order(want[1].cpu().numpy(), E, *want[2:5])


@pytest.mark.parametrize("T", [10, 200, 4200])
def test_route_ties_go_to_the_lowest_index(spg, T):
    x = np.random.default_rng(5).integers(-1, 2, (T, 96)).astype(np.float32)
    x[0] = 0
    x[1] = -0.0
    x[1, ::2] = 0.0
    for score in ("softmax", "sigmoid"):
        check_route(spg, x, 12, score=score)
        check_route(spg, x, 12, score=score, groups=8, top_groups=3)
        check_route(spg, x, 12, score=score, bias=np.zeros(96, np.float32))


@pytest.mark.parametrize("T", [12, 100, 4200])
def test_route_masks(spg, T):
    # masked experts, rows with fewer experts left than places, rows with
    # none, values of the type's lowest, infinite logits, NaN
    x = logits(T, 64, 8)
    x[0] = -np.inf
    x[1, 3:] = -np.inf
    x[2, ::2] = -np.inf
    x[3] = -3.3895313892515355e38              # bf16's lowest finite value: not a mask
    x[4, 7] = np.inf
    x[5, [7, 9]] = np.inf
    x[6, 5] = np.nan
    x[7, 5:] = np.nan
    x[8, 1:] = -3.3895313892515355e38
    bias = np.zeros(64, np.float32)
    bias[10:20] = -np.inf
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check_route(spg, x, 8, score=score, renormalize=renorm)
            check_route(spg, x, 8, score=score, renormalize=renorm, bias=bias)
            check_route(spg, x, 8, score=score, renormalize=renorm, groups=8, top_groups=2, bias=bias)


@pytest.mark.parametrize("T", [6, 300, 4200])
@pytest.mark.parametrize("gap", [300, 590, 640, 710, 740, 800, 2.0 ** 100])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_chosen_far_below_the_largest_logit(spg, T, gap, groups):
    # the bias steers to experts whose softmax scores are tiny, or 0 even in 64
    # bits: their shares are the softmax over the chosen ones all the same
    E, top = 64, 5
    x = logits(T, E, 12)
    x[:, 16:] = (x[:, 16:] - np.float32(gap)).astype(np.float32)
    x[:, 22] -= 70
    x = torch.from_numpy(x).bfloat16().float().numpy()
    bias = np.zeros(E, np.float32)
    bias[:16] = -4.0
    bias[20:25] = 8.0
    X = np.tile(np.arange(20, 25), (T, 1))
    l = x[:, 20:25].astype(np.float64)   # noqa: E741
    q = np.exp(l - l.max(1, keepdims=True))
    q /= q.sum(1, keepdims=True)
    g = np.random.default_rng(T).standard_normal((T, top)).astype(np.float32)
    for dt, step in ((torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8)):
        lg = torch.from_numpy(x).cuda().to(dt)
        r = spg.expert_route(lg, top, bias=torch.from_numpy(bias).cuda(), groups=groups, top_groups=1, scale=1.5)
        ids = r.experts.cpu().numpy()
        assert np.array_equal(np.sort(ids, 1), X)
        order = ids - 20
        # fp64 scores (a few 2^-52) and one rounding to fp32
        np.testing.assert_allclose(r.weights.cpu().numpy(), 1.5 * np.take_along_axis(q, order, 1), rtol=1.01 * 2.0 ** -24,
                                   atol=2.0 ** -140)
        got = spg.expert_route_backward(torch.from_numpy(g).cuda(), lg, r.experts, scale=1.5).double().cpu().numpy()
        qo, lo = np.take_along_axis(q, order, 1), np.take_along_axis(l, order, 1)
        want = 1.5 * qo * (g - (g * qo).sum(1, keepdims=True))
        # the bound of test_route_backward with the chosen logits' reach
        tol = qo * 3.0 * np.abs(g).max(1, keepdims=True) * (2 * np.ptp(lo, 1)[:, None] + 42) * 2.0 ** -24
        assert (np.abs(np.take_along_axis(got, ids, 1) - want) <= tol + np.abs(want) * step + 2.0 ** -126).all()


@pytest.mark.parametrize("T", [5, 4200])
@pytest.mark.parametrize("base", [-596.0, -604.0, -700.0, -708.0, -712.0])
def test_route_of_small_sigmoid_scores(spg, T, base):
    # scores at the lower end of 64 bits: ordinary shares down to where exp(-l)
    # of the largest chosen one overflows (-709.78), weights and gradients of 0 below
    E, top = 40, 8
    x = np.full((T, E), -np.inf, np.float32)
    x[:, 3:23] = np.random.default_rng(1).permuted(np.tile(base - 4.0 * np.arange(20), (T, 1)), axis=1)   # exact in bf16
    l = base - 4.0 * np.arange(top)   # noqa: E741
    q = np.exp(l - base) / np.exp(l - base).sum() if base > -709 else np.zeros(top)
    g = np.random.default_rng(T).standard_normal((T, top)).astype(np.float32)
    want = 2.5 * q * (g - (g * q).sum(1, keepdims=True))
    tol = 5.0 * q * np.abs(g).max(1, keepdims=True) * (2 * np.ptp(l) + 42) * 2.0 ** -24 + 2.0 ** -126
    for dt, step in ((torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8)):
        lg = torch.from_numpy(x).cuda().to(dt)
        r = spg.expert_route(lg, top, score="sigmoid", scale=2.5)
        ids = r.experts.cpu().numpy()
        assert np.array_equal(np.take_along_axis(x, ids, 1), np.tile(l, (T, 1)))
        np.testing.assert_allclose(r.weights.cpu().numpy(), np.tile(2.5 * q, (T, 1)), rtol=1.01 * 2.0 ** -24, atol=2.0 ** -140)
        got = spg.expert_route_backward(torch.from_numpy(g).cuda(), lg, r.experts, score="sigmoid", scale=2.5)
        got = np.take_along_axis(got.double().cpu().numpy(), ids, 1)
        assert (np.abs(got - want) <= tol + np.abs(want) * step).all()


def test_route_strided_logits_and_no_order(spg):
    x = logits(90, 128, 3)
    wide = torch.zeros((90, 200), device="cuda")
    wide[:, 33:161] = torch.from_numpy(x).cuda()
    W, X, _ = route_ref(x, 6)
    r = spg.expert_route(wide[:, 33:161], 6, order=False)
    assert np.array_equal(r.experts.cpu().numpy(), X) and r.offsets is None and r.rows is None and r.slots is None
    assert spg.expert_workspace(90, 6, 128) is None
    r2 = spg.expert_route(wide[:, 33:161], 6)
    assert torch.equal(r2.weights, r.weights)
    check_order(X, 128, r2.offsets, r2.rows, r2.slots)
    x = torch.from_numpy(logits(3000, 128, 4)).cuda()      # a given workspace, whatever it holds
    ws = spg.expert_workspace(3000, 6, 128)
    ws.fill_(0xA5)
    r, r2 = spg.expert_route(x, 6), spg.expert_route(x, 6, workspace=ws)
    for a, b in zip(r, r2):
        assert torch.equal(a, b)
    check_order(r.experts.cpu().numpy(), 128, r.offsets, r.rows, r.slots)


@pytest.mark.parametrize("T,top,E", [(1, 1, 1), (7, 3, 5), (64, 8, 256), (65, 8, 256), (3000, 5, 1000), (17000, 2, 33)])
def test_sort_of_given_experts(spg, T, top, E):
    # any experts, the same one twice in a row and invalid ones included
    x = np.random.default_rng(T).integers(-1, E + 1, (T, top))
    offsets, rows, slots = spg.expert_sort(i32(x), E)
    check_order(np.where(x >= E, -1, x), E, offsets, rows, slots)


def test_sort_of_no_tokens(spg):
    offsets, rows, slots = spg.expert_sort(torch.zeros((0, 4), dtype=torch.int32, device="cuda"), 10)
    assert offsets.cpu().tolist() == [0] * 11 and rows.shape == (0,) and slots.shape == (0, 4)


# ---- gradient of the routing ---------------------------------------------------------

def route_grad_ref(x, experts, g, score, renorm, scale):
    """dl of sum_j g_j w_j in fp64 from the definition's derivative, and the
    size that fp32 errors scale with."""
    x = x.astype(np.float64)
    T, E = x.shape
    d, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        ids = [int(e) for e in experts[t] if e >= 0]
        gt = g[t].astype(np.float64)[:len(ids)] * scale
        if not ids:
            continue
        if score == "softmax":
            p = np.exp(x[t] - x[t].max())
            p /= p.sum()
        else:
            p = 1 / (1 + np.exp(-x[t]))
        pc = p[ids]
        z = pc.sum()
        gp = (gt - (gt * pc).sum() / z) / z if renorm else gt
        dp = np.zeros(E)
        np.add.at(dp, ids, gp)
        big = np.zeros(E)
        np.add.at(big, ids, np.full(len(ids), 2 * np.abs(gt).max() / (z if renorm else 1.0)))
        if score == "softmax":
            # renormalised: sum gp pc = (sum gt pc - (sum gt pc / z) sum pc) / z = 0
            d[t] = p * (dp - (0.0 if renorm else (gp * pc).sum()))
            size[t] = p * (big + (0 if renorm else 2 * np.abs(gt).max()))
        else:
            d[t] = dp * p * (1 - p)
            size[t] = big * p * (1 - p)
    return d, size


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,top", [(1, 1, 1), (5, 7, 7), (33, 128, 8), (9, 300, 32), (70, 1024, 3)])
def test_route_backward(spg, score, renorm, T, E, top):
    x = logits(T, E, 3 + E, 2.0)
    if T > 3 and E > 8:
        x[2, 4:] = -np.inf                       # fewer experts than places
    g = np.random.default_rng(E).standard_normal((T, top)).astype(np.float32)
    for dt, step in ((torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8)):
        lg = torch.from_numpy(x).cuda().to(dt)
        r = spg.expert_route(lg, top, score=score, renormalize=renorm, scale=1.7)
        got = spg.expert_route_backward(torch.from_numpy(g).cuda(), lg, r.experts, score=score, renormalize=renorm,
                                        scale=1.7)
        assert got.dtype == dt and got.shape == (T, E)
        got = got.double().cpu().numpy()
        for t in range(T):
            fin = np.isfinite(x[t])
            d, size = route_grad_ref(np.where(fin, x[t], -1e30)[None], r.experts[t:t + 1].cpu().numpy(), g[t:t + 1],
                                     score, renorm, 1.7)
            # exp: the argument l - max (up to `reach`) is rounded (reach
            # 2^-24 relative), 2 ulp for exp itself; sums of up to E terms in
            # a tree of 6 + E / 64 steps; a dozen products and quotients
            reach = np.ptp(x[t][fin]) if score == "softmax" else np.abs(x[t][fin]).max()
            tol = size * (2 * reach + 2 * E / 64 + 40) * 2.0 ** -24 + np.abs(d) * step + 2.0 ** -126
            assert (np.abs(got[t] - d[0]) <= tol[0]).all(), (t, np.abs(got[t] - d[0]).max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_against_differences(spg, score, renorm):
    # central differences of the fp64 definition with the choice held fixed;
    # step h = 2^-12: the third derivative of the scores is at most 1, so the
    # difference is off by h^2 scale sum |g| / 6 * (1 + 1 / z^3-like factors),
    # below 2^-18 for these inputs (z > 0.5)
    T, E, top, h = 6, 20, 4, 2.0 ** -12
    x = logits(T, E, 77, 1.0)
    g = np.random.default_rng(2).standard_normal((T, top)).astype(np.float32)
    lg = torch.from_numpy(x).cuda()
    r = spg.expert_route(lg, top, score=score, renormalize=renorm)
    got = spg.expert_route_backward(torch.from_numpy(g).cuda(), lg, r.experts, score=score, renormalize=renorm)
    ids = r.experts.cpu().numpy()

    def f(t, l):
        p = np.exp(l) / np.exp(l).sum() if score == "softmax" else 1 / (1 + np.exp(-l))
        pc = p[ids[t]]
        return (g[t].astype(np.float64) * (pc / pc.sum() if renorm else pc)).sum()

    for t in range(T):
        for e in range(E):
            up, dn = x[t].astype(np.float64), x[t].astype(np.float64)
            up[e] += h
            dn[e] -= h
            assert abs((f(t, up) - f(t, dn)) / (2 * h) - float(got[t, e])) < 2.0 ** -18


@pytest.mark.parametrize("base", [0.0, -80.0, -87.0, -88.5, -89.0, -110.0, -200.0, -700.0])
@pytest.mark.parametrize("T,E,top", [(4, 8, 2), (9, 64, 8), (5, 300, 32)])
def test_route_backward_of_small_sigmoid_scores(spg, base, T, E, top):
    # every score of a token far below the smallest fp32 number, or around
    # it: the shares, and so the gradient, are ordinary numbers
    x = torch.from_numpy(logits(T, E, E, 0.6) + np.float32(base)).bfloat16().float().numpy()
    x[0, 3:] = -np.inf
    g = np.random.default_rng(E).standard_normal((T, top)).astype(np.float32)
    for dt, step in ((torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8)):
        lg = torch.from_numpy(x).cuda().to(dt)
        r = spg.expert_route(lg, top, score="sigmoid", scale=2.5)
        ids = r.experts.cpu().numpy()
        got = spg.expert_route_backward(torch.from_numpy(g).cuda(), lg, r.experts, score="sigmoid", scale=2.5)
        got = got.double().cpu().numpy()
        assert np.isfinite(got).all()
        with np.errstate(over="ignore"):
            d, size = route_grad_ref(np.where(np.isfinite(x), x, -700.0), ids, g, "sigmoid", True, 2.5)
        # the bound of test_route_backward: the logits' differences (up to `reach`)
        # rounded, two exps, sums of `top` terms, a dozen products and quotients
        reach = np.where(ids >= 0, np.take_along_axis(x, np.maximum(ids, 0), 1), np.nan)
        reach = (np.nanmax(reach, 1) - np.nanmin(reach, 1))[:, None]
        assert (np.abs(got - d) <= (2 * reach + 42) * 2.0 ** -24 * size + np.abs(d) * step + 2.0 ** -126).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_route_backward_of_nan_logits(spg, score, renorm, dt):
    # a NaN logit makes all weights of its token NaN, and so its gradient;
    # chosen or not, the only one, with fewer experts than places; other
    # tokens keep theirs
    for E, top in ((1, 1), (7, 3), (300, 8)):
        x = logits(6, E, E)
        clean = torch.from_numpy(x).cuda().to(dt)
        x[1, E - 1] = x[4, 0] = np.nan
        x[5] = np.nan
        if E > 2:
            x[2, 1:] = -np.inf
            x[3] = -np.inf
            x[4, 2:] = -np.inf
            clean[2, 1:] = clean[3] = -np.inf
        lg = torch.from_numpy(x).cuda().to(dt)
        g = torch.randn(6, top, generator=torch.Generator().manual_seed(E)).cuda()
        how = dict(score=score, renormalize=renorm, scale=1.7)
        r = spg.expert_route(lg, top, **how)
        assert bool(r.weights[[1, 4, 5]].isnan().all()) and not bool(r.weights[[0, 2, 3]].isnan().any())
        got = spg.expert_route_backward(g, lg, r.experts, **how)
        assert bool(got[[1, 4, 5]].isnan().all())
        want = spg.expert_route_backward(g, clean, spg.expert_route(clean, top, **how).experts, **how)
        assert torch.equal(got[[0, 2, 3]], want[[0, 2, 3]]) and bool(got[[0, 2, 3]].isfinite().all())


def test_route_backward_repeated_and_missing_experts(spg):
    # experts chosen elsewhere: the same one twice gets both parts, -1 none
    x = logits(2, 8, 1)
    ids = np.array([[3, 3, 5], [-1, 2, -1]])
    g = np.array([[1.0, 2.0, 3.0], [4.0, 5.0, 6.0]], np.float32)
    got = spg.expert_route_backward(torch.from_numpy(g).cuda(), torch.from_numpy(x).cuda(), i32(ids), score="sigmoid",
                                    renormalize=False).cpu().numpy()
    p = 1 / (1 + np.exp(-x.astype(np.float64)))
    want = np.zeros((2, 8))
    want[0, 3], want[0, 5], want[1, 2] = 3.0, 3.0, 5.0
    np.testing.assert_allclose(got, want * p * (1 - p), rtol=2.0 ** -20, atol=0)


# ---- combine -------------------------------------------------------------------------

def combine_ref(y, w, slots, res):
    y, w = y.astype(np.float64), w.astype(np.float64)
    out, S = res.astype(np.float64).copy(), np.abs(res.astype(np.float64))
    for t in range(slots.shape[0]):
        for j in range(slots.shape[1]):
            if 0 <= slots[t, j] < y.shape[0]:
                out[t] += w[t, j] * y[slots[t, j]]
                S[t] += np.abs(w[t, j] * y[slots[t, j]])
    return out, S


@pytest.mark.parametrize("T,top,H", [(1, 1, 1), (3, 8, 64), (16, 8, 2048), (5, 3, 777), (7, 13, 2056), (2, 32, 5000),
                                     (600, 2, 72)])
@pytest.mark.parametrize("with_res", [True, False])
def test_combine(spg, T, top, H, with_res):
    rng = np.random.default_rng(H)
    R = T * top
    y16, r16 = bf16_normal((R, H), 1.0, 1), bf16_normal((T, H), 1.0, 2)
    w = rng.standard_normal((T, top)).astype(np.float32)
    slots = rng.permutation(R).reshape(T, top)
    if T > 2:
        slots[1] = -1                            # a token without experts
        slots[2, 0] = R                          # outside: no term
    out = spg.expert_combine(dev(y16), torch.from_numpy(w).cuda(), i32(slots), residual=dev(r16) if with_res else None)
    res = oracle.bf16_to_f64(r16) if with_res else np.zeros((T, H))
    want, S = combine_ref(oracle.bf16_to_f64(y16), w, slots, res)
    # one multiply-add per term in fp32 (top + 1 roundings of 2^-24 S), one rounding to bf16
    err = np.abs(oracle.bf16_to_f64(host(out)) - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + (top + 2) * 2.0 ** -24 * S * (1 + 2.0 ** -8)).all()


@pytest.mark.parametrize("H", [64, 77])
def test_combine_strides_and_in_place(spg, H):
    T, top, R = 9, 3, 40
    big = dev(bf16_normal((R, H + 24), 1.0, 1))
    y = big[:, 8:8 + H]
    r16 = bf16_normal((T, H), 1.0, 2)
    w = torch.rand(T, top, device="cuda")
    slots = i32(np.random.default_rng(0).permutation(R)[:T * top].reshape(T, top))
    want = spg.expert_combine(y.contiguous(), w, slots, residual=dev(r16))
    frame = torch.full((T, H + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    buf = frame[:, 8:8 + H]
    buf.copy_(dev(r16))
    spg.expert_combine(y, w, slots, residual=buf, out=buf)
    assert torch.equal(buf, want)
    buf.fill_(3.0)
    assert bool((frame == 3.0).all())


@pytest.mark.parametrize("T,top,H", [(1, 1, 1), (16, 8, 2048), (5, 3, 777), (7, 13, 2056), (3, 32, 4104), (600, 2, 72)])
def test_combine_backward(spg, T, top, H):
    rng = np.random.default_rng(H)
    R = T * top + 4
    y16, g16 = bf16_normal((R, H), 1.0, 1), bf16_normal((T, H), 0.01, 2)
    w = rng.standard_normal((T, top)).astype(np.float32)
    slots = rng.permutation(R)[:T * top].reshape(T, top)
    if T > 2:
        slots[1, 0] = -1
    gy0 = torch.full((R, H), 3.0, dtype=torch.bfloat16, device="cuda")
    gy, gw = spg.expert_combine_backward(dev(g16), dev(y16), torch.from_numpy(w).cuda(), i32(slots), grad_y=gy0)
    gy, gw = oracle.bf16_to_f64(host(gy)), gw.cpu().numpy()
    y, g = oracle.bf16_to_f64(y16), oracle.bf16_to_f64(g16)
    seen = np.zeros(R, bool)
    for t in range(T):
        for j in range(top):
            s = slots[t, j]
            if s < 0:
                assert gw[t, j] == 0
                continue
            seen[s] = True
            want = np.float64(w[t, j]) * g[t]
            # the fp32 product, then bf16
            assert (np.abs(gy[s] - want) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want)).all()
            # sums of at most H / 256 + 8 terms per lane, 6 + 4 steps across
            tol = (H / 256 + 20) * 2.0 ** -24 * (np.abs(g[t]) * np.abs(y[s])).sum()
            assert abs(gw[t, j] - (g[t] * y[s]).sum()) <= tol
    assert (gy[~seen] == 3.0).all()              # rows that no slot names


# ---- the layer -----------------------------------------------------------------------

def layer(spg, x, gate, w1, s1, w2, s2, top, groups):
    r = spg.expert_route(gate, top, score="sigmoid", groups=groups, top_groups=max(1, groups // 2), scale=2.5)
    qx, sx = spg.quantize_block128(x, "row")
    h = spg.gemm_grouped(qx, sx, w1, s1, r.offsets, "swiglu", rows=r.rows)
    qh, sh = spg.quantize_block128(h, "row")
    y = spg.gemm_grouped(qh, sh, w2, s2, r.offsets)
    return r, (qx, sx), h, (qh, sh), y, spg.expert_combine(y, r.weights, r.slots, residual=x)


@pytest.mark.parametrize("T,E,top,groups", [(1, 8, 2, 1), (16, 16, 4, 4), (150, 8, 3, 2), (900, 4, 2, 1)])
def test_experts_layer(spg, T, E, top, groups):
    H, I = 400, 256
    x = dev(bf16_normal((T, H), 1.0, 1))
    gate = torch.from_numpy(logits(T, E, 5)).cuda()
    w1, s1 = spg.quantize_block128(dev(bf16_normal((E, 2 * I, H), 0.05, 2)), "block")
    w2, s2 = spg.quantize_block128(dev(bf16_normal((E, H, I), 0.05, 3)), "block")
    r, (qx, sx), h, (qh, sh), y, out = layer(spg, x, gate, w1, s1, w2, s2, top, groups)
    ids = r.experts.cpu().numpy()
    assert (ids >= 0).all()
    check_order(ids, E, r.offsets, r.rows, r.slots)
    off = r.offsets.cpu().numpy()
    for lo, hi, want, S in grouped_ref(qx, sx, w1, s1, off, r.rows.cpu().numpy(), "swiglu").values():
        check(h[lo:hi], want, S, "gate and up")
    for lo, hi, want, S in grouped_ref(qh, sh, w2, s2, off, None, "store").values():
        check(y[lo:hi], want, S, "down")
    want, S = combine_ref(oracle.bf16_to_f64(host(y)), r.weights.cpu().numpy(), r.slots.cpu().numpy(),
                          oracle.bf16_to_f64(host(x)))
    err = np.abs(oracle.bf16_to_f64(host(out)) - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + (top + 2) * 2.0 ** -24 * S * (1 + 2.0 ** -8)).all()


@pytest.mark.parametrize("T", [16, 200])
def test_experts_layer_captured(spg, T):
    # the whole layer in a graph, replayed on new tokens and logits with eager
    # runs in between; gradients of routing and combining in the same graph
    H, I, E, top = 256, 128, 16, 4
    x = dev(bf16_normal((T, H), 1.0, 1))
    gate = torch.from_numpy(logits(T, E, 5)).cuda()
    w1, s1 = spg.quantize_block128(dev(bf16_normal((E, 2 * I, H), 0.05, 2)), "block")
    w2, s2 = spg.quantize_block128(dev(bf16_normal((E, H, I), 0.05, 3)), "block")
    go = dev(bf16_normal((T, H), 0.01, 9))

    def step():
        r, _, _, _, y, out = layer(spg, x, gate, w1, s1, w2, s2, top, 4)
        gy, gw = spg.expert_combine_backward(go, y, r.weights, r.slots)
        return out, gy, spg.expert_route_backward(gw, gate, r.experts, score="sigmoid", scale=2.5)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(3):
        x.copy_(dev(bf16_normal((T, H), 1.0, 20 + k)))
        gate.copy_(torch.from_numpy(logits(T, E, 30 + k)).cuda())
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), f"replay {k}"


def test_experts_layer_on_two_streams(spg):
    H, I, E, top = 256, 128, 16, 4
    w1, s1 = spg.quantize_block128(dev(bf16_normal((E, 2 * I, H), 0.05, 2)), "block")
    w2, s2 = spg.quantize_block128(dev(bf16_normal((E, H, I), 0.05, 3)), "block")
    ins = [(dev(bf16_normal((T, H), 1.0, T)), torch.from_numpy(logits(T, E, T)).cuda()) for T in (16, 200, 70, 700)]
    want = [layer(spg, x, g, w1, s1, w2, s2, top, 1)[-1].clone() for x, g in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for rep in range(3):
        got = []
        for i, (x, g) in enumerate(ins):
            with torch.cuda.stream(streams[(i + rep) % 2]):
                got.append(layer(spg, x, g, w1, s1, w2, s2, top, 1)[-1])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
