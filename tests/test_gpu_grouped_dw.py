"""GPU tests of gemm_grouped_dw against a plain product in 64 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def spg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import scaled_precision_gemm_amd as m
    return m


def rand(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def ref(dy, x, offsets, rows=None, add=None):
    """y and the sum of |terms| in fp64, [E, N, K]."""
    E, N, K, T = len(offsets) - 1, dy.shape[1], x.shape[1], x.shape[0]
    y = torch.zeros((E, N, K), dtype=torch.float64, device="cuda")
    S = torch.zeros_like(y)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            a, at = dy[lo:hi].double(), torch.arange(lo, hi, device="cuda")
            if rows is not None:
                at = i32(rows)[lo:hi].long()
            ok = (at >= 0) & (at < T)
            b = torch.where(ok[:, None], x[at.clamp(0, max(T - 1, 0))].double() if T else torch.zeros(hi - lo, K, device="cuda").double(), 0.0)
            y[e] = torch.matmul(a.t(), b)
            S[e] = torch.matmul(a.abs().t(), b.abs())
    if add is not None:
        y, S = y + add.double(), S + add.double().abs()
    return y, S


def check(out, y, S, terms):
    # an fp32 sum of `terms` exact products in any order and with the matrix core's own: each join at most one
    # step, 2^-23 of the sum of |terms| (fewer than 4096 of them; the rest by their square root would do);
    # then half a step of the output's type
    half = 2.0 ** -8 if out.dtype == BF else 2.0 ** -24
    bound = half * y.abs() + min(terms + 2, 4096) * 2.0 ** -23 * S + 2.0 ** -134
    off = (out.double() - y).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside, at {bad.nonzero()[:4].tolist()}"


def run(spg, counts, N, K, gather=False, dtype=BF, add=False, tail=0, head=0, seed=0, tokens=None):
    counts = list(counts)
    R = head + sum(counts) + tail
    off = np.concatenate([[0], np.cumsum(counts)]) + head
    T = tokens or (max(1, R // 2) if gather else R)
    dy, x = rand((R, N), seed), rand((T, K), seed + 1)
    rows = None
    if gather:
        rows = np.random.default_rng(seed).integers(0, T, R)
    if tail:        # what stands behind the last expert's rows is not read
        dy[R - tail:] = float("nan")
        if rows is not None:
            rows[R - tail:] = -1
    if head:
        dy[:head] = float("inf")
    a = rand((len(counts), N, K), seed + 2, 3.0, dtype) if add else None
    out = spg.gemm_grouped_dw(dy, x, i32(off), rows=None if rows is None else i32(rows), add=a, dtype=dtype)
    assert out.dtype == dtype and out.shape == (len(counts), N, K)
    y, S = ref(dy, x, off, rows, a)
    check(out, y, S, max(counts + [1]))
    return out


# rows of an expert: none, one, stages of 32 that end inside, on and behind their last row
COUNTS = {"one": [1], "none": [0, 0], "mixed": [0, 1, 0, 31, 32, 33, 0], "stages": [64, 96, 97, 127, 128, 129],
          "long": [700, 0, 1500, 3]}


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("add", [False, True], ids=["", "add"])
@pytest.mark.parametrize("gather", [False, True], ids=["in_order", "gathered"])
@pytest.mark.parametrize("counts", COUNTS.values(), ids=COUNTS.keys())
def test_parity(spg, counts, gather, add, dtype):
    run(spg, counts, 264, 328, gather, dtype, add, tail=5, head=3, seed=len(counts))


@pytest.mark.parametrize("N,K", [(8, 8), (8, 512), (512, 8), (128, 64), (248, 256), (256, 264), (520, 1032), (1024, 768)])
def test_sizes(spg, N, K):
    run(spg, [40, 0, 100, 9], N, K, True, seed=N)
    run(spg, [40, 0, 100, 9], N, K, False, F32, True, seed=K)


@pytest.mark.parametrize("E", [1, 3, 8, 9, 64, 130])
def test_experts(spg, E):
    # rows of tiles that fill the XCDs' rounds and not, and workgroups without one
    rng = np.random.default_rng(E)
    run(spg, rng.integers(0, 80, E), 520, 264, True, seed=E)


@pytest.mark.parametrize("R,N,K,E", [(256, 256, 256, 1), (512, 256, 256, 1), (513, 264, 248, 1), (4000, 1024, 512, 1),
                                     (5000, 256, 256, 1), (9000, 128, 136, 1), (3000, 264, 512, 3)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_rows_in_slices(spg, R, N, K, E, dtype):
    # few tiles: each expert's rows are cut, the parts summed by a second launch
    need = spg.grouped_dw_workspace(R, E, N, K)
    assert (need is not None) == (R // E >= 512)
    counts = [R] if E == 1 else [R // 2, 0, R - R // 2]
    run(spg, counts, N, K, E == 3, dtype, False, seed=R)
    run(spg, counts, N, K, False, dtype, True, seed=R + 1)
    # an expert with fewer rows than slices and none at all
    run(spg, [R - 1, 1] + [0] * (E - 1) if E > 1 else [R], N, K, False, dtype, seed=R + 2)


@pytest.mark.parametrize("gather", [False, True], ids=["in_order", "gathered"])
@pytest.mark.parametrize("counts,N,K", [([40, 0, 1000, 33], 1800, 2056), ([300] * 150, 264, 248), ([5, 0] * 80, 264, 264),
                                        ([0] * 70 + [2000] + [3] * 70, 256, 264), ([1100, 900] * 40, 520, 264)])
def test_more_tiles_than_compute_units(spg, counts, N, K, gather):
    # 256-row tiles, several a workgroup; experts without rows, shorter than the copies run ahead, and of several
    # chunks of row numbers, next to each other in every order
    run(spg, counts, N, K, gather, seed=N, tail=3, head=1)


@pytest.mark.parametrize("gather", [False, True], ids=["in_order", "gathered"])
@pytest.mark.parametrize("counts,N,K", [([40, 0, 70] * 23, 1288, 264), ([300, 1, 64, 0] * 17, 1032, 520), ([50] * 43, 776, 264),
                                        ([0] * 31 + [900] + [0] * 33, 2048, 264)])
def test_rows_of_tiles_dealt_together(spg, counts, N, K, gather):
    # two or four rows of tiles an XCD, across experts' borders, the last unit not whole
    run(spg, counts, N, K, gather, seed=K, tail=2)


@pytest.mark.parametrize("gather", [False, True], ids=["in_order", "gathered"])
@pytest.mark.parametrize("counts,N,K", [([130], 4096, 4096), ([130], 2048, 4096), ([99], 2056, 4096), ([70], 4096, 8192),
                                        ([40, 0, 130, 33, 1, 64, 7], 4096, 4096), ([20] * 9, 2312, 4104), ([33], 1024, 8200)])
def test_parts_of_rows_of_tiles(spg, counts, N, K, gather):
    # wide outputs: a row of tiles in two or four parts, or whole, on several XCDs
    run(spg, counts, N, K, gather, seed=N, tail=1)


@pytest.mark.parametrize("R,N,K,E", [(32768, 2048, 256, 1), (16384, 1024, 256, 2)])
def test_parts_dealt_together(spg, R, N, K, E):
    assert spg.grouped_dw_workspace(R, E, N, K) is not None
    run(spg, [R] if E == 1 else [R - 77, 77], N, K, E == 2, F32, seed=E)


@pytest.mark.parametrize("last", [1, 33, 97, 129, 161, 1025, 1057, 1153])
def test_chunks_of_row_numbers(spg, last):
    # 1024 rows a chunk: tiles that end right behind a border, followed by others
    for counts in ([last, 1024, 70], [1024 + last] * 3, [2048, last, 1, 1024]):
        run(spg, counts, 1288, 4104, True, seed=last)


def test_offsets_and_indices_out_of_range(spg):
    N, K, R, T = 256, 128, 64, 20
    dy, x = rand((R, N), 1), rand((T, K), 2)
    rows = np.random.default_rng(0).integers(0, T, R)
    rows[[3, 20, 40]] = [-1, T, 2 ** 31 - 1]
    out = spg.gemm_grouped_dw(dy, x, i32([-7, 10, 5, 30, 2 ** 31 - 1]), rows=i32(rows), dtype=F32)
    # expert 0: [0, 10), 1: none, 2: [5, 30), 3: [30, 64)
    for e, (lo, hi) in enumerate([(0, 10), (0, 0), (5, 30), (30, 64)]):
        y, S = ref(dy, x, [lo, hi], rows)
        check(out[e:e + 1], y, S, 64)
    out = spg.gemm_grouped_dw(dy, x[:0], i32([0, 30, 64]), rows=i32(rows))
    assert bool((out == 0).all())
    out = spg.gemm_grouped_dw(dy[:0], x, i32([0, 0, 0]), rows=i32(rows[:0]))
    assert out.shape == (2, N, K) and bool((out == 0).all())
    a = rand((2, N, K), 3)
    assert torch.equal(spg.gemm_grouped_dw(dy[:0], x, i32([0, 0, 0]), add=a), a)
    assert spg.gemm_grouped_dw(dy[:, :0], x, i32([0, 64]), rows=i32(rows)).shape == (1, 0, K)


def test_values_behind_the_last_row_are_not_multiplied(spg):
    # NaN in both operands' rows past each expert's end, at every place of a stage
    N, K = 264, 136
    for n in (1, 5, 31, 32, 33, 63):
        dy, x = rand((200, N), n), rand((200, K), n + 1)
        dy[n:64], x[n:64] = float("nan"), float("nan")
        out = spg.gemm_grouped_dw(dy, x, i32([0, n, n, n]), dtype=F32)
        y, S = ref(dy[:n], x[:n], [0, n, n, n])
        check(out, y, S, n)
        # and NaN rows of their own expert reach that expert only
        out = spg.gemm_grouped_dw(dy, x, i32([0, n, 64, 200]), dtype=F32)
        check(out[:1], y[:1], S[:1], n)
        assert bool(torch.isnan(out[1]).all())
        y, S = ref(dy, x, [64, 200])
        check(out[2:], y, S, 136)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_strides_guards_and_in_place(spg, dtype):
    R, T, E, N, K = 300, 90, 3, 136, 264
    wide_y, wide_x = rand((R, N + 24), 1), rand((T, K + 16), 2)
    dy, x = wide_y[:, 8:8 + N], wide_x[:, 16:16 + K]
    rows, off = np.random.default_rng(1).integers(0, T, R), [5, 100, 220, 290]
    big = torch.full((E + 1, N + 3, K + 24), 3.0, dtype=dtype, device="cuda")
    out = big[:E, 2:2 + N, 8:8 + K]
    got = spg.gemm_grouped_dw(dy, x, i32(off), rows=i32(rows), out=out, dtype=dtype)
    assert got is out
    y, S = ref(dy, x, off, rows)
    check(out, y, S, 120)
    # gradients of a second chunk, added in place
    first = out.clone()
    spg.gemm_grouped_dw(dy, x, i32(off), rows=i32(rows), add=out, out=out, dtype=dtype)
    y, S = ref(dy, x, off, rows, first)
    check(out, y, S, 121)
    out.fill_(3.0)
    assert bool((big == 3.0).all())
    # a dense layer's in slices, in place
    dy, x = rand((2000, 256), 3), rand((2000, 256), 4)
    acc = rand((1, 256, 256), 5, dtype=dtype)
    y, S = ref(dy, x, [0, 2000], None, acc)
    ws = spg.grouped_dw_workspace(2000, 1, 256, 256)
    spg.gemm_grouped_dw(dy, x, i32([0, 2000]), add=acc, out=acc, dtype=dtype, workspace=ws)
    check(acc, y, S, 2001)


def test_overlapping_ranges_count_for_both(spg):
    dy, x = rand((100, 64), 1), rand((100, 72), 2)
    off = [0, 80, 40, 100]          # [0, 80), none, [40, 100)
    out = spg.gemm_grouped_dw(dy, x, i32(off), dtype=F32)
    for e, (lo, hi) in enumerate([(0, 80), (0, 0), (40, 100)]):
        y, S = ref(dy, x, [lo, hi])
        check(out[e:e + 1], y, S, 100)


def test_against_differences_of_the_products(spg):
    # the loss sum(dY * (X W^T)) of every expert is linear in W: its difference along a direction
    E, N, K, T = 4, 64, 48, 50
    rng = np.random.default_rng(3)
    rows, off = rng.integers(0, T, 150), [0, 40, 40, 111, 150]
    dy, x = rand((150, N), 1), rand((T, K), 2)
    out = spg.gemm_grouped_dw(dy, x, i32(off), rows=i32(rows), dtype=F32)
    S = ref(dy, x, off, rows)[1]
    w = rand((E, N, K), 4, dtype=torch.float64)

    def loss(w):
        return sum((dy[off[e]:off[e + 1]].double() * torch.matmul(x[i32(rows)[off[e]:off[e + 1]].long()].double(), w[e].t())).sum()
                   for e in range(E))

    for seed in range(3):
        v = rand((E, N, K), 10 + seed, dtype=torch.float64)
        d = (loss(w + v) - loss(w - v)) / 2
        assert abs(d - (out.double() * v).sum()) <= (152 * 2.0 ** -23 * S * v.abs()).sum()


def test_large_operands(spg):
    # offsets past 2^31 bytes in dY and X (rows far into them) and in the output
    R, N, K = 600000, 2048, 2048
    dy, x = torch.empty((R, N), dtype=BF, device="cuda"), torch.empty((R, K), dtype=BF, device="cuda")
    lo, hi = R - 70, R - 3
    dy[lo:], x[lo:] = rand((70, N), 1), rand((70, K), 2)
    off = [lo] * 300 + [hi]                # the last of 300 experts
    out = spg.gemm_grouped_dw(dy, x, i32(off))
    y, S = ref(dy, x, [lo, hi])
    check(out[299:], y, S, 67)
    assert bool((out[:299] == 0).all())


def test_gathered_to_the_last_row_below_the_limit(spg):
    # X of 2^30 - 2048 elements: byte offsets up to 2^31
    T, K, N = (1 << 19) - 1, 2048, 264
    x = torch.empty((T, K), dtype=BF, device="cuda")
    at = [T - 1, 0, T - 2, T // 2, T - 1, T - 33, T, 1 << 30]      # the last two stand for zeros
    dy, rows = rand((len(at), N), 1), i32(at)
    for i, r in enumerate(sorted(set(at[:6]))):
        x[r] = rand((K,), 10 + i)
    out = spg.gemm_grouped_dw(dy, x, i32([0, 3, 8]), rows=rows, dtype=F32)
    some = torch.stack([x[r] if r < T else torch.zeros_like(x[0]) for r in at])
    y, S = ref(dy, some, [0, 3, 8])
    check(out, y, S, 5)


def test_most_experts(spg):
    # 65536 experts in groups of 64 sorted by their rows; nearly all without any
    E, N, K, R = 65536, 8, 16, 3000
    counts = np.zeros(E, dtype=np.int64)
    np.add.at(counts, np.random.default_rng(1).integers(0, E, 300), 10)
    off = np.concatenate([[0], np.cumsum(counts)])
    dy, x = rand((R, N), 1), rand((R, K), 2)
    add = rand((E, N, K), 3)
    out = spg.gemm_grouped_dw(dy, x, i32(off), add=add)
    full = np.nonzero(counts)[0]
    y, S = ref(dy, x, np.concatenate([[0], np.cumsum(counts[full])]), None, add[torch.as_tensor(full, device="cuda")])
    check(out[torch.as_tensor(full, device="cuda")], y, S, int(counts.max()))
    empty = torch.as_tensor(counts == 0, device="cuda")
    assert torch.equal(out[empty], add[empty])


def test_captured_and_replayed_with_other_routings(spg):
    E, N, K, T, top = 8, 264, 512, 100, 2
    dy, x = rand((T * top, N), 1), rand((T, K), 2)
    big_dy, big_x = rand((3000, 256), 3), rand((3000, 256), 4)
    off, rows, all_ = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(T * top, dtype=torch.int32, device="cuda"), i32([0, 3000])

    def route(seed):
        ids = np.random.default_rng(seed).integers(0, E, T * top)
        off.copy_(i32(np.concatenate([[0], np.cumsum(np.bincount(ids, minlength=E))])))
        rows.copy_(i32(np.argsort(ids, kind="stable") // top))

    ws = spg.grouped_dw_workspace(3000, 1, 256, 256)

    def step():
        return spg.gemm_grouped_dw(dy, x, off, rows=rows), spg.gemm_grouped_dw(big_dy, big_x, all_, dtype=F32, workspace=ws)

    route(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = step()
    for i in range(4):
        route(i + 1)
        dy.copy_(rand((T * top, N), 20 + i))
        big_x.copy_(rand((3000, 256), 30 + i))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept[0], want[0]) and torch.equal(kept[1], want[1])


def test_two_streams(spg):
    streams = [torch.cuda.Stream() for _ in range(2)]
    args = [(rand((2000, 512), i), rand((2000, 256), 5 + i), i32([0, 900 + i, 2000])) for i in range(2)]
    want = [spg.gemm_grouped_dw(*a) for a in args]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(spg.gemm_grouped_dw(*args[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])


@pytest.mark.parametrize("gather", [False, True], ids=["in_order", "gathered"])
@pytest.mark.parametrize("counts,N,K", [([40], 3584, 28672), ([33], 3328, 28672), ([33, 0, 7], 1280, 32768), ([9, 1, 0, 40, 3], 1280, 20480)])
def test_wide_outputs_are_whole(spg, counts, N, K, gather):
    # rows of tiles in eight parts and more, the last unit of rows of tiles not whole; every element written
    E, R = len(counts), sum(counts) + 2
    off, T = np.concatenate([[0], np.cumsum(counts)]), R // 2 if gather else R
    dy, x = rand((R, N), 1), rand((T, K), 2)
    rows = np.random.default_rng(N).integers(0, T, R) if gather else None
    idx = None if rows is None else i32(rows)
    out = torch.full((E, N, K), float("nan"), dtype=BF, device="cuda")
    spg.gemm_grouped_dw(dy, x, i32(off), rows=idx, out=out)
    y, S = ref(dy, x, off, rows)
    check(out, y, S, max(counts))
    # a second chunk, added in place
    first = out.clone()
    spg.gemm_grouped_dw(dy, x, i32(off), rows=idx, add=out, out=out)
    y, S = ref(dy, x, off, rows, first)
    check(out, y, S, max(counts) + 1)


@pytest.mark.parametrize("kind", ["alike", "outlier", "random"])
@pytest.mark.parametrize("R", [16384, 32768 + 16, 131072, 1 << 20, (1 << 21) - 40])
@pytest.mark.parametrize("E", [1, 129], ids=["in_parts", "whole"])
def test_long_sums(spg, R, E, kind):
    # sums whose roundings all fall the same way: rows that are alike, and rows each below half a step of a first
    # one's product.  Per element half a step of fp32, and per eight products one rounding of the sum so far,
    # 2^-24 of it, with up to 2^-4 of a step lost where they are aligned: rows / 8 of them, 1.125 2^-24 S each,
    # below rows 2^-26 S (rows in parts: at most 16 further ones, below 2^-19 S, within what is left of that)
    dy, x = rand((R, 8), 1), rand((R, 16), 2)
    if kind != "random":
        dy.fill_(1 + 7 / 128 if kind == "alike" else 0.124)
        x.fill_(1 + 9 / 128 if kind == "alike" else 1.0)
    if kind == "outlier":
        dy[0], x[0] = 4096.0, 4096.0
    off = [0] + [R] * E
    assert (spg.grouped_dw_workspace(R, E, 8, 16) is None) == (E > 1)
    out = spg.gemm_grouped_dw(dy, x, i32(off), dtype=F32)
    y, S = torch.matmul(dy.double().t(), x.double()), torch.matmul(dy.double().abs().t(), x.double().abs())
    off_by = (out[0].double() - y).abs()
    assert bool((off_by <= 2.0 ** -24 * y.abs() + max(2.0 ** -12, R * 2.0 ** -26) * S).all()), float((off_by / S).max())
    assert not bool(out[1:].any())
