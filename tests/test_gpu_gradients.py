"""GPU tests of gradient_norm and clip_gradients against plain sums in 64 bits."""
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


def rand(n, seed, std=1.0, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * std).to(dtype)


def norm_of(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads if g is not None))


def check_norm(got, want):
    # the sum in 64 bits (10^9 terms: 2^-30 in relation to fp32's half step), one rounding; below fp32's
    # normal range its steps are 2^-149 apart, so that half a step is 2^-150 whatever the norm is
    assert got.shape == (1,) and got.dtype == F32
    if want >= 2.0 ** 128:             # past fp32's largest number, (2 - 2^-23) 2^127: rounded to infinity
        assert math.isinf(float(got))
        return
    assert abs(float(got) - want) <= 1.01 * HALF * want + 2.0 ** -150, (float(got), want)


def check_scaled(after, before, n, limit):
    f = limit / n if n > limit else 1.0
    for a, b in zip(after, before):
        want = b.double() * f
        # the factor's rounding and the product's, then the type's half step; a factor of 1 changes nothing
        half = 2.0 ** -8 if a.dtype == BF else 0.0
        tiny = (2.0 ** -134 if a.dtype == BF else 0.0) + 2.0 ** -150
        off = (a.double() - want).abs()
        assert bool((off <= (0.0 if f == 1.0 else half + 2.01 * HALF) * want.abs() + (0.0 if f == 1.0 else tiny)).all())


def run(spg, grads, ratio):
    n = norm_of(grads)
    check_norm(spg.gradient_norm(grads), n)
    limit = ratio * n
    before = [g.clone() for g in grads]
    out = [torch.full_like(g, 7.0) for g in grads]
    check_norm(spg.clip_gradients(grads, limit, out=out), n)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    check_scaled(out, before, n, limit)
    check_norm(spg.clip_gradients(grads, limit), n)
    assert all(torch.equal(a, b) for a, b in zip(grads, out))


SIZES = [1, 2, 3, 7, 8, 9, 255, 256, 2047, 2048, 2049, 16383, 16384, 16385, 32768, 100001]


@pytest.mark.parametrize("ratio", [0.5, 2.0])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["fp32", "bf16"])
def test_one_tensor(spg, dtype, ratio):
    for n in SIZES:
        run(spg, [rand(n, n, 0.1, dtype)], ratio)


@pytest.mark.parametrize("count", [2, 119, 120, 121, 400, 1000])
def test_many_tensors_of_both_types(spg, count):
    rng = np.random.default_rng(count)
    sizes = np.exp(rng.uniform(0, math.log(40000), count)).astype(int)
    grads = [rand(int(n), i, 0.1, (F32, BF)[i % 2]) for i, n in enumerate(sizes)]
    run(spg, grads, 0.3)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["fp32", "bf16"])
def test_large_tensors(spg, dtype):
    # more chunks than workgroups
    run(spg, [rand(70_000_001, 1, 0.01, dtype), rand(33, 2, 100.0, dtype), rand(5_000_000, 3, 1e-3, dtype)], 0.7)


def test_past_32_bits(spg):
    n = (1 << 31) + 4097          # bytes past 2^32, elements past 2^31
    g = torch.zeros(n, dtype=BF, device="cuda")
    g[-3:] = 2.0
    g[1 << 20] = 1.0
    norm = spg.clip_gradients([g], 1.0)
    check_norm(norm, math.sqrt(13.0))
    f = 1 / math.sqrt(13.0)
    assert abs(float(g[-1]) - 2 * f) <= 2.0 ** -8 and abs(float(g[1 << 20]) - f) <= 2.0 ** -8
    assert int((g != 0).sum()) == 4


@pytest.mark.parametrize("offset", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["fp32", "bf16"])
def test_any_alignment_and_guards(spg, dtype, offset):
    for n in (1, 9, 1000, 16384, 40000):
        a = torch.full((n + 32,), 3.0, dtype=dtype, device="cuda")
        b = torch.full((n + 32,), 3.0, dtype=dtype, device="cuda")
        src, dst = a[offset:offset + n], b[offset + 1:offset + 1 + n]
        src.copy_(rand(n, n, 0.1))
        total = norm_of([src])
        check_norm(spg.clip_gradients([src], total / 3, out=[dst]), total)
        check_scaled([dst], [src], total, total / 3)
        dst.fill_(3.0)
        assert bool((b == 3.0).all())


def test_range(spg):
    # squares past fp32's range at both ends
    for std in (1e-42, 1e-30, 1e20, 1e37):
        run(spg, [rand(1000, 1, std), rand(300, 2, min(std, 1e37), BF)], 0.5)
    big = torch.full((4,), 3e38, device="cuda")
    n = spg.clip_gradients([big], 1.0)                 # 6e38: past fp32, and scaled all the same
    assert bool(torch.isinf(n).all()) and bool(((big - 0.5).abs() <= 2 * HALF).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_norm_that_is_not_finite_scales_nothing(spg, bad):
    grads = [rand(1000, 1), rand(50, 2, dtype=BF)]
    grads[0][17] = bad
    before = [g.clone() for g in grads]
    n = spg.clip_gradients(grads, 1e-3)
    assert not bool(torch.isfinite(n).any()) and bool(torch.isnan(n).all()) == math.isnan(bad)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(grads, before))


def test_zeros_empty_tensors_and_none(spg):
    z = [torch.zeros(100, device="cuda"), torch.empty(0, device="cuda"), None, torch.empty((0, 3), dtype=BF, device="cuda")]
    assert float(spg.gradient_norm(z)) == 0.0 and float(spg.clip_gradients(z, 0.0)) == 0.0
    assert float(spg.gradient_norm(z[1:2])) == 0.0 and float(spg.clip_gradients(z[1:2], 1.0)) == 0.0
    g = [None, rand(10, 1), torch.empty(0, device="cuda"), rand((3, 4), 2)]
    n = norm_of(g)
    check_norm(spg.clip_gradients(g, 0.0), n)
    assert not bool(g[1].any()) and not bool(g[3].any())
    # the norm of a tensor listed twice counts it twice
    a = rand(100, 3)
    check_norm(spg.gradient_norm([a, a]), math.sqrt(2) * norm_of([a]))


def test_shared_memory_is_refused(spg):
    a = rand(100, 1)
    for grads, out in (([a, a], None), ([a[:60], a[40:]], None), ([a[:50], rand(50, 2)], [a[50:], a[:50]]),
                       ([a[:50]], [a[10:60]]), ([a[:50], a[50:]], [a[50:], a[:50]])):
        before = a.clone()
        with pytest.raises(spg.SpgError):
            spg.clip_gradients(grads, 1e-3, out=out)
        assert torch.equal(a, before)
    # neighbours in one buffer, in any order
    want = a * (1.0 / norm_of([a]))
    spg.clip_gradients([a[60:], a[:25], a[25:60]], 1.0)
    assert bool(((a - want).abs() <= 3 * HALF * want.abs()).all())


def test_captured_and_replayed(spg):
    grads = [rand(3000 * (i + 1) + i, i, 0.1, (F32, BF)[i % 2]) for i in range(130)]
    outs = [torch.empty_like(g) for g in grads]

    def step():
        return spg.clip_gradients(grads, 5.0, out=outs)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = step()
    for i in range(4):
        for k, t in enumerate(grads):
            t.copy_(rand(t.numel(), 100 * i + k, 0.05 * (i + 1)))
        want = step().clone()
        copies = [o.clone() for o in outs]
        torch.cuda.synchronize()
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, want) and all(torch.equal(p, q) for p, q in zip(outs, copies))


def test_same_bits_and_two_streams(spg):
    sets = [[rand(50000 + i, 10 * k + i, 0.1, (F32, BF)[i % 2]) for i in range(20)] for k in range(2)]
    want = [spg.gradient_norm(s) for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k].append(spg.gradient_norm(sets[k]))
    torch.cuda.synchronize()
    assert all(torch.equal(n, want[k]) for k in range(2) for n in got[k])


@pytest.mark.parametrize("size", [1000, 9_000_000], ids=["few_parts", "many_parts"])
@pytest.mark.parametrize("std,limit", [(1e36, 1.0), (1e37, 1e-3), (1e36, 1e-10), (1e37, 1e-30), (1e30, 1e-36)])
def test_factors_below_the_normal_range(spg, std, limit, size):
    # max_norm / norm from 2^-124, the last normal ones, down to 2^-234, of gradients whose scaled values are
    # ordinary numbers and small ones
    for dtype in (F32, BF):
        grads = [rand(size, 1, std, dtype), rand(77, 2, std, dtype)]
        n = norm_of(grads)
        assert 2.0 ** -235 < limit / n < 2.0 ** -124
        before = [g.clone() for g in grads]
        out = [torch.full_like(g, 7.0) for g in grads]
        spg.clip_gradients(grads, limit, out=out)
        check_scaled(out, before, n, limit)
        spg.clip_gradients(grads, limit)
        assert all(torch.equal(a, b) for a, b in zip(grads, out))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("n", [1000, 9_000_000], ids=["few_parts", "many_parts"])
def test_an_infinite_norm_tells_two_things(spg, n, dtype):
    # finite gradients whose norm is past fp32's range: scaled.  An infinite one among them: left as they are
    g, out = torch.full((n,), 2.0 ** 127, dtype=dtype, device="cuda"), torch.zeros(n, dtype=dtype, device="cuda")
    assert math.isinf(float(spg.gradient_norm([g])))
    assert math.isinf(float(spg.clip_gradients([g], 1.0, out=[out])))
    check_scaled([out], [g], norm_of([g]), 1.0)
    before = g.clone()
    g[n // 2] = before[n // 2] = math.inf
    assert math.isinf(float(spg.clip_gradients([g], 1.0))) and torch.equal(g, before)
    assert math.isinf(float(spg.clip_gradients([g], 1.0, out=[out]))) and torch.equal(out, before)
