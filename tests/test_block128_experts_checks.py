"""Refusals of the block-128 and experts' entry points (CPU only, nothing is
launched): the C ABI with pointers that are never dereferenced, and the
Python binding with tensors on torch's "meta" device.
"""
import ctypes

import pytest
import torch

import scaled_precision_gemm_amd as spg

P = ctypes.c_void_p
FAKE, FAR = P(0x100000), P(0x40000000000)
MIS16, MIS4 = P(0x100008), P(0x100002)
EINVAL, EUNSUP, EWS = 1, 2, 3
BF, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32


# ---- C ABI ------------------------------------------------------------------

def quant(x=FAKE, batch=1, rows=32, K=256, ldx=256, bs=0, q=FAKE, ldq=256, qbs=0, scale=FAKE, tiling=0):
    return spg.lib.quantize_block128(x, batch, rows, K, ldx, bs, q, ldq, qbs, scale, tiling, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tiling=3), EINVAL), (dict(batch=0), EINVAL), (dict(rows=-1), EINVAL), (dict(K=24, ldx=24, ldq=32), EINVAL),
    (dict(K=0), EINVAL), (dict(x=None), EINVAL), (dict(q=None), EINVAL), (dict(scale=None), EINVAL),
    (dict(ldx=248), EINVAL), (dict(ldx=260), EINVAL), (dict(ldq=264), EINVAL), (dict(ldq=240), EINVAL),
    (dict(x=MIS16), EINVAL), (dict(q=MIS16), EINVAL), (dict(scale=MIS4), EINVAL),
    (dict(batch=2, bs=8184, qbs=8192), EINVAL), (dict(batch=2, bs=8196, qbs=8192), EINVAL),
    (dict(batch=2, bs=8192, qbs=8176), EINVAL), (dict(batch=2, bs=8192, qbs=8200), EINVAL),
    (dict(batch=65536, bs=8192, qbs=8192), EUNSUP), (dict(rows=2 ** 24, tiling=2), EUNSUP),
    (dict(K=2 ** 26, ldx=2 ** 26, ldq=2 ** 26), EUNSUP), (dict(rows=0, x=None, q=None, scale=None), 0),
])
def test_quantize_refusals(kw, want):
    assert quant(**kw) == want


def gemm(d, epi=0, res=None):
    return spg.lib.gemm_scaled(FAKE, FAR, FAR, FAR, FAR, res, epi, ctypes.byref(d), None, 0, None)


def desc(M, N, K):
    d = spg.GemmDesc()
    spg.lib.spg_gemm_desc_init(ctypes.byref(d), M, N, K, spg.FMT_E4M3_BLOCK128)
    return d


def test_gemm_refusals():
    assert gemm(desc(64, 64, 24)) == EINVAL
    assert gemm(desc(64, 384, 256), epi=2) == EINVAL          # the up rows would start inside a block
    d = desc(64, 64, 256)
    d.scale_layout = 1
    assert gemm(d) == EINVAL
    assert gemm(desc(2 ** 29, 64, 256)) == EUNSUP
    d = desc(96, 512, 8192)                                    # split along K: needs a workspace
    assert spg.lib.gemm_scaled_workspace_bytes(ctypes.byref(d), 0) > 0
    assert gemm(d) == EWS
    d = desc(64, 64, 2 ** 20 * 16)
    assert gemm(d) == EUNSUP                                   # row stride


@pytest.mark.parametrize("M,N,most", [(16, 16, 2 ** 24), (33, 16, 2 ** 23), (200, 256, 2 ** 23)])
def test_more_workgroups_than_a_launch_takes(M, N, most):
    # 2^32 threads: refused before anything is enqueued (the pointers are not real)
    for batch, want in ((most - 1, 0), (most, EUNSUP)):
        d = desc(M, N, 16)
        d.batch, d.stride_a, d.stride_w, d.stride_o = batch, M * 16, N * 16, M * N
        plan = spg.Plan()
        assert spg.lib.spg_gemm_plan(ctypes.byref(d), 0, 256, ctypes.byref(plan)) == want
    assert plan.workgroups == {16: 2 ** 24, 33: 2 ** 23, 200: 2 ** 23}[M]
    assert gemm(d) == EUNSUP


def test_scales_of_each_entry_flags():
    d = desc(64, 64, 256)
    plan = spg.Plan()
    check = lambda: spg.lib.spg_gemm_plan(ctypes.byref(d), 0, 256, ctypes.byref(plan))  # noqa: E731
    for flags, want in ((0, 0), (1, 0), (2, 0), (3, 0), (4, EINVAL), (-1, EINVAL)):
        d.scale_batch = flags
        assert check() == want
    spg.lib.spg_gemm_desc_init(ctypes.byref(d), 64, 64, 256, spg.FMT_E4M3_ROW)
    d.scale_batch = 1
    assert check() == EUNSUP


@pytest.mark.parametrize("M", [1, 16, 17, 32, 33, 128, 129, 1000, 4096, 100000])
@pytest.mark.parametrize("N", [16, 512, 5120, 34816])
@pytest.mark.parametrize("K", [16, 1024, 5120, 17408])
def test_plans(M, N, K):
    p = spg.gemm_plan(M, N, K, fmt="e4m3_block128")
    tiles = {4: (256, 256), 5: (128, 256), 6: (p["bm"], 32)}
    bm, bn = tiles[p["kernel"]]
    assert (p["bm"], p["bn"]) == (bm, bn) and (p["kernel"] != 6 or p["bm"] in (16, 32) and p["bm"] >= min(M, 32))
    assert p["tiles"] == -(-M // bm) * -(-N // bn)
    assert p["workgroups"] == (p["tiles"] - p["tail_tiles"]) * p["split_k"]
    assert p["tail_tiles"] == 0 or (p["kernel"], p["split_k"], p["tail_bm"], p["tail_split"]) == (4, 1, 128, 1)
    chunk = -(--(-K // p["split_k"]) // 128) * 128
    assert 1 <= p["split_k"] and (p["split_k"] - 1) * chunk < K     # no empty slice
    assert p["split_k"] == 1 or p["kernel"] != 6


def grouped_desc(**kw):
    d = dict(rows=64, a_rows=64, N=512, K=256, lda=256, ldw=256, stride_w=512 * 256, ldo=512, experts=4)
    d.update(kw)
    return spg.GroupedDesc(*[d[k] for k in ("rows", "a_rows", "N", "K", "lda", "ldw", "stride_w", "ldo", "experts")], 0)


def grouped(d, epi=0, out=FAKE, A=FAR, sa=FAR, W=FAR, sw=FAR, off=FAR, idx=None):
    return spg.lib.gemm_grouped(out, A, sa, W, sw, off, idx, epi, ctypes.byref(d) if d else None, None)


@pytest.mark.parametrize("kw,call,want", [
    ({}, dict(epi=5), EINVAL), ({}, dict(epi=1), EUNSUP), (dict(rows=-1), {}, EINVAL), (dict(K=24), {}, EINVAL),
    (dict(experts=0), {}, EINVAL), (dict(experts=65537), {}, EUNSUP), (dict(N=384), dict(epi=2), EINVAL),
    (dict(a_rows=63), {}, EINVAL), (dict(lda=240), {}, EINVAL), (dict(lda=264), {}, EINVAL), (dict(ldw=240), {}, EINVAL),
    (dict(lda=2 ** 24), {}, EUNSUP), (dict(stride_w=512 * 256 - 16), {}, EINVAL), (dict(stride_w=-16), {}, EINVAL),
    (dict(ldo=500), {}, EINVAL), (dict(ldo=2 ** 26), {}, EUNSUP), (dict(rows=2 ** 29, a_rows=2 ** 29), {}, EUNSUP),
    (dict(a_rows=2 ** 23), dict(idx=FAR), EUNSUP), ({}, dict(out=None), EINVAL), ({}, dict(A=None), EINVAL),
    ({}, dict(sa=None), EINVAL), ({}, dict(sw=None), EINVAL), ({}, dict(off=None), EINVAL), ({}, dict(A=MIS16), EINVAL),
    ({}, dict(W=MIS16), EINVAL), ({}, dict(sa=MIS4), EINVAL), ({}, dict(idx=MIS4), EINVAL), ({}, dict(A=FAKE), EINVAL),
    ({}, dict(sw=FAKE), EINVAL), ({}, dict(off=FAKE), EINVAL), ({}, dict(idx=FAKE), EINVAL),
    (dict(rows=0), dict(out=None, A=None), 0),
])
def test_grouped_refusals(kw, call, want):
    assert grouped(grouped_desc(**kw), **call) == want


def test_grouped_null_desc_and_tile_rows():
    assert grouped(None) == EINVAL
    rows = (1, 8 * 8, 8 * 9, 8 * 96, 8 * 97)
    assert [spg.grouped_tile_rows(n, 8, 512, 256) for n in rows] == [16, 16, 128, 128, 128]
    assert [spg.grouped_tile_rows(16 * n, 128, 512, 256) for n in rows] == [16, 128, 128, 128, 256]
    assert spg.grouped_tile_rows(64 * 5, 64, 2048, 256) == 128
    assert spg.grouped_tile_rows(8, 8, 500, 24) == 0


@pytest.mark.parametrize("a_rows", [0, 4096, 32768, 2 ** 28])
def test_tile_rows_of_gathered_rows(a_rows):
    # the first product of an experts' layer: more output rows than rows of A
    d = grouped_desc(rows=32768, a_rows=a_rows, N=2048, K=2048, lda=2048, ldw=2048, stride_w=2048 * 2048, ldo=2048,
                     experts=64)
    assert spg.lib.spg_grouped_tile_rows(ctypes.byref(d), 0) == 256
    assert spg.grouped_tile_rows(32768, 64, 2048, 2048) == 256


def route_desc(**kw):
    d = dict(T=100, ld=64, E=64, top=8, groups=1, top_groups=1, score=0, renormalize=1, logits_bf16=0, scale=1.0)
    d.update(kw)
    return spg.RouteDesc(*[d[k] for k in ("T", "ld", "E", "top", "groups", "top_groups", "score", "renormalize",
                                          "logits_bf16", "scale")])


def route(d, logits=FAKE, bias=None, w=FAR, x=FAR, off=FAR, rows=FAR, slots=FAR, ws=FAR, nws=1 << 20):
    return spg.lib.expert_route(logits, bias, w, x, off, rows, slots, ctypes.byref(d), ws, nws, None)


@pytest.mark.parametrize("kw,call,want", [
    (dict(T=-1), {}, EINVAL), (dict(E=0), {}, EINVAL), (dict(top=0), {}, EINVAL), (dict(top=65), {}, EINVAL),
    (dict(ld=63), {}, EINVAL), (dict(groups=0), {}, EINVAL), (dict(groups=3), {}, EINVAL),
    (dict(groups=4, top_groups=5), {}, EINVAL), (dict(top_groups=0), {}, EINVAL), (dict(score=2), {}, EINVAL),
    (dict(scale=float("inf")), {}, EINVAL), (dict(scale=float("nan")), {}, EINVAL), (dict(E=1025, ld=1025), {}, EUNSUP),
    (dict(top=33), {}, EUNSUP), (dict(E=128, ld=128, groups=128), {}, EUNSUP), (dict(T=2 ** 28), {}, EUNSUP),
    ({}, dict(logits=None), EINVAL), ({}, dict(w=None), EINVAL), ({}, dict(x=None), EINVAL), ({}, dict(off=None), EINVAL),
    ({}, dict(rows=None), EINVAL), ({}, dict(slots=None), EINVAL), ({}, dict(logits=MIS4), EINVAL),
    ({}, dict(bias=MIS4), EINVAL), ({}, dict(slots=MIS4), EINVAL), (dict(T=2100), dict(ws=None), EWS),
    (dict(T=2100), dict(nws=132 * 64 * 4 - 1), EWS), (dict(T=2100), dict(ws=MIS4), EWS),
    (dict(T=0), dict(off=None, rows=None, slots=None), 0),
])
def test_route_refusals(kw, call, want):
    assert route(route_desc(**kw), **call) == want


@pytest.mark.parametrize("T,want", [(2 ** 25 - 1, EINVAL), (2 ** 25, EUNSUP)])
def test_route_token_limit(T, want):
    # fewer than 2^25 tokens are within the limits: what is then wrong is the missing pointer
    d = route_desc(T=T, top=1)
    assert route(d, logits=None) == want
    assert spg.lib.expert_route_backward(FAR, None, FAR, FAKE, ctypes.byref(d), None) == want


def test_order_workspace():
    n = spg.lib.expert_order_workspace_bytes
    assert n(2048, 8, 256) == 0 and n(0, 8, 8) == 0 and n(3000, 8, 0) == 0 and n(3000, 8, 1025) == 0 and n(3000, 0, 8) == 0
    assert n(2049, 8, 256) == 129 * 256 * 4                    # chunks of 16 tokens
    assert n(8192, 8, 128) == 256 * 128 * 4                    # of 32
    assert n(10 ** 6, 8, 1024) == 255 * 1024 * 4               # of 3936: at most 256 chunks


def test_sort_and_backward_refusals():
    sort = lambda x=FAKE, T=100, top=4, E=64, off=FAR, rows=FAR, slots=FAR, ws=FAR, nws=1 << 20: spg.lib.expert_sort(  # noqa: E731
        x, T, top, E, off, rows, slots, ws, nws, None)
    assert [sort(T=-1), sort(top=0), sort(E=0), sort(x=None), sort(off=None), sort(rows=None), sort(slots=None),
            sort(x=MIS4), sort(E=1025), sort(T=2 ** 30), sort(T=5000, ws=None), sort(T=5000, nws=8)] == \
        [EINVAL] * 8 + [EUNSUP] * 2 + [EWS] * 2
    back = lambda d, g=FAR, l=FAKE, x=FAR, o=P(0x8000000): spg.lib.expert_route_backward(g, l, x, o, ctypes.byref(d), None)  # noqa: E731,E741
    assert [back(route_desc(top=33)), back(route_desc(top=65)), back(route_desc(), g=None), back(route_desc(), l=None),
            back(route_desc(), x=None), back(route_desc(), o=None), back(route_desc(), o=FAKE),
            back(route_desc(), l=MIS4), back(route_desc(T=0), g=None)] == [EUNSUP] + [EINVAL] * 7 + [0]


def combine(y=FAR, R=80, ldy=64, w=FAR, s=FAR, T=10, top=8, H=64, res=None, ldr=64, out=FAKE, ldo=64):
    return spg.lib.expert_combine(y, R, ldy, w, s, T, top, H, res, ldr, out, ldo, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), EINVAL), (dict(R=-1), EINVAL), (dict(H=-1), EINVAL), (dict(top=0), EINVAL), (dict(top=33), EUNSUP),
    (dict(ldy=63), EINVAL), (dict(ldo=63), EINVAL), (dict(res=FAR, ldr=63), EINVAL), (dict(y=None), EINVAL),
    (dict(w=None), EINVAL), (dict(s=None), EINVAL), (dict(out=None), EINVAL), (dict(w=MIS4), EINVAL),
    (dict(y=P(0x100001)), EINVAL), (dict(y=FAKE), EINVAL), (dict(w=FAKE), EINVAL), (dict(s=FAKE), EINVAL),
    (dict(res=P(0x100002)), EINVAL), (dict(res=FAKE, ldr=72), EINVAL), (dict(T=0, y=None, out=None), 0),
    (dict(H=0), 0),
])
def test_combine_refusals(kw, want):
    assert combine(**kw) == want


def test_combine_backward_refusals():
    def back(g=FAR, ldg=64, y=FAR, R=80, ldy=64, w=FAR, s=FAR, T=10, top=8, H=64, gy=FAKE, ldgy=64, gw=P(0x8000000)):
        return spg.lib.expert_combine_backward(g, ldg, y, R, ldy, w, s, T, top, H, gy, ldgy, gw, None)
    bad = [dict(T=-1), dict(top=0), dict(ldg=63), dict(ldy=63), dict(ldgy=63), dict(g=None), dict(y=None), dict(w=None),
           dict(s=None), dict(gy=None), dict(gw=None), dict(gw=MIS4), dict(y=FAKE), dict(g=FAKE), dict(w=FAKE),
           dict(s=FAKE), dict(gw=FAKE), dict(gw=FAR)]
    assert [back(**k) for k in bad] == [EINVAL] * len(bad)
    assert back(top=33) == EUNSUP and back(T=0, g=None) == 0


def test_outputs_overlap_nothing():
    at = lambda n: P(0x100000 + n)                             # noqa: E731
    assert [quant(q=at(0)), quant(q=at(2 * 32 * 256 - 16), scale=FAR), quant(q=FAR, scale=at(16380)),
            quant(q=FAR, scale=P(FAR.value + 32 * 256 - 4)), quant(tiling=2, q=FAR, scale=P(FAR.value - 4))] == [EINVAL] * 5
    outs = [P(0x40000000 + (i << 24)) for i in range(6)]       # weights, experts, offsets, rows, slots, workspace
    d = route_desc(T=3000)
    for i in range(6):
        for j in range(i):
            o = list(outs)
            o[i] = o[j]
            assert route(d, FAKE, FAR, *o) == EINVAL, (i, j)
            if j >= 2:
                assert spg.lib.expert_sort(FAKE, 3000, 8, 64, *o[2:], 1 << 20, None) == EINVAL
        assert route(d, outs[i], FAR, *outs) == EINVAL and route(d, FAKE, outs[i], *outs) == EINVAL
        if i >= 2:
            assert spg.lib.expert_sort(outs[i], 3000, 8, 64, *outs[2:], 1 << 20, None) == EINVAL
    for g, l, x in ((FAR, FAR, FAKE), (FAKE, FAR, FAR), (FAR, FAKE, FAR)):   # noqa: E741
        assert spg.lib.expert_route_backward(g, l, x, FAKE, ctypes.byref(route_desc()), None) == EINVAL


def test_strides_past_64_bits():
    big = 2 ** 62
    assert quant(ldx=big) == EUNSUP and quant(ldq=big) == EUNSUP
    assert quant(batch=4, bs=big, qbs=8192) == EUNSUP and quant(batch=4, bs=8192, qbs=big) == EUNSUP
    assert grouped(grouped_desc(stride_w=big)) == EUNSUP
    assert route(route_desc(ld=big)) == EUNSUP and route(route_desc(T=2 ** 25, top=1)) == EUNSUP
    assert combine(ldy=big) == EUNSUP and combine(ldo=big) == EUNSUP and combine(res=FAR, ldr=big) == EUNSUP
    assert combine(T=2 ** 23, top=1) == EUNSUP and combine(R=2 ** 31) == EUNSUP


# ---- Python binding -----------------------------------------------------------

def t(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="meta")


def refuses(match, f, *a, **k):
    with pytest.raises(ValueError, match=match):
        f(*a, **k)


def test_quantize_binding():
    q = spg.quantize_block128
    refuses("CUDA", q, t((4, 256), BF))
    refuses("CUDA", q, t((2, 4, 256), BF), "block", out=t((2, 4, 256), U8), scale=t((2, 1, 2), F32))
    refuses("bf16", q, t((4, 256), F32))
    refuses("2-D or 3-D", q, t((256,), BF))
    refuses("tiling", q, t((4, 256), BF), "tile")
    refuses("multiple of 16", q, t((4, 250), BF))
    refuses("contiguous", q, t((256, 4), BF).t())
    refuses("row stride", q, t((4, 260), BF)[:, :256])
    refuses("must not overlap", q, t((4, 256), BF).expand(3, 4, 256))
    refuses("out must be", q, t((4, 256), BF), out=t((4, 128), U8))
    refuses("scale must be", q, t((4, 256), BF), scale=t((4, 2), F32))
    refuses("out rows", q, t((4, 256), BF), out=t((4, 264), U8)[:, :256])


def test_gemm_binding():
    def g(M=64, N=256, K=400, sa=None, sw=None, **k):
        return spg.gemm_scaled(t((M, K), U8), sa if sa is not None else t((4, M), F32), t((N, K), U8),
                               sw if sw is not None else t((2, 4), F32), fmt="e4m3_block128", **k)
    refuses("CUDA", g)
    refuses("CUDA", g, epilogue="swiglu")
    refuses("multiple of 256", g, N=384, sw=t((3, 4), F32), epilogue="swiglu")
    refuses("sa must be", g, sa=t((64, 4), F32))
    refuses("sw must be", g, sw=t((4, 2), F32))
    refuses("fp32", g, sa=t((4, 64), BF))
    refuses("sa must be", g, sa=t((64, 4), F32).t())
    f = spg.gemm_scaled
    refuses("CUDA", f, t((400, 64), U8), t((4, 64), F32), t((400, 256), U8), t((4, 2), F32), fmt="e4m3_block128",
            a_kmajor=True, w_kmajor=True)
    refuses("sw must be", f, t((64, 400), U8), t((4, 64), F32), t((400, 256), U8), t((2, 4), F32), fmt="e4m3_block128",
            w_kmajor=True)


def test_grouped_binding():
    def g(A=None, sa=None, W=None, sw=None, off=None, **k):
        return spg.gemm_grouped(A if A is not None else t((10, 400), U8), sa if sa is not None else t((4, 10), F32),
                                W if W is not None else t((3, 256, 400), U8), sw if sw is not None else t((3, 2, 4), F32),
                                off if off is not None else t((4,), I32), **k)
    refuses("CUDA", g)
    refuses("CUDA", g, epilogue="swiglu", rows=t((33,), I32), out=t((33, 128), BF))
    refuses("store or swiglu", g, epilogue="add")
    refuses("disagree on K", g, A=t((10, 384), U8))
    refuses("A must be", g, A=t((10, 400), F32))
    refuses("W must be", g, W=t((256, 400), U8))
    refuses("multiple of 16", g, A=t((10, 392), U8), W=t((3, 256, 392), U8))
    refuses("multiple of 256", g, W=t((3, 384, 400), U8), sw=t((3, 3, 4), F32), epilogue="swiglu")
    refuses("sa must be", g, sa=t((10, 4), F32))
    refuses("sw must be", g, sw=t((2, 4), F32))
    refuses("offsets must be", g, off=t((3,), I32))
    refuses("offsets must be", g, off=t((4,), torch.int64))
    refuses("rows must be", g, rows=t((2, 5), I32))
    refuses("rows must be", g, rows=t((5,), torch.int64))
    refuses("out must have", g, out=t((10, 128), BF))
    refuses("out must be", g, out=t((10, 256), F32))
    refuses("must not overlap", g, out=t((1, 256), BF).expand(10, 256))
    refuses("16-byte", g, A=t((10, 408), U8)[:, :400])


def test_route_binding():
    r = spg.expert_route
    refuses("CUDA", r, t((5, 64), F32), 8)
    refuses("CUDA", r, t((5, 64), BF), 8, score="sigmoid", bias=t((64,), F32), groups=8, top_groups=4)
    refuses("fp32 or bf16", r, t((5, 64), torch.float16), 8)
    refuses("2-D", r, t((64,), F32), 8)
    refuses("contiguous", r, t((64, 5), F32).t(), 8)
    refuses("overlap", r, t((1, 64), F32).expand(5, 64), 8)
    refuses("score", r, t((5, 64), F32), 8, score="relu")
    refuses("top must", r, t((5, 64), F32), 65)
    refuses("top must", r, t((5, 64), F32), 0)
    refuses("groups", r, t((5, 64), F32), 8, groups=7)
    refuses("groups", r, t((5, 64), F32), 8, groups=8, top_groups=9)
    refuses("finite", r, t((5, 64), F32), 8, scale=float("inf"))
    # a tensor's value may change while its place in a signature does not
    refuses("number", r, t((5, 64), F32), 8, scale=torch.tensor(2.5))
    refuses("ints", r, t((5, 64), F32), torch.tensor(8))
    refuses("ints", r, t((5, 64), F32), 8.0)
    refuses("bias", r, t((5, 64), F32), 8, bias=t((64,), BF))
    refuses("bias", r, t((5, 64), F32), 8, bias=t((63,), F32))
    s = spg.expert_sort
    refuses("CUDA", s, t((5, 8), I32), 64)
    refuses("int32", s, t((5, 8), torch.int64), 64)
    refuses("at least one", s, t((5, 8), I32), 0)
    b = spg.expert_route_backward
    refuses("CUDA", b, t((5, 8), F32), t((5, 64), BF), t((5, 8), I32))
    refuses("grad_weights", b, t((5, 8), BF), t((5, 64), BF), t((5, 8), I32))
    refuses("number", b, t((5, 8), F32), t((5, 64), BF), t((5, 8), I32), scale=torch.tensor(2.5))
    refuses("grad_weights", b, t((5, 7), F32), t((5, 64), BF), t((5, 8), I32))
    refuses("experts", b, t((5, 8), F32), t((6, 64), BF), t((5, 8), I32))


def test_combine_binding():
    c = spg.expert_combine
    y, w, s = t((40, 64), BF), t((5, 8), F32), t((5, 8), I32)
    refuses("CUDA", c, y, w, s)
    refuses("CUDA", c, y, w, s, residual=t((5, 64), BF), out=t((5, 64), BF))
    refuses("y must be", c, t((40, 64), F32), w, s)
    refuses("weights", c, y, t((5, 8), BF), s)
    refuses("weights", c, y, t((5, 7), F32), s)
    refuses("slots", c, y, w, t((40,), I32))
    refuses("slots", c, y, w, t((5, 8), torch.int64))
    refuses("residual", c, y, w, s, residual=t((5, 63), BF))
    refuses("residual", c, y, w, s, residual=t((5, 64), F32))
    refuses("out", c, y, w, s, out=t((4, 64), BF))
    b = spg.expert_combine_backward
    refuses("CUDA", b, t((5, 64), BF), y, w, s)
    refuses("disagree", b, t((6, 64), BF), y, w, s)
    refuses("grad_out", b, t((5, 60), BF), y, w, s)
    refuses("grad_y", b, t((5, 64), BF), y, w, s, grad_y=t((39, 64), BF))
