"""Refusals of gemm_grouped_dw (CPU only, nothing is launched): the C ABI with
pointers that are never dereferenced, and the Python binding with tensors on
torch's "meta" device.
"""
import ctypes

import pytest
import torch

import scaled_precision_gemm_amd as spg

P = ctypes.c_void_p
EINVAL, EUNSUP, EWS = 1, 2, 3
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def at(k, off=0):
    """Addresses 2^42 apart that are never dereferenced."""
    return P((k + 1 << 42) + off)


def desc(**kw):
    d = dict(rows=1024, x_rows=1024, N=512, K=256, ldy=None, ldx=None, ldo=None, stride_o=None, lda=None, stride_a=None,
             experts=4, out_fp32=0)
    d.update(kw)
    for name, v in (("ldy", d["N"]), ("ldx", d["K"]), ("ldo", d["K"]), ("lda", d["K"]), ("stride_o", d["N"] * d["K"]),
                    ("stride_a", d["N"] * d["K"])):
        if d[name] is None:
            d[name] = v
    return spg.GroupedDwDesc(**d)


def call(d, out=at(0), dy=at(1), x=at(2), off=at(3), idx=None, add=None, ws=at(6), ws_bytes=None):
    n = spg.lib.gemm_grouped_dw_workspace_bytes(ctypes.byref(d)) if ws_bytes is None else ws_bytes
    return spg.lib.gemm_grouped_dw(out, dy, x, off, idx, add, ctypes.byref(d), ws, n, None)


DENSE = dict(rows=4096, x_rows=4096, experts=1)     # eight tiles, cut into slices: needs a workspace


@pytest.mark.parametrize("kw,args,want", [
    (dict(rows=-1), {}, EINVAL), (dict(x_rows=-1), {}, EINVAL), (dict(N=-8), {}, EINVAL), (dict(K=-8), {}, EINVAL),
    (dict(N=516), {}, EINVAL), (dict(K=260), {}, EINVAL), (dict(experts=0), {}, EINVAL), (dict(experts=65537), {}, EUNSUP),
    (dict(ldy=504), {}, EINVAL), (dict(ldx=248), {}, EINVAL), (dict(ldy=516), {}, EINVAL), (dict(ldx=260), {}, EINVAL),
    (dict(ldy=2 ** 24 + 8), {}, EUNSUP), (dict(ldx=2 ** 24 + 8), {}, EUNSUP), (dict(ldo=248), {}, EINVAL),
    (dict(ldo=260), {}, EINVAL), (dict(ldo=258, out_fp32=1), {}, EINVAL), (dict(stride_o=512 * 256 + 4), {}, EINVAL),
    (dict(stride_o=512 * 256 - 8), {}, EINVAL), (dict(stride_o=0), {}, EINVAL), (dict(stride_o=2 ** 56), {}, EUNSUP),
    (dict(ldo=2 ** 50), {}, EUNSUP), (dict(stride_o=-512 * 256), {}, EINVAL),
    (dict(lda=248), dict(add=at(5)), EINVAL), (dict(lda=260), dict(add=at(5)), EINVAL),
    (dict(stride_a=0), dict(add=at(5)), EINVAL), (dict(stride_a=2 ** 56), dict(add=at(5)), EUNSUP),
    (dict(rows=2 ** 31, x_rows=2 ** 31), {}, EUNSUP), (dict(x_rows=2 ** 31), {}, EUNSUP), (dict(N=2 ** 29), {}, EUNSUP),
    (dict(x_rows=1023), {}, EINVAL), (dict(x_rows=2 ** 22), dict(idx=at(4)), EUNSUP),
    (dict(experts=65536, N=2 ** 16, K=4096), {}, EUNSUP),                                  # tiles
    ({}, dict(out=None), EINVAL), ({}, dict(dy=None), EINVAL), ({}, dict(x=None), EINVAL), ({}, dict(off=None), EINVAL),
    ({}, dict(out=at(0, 8)), EINVAL), ({}, dict(dy=at(1, 8)), EINVAL), ({}, dict(x=at(2, 8)), EINVAL),
    ({}, dict(off=at(3, 2)), EINVAL), ({}, dict(idx=at(4, 2)), EINVAL), ({}, dict(add=at(5, 8)), EINVAL),
    (DENSE, dict(ws=None), EWS), (DENSE, dict(ws_bytes=64), EWS), (DENSE, dict(ws=at(6, 8)), EWS),
    ({}, dict(out=at(1)), EINVAL), ({}, dict(out=at(2, 4096)), EINVAL), ({}, dict(out=at(3)), EINVAL),
    ({}, dict(out=at(4), idx=at(4)), EINVAL), ({}, dict(add=at(0, 16)), EINVAL), (dict(lda=264, stride_a=2 ** 20), dict(add=at(0)), EINVAL),
    (DENSE, dict(ws=at(0)), EINVAL), (DENSE, dict(ws=at(1)), EINVAL), (DENSE, dict(ws=at(2)), EINVAL),
    (DENSE, dict(ws=at(5), add=at(5)), EINVAL), (DENSE, dict(ws=at(3)), EINVAL),
    (dict(N=0), {}, 0), (dict(K=0), {}, 0), (dict(N=0), dict(out=None, dy=None, x=None, off=None), 0),
])
def test_refusals(kw, args, want):
    assert call(desc(**kw), **args) == want


def test_needs_a_desc():
    assert spg.lib.gemm_grouped_dw(at(0), at(1), at(2), at(3), None, None, None, None, 0, None) == EINVAL
    assert spg.lib.gemm_grouped_dw_workspace_bytes(None) == 0


def test_workspace():
    f = lambda **kw: spg.lib.gemm_grouped_dw_workspace_bytes(ctypes.byref(desc(**kw)))  # noqa: E731
    tile = 256 * 256 * 4
    assert f() == 0 and f(N=516) == 0                       # 256 rows an expert; an invalid call
    assert f(**DENSE) == 4 * 15 * tile // 2                 # four tiles of 128 x 256 in fifteen parts
    assert f(rows=4000, x_rows=4000, N=2048, K=2048, experts=1) == 128 * 2 * tile // 2
    assert f(rows=4000, x_rows=4000, N=4096, K=2048, experts=1) == 0
    assert f(rows=4000, x_rows=4000, N=4096, K=2304, experts=1) == 0    # 144 tiles of 256 x 256
    assert spg.grouped_dw_workspace(4096, 1, 512, 256, "cpu").numel() == 4 * 15 * tile // 2
    assert spg.grouped_dw_workspace(1024, 4, 512, 256, "cpu") is None


# ---- binding ------------------------------------------------------------------------

def T(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("kw", [
    dict(dY=T(100, 64, dtype=F32)), dict(dY=T(64)), dict(dY=None), dict(dY=T(64, 100).t()), dict(dY=T(100, 60)),
    dict(dY=T(100, 68)[:, :64]), dict(X=T(100, 44)), dict(X=T(99, 48)), dict(X=T(100, 48, dtype=F32)),
    dict(X=torch.empty(100, 48, dtype=BF)), dict(offsets=T(5, dtype=torch.int64)), dict(offsets=T(1, dtype=I32)),
    dict(offsets=T(10, dtype=I32)[::2]), dict(offsets=None), dict(rows=T(99, dtype=I32)), dict(rows=T(100)),
    dict(dtype=torch.float16), dict(out=T(4, 64, 48, dtype=F32)), dict(out=T(3, 64, 48)), dict(out=T(4, 64, 52)[:, :, :48]),
    dict(out=T(64, 48).expand(4, 64, 48)), dict(out=T(4, 48, 64).transpose(1, 2)), dict(add=T(4, 64, 48, dtype=F32)),
    dict(add=T(4, 64, 40)), dict(add=T(64, 48).expand(4, 64, 48)), dict(dtype=F32, add=T(4, 64, 48)),
])
def test_binding_refusals(kw):
    args = dict(dY=T(100, 64), X=T(100, 48), offsets=T(5, dtype=I32))
    args.update(kw)
    with pytest.raises((ValueError, TypeError)) as e:
        spg.gemm_grouped_dw(**args)
    assert "CUDA" not in str(e.value)


def test_binding_wants_a_gpu_tensor():
    for kw in (dict(), dict(rows=T(100, dtype=I32), X=T(7, 48)), dict(dtype=F32, add=T(4, 64, 48, dtype=F32))):
        with pytest.raises(ValueError, match="CUDA"):
            spg.gemm_grouped_dw(**{"dY": T(100, 64), "X": T(100, 48), "offsets": T(5, dtype=I32), **kw})
