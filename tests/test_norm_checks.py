"""Refusals of rms_norm and rms_norm_backward (CPU only, nothing is launched):
the C ABI with pointers that are never dereferenced, and the Python binding
with tensors on torch's "meta" device.
"""
import ctypes
import math

import pytest
import torch

import scaled_precision_gemm_amd as spg

P = ctypes.c_void_p
EINVAL, EUNSUP, EWS = 1, 2, 3
BF, U8, F32 = torch.bfloat16, torch.uint8, torch.float32


def at(k, off=0):
    """Addresses 2^36 apart that are never dereferenced."""
    return P((k + 1 << 36) + off)


def norm(output=0, R=32, H=256, x=at(0), residual=None, weight=at(1), h=None, normed=at(3), q=None, scale=None,
         rstd=None, call=spg.lib.rms_norm, **kw):
    if output:
        q, scale = kw.pop("q_", at(4)), kw.pop("scale_", at(5))
    d = dict(R=R, H=H, ldx=H, ldr=H, ldh=H, ldn=H, ldq=H, eps=1e-6, weight_offset=0.0, weight_fp32=0, output=output)
    d.update(kw)
    desc = spg.NormDesc(**d)
    return call(x, residual, weight, h, normed, q, scale, rstd, ctypes.byref(desc), None)


@pytest.mark.parametrize("kw,want", [
    (dict(output=3), EINVAL), (dict(output=-1), EINVAL), (dict(R=-1), EINVAL), (dict(H=0), EINVAL),
    (dict(H=32769), EUNSUP), (dict(H=256, R=2 ** 26), EUNSUP), (dict(H=2049, R=2 ** 24), EUNSUP),
    (dict(H=8193, R=2 ** 22), EUNSUP), (dict(eps=-1e-6), EINVAL), (dict(eps=math.nan), EINVAL),
    (dict(eps=math.inf), EINVAL), (dict(weight_offset=math.nan), EINVAL), (dict(weight_offset=math.inf), EINVAL),
    (dict(ldx=255), EINVAL), (dict(ldn=255), EINVAL), (dict(ldx=2 ** 56), EUNSUP), (dict(ldn=2 ** 56), EUNSUP),
    (dict(x=None), EINVAL), (dict(weight=None), EINVAL), (dict(normed=None), EINVAL),
    (dict(q=at(4)), EINVAL), (dict(scale=at(5)), EINVAL),                      # a bf16 output has neither
    (dict(residual=at(6)), EINVAL), (dict(h=at(7)), EINVAL),                   # both or none
    (dict(residual=at(6), h=at(7), ldr=255), EINVAL), (dict(residual=at(6), h=at(7), ldh=255), EINVAL),
    (dict(x=at(0, 1)), EINVAL), (dict(normed=at(3, 1)), EINVAL), (dict(weight=at(1, 1)), EINVAL),
    (dict(weight=at(1, 2), weight_fp32=1), EINVAL), (dict(rstd=at(8, 2)), EINVAL),
    (dict(output=1, H=264), EINVAL), (dict(output=1, ldq=240), EINVAL), (dict(output=2, ldq=264), EINVAL),
    (dict(output=1, q_=None), EINVAL), (dict(output=2, scale_=None), EINVAL), (dict(output=1, q_=at(4, 8)), EINVAL),
    (dict(output=1, scale_=at(5, 2)), EINVAL),
    # overlaps: an output inside an input or another output, shifted copies of the tensor it may replace
    (dict(normed=at(0, 512)), EINVAL), (dict(normed=at(0), ldn=264), EINVAL), (dict(normed=at(1)), EINVAL),
    (dict(residual=at(6), h=at(0, 2)), EINVAL), (dict(residual=at(6), h=at(6), ldh=264), EINVAL),
    (dict(residual=at(6), h=at(3)), EINVAL), (dict(residual=at(6), h=at(1)), EINVAL),
    (dict(output=1, q_=at(0)), EINVAL), (dict(output=1, q_=at(3)), EINVAL), (dict(output=1, scale_=at(4)), EINVAL),
    (dict(output=2, scale_=at(0)), EINVAL), (dict(rstd=at(3)), EINVAL), (dict(rstd=at(1)), EINVAL),
    (dict(output=1, rstd=at(5)), EINVAL),
    (dict(R=0), 0), (dict(R=0, x=None, weight=None), 0), (dict(R=0, output=2), 0),
])
def test_norm_refusals(kw, want):
    assert norm(**kw) == want


def test_norm_needs_a_desc():
    assert spg.lib.rms_norm(at(0), None, at(1), None, at(3), None, None, None, None, None) == EINVAL
    assert spg.lib.rms_norm_backward(at(0), at(1), None, at(2), at(3), at(4), None, None, None, 0, None) == EINVAL


def backward(R=256, H=256, dy=at(0), h=at(1), dres=None, weight=at(2), rstd=at(3), dx=at(4), dw=at(5), ws=at(6),
             ws_bytes=None, **kw):
    d = dict(R=R, H=H, ldg=H, ldh=H, ldr=H, ldx=H, weight_offset=0.0, weight_fp32=0)
    d.update(kw)
    desc = spg.NormGradDesc(**d)
    n = spg.lib.rms_norm_backward_workspace_bytes(R, H) if ws_bytes is None else ws_bytes
    return spg.lib.rms_norm_backward(dy, h, dres, weight, rstd, dx, dw, ctypes.byref(desc), ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(R=-1), EINVAL), (dict(H=0), EINVAL), (dict(H=32769), EUNSUP), (dict(R=2 ** 26), EUNSUP),
    (dict(weight_offset=math.nan), EINVAL), (dict(ldg=255), EINVAL), (dict(ldh=255), EINVAL), (dict(ldx=255), EINVAL),
    (dict(dres=at(7), ldr=255), EINVAL), (dict(ldg=2 ** 56), EUNSUP), (dict(dres=at(7), ldr=2 ** 56), EUNSUP),
    (dict(dy=None), EINVAL), (dict(h=None), EINVAL), (dict(weight=None), EINVAL), (dict(rstd=None), EINVAL),
    (dict(dx=None), EINVAL), (dict(dy=at(0, 1)), EINVAL), (dict(rstd=at(3, 2)), EINVAL), (dict(dw=at(5, 2)), EINVAL),
    (dict(weight=at(2, 2), weight_fp32=1), EINVAL),
    (dict(ws=None), EWS), (dict(ws_bytes=16), EWS), (dict(ws=at(6, 2)), EWS),
    (dict(dx=at(0, 2)), EINVAL), (dict(dx=at(0), ldx=264), EINVAL), (dict(dx=at(1, 512)), EINVAL),
    (dict(dres=at(7), dx=at(7, 4)), EINVAL), (dict(dx=at(2)), EINVAL), (dict(dx=at(3)), EINVAL),
    (dict(dw=at(0)), EINVAL), (dict(dw=at(4)), EINVAL), (dict(dw=at(2)), EINVAL), (dict(dw=at(6)), EINVAL),
    (dict(ws=at(1)), EINVAL), (dict(ws=at(4)), EINVAL),
    (dict(R=0, dw=None), 0), (dict(R=0, dw=None, dy=None, h=None, rstd=None, dx=None), 0),
])
def test_backward_refusals(kw, want):
    assert backward(**kw) == want


def test_backward_workspace():
    f = spg.lib.rms_norm_backward_workspace_bytes
    assert f(0, 256) == f(1, 5120) == f(8, 5120) == f(-1, 256) == f(9, 0) == f(9, 40000) == 0
    assert f(9, 4096) == 5 * 4096 * 4          # two rows a workgroup, one partial sum each
    for H, parts in ((128, 512), (640, 512), (4096, 512), (5120, 256), (20000, 256)):
        assert parts * H * 4 <= f(10 ** 6, H) <= parts * 2 * H * 4
    assert spg.norm_workspace(1, 5120, "cpu") is None and spg.norm_workspace(9, 5120, "cpu").numel() == f(9, 5120)


# ---- binding ------------------------------------------------------------------------

def T(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


X, W = T(8, 256), T(256)


@pytest.mark.parametrize("kw", [
    dict(x=T(256)), dict(x=T(2, 8, 256)), dict(x=T(8, 256, dtype=torch.float16)), dict(x=T(256, 8).t()),
    dict(x=T(8, 0), weight=T(0)), dict(x=T(1, 256).expand(8, 256)),
    dict(weight=T(255)), dict(weight=T(256, dtype=torch.float64)), dict(weight=T(512)[::2]), dict(weight=None),
    dict(weight=torch.empty(256, dtype=BF)),
    dict(output="e4m3"), dict(output=1), dict(output="e4m3_row", x=T(8, 264), weight=T(264)),
    dict(eps=-1.0), dict(eps=math.nan), dict(eps=torch.tensor(1e-6)), dict(weight_offset=math.inf),
    dict(residual=T(8, 255)), dict(residual=T(8, 256, dtype=F32)), dict(residual=T(9, 256)), dict(h=T(8, 256)),
    dict(residual=X, h=T(8, 255)), dict(normed=True), dict(normed=T(8, 256)), dict(scale=T(8, dtype=F32)),
    dict(out=T(8, 256, dtype=U8)), dict(out=T(8, 255)), dict(output="e4m3_row", out=T(8, 256)),
    dict(output="e4m3_row", out=T(8, 264, dtype=U8)[:, :256]), dict(output="e4m3_row", scale=T(2, 8, dtype=F32)),
    dict(output="e4m3_block128", scale=T(8, dtype=F32)), dict(output="e4m3_block128", scale=T(8, 2, dtype=F32).t()),
    dict(output="e4m3_block128", normed=T(8, 255)),
])
def test_norm_binding_refusals(kw):
    args = dict(x=X, weight=W)
    args.update(kw)
    with pytest.raises((ValueError, TypeError)) as e:
        spg.rms_norm(**args)
    assert "CUDA" not in str(e.value)      # refused before the device is looked at


def test_norm_binding_wants_a_gpu_tensor():
    for kw in (dict(), dict(output="e4m3_row", residual=X, normed=True), dict(output="e4m3_block128", weight=T(256, dtype=F32))):
        with pytest.raises(ValueError, match="CUDA"):
            spg.rms_norm(**{"x": X, "weight": W, **kw})
    with pytest.raises(ValueError, match="CUDA"):
        spg.rms_norm_backward(X, X, W, T(8, dtype=F32), grad_residual=X)


@pytest.mark.parametrize("kw", [
    dict(grad_out=T(256)), dict(grad_out=T(8, 256, dtype=F32)), dict(h=T(8, 255)), dict(h=None), dict(h=T(8, 256, dtype=F32)),
    dict(weight=T(255)), dict(rstd=T(8)), dict(rstd=T(9, dtype=F32)), dict(rstd=None), dict(rstd=T(8, 1, dtype=F32)),
    dict(grad_residual=T(7, 256)), dict(grad_x=T(8, 257)), dict(grad_x=T(8, 256, dtype=F32)), dict(weight_offset=math.nan),
    dict(grad_weight=None), dict(grad_weight=T(256, dtype=F32)),
])
def test_backward_binding_refusals(kw):
    args = dict(grad_out=X, h=X, weight=W, rstd=T(8, dtype=F32))
    args.update(kw)
    with pytest.raises((ValueError, TypeError)) as e:
        spg.rms_norm_backward(**args)
    assert "CUDA" not in str(e.value)


@pytest.mark.parametrize("H,most", [(513, 2 ** 26 - 4), (1024, 2 ** 26 - 4), (2048, 2 ** 26 - 4), (2049, 2 ** 24 - 1), (32768, 2 ** 22 - 1)])
def test_rows_of_a_launch(H, most):
    # 64 lanes a row and four rows a workgroup up to 2048 elements: 2^26 - 3 rows would be 2^32 threads, one too many
    # for a launch.  (Nothing is launched here: the calls without an input are refused behind the sizes' check)
    for output in (0, 1) if H % 16 == 0 else (0,):
        assert norm(output=output, H=H, R=most + 1) == EUNSUP
        assert norm(output=output, H=H, R=most, x=None) == EINVAL
    # the gradients walk over their rows
    assert backward(H=H, R=(2 ** 26 if H <= 2048 else 2 ** 24 if H <= 8192 else 2 ** 22) - 1, dy=None) == EINVAL
