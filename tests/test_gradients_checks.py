"""Refusals of gradient_norm and clip_gradients (CPU only, nothing is
launched): the C ABI with pointers that are never dereferenced, and the Python
binding with tensors on torch's "meta" device.
"""
import ctypes
import math

import pytest
import torch

import scaled_precision_gemm_amd as spg

P = ctypes.c_void_p
EINVAL, EUNSUP, EWS = 1, 2, 3
BF, F32 = torch.bfloat16, torch.float32
NORM, WS = P(1 << 44), P(2 << 44)


def entries(*rows):
    """(src, dst, n, bf16) each, addresses that are never dereferenced."""
    flat = [v for r in rows for v in r]
    return (ctypes.c_int64 * len(flat))(*flat)


def at(k):
    return (k + 1) << 32


def clip(rows, max_norm=1.0, norm=NORM, ws=WS, ws_bytes=1 << 20, count=None):
    e = entries(*rows)
    return spg.lib.clip_gradients(e, len(rows) if count is None else count, max_norm, norm, ws, ws_bytes, None)


GOOD = (at(0), at(1), 100, 0)


@pytest.mark.parametrize("rows,kw,want", [
    ([(at(0), at(1), -1, 0)], {}, EINVAL), ([(0, at(1), 100, 0)], {}, EINVAL), ([(at(0), 0, 100, 0)], {}, EINVAL),
    ([(at(0) + 2, at(1), 100, 0)], {}, EINVAL), ([(at(0), at(1) + 2, 100, 0)], {}, EINVAL),
    ([(at(0) + 1, at(1), 100, 1)], {}, EINVAL), ([(at(0), at(1) + 1, 100, 1)], {}, EINVAL),
    ([(at(0), at(1), 2 ** 44, 0)], {}, EUNSUP), ([GOOD], dict(count=-1), EINVAL),
    ([GOOD], dict(max_norm=-1.0), EINVAL), ([GOOD], dict(max_norm=math.nan), EINVAL), ([GOOD], dict(max_norm=math.inf), EINVAL),
    ([GOOD], dict(norm=None), EINVAL), ([GOOD], dict(norm=P((1 << 44) + 2)), EINVAL),
    ([GOOD], dict(ws=None), EWS), ([GOOD], dict(ws_bytes=23), EWS), ([GOOD], dict(ws=P((2 << 44) + 8)), EWS),
    # shared memory: with another tensor's src or dst, shifted against its own src, with norm and workspace
    ([GOOD, (at(0), at(2), 100, 0)][1:] + [(at(3), at(2) + 396, 100, 0)], {}, EINVAL),
    ([GOOD, (at(1) + 396, at(2), 100, 0)], {}, EINVAL), ([(at(0), at(0) + 4, 100, 0)], {}, EINVAL),
    ([(at(0), at(0), 100, 0), (at(0) + 396, at(0) + 396, 100, 0)], {}, EINVAL),
    ([(at(0), at(0), 100, 1), (at(0), at(0), 100, 1)], {}, EINVAL),
    ([GOOD], dict(norm=P(at(0) + 8)), EINVAL), ([GOOD], dict(norm=P(at(1) + 396)), EINVAL),
    ([GOOD], dict(ws=P(at(0) - 16)), EINVAL), ([GOOD], dict(ws=P(at(1) + 384)), EINVAL), ([GOOD], dict(norm=P((2 << 44) + 4)), EINVAL),
])
def test_clip_refusals(rows, kw, want):
    assert clip(rows, **kw) == want


def test_norm_refusals():
    e = entries(GOOD)
    assert spg.lib.gradient_norm(None, 1, NORM, WS, 1 << 20, None) == EINVAL
    assert spg.lib.gradient_norm(e, 1, None, WS, 1 << 20, None) == EINVAL
    assert spg.lib.gradient_norm(e, 1, NORM, WS, 0, None) == EWS
    assert spg.lib.gradient_norm(e, 2 ** 24 + 1, NORM, WS, 1 << 20, None) == EUNSUP
    assert spg.lib.gradient_norm(e, 1, P(at(0)), WS, 1 << 20, None) == EINVAL
    assert spg.lib.gradient_norm(entries((at(0) + 2, 0, 4, 0)), 1, NORM, WS, 1 << 20, None) == EINVAL


def test_workspace():
    f = lambda *rows: spg.lib.gradient_workspace_bytes(entries(*rows), len(rows))  # noqa: E731
    assert f() == 16 and f((0, 0, 0, 0)) == 16
    assert f(GOOD) == 16 + 8 and f((at(0), 0, 16385, 1)) == 16 + 16
    assert f(*[GOOD] * 121) == 16 + 8 * 121
    assert f((at(0), 0, 10 ** 10, 0)) == 16 + 8 * 2048
    assert f((at(0), 0, -1, 0)) == 0


# ---- binding ------------------------------------------------------------------------

def T(*shape, dtype=F32):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("grads,out", [
    (T(8), None), ([], None), ([None], None), ([3.0], None), ([T(8, dtype=torch.float16)], None),
    ([T(8, dtype=torch.float64)], None), ([T(8, 4).t()], None), ([T(16)[::2]], None), ([T(8), torch.empty(8)], None),
    ([T(8)], T(8)), ([T(8)], []), ([T(8)], [None]), ([T(8)], [T(9)]), ([T(8)], [T(8, dtype=BF)]), ([T(8)], [T(16)[::2]]),
    ([T(8)], [torch.empty(8)]), ([None, T(8)], [T(8), T(8)]),
])
def test_binding_refusals(grads, out):
    with pytest.raises((ValueError, TypeError)) as e:
        spg.clip_gradients(grads, 1.0, out=out)
    assert "CUDA" not in str(e.value)


def test_binding_limits():
    for limit in (-1.0, math.nan, math.inf, None, torch.tensor(1.0)):
        with pytest.raises(ValueError, match="max_norm"):
            spg.clip_gradients([T(8)], limit)
    with pytest.raises(ValueError, match="CUDA"):
        spg.clip_gradients([T(8), None, T(3, 4, dtype=BF)], 1)
    with pytest.raises(ValueError, match="CUDA"):
        spg.gradient_norm([T(8)])
