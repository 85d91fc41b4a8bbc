"""Python binding of the gfx950 scaled low-precision GEMM library.

Argument marshalling only: each function checks dtypes and shapes, allocates
outputs with torch on the input's device (torch is the memory and stream
provider), and calls the C ABI of ``libspg.so`` (declared in
``include/spg.h``) on torch's current stream.  Every step of the path runs in
the library's HIP kernels; there is no fallback.  Importing this package
fails loudly when the library is not built.
"""
from __future__ import annotations

import array
import collections
import ctypes
import itertools
import math
import operator
import os

import torch

__all__ = [
    "quantize_rowwise", "quantize_tensor", "quantize_block16", "quantize_block128", "gemm_scaled", "gemm_grouped",
    "expert_route", "expert_sort", "expert_route_backward", "expert_combine", "expert_combine_backward",
    "ExpertRoute", "expert_workspace", "grouped_tile_rows", "block128_scale_shape",
    "gemm_grouped_dw", "grouped_dw_workspace", "rms_norm", "rms_norm_backward", "RmsNorm", "norm_workspace",
    "gradient_norm", "clip_gradients",
    "gemm_plan", "gemm_workspace", "route_select", "route_cost", "probe_mfma", "probe_read", "probe_fp4_rounding",
    "lib", "LIB_PATH",
    "FMT_E4M3_ROW", "FMT_E4M3_TENSOR", "FMT_NVFP4", "FMT_E4M3_BLOCK128", "EPI_STORE", "EPI_ADD", "EPI_SWIGLU",
    "SpgError", "check_operands", "block16_scale_shape", "SCALES_ROW_MAJOR", "SCALES_BLOCKED", "QUANT_SINGLE_LAUNCH",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspg.so")

FMT_E4M3_ROW, FMT_E4M3_TENSOR, FMT_NVFP4, FMT_E4M3_BLOCK128 = 0, 1, 2, 3
EPI_STORE, EPI_ADD, EPI_SWIGLU = 0, 1, 2
SCALES_ROW_MAJOR, SCALES_BLOCKED = 0, 1
QUANT_SINGLE_LAUNCH = 0x100
_LAYOUT = {"row": SCALES_ROW_MAJOR, "blocked": SCALES_BLOCKED}
_EPI = {"store": EPI_STORE, "add": EPI_ADD, "swiglu": EPI_SWIGLU}
_FMT = {"e4m3_row": FMT_E4M3_ROW, "e4m3_tensor": FMT_E4M3_TENSOR, "nvfp4": FMT_NVFP4,
        "e4m3_block128": FMT_E4M3_BLOCK128}
_TILING = {"row": 0, "column": 1, "block": 2}
_SCORE = {"softmax": 0, "sigmoid": 1}
_NORM = {"bf16": 0, "e4m3_row": 1, "e4m3_block128": 2}


class SpgError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {lib.spg_status_string(status).decode()} (status {status})")
        self.status = status


MAX_OUT_SPLITS = 8
LAYOUT_NT, LAYOUT_A_KMAJOR, LAYOUT_W_KMAJOR = 0, 1, 2
SCALE_BATCH_A, SCALE_BATCH_W = 1, 2


class OutSplit(ctypes.Structure):
    _fields_ = [
        ("count", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("col_end", ctypes.c_int64 * MAX_OUT_SPLITS), ("out", ctypes.c_void_p * MAX_OUT_SPLITS),
        ("ldo", ctypes.c_int64 * MAX_OUT_SPLITS), ("stride_o", ctypes.c_int64 * MAX_OUT_SPLITS),
    ]


class GemmDesc(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("batch", ctypes.c_int64),
        ("lda", ctypes.c_int64), ("ldw", ctypes.c_int64), ("ldo", ctypes.c_int64), ("ldr", ctypes.c_int64),
        ("stride_a", ctypes.c_int64), ("stride_w", ctypes.c_int64),
        ("stride_o", ctypes.c_int64), ("stride_r", ctypes.c_int64),
        ("format", ctypes.c_int32), ("scale_layout", ctypes.c_int32),
        ("tscale_a", ctypes.c_void_p), ("tscale_w", ctypes.c_void_p),
        ("clock_probe", ctypes.c_void_p), ("bias_scale", ctypes.c_void_p),
        ("out_split", ctypes.POINTER(OutSplit)), ("layout", ctypes.c_int32), ("scale_batch", ctypes.c_int32),
    ]


class Plan(ctypes.Structure):
    _fields_ = [
        ("bm", ctypes.c_int32), ("bn", ctypes.c_int32), ("bk", ctypes.c_int32), ("split_k", ctypes.c_int32),
        ("tiles", ctypes.c_int64), ("workgroups", ctypes.c_int64), ("kernel", ctypes.c_int32),
        ("tail_split", ctypes.c_int32), ("tail_tiles", ctypes.c_int64),
        ("tail_bm", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class RouteCandidate(ctypes.Structure):
    _fields_ = [("bm", ctypes.c_int32), ("bn", ctypes.c_int32), ("per_unit", ctypes.c_int32),
                ("factor", ctypes.c_double)]


class GroupedDesc(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("a_rows", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("lda", ctypes.c_int64), ("ldw", ctypes.c_int64), ("stride_w", ctypes.c_int64), ("ldo", ctypes.c_int64),
        ("experts", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class RouteDesc(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int64), ("ld", ctypes.c_int64),
        ("E", ctypes.c_int32), ("top", ctypes.c_int32), ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
        ("score", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("logits_bf16", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class GroupedDwDesc(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("x_rows", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("ldy", ctypes.c_int64), ("ldx", ctypes.c_int64), ("ldo", ctypes.c_int64), ("stride_o", ctypes.c_int64),
        ("lda", ctypes.c_int64), ("stride_a", ctypes.c_int64), ("experts", ctypes.c_int32), ("out_fp32", ctypes.c_int32),
    ]


class NormDesc(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int64), ("H", ctypes.c_int64), ("ldx", ctypes.c_int64), ("ldr", ctypes.c_int64),
        ("ldh", ctypes.c_int64), ("ldn", ctypes.c_int64), ("ldq", ctypes.c_int64), ("eps", ctypes.c_double),
        ("weight_offset", ctypes.c_float), ("weight_fp32", ctypes.c_int32), ("output", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class NormGradDesc(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int64), ("H", ctypes.c_int64), ("ldg", ctypes.c_int64), ("ldh", ctypes.c_int64),
        ("ldr", ctypes.c_int64), ("ldx", ctypes.c_int64), ("weight_offset", ctypes.c_float),
        ("weight_fp32", ctypes.c_int32),
    ]


# Exported symbols and their signatures (mirrors include/spg.h).
_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
SIGNATURES = {
    "quantize_block128": (ctypes.c_int, [_P, _I64, _I64, _I64, _I64, _I64, _P, _I64, _I64, _P, ctypes.c_int, _P]),
    "gemm_grouped": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.POINTER(GroupedDesc), _P]),
    "spg_grouped_tile_rows": (ctypes.c_int, [ctypes.POINTER(GroupedDesc), ctypes.c_int]),
    "expert_order_workspace_bytes": (_SZ, [_I64, _I32, _I32]),
    "expert_route": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(RouteDesc), _P, _SZ, _P]),
    "expert_sort": (ctypes.c_int, [_P, _I64, _I32, _I32, _P, _P, _P, _P, _SZ, _P]),
    "expert_route_backward": (ctypes.c_int, [_P, _P, _P, _P, ctypes.POINTER(RouteDesc), _P]),
    "expert_combine": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _I64, _I32, _I64, _P, _I64, _P, _I64, _P]),
    "expert_combine_backward": (ctypes.c_int, [_P, _I64, _P, _I64, _I64, _P, _P, _I64, _I32, _I64, _P, _I64, _P, _P]),
    "gemm_grouped_dw_workspace_bytes": (_SZ, [ctypes.POINTER(GroupedDwDesc)]),
    "gemm_grouped_dw": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.POINTER(GroupedDwDesc), _P, _SZ, _P]),
    "rms_norm": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(NormDesc), _P]),
    "rms_norm_backward_workspace_bytes": (_SZ, [_I64, _I64]),
    "rms_norm_backward": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(NormGradDesc), _P, _SZ, _P]),
    "gradient_workspace_bytes": (_SZ, [_P, _I64]),
    "gradient_norm": (ctypes.c_int, [_P, _I64, _P, _P, _SZ, _P]),
    "clip_gradients": (ctypes.c_int, [_P, _I64, ctypes.c_double, _P, _P, _SZ, _P]),
    "spg_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "quantize_rowwise": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I64, _P, _P]),
    "quantize_tensor_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "quantize_tensor": (ctypes.c_int, [_P, _I64, _I64, _I64, _I64, _P, _P, _P, _SZ, _P]),
    "quantize_block16_workspace_bytes": (_SZ, [_I64, _I64]),
    "quantize_block16_path": (ctypes.c_int, [_I64, _I64]),
    "quantize_block16": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _P, ctypes.c_int, _P, _SZ, _P]),
    "quantize_block16_noalloc": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _P, ctypes.c_int, _P]),
    "spg_gemm_desc_init": (None, [ctypes.POINTER(GemmDesc), _I64, _I64, _I64, _I32]),
    "gemm_scaled_workspace_bytes": (_SZ, [ctypes.POINTER(GemmDesc), ctypes.c_int]),
    "gemm_scaled": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.POINTER(GemmDesc), _P, _SZ, _P]),
    "spg_route_cost": (ctypes.c_double, [ctypes.POINTER(RouteCandidate), _I64, _I64, _I64, _I32]),
    "spg_route_select": (ctypes.c_int, [ctypes.POINTER(RouteCandidate), _I32, _I64, _I64, _I64, _I32]),
    "spg_gemm_plan": (ctypes.c_int, [ctypes.POINTER(GemmDesc), ctypes.c_int, _I32, ctypes.POINTER(Plan)]),
    "spg_probe_mfma": (ctypes.c_int, [ctypes.c_int, _I64, _I32, _P, _P, _P]),
    "spg_probe_read": (ctypes.c_int, [_P, _I64, _I32, _P, _P]),
    "spg_probe_fp4_rounding": (ctypes.c_int, [_P, _P]),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run scaled_precision_gemm_amd/build.py (hipcc, gfx950)")
    handle = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle


lib = _load()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t: torch.Tensor):
    """torch's current stream on t's device, as a raw hipStream_t value."""
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(status: int, what: str):
    if status != 0:
        raise SpgError(status, what)


def _need(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run(fn, what: str, t: torch.Tensor, *args):
    """Calls the library with t's device current, on that device's current
    stream (the last argument of every launching entry point)."""
    if _current_device() == t.get_device():
        status = fn(*args, _stream(t))
    else:
        with torch.cuda.device(t.device):
            status = fn(*args, _stream(t))
    if status != 0:
        raise SpgError(status, what)


# The checks of a call depend only on what _sig reads of its tensors (and on
# its options), so a call that repeats an earlier one's signature reuses what
# the checks worked out.
_CALLS: dict = {}
_CALLS_MAX = 512


def _checked(key, check):
    hit = _CALLS.get(key)
    if hit is None:
        hit = check()
        if len(_CALLS) >= _CALLS_MAX:
            _CALLS.clear()
        _CALLS[key] = hit
    return hit


def _sig(t):
    """What the argument checks read of a tensor: shape, strides, dtype,
    device and the pointer's alignment (TypeError for a non-tensor)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("arguments must be tensors")
    return (t.shape, t.stride(), t.dtype, t.device, t.data_ptr() & 15)


# ---------------------------------------------------------------------------
# quantizers
# ---------------------------------------------------------------------------

def quantize_rowwise(x: torch.Tensor, out: torch.Tensor | None = None, scale: torch.Tensor | None = None):
    """Per-row E4M3: x bf16 [R, K] -> (codes uint8 [R, K], scales fp32 [R])."""
    _need(x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_cuda, "x must be a 2-D bf16 CUDA tensor")
    _need(x.stride(1) == 1, "x rows must be contiguous")
    R, K = x.shape
    q = out if out is not None else torch.empty((R, K), dtype=torch.uint8, device=x.device)
    s = scale if scale is not None else torch.empty((R,), dtype=torch.float32, device=x.device)
    _check(lib.quantize_rowwise(_ptr(x), R, K, x.stride(0), _ptr(q), q.stride(0), _ptr(s), _stream(x)),
           "quantize_rowwise")
    return q, s


def quantize_tensor(x: torch.Tensor):
    """Per-matrix E4M3: x bf16 [R, K] or [B, R, K] -> (codes, scales fp32 [B])."""
    _need(x.dtype == torch.bfloat16 and x.dim() in (2, 3) and x.is_cuda and x.is_contiguous(),
          "x must be a contiguous 2-D or 3-D bf16 CUDA tensor")
    xb = x.unsqueeze(0) if x.dim() == 2 else x
    B, R, K = xb.shape
    q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    s = torch.empty((B,), dtype=torch.float32, device=x.device)
    nws = lib.quantize_tensor_workspace_bytes(B, R, K)
    ws = torch.empty((max(nws, 16),), dtype=torch.uint8, device=x.device)
    _check(lib.quantize_tensor(_ptr(xb), B, R, K, R * K, _ptr(q), _ptr(s), _ptr(ws), ws.numel(), _stream(x)),
           "quantize_tensor")
    return q, s


def block16_scale_shape(R: int, K: int, layout="row") -> tuple:
    """Shape of the NVFP4 block-scale plane: [R, K/16] row-major, or the
    blocked plane of ceil(R/256) row tiles x K/256 stages x 4096 bytes."""
    if _LAYOUT.get(layout, layout) == SCALES_BLOCKED:
        return ((R + 255) // 256, K // 256, 4096)
    return (R, K // 16)


def quantize_block16(x: torch.Tensor, layout="row", single_launch=False):
    """NVFP4: x bf16 [R, K] -> (codes uint8 [R, K/2], block scales uint8
    (E4M3; [R, K/16] row-major, or the blocked plane of block16_scale_shape),
    tensor scale fp32 [1]).  single_launch requests the one-launch quantizer
    (same results)."""
    _need(x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_cuda and x.is_contiguous(),
          "x must be a contiguous 2-D bf16 CUDA tensor")
    lay = _LAYOUT.get(layout, layout)
    R, K = x.shape
    q = torch.empty((R, K // 2), dtype=torch.uint8, device=x.device)
    bs = torch.empty(block16_scale_shape(R, K, lay), dtype=torch.uint8, device=x.device)
    t = torch.empty((1,), dtype=torch.float32, device=x.device)
    nws = lib.quantize_block16_workspace_bytes(R, K)
    ws = torch.empty((max(nws, 16),), dtype=torch.uint8, device=x.device)
    flags = lay | (QUANT_SINGLE_LAUNCH if single_launch else 0)
    _check(lib.quantize_block16(_ptr(x), R, K, _ptr(q), _ptr(bs), _ptr(t), flags, _ptr(ws), ws.numel(), _stream(x)),
           "quantize_block16")
    return q, bs, t


def block128_scale_shape(R: int, K: int, tiling="row") -> tuple:
    """Shape of quantize_block128's scale plane for one [R, K] matrix: row
    groups [ceil(K/128), R], column groups [ceil(R/128), K], blocks
    [ceil(R/128), ceil(K/128)]."""
    gr, gk = (R + 127) // 128, (K + 127) // 128
    return {"row": (gk, R), "column": (gr, K), "block": (gr, gk)}[tiling]


def _check_block128(x, tiling, out, scale):
    _need(isinstance(x, torch.Tensor) and x.dtype == torch.bfloat16 and x.dim() in (2, 3),
          "x must be a 2-D or 3-D bf16 tensor")
    _need(tiling in _TILING, f"unknown tiling {tiling}")
    _need(x.numel() == 0 or x.stride(-1) == 1, "x rows must be contiguous")
    R, K = x.shape[-2:]
    lead = tuple(x.shape[:-2])
    B = lead[0] if lead else 1
    _need(B >= 1, "x must hold at least one matrix")
    _need(K % 16 == 0, "rows must be a multiple of 16 elements")
    _need(R <= 1 or x.stride(-2) % 8 == 0 and x.stride(-2) >= K, "the row stride must be a multiple of 8, at least K")
    _need(R == 0 or B == 1 or x.stride(0) % 8 == 0 and x.stride(0) >= (R - 1) * x.stride(-2) + K,
          "matrices must not overlap, their stride a multiple of 8")
    shape = lead + block128_scale_shape(R, K, tiling)
    for name, t, want, dt in (("out", out, tuple(x.shape), torch.uint8), ("scale", scale, shape, torch.float32)):
        _need(t is None or (isinstance(t, torch.Tensor) and t.device == x.device and t.dtype == dt
                            and tuple(t.shape) == want), f"{name} must be {dt} {want} on {x.device}")
    ldq, qbs = K, R * K
    if out is not None and R > 0:
        _need(out.stride(-1) == 1 and (R == 1 or out.stride(-2) % 16 == 0 and out.stride(-2) >= K)
              and (B == 1 or out.stride(0) % 16 == 0 and out.stride(0) >= (R - 1) * out.stride(-2) + K),
              "out rows must be contiguous, 16-byte aligned and must not overlap")
        ldq, qbs = out.stride(-2) if R > 1 else K, out.stride(0) if B > 1 else 0
    _need(scale is None or scale.is_contiguous(), "scale must be contiguous")
    _need(x.is_cuda, "x must be a CUDA tensor")
    return (B, R, K, x.stride(-2) if R > 1 else K, x.stride(0) if B > 1 else 0), (ldq, qbs), shape


def quantize_block128(x: torch.Tensor, tiling="row", out: torch.Tensor | None = None,
                      scale: torch.Tensor | None = None):
    """E4M3 with an fp32 scale per 128 elements: x bf16 [R, K] or [B, R, K] ->
    (codes uint8 like x, scales fp32).  tiling "row": 1 x 128 (activations;
    scales group-major [ceil(K/128), R]); "column": 128 x 1 (a K-major A, as
    the weight-gradient product reads it; [ceil(R/128), K]); "block": 128 x
    128 (weights; [ceil(R/128), ceil(K/128)])."""
    dims, strides, shape = _checked(("quantize", tiling, _sig(x), _sig(out), _sig(scale)),
                                    lambda: _check_block128(x, tiling, out, scale))
    q = out if out is not None else x.new_empty(x.shape, dtype=torch.uint8)
    s = scale if scale is not None else x.new_empty(shape, dtype=torch.float32)
    if dims[1] > 0:
        _run(lib.quantize_block128, "quantize_block128", x, x.data_ptr(), *dims, q.data_ptr(), *strides, s.data_ptr(),
             _TILING[tiling])
    return q, s


# ---------------------------------------------------------------------------
# GEMM
# ---------------------------------------------------------------------------

def _desc(fmt: int, M: int, N: int, K: int) -> GemmDesc:
    d = GemmDesc()
    lib.spg_gemm_desc_init(ctypes.byref(d), M, N, K, fmt)
    return d


def _logical_dims(A, W, a_kmajor, w_kmajor):
    """(M, N, K in code bytes) of the product from the stored operands: A is
    [M, K] or, K-major, [K, M]; W is [N, K] or, K-major, [K, N]."""
    M, Ka = (A.shape[-1], A.shape[-2]) if a_kmajor else (A.shape[-2], A.shape[-1])
    N, Kw = (W.shape[-1], W.shape[-2]) if w_kmajor else (W.shape[-2], W.shape[-1])
    return M, N, Ka, Kw


def make_desc(A: torch.Tensor, W: torch.Tensor, fmt, epilogue, out=None, residual=None,
              tscale_a=None, tscale_w=None, a_kmajor=False, w_kmajor=False) -> tuple[GemmDesc, int, int]:
    fmt = _FMT.get(fmt, fmt)
    epi = _EPI.get(epilogue, epilogue)
    _need(A.dtype == torch.uint8 and W.dtype == torch.uint8, "A and W must be uint8 code tensors")
    batched = A.dim() == 3 or W.dim() == 3
    A3 = A if A.dim() == 3 else A.unsqueeze(0)
    W3 = W if W.dim() == 3 else W.unsqueeze(0)
    _need(A3.stride(2) == 1 and W3.stride(2) == 1, "rows must be contiguous")
    batch = max(A3.shape[0], W3.shape[0])
    _need(A3.shape[0] in (1, batch) and W3.shape[0] in (1, batch), "batch sizes must match or be 1")
    M, N, Kc, Kw = _logical_dims(A3, W3, a_kmajor, w_kmajor)
    K = 2 * Kc if fmt == FMT_NVFP4 else Kc
    _need(Kw == Kc, "A and W disagree on K")
    d = _desc(fmt, M, N, K)
    d.layout = (LAYOUT_A_KMAJOR if a_kmajor else 0) | (LAYOUT_W_KMAJOR if w_kmajor else 0)
    d.batch = batch
    d.lda, d.ldw = A3.stride(1), W3.stride(1)
    d.stride_a = A3.stride(0) if A3.shape[0] > 1 else 0
    d.stride_w = W3.stride(0) if W3.shape[0] > 1 else 0
    if fmt == FMT_E4M3_BLOCK128:
        # an operand expanded over the batch: one matrix of codes, a scale plane for each entry
        d.scale_batch = ((SCALE_BATCH_A if A3.shape[0] > 1 and d.stride_a == 0 else 0)
                         | (SCALE_BATCH_W if W3.shape[0] > 1 and d.stride_w == 0 else 0))
    n_out = N // 2 if epi == EPI_SWIGLU else N
    if out is not None:
        o3 = out if out.dim() == 3 else out.unsqueeze(0)
        d.ldo = o3.stride(1)
        d.stride_o = o3.stride(0) if batch > 1 else 0
    else:
        d.ldo = n_out
        d.stride_o = M * n_out if batch > 1 else 0
    if residual is not None and residual.dim() == 1:
        # one row [N]: a bias added to every token row of every batch entry
        _need(residual.shape[0] == n_out and residual.stride(0) == 1, "a bias row must be contiguous [N]")
        d.ldr, d.stride_r = 0, 0
    elif residual is not None:
        r3 = residual if residual.dim() == 3 else residual.unsqueeze(0)
        d.ldr = r3.stride(1)
        d.stride_r = r3.stride(0) if r3.shape[0] > 1 else 0
    if fmt == FMT_NVFP4:
        d.tscale_a = tscale_a.data_ptr() if tscale_a is not None else None
        d.tscale_w = tscale_w.data_ptr() if tscale_w is not None else None
    return d, epi, batched


def check_out_split(segs, M, n_out, batch, batched, dev):
    """The segments of a split output: bf16 tensors [M, w] ([B, M, w] when
    batched), rows contiguous, 16-byte aligned with a row stride that is a
    multiple of 8, widths adding up to the output width with every boundary
    but the last a multiple of 64."""
    _need(isinstance(segs, (list, tuple)) and 1 <= len(segs) <= MAX_OUT_SPLITS,
          f"out_split takes 1 to {MAX_OUT_SPLITS} output tensors")
    end = 0
    for i, t in enumerate(segs):
        _need(isinstance(t, torch.Tensor) and t.device == dev and t.dtype == torch.bfloat16,
              f"output segment {i} must be a bf16 tensor on {dev}")
        _need(t.dim() == (3 if batched else 2), f"output segment {i} must be {'3' if batched else '2'}-D")
        _need(t.shape[-2] == M and (not batched or t.shape[0] == batch), f"output segment {i} has the wrong rows")
        _need(t.stride(-1) == 1 and t.stride(-2) % 8 == 0 and t.data_ptr() % 16 == 0,
              f"output segment {i}: contiguous rows, 16-byte aligned, row stride a multiple of 8")
        end += t.shape[-1]
        _need(t.shape[-1] > 0 and (i + 1 == len(segs) or end % 64 == 0),
              "every output segment boundary but the last must be a multiple of 64 columns")
    _need(end == n_out, f"the output segments must add up to {n_out} columns")


def check_operands(A, sa, W, sw, fmt, epilogue, out=None, residual=None, tscale_a=None, tscale_w=None,
                   scale_layout="row", bias_scale=None, out_split=None, a_kmajor=False, w_kmajor=False):
    """Shapes, dtypes, strides and devices of a gemm_scaled call, checked
    before anything reaches the library (raises ValueError).  The library
    trusts the sizes it is given, so an output, residual or scale tensor
    smaller than the descriptor says would be read or written out of
    bounds."""
    fmt = _FMT.get(fmt, fmt)
    epi = _EPI.get(epilogue, epilogue)
    _need(fmt in (FMT_E4M3_ROW, FMT_E4M3_TENSOR, FMT_NVFP4, FMT_E4M3_BLOCK128), f"unknown format {fmt}")
    _need(epi in (EPI_STORE, EPI_ADD, EPI_SWIGLU), f"unknown epilogue {epilogue}")
    _need(isinstance(A, torch.Tensor) and isinstance(W, torch.Tensor), "A and W must be tensors")
    _need(A.dtype == torch.uint8 and W.dtype == torch.uint8, "A and W must be uint8 code tensors")
    _need(A.dim() in (2, 3) and W.dim() in (2, 3), "A and W must be 2-D or 3-D")
    _need(A.stride(-1) == 1 and W.stride(-1) == 1, "rows of A and W must be contiguous")
    dev = A.device
    for name, t in (("W", W), ("sa", sa), ("sw", sw), ("out", out), ("residual", residual),
                    ("tscale_a", tscale_a), ("tscale_w", tscale_w), ("bias_scale", bias_scale)):
        _need(t is None or (isinstance(t, torch.Tensor) and t.device == dev), f"{name} must be on {dev}")
    Ab = A.shape[0] if A.dim() == 3 else 1
    Wb = W.shape[0] if W.dim() == 3 else 1
    batch = max(Ab, Wb)
    _need(Ab in (1, batch) and Wb in (1, batch), "batch sizes of A and W must match or be 1")
    batched = A.dim() == 3 or W.dim() == 3
    _need(fmt != FMT_NVFP4 or not (a_kmajor or w_kmajor), "K-major operands are taken only by the FP8 formats")
    M, N, Kc, Kw = _logical_dims(A, W, a_kmajor, w_kmajor)
    _need(Kw == Kc, "A and W disagree on K")
    for name, t, km in (("A", A, a_kmajor), ("W", W, w_kmajor)):
        _need(not km or (t.stride(-2) % 16 == 0 and t.data_ptr() % 16 == 0),
              f"a K-major {name} needs 16-byte aligned rows")
    n_out = N // 2 if epi == EPI_SWIGLU else N
    _need(sa is not None and sw is not None, "sa and sw are required")
    if fmt == FMT_E4M3_ROW:
        _need(sa.dtype == torch.float32 and sw.dtype == torch.float32, "row scales must be fp32")
        _need(sa.is_contiguous() and sa.numel() == Ab * M, f"sa must hold {Ab * M} fp32 row scales")
        _need(sw.is_contiguous() and sw.numel() == Wb * N, f"sw must hold {Wb * N} fp32 row scales")
    elif fmt == FMT_E4M3_TENSOR:
        _need(sa.dtype == torch.float32 and sw.dtype == torch.float32, "tensor scales must be fp32")
        _need(sa.is_contiguous() and sa.numel() == Ab, f"sa must hold {Ab} fp32 tensor scale(s)")
        _need(sw.is_contiguous() and sw.numel() == Wb, f"sw must hold {Wb} fp32 tensor scale(s)")
    elif fmt == FMT_E4M3_BLOCK128:
        _need(sa.dtype == torch.float32 and sw.dtype == torch.float32, "block scales must be fp32")
        _need(epi != EPI_SWIGLU or N % 256 == 0, "block-scaled SwiGLU needs N to be a multiple of 256")
        sa_shape = A.shape[:-2] + ((Kc + 127) // 128, M)
        sw_shape = W.shape[:-2] + block128_scale_shape(W.shape[-2], W.shape[-1], "block")
        _need(tuple(sa.shape) == tuple(sa_shape) and sa.is_contiguous(),
              f"sa must be a contiguous {tuple(sa_shape)} plane")
        _need(tuple(sw.shape) == tuple(sw_shape) and sw.is_contiguous(),
              f"sw must be a contiguous {tuple(sw_shape)} plane")
    else:
        _need(not batched, "NVFP4 takes one product (2-D operands)")
        _need(sa.dtype == torch.uint8 and sw.dtype == torch.uint8, "NVFP4 block scales are uint8 E4M3 codes")
        lay = _LAYOUT.get(scale_layout, scale_layout)
        _need(lay in (SCALES_ROW_MAJOR, SCALES_BLOCKED), f"unknown scale layout {scale_layout}")
        _need(lay == SCALES_ROW_MAJOR or (2 * Kc) % 256 == 0, "blocked scale planes need K % 256 == 0")
        sa_shape, sw_shape = block16_scale_shape(M, 2 * Kc, lay), block16_scale_shape(N, 2 * Kc, lay)
        _need(tuple(sa.shape) == sa_shape and sa.is_contiguous(), f"sa must be a contiguous {sa_shape} plane")
        _need(tuple(sw.shape) == sw_shape and sw.is_contiguous(), f"sw must be a contiguous {sw_shape} plane")
        for name, t in (("tscale_a", tscale_a), ("tscale_w", tscale_w)):
            _need(t is not None and t.dtype == torch.float32 and t.numel() == 1, f"{name} must be one fp32 value")
    if out is not None:
        want = (batch, M, n_out) if batched else (M, n_out)
        _need(out.dtype == torch.bfloat16, "out must be bf16")
        _need(tuple(out.shape) == want, f"out must have shape {want}")
        _need(out.stride(-1) == 1, "rows of out must be contiguous")
    if out_split is not None:
        _need(out is None, "out and out_split are exclusive")
        segs = list(out_split)
        if segs and all(isinstance(w, int) for w in segs):
            _need(len(segs) <= MAX_OUT_SPLITS and all(w > 0 for w in segs) and sum(segs) == n_out,
                  f"out_split widths: 1 to {MAX_OUT_SPLITS} positive widths adding up to {n_out}")
            _need(all(sum(segs[:i + 1]) % 64 == 0 for i in range(len(segs) - 1)),
                  "every output segment boundary but the last must be a multiple of 64 columns")
        else:
            check_out_split(segs, M, n_out, batch, batched, dev)
    if bias_scale is not None:
        # an E4M3 bias row: uint8 codes [N], one fp32 scale
        _need(epi == EPI_ADD, "a bias scale is taken only by the add epilogue")
        _need(bias_scale.dtype == torch.float32 and bias_scale.numel() == 1, "bias_scale must be one fp32 value")
        _need(residual is not None and residual.dtype == torch.uint8 and residual.dim() == 1
              and residual.shape[0] == n_out and residual.stride(0) == 1,
              f"with a bias scale the residual must be contiguous uint8 E4M3 codes [{n_out}]")
    elif epi == EPI_ADD:
        _need(residual is not None, "the add epilogue needs a residual")
        _need(residual.dtype == torch.bfloat16, "residual must be bf16")
        _need(residual.stride(-1) == 1, "rows of the residual must be contiguous")
        shapes = [(n_out,), (M, n_out)] + ([(batch, M, n_out), (1, M, n_out)] if batched else [])
        _need(tuple(residual.shape) in shapes, f"residual must have one of the shapes {shapes}")
    else:
        _need(residual is None, "a residual is taken only by the add epilogue")
    return fmt, epi


def gemm_scaled(A, sa, W, sw, epilogue="store", residual=None, fmt="e4m3_row",
                out=None, tscale_a=None, tscale_w=None, workspace=None, clock_probe=None, scale_layout="row",
                bias_scale=None, out_split=None, a_kmajor=False, w_kmajor=False):
    """out = epilogue(scale * A W^T) in bf16.

    e4m3_row: A uint8 [M,K], sa fp32 [M]; W uint8 [N,K], sw fp32 [N]
    e4m3_tensor: A [B,M,K] or [M,K], sa fp32 [B]; W likewise, sw fp32 [B]
    nvfp4: A uint8 [M,K/2], sa uint8 [M,K/16]; W [N,K/2], sw [N,K/16];
           tscale_a, tscale_w fp32 [1]; scale_layout "row" or "blocked" (both
           planes, as quantize_block16 wrote them)
    e4m3_block128: A uint8 [M,K], sa fp32 [ceil(K/128),M]; W [N,K], sw fp32
           [ceil(N/128),ceil(K/128)] ([B, ...] each when batched), as
           quantize_block128 wrote them with tiling "row" (a K-major A:
           "column") and "block" (a K-major W keeps the blocks of its stored
           [K,N]: sw [ceil(K/128),ceil(N/128)]); "swiglu" needs N % 256 == 0.
           Entries of an operand that is expanded over the batch have their
           own scales (in the other formats those of its first entry)
    clock_probe: optional int64 tensor of 4 elements on the same device; the
           main GEMM launch records its clock counters there (see
           spg_gemm_desc.clock_probe): shader clock in GHz =
           (c[1] - c[0]) / (c[3] - c[2]) / 10
    bias_scale: optional fp32 [1] on the same device; with "add" and a
           residual of uint8 E4M3 codes [N], the bias added to every row is
           dec(code) * bias_scale (see spg_gemm_desc.bias_scale); without it
           a 1-D residual is a bf16 bias row
    out_split: optional list of output column widths (ints) or of bf16
           output tensors, one per column segment (see spg_out_split): the
           output goes to them instead of one tensor, and they are returned
           as a list (out must then be None)
    a_kmajor, w_kmajor: the operand is stored K-major - A as [K, M], W as
           [K, N] ([B, K, .] batched), as the backward products read them
           (dX = dY W: w_kmajor; dW = dY^T X: both); FP8 formats only
    """
    segs = None
    if out_split is None:
        # the checks and the descriptor depend only on what _sig reads, so a
        # call that repeats an earlier call's signature reuses its checked
        # descriptor (the per-call pointers are filled in below)
        try:
            key = (fmt, epilogue, scale_layout, a_kmajor, w_kmajor, _sig(A), _sig(sa), _sig(W), _sig(sw),
                   _sig(out), _sig(residual), _sig(tscale_a), _sig(tscale_w), _sig(bias_scale))
            hit = _GEMM_CACHE.get(key)
        except TypeError:      # a non-tensor argument or an unhashable option: the full checks report it
            key = hit = None
        if hit is None:
            hit = _prepare(A, sa, W, sw, fmt, epilogue, out, residual, tscale_a, tscale_w, scale_layout,
                           bias_scale, a_kmajor, w_kmajor)
            if key is not None:
                if len(_GEMM_CACHE) >= _GEMM_CACHE_MAX:
                    _GEMM_CACHE.clear()
                _GEMM_CACHE[key] = hit
        tmpl, epi, out_shape, nws = hit
        d = GemmDesc.from_buffer_copy(tmpl)
    else:
        check_operands(A, sa, W, sw, fmt, epilogue, out, residual, tscale_a, tscale_w, scale_layout, bias_scale,
                       out_split, a_kmajor, w_kmajor)
        _need(A.is_cuda, "operands must be CUDA tensors")
        d, epi, batched = make_desc(A, W, fmt, epilogue, out, residual, tscale_a, tscale_w, a_kmajor, w_kmajor)
        d.scale_layout = _LAYOUT.get(scale_layout, scale_layout)
        segs = list(out_split)
        if all(isinstance(w, int) for w in segs):
            # row strides rounded up to 8 elements (the library's alignment rule)
            segs = [torch.empty((d.batch, d.M, (w + 7) // 8 * 8) if batched else (d.M, (w + 7) // 8 * 8),
                                dtype=torch.bfloat16, device=A.device)[..., :w] for w in segs]
        split = OutSplit()
        split.count = len(segs)
        end = 0
        for i, t in enumerate(segs):
            end += t.shape[-1]
            split.col_end[i] = end
            split.out[i] = t.data_ptr()
            split.ldo[i] = t.stride(-2)
            split.stride_o[i] = t.stride(0) if batched else 0
        d.out_split = ctypes.pointer(split)
        out_shape = None
        nws = lib.gemm_scaled_workspace_bytes(ctypes.byref(d), epi)
    if clock_probe is not None:
        _need(isinstance(clock_probe, torch.Tensor) and clock_probe.dtype == torch.int64 and clock_probe.numel() == 4
              and clock_probe.is_contiguous() and clock_probe.device == A.device,
              "clock_probe must be 4 contiguous int64 values on A's device")
    if tscale_a is not None:
        d.tscale_a = tscale_a.data_ptr()
    if tscale_w is not None:
        d.tscale_w = tscale_w.data_ptr()
    if clock_probe is not None:
        d.clock_probe = clock_probe.data_ptr()
    if bias_scale is not None:
        d.bias_scale = bias_scale.data_ptr()
    if out is None and out_shape is not None:
        out = torch.empty(out_shape, dtype=torch.bfloat16, device=A.device)
    _need(workspace is None or workspace.device == A.device, f"the workspace must be on {A.device}")
    if nws > 0:
        if workspace is None or workspace.numel() < nws:
            workspace = torch.empty((nws,), dtype=torch.uint8, device=A.device)
        wsp, wsn = workspace.data_ptr(), workspace.numel()
    else:
        wsp, wsn = None, 0
    _run(lib.gemm_scaled, "gemm_scaled", A, _ptr(out), A.data_ptr(), _ptr(sa), W.data_ptr(), _ptr(sw), _ptr(residual),
         epi, ctypes.byref(d), wsp, wsn)
    return segs if segs is not None else out


_GEMM_CACHE: dict = {}
_GEMM_CACHE_MAX = 256


def _prepare(A, sa, W, sw, fmt, epilogue, out, residual, tscale_a, tscale_w, scale_layout, bias_scale,
             a_kmajor, w_kmajor):
    """Checks a gemm_scaled call without an output split and returns its
    descriptor with the pointer fields cleared (as bytes), the epilogue code,
    the shape of the output to allocate when none is given, and the
    workspace bytes the library asks for."""
    check_operands(A, sa, W, sw, fmt, epilogue, out, residual, tscale_a, tscale_w, scale_layout, bias_scale,
                   None, a_kmajor, w_kmajor)
    _need(A.is_cuda, "operands must be CUDA tensors")
    d, epi, batched = make_desc(A, W, fmt, epilogue, out, residual, tscale_a, tscale_w, a_kmajor, w_kmajor)
    d.scale_layout = _LAYOUT.get(scale_layout, scale_layout)
    if bias_scale is not None:
        d.bias_scale = bias_scale.data_ptr()
    nws = lib.gemm_scaled_workspace_bytes(ctypes.byref(d), epi)
    d.tscale_a = d.tscale_w = d.bias_scale = None
    n_out = d.N // 2 if epi == EPI_SWIGLU else d.N
    out_shape = (d.batch, d.M, n_out) if batched else (d.M, n_out)
    return bytes(d), epi, out_shape, nws


def gemm_workspace(A, W, fmt="e4m3_row", epilogue="store", out=None, residual=None, a_kmajor=False,
                   w_kmajor=False):
    """A device workspace large enough for gemm_scaled on these operands, or
    None when the plan needs none."""
    d, epi, _ = make_desc(A, W, fmt, epilogue, out, residual, a_kmajor=a_kmajor, w_kmajor=w_kmajor)
    nws = lib.gemm_scaled_workspace_bytes(ctypes.byref(d), epi)
    return torch.empty((nws,), dtype=torch.uint8, device=A.device) if nws > 0 else None


def gemm_plan(M, N, K, fmt="e4m3_row", epilogue="store", batch=1, units=256) -> dict:
    fmt = _FMT.get(fmt, fmt)
    epi = _EPI.get(epilogue, epilogue)
    d = _desc(fmt, M, N, K)
    d.batch = batch
    if batch > 1:
        d.stride_a, d.stride_w = M * d.lda, N * d.ldw
    p = Plan()
    _check(lib.spg_gemm_plan(ctypes.byref(d), epi, units, ctypes.byref(p)), "spg_gemm_plan")
    return {f: getattr(p, f) for f, _ in Plan._fields_}


# ---------------------------------------------------------------------------
# Experts: routing, one product per expert, the weighted sum
# ---------------------------------------------------------------------------

ExpertRoute = collections.namedtuple("ExpertRoute", "weights experts offsets rows slots")


def _index(name, t, shape, dev):
    _need(isinstance(t, torch.Tensor) and t.dtype == torch.int32 and t.device == dev and tuple(t.shape) == tuple(shape)
          and t.is_contiguous(), f"{name} must be a contiguous int32 {tuple(shape)} tensor on {dev}")


def _rows_ok(name, t, dt, dev):
    _need(isinstance(t, torch.Tensor) and t.dim() == 2 and t.dtype == dt and t.device == dev,
          f"{name} must be a 2-D {dt} tensor on {dev}")
    _need(t.numel() == 0 or t.shape[1] == 1 or t.stride(1) == 1, f"rows of {name} must be contiguous")
    _need(t.numel() == 0 or t.shape[0] == 1 or t.stride(0) >= t.shape[1], f"rows of {name} must not overlap")


def _ld(t):
    """Row stride of a 2-D tensor; the row length where it has at most one row."""
    return t.stride(0) if t.shape[0] > 1 and t.numel() else t.shape[1]


def _grouped(A, sa, W, sw, offsets, epilogue, rows, out):
    epi = _EPI.get(epilogue, epilogue)
    _need(epi in (EPI_STORE, EPI_SWIGLU), "the epilogue of experts' products is store or swiglu")
    _need(isinstance(A, torch.Tensor), "A must be a tensor")
    dev = A.device
    _rows_ok("A", A, torch.uint8, dev)
    _need(isinstance(W, torch.Tensor) and W.dim() == 3 and W.dtype == torch.uint8 and W.device == dev,
          f"W must be uint8 codes [experts, N, K] on {dev}")
    E, N, K = W.shape
    a_rows = A.shape[0]
    _need(E >= 1 and A.shape[1] == K, "A and W disagree on K, or W holds no expert")
    _need(K % 16 == 0, "K must be a multiple of 16")
    _need(epi != EPI_SWIGLU or N % 256 == 0, "block-scaled SwiGLU needs N to be a multiple of 256")
    _need(W.stride(2) == 1 or K <= 1, "rows of W must be contiguous")
    for name, t, ld in (("A", A, _ld(A)), ("W", W, W.stride(1) if N > 1 else K)):
        _need(ld % 16 == 0 and ld >= K and t.data_ptr() % 16 == 0, f"rows of {name} must be 16-byte aligned")
    _need(E == 1 or N == 0 or W.stride(0) % 16 == 0 and
          (W.stride(0) == 0 or W.stride(0) >= (N - 1) * (W.stride(1) if N > 1 else K) + K),
          "experts' weights must be 16-byte aligned and must not overlap")
    G = (K + 127) // 128
    for name, t, want in (("sa", sa, (G, a_rows)), ("sw", sw, (E, (N + 127) // 128, G))):
        _need(isinstance(t, torch.Tensor) and t.dtype == torch.float32 and t.device == dev and tuple(t.shape) == want
              and t.is_contiguous(), f"{name} must be a contiguous fp32 {want} plane on {dev}")
    _index("offsets", offsets, (E + 1,), dev)
    R = a_rows
    if rows is not None:
        _need(isinstance(rows, torch.Tensor) and rows.dim() == 1, "rows must be a 1-D int32 tensor")
        R = rows.shape[0]
        _index("rows", rows, (R,), dev)
    n_out = N // 2 if epi == EPI_SWIGLU else N
    if out is not None:
        _rows_ok("out", out, torch.bfloat16, dev)
        _need(tuple(out.shape) == (R, n_out), f"out must have shape {(R, n_out)}")
    d = GroupedDesc(R, a_rows, N, K, _ld(A), W.stride(1) if N > 1 else K, W.stride(0) if E > 1 else 0,
                    n_out if out is None else _ld(out), E, 0)
    _need(A.is_cuda, "operands must be CUDA tensors")
    return d, epi, n_out


def gemm_grouped(A, sa, W, sw, offsets, epilogue="store", rows=None, out=None):
    """One e4m3_block128 product per expert over rows grouped by expert: for
    r in [offsets[e], offsets[e + 1]), out[r] = epilogue(A[rows[r]] W[e]^T)
    (A[r] without rows), bf16 [R, N] ("store") or [R, N/2] ("swiglu").

    A uint8 [T, K], sa fp32 [ceil(K/128), T] (quantize_block128 "row"); W uint8
    [E, N, K], sw fp32 [E, ceil(N/128), ceil(K/128)] ("block"); offsets int32
    [E + 1] and rows int32 [R] as expert_route returns them.  Rows of no
    expert are left as they were (undefined in an output allocated here)."""
    d, epi, n_out = _checked(("grouped", epilogue, _sig(A), _sig(sa), _sig(W), _sig(sw), _sig(offsets), _sig(rows),
                              _sig(out)), lambda: _grouped(A, sa, W, sw, offsets, epilogue, rows, out))
    if out is None:
        out = A.new_empty((d.rows, n_out), dtype=torch.bfloat16)
    if d.rows > 0 and n_out > 0:
        _run(lib.gemm_grouped, "gemm_grouped", A, out.data_ptr(), A.data_ptr(), sa.data_ptr(), W.data_ptr(),
             sw.data_ptr(), offsets.data_ptr(), _ptr(rows), epi, ctypes.byref(d))
    return out


def _grouped_dw(dY, X, offsets, rows, add, out, dtype):
    _need(isinstance(dY, torch.Tensor) and isinstance(X, torch.Tensor), "dY and X must be tensors")
    dev = dY.device
    _rows_ok("dY", dY, torch.bfloat16, dev)
    _rows_ok("X", X, torch.bfloat16, dev)
    (R, N), (x_rows, K) = dY.shape, X.shape
    _need(N % 8 == 0 and K % 8 == 0, "columns of dY and X must be multiples of 8")
    for name, t in (("dY", dY), ("X", X)):
        _need(_ld(t) % 8 == 0 and t.data_ptr() % 16 == 0, f"rows of {name} must be 16-byte aligned")
    _need(isinstance(offsets, torch.Tensor) and offsets.dim() == 1 and offsets.shape[0] >= 2,
          "offsets must be int32 [experts + 1]")
    E = offsets.shape[0] - 1
    _index("offsets", offsets, (E + 1,), dev)
    if rows is None:
        _need(x_rows >= R, "X has fewer rows than dY")
    else:
        _index("rows", rows, (R,), dev)
    _need(dtype in (torch.bfloat16, torch.float32), "dtype must be torch.bfloat16 or torch.float32")
    strides = []
    for name, t in (("out", out), ("add", add)):
        if t is None:
            strides.append((K, N * K))
            continue
        _need(isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == dev and tuple(t.shape) == (E, N, K),
              f"{name} must be a {dtype} {(E, N, K)} tensor on {dev}")
        ld, st, unit = t.stride(1) if N > 1 else K, t.stride(0) if E > 1 else 0, 16 // t.element_size()
        _need(t.numel() == 0 or (t.stride(2) == 1 or K == 1) and ld >= K and ld % unit == 0 and st % unit == 0
              and t.data_ptr() % 16 == 0 and (E == 1 or st >= (N - 1) * ld + K),
              f"rows of {name} must be contiguous, 16-byte aligned and must not overlap")
        strides.append((ld, st))
    d = GroupedDwDesc(R, x_rows, N, K, _ld(dY), _ld(X), *strides[0], *strides[1], E, int(dtype == torch.float32))
    _need(dY.is_cuda, "operands must be CUDA tensors")
    return d, lib.gemm_grouped_dw_workspace_bytes(ctypes.byref(d))


def gemm_grouped_dw(dY, X, offsets, rows=None, add=None, out=None, dtype=torch.bfloat16, workspace=None):
    """The weight gradients of gemm_grouped's products, from bf16 operands:
    out[e] = add[e] + sum over r in [offsets[e], offsets[e + 1]) of dY[r]^T
    X[rows[r]] (X[r] without rows), [experts, N, K] in `dtype` (bf16 or fp32);
    fp32 sums, one rounding at their end (an expert of far more than 16384 rows
    that are alike is better cut into calls that add in fp32).

    dY bf16 [R, N] in expert order; X bf16 [T, K]; offsets int32 [experts + 1]
    and rows int32 [R] as expert_route returns them (an index outside X stands
    for a row of zeros); N and K multiples of 8.  add [experts, N, K] in
    `dtype`, which may be `out` itself (gradients of several chunks).  An
    expert without rows gets add, or zeros.  offsets [0, R] makes it a dense
    layer's weight gradient.  workspace: grouped_dw_workspace(...), else
    allocated where the call needs one."""
    d, nws = _checked(("grouped dw", _sig(dY), _sig(X), _sig(offsets), _sig(rows), _sig(add), _sig(out), dtype),
                      lambda: _grouped_dw(dY, X, offsets, rows, add, out, dtype))
    if out is None:
        out = dY.new_empty((d.experts, d.N, d.K), dtype=dtype)
    if d.N > 0 and d.K > 0:
        ws = _order_ws(workspace, nws, dY)
        _run(lib.gemm_grouped_dw, "gemm_grouped_dw", dY, out.data_ptr(), dY.data_ptr(), X.data_ptr(), offsets.data_ptr(),
             _ptr(rows), _ptr(add), ctypes.byref(d), _ptr(ws), nws)
    return out


def grouped_dw_workspace(rows: int, experts: int, N: int, K: int, device="cuda"):
    """A device workspace for gemm_grouped_dw of `rows` rows, or None when it
    needs none."""
    d = GroupedDwDesc(rows, rows, N, K, N, K, K, N * K, K, N * K, experts, 1)
    n = lib.gemm_grouped_dw_workspace_bytes(ctypes.byref(d))
    return torch.empty((n,), dtype=torch.uint8, device=device) if n > 0 else None


def grouped_tile_rows(rows: int, experts: int, N: int, K: int, epilogue="store") -> int:
    """Rows of the tiles gemm_grouped takes (16, 128 or 256)."""
    epi = _EPI.get(epilogue, epilogue)
    d = GroupedDesc(rows, rows, N, K, K, K, N * K, N // 2 if epi == EPI_SWIGLU else N, experts, 0)
    return lib.spg_grouped_tile_rows(ctypes.byref(d), epi)


def expert_workspace(T: int, top: int, E: int, device="cuda"):
    """A device workspace for the row order of T tokens with `top` of E
    experts each, or None when it needs none."""
    n = lib.expert_order_workspace_bytes(T, top, E)
    return torch.empty((n,), dtype=torch.uint8, device=device) if n > 0 else None


def _order_ws(workspace, n, like):
    if n == 0:
        return None
    if workspace is None:
        return like.new_empty((n,), dtype=torch.uint8)
    _need(isinstance(workspace, torch.Tensor) and workspace.device == like.device and workspace.is_contiguous()
          and workspace.numel() * workspace.element_size() >= n, f"the workspace must hold {n} bytes on {like.device}")
    return workspace


def _route_desc(logits, top, score, groups, top_groups, renormalize, scale):
    _need(isinstance(logits, torch.Tensor) and logits.dim() == 2 and logits.dtype in (torch.float32, torch.bfloat16),
          "logits must be a 2-D fp32 or bf16 tensor")
    _rows_ok("logits", logits, logits.dtype, logits.device)
    T, E = logits.shape
    _need(isinstance(score, str) and score in _SCORE, f"unknown score {score}")
    # plain numbers: they are part of the checked signature by value
    _need(all(isinstance(v, int) for v in (top, groups, top_groups)) and isinstance(scale, (int, float)),
          "top, groups and top_groups must be ints, scale a number")
    _need(1 <= top <= E, "top must be between 1 and the number of experts")
    _need(1 <= top_groups <= groups and E % groups == 0, "groups must divide the experts, top_groups be 1 .. groups")
    _need(math.isfinite(scale), "scale must be finite")
    return RouteDesc(T, _ld(logits), E, top, groups, top_groups, _SCORE[score], int(bool(renormalize)),
                     int(logits.dtype == torch.bfloat16), scale)


def expert_route(logits, top, score="softmax", bias=None, groups=1, top_groups=1, renormalize=True, scale=1.0,
                 order=True, workspace=None):
    """Experts and weights of each token, and the row order of the experts'
    products, from logits [T, E] (fp32 or bf16): ExpertRoute(weights fp32 [T,
    top], experts int32 [T, top], offsets int32 [E + 1], rows int32 [T top],
    slots int32 [T, top]); the last three None with order=False.

    p = softmax or sigmoid of the logits, c = p + bias (fp32 [E]); of `groups`
    runs of consecutive experts, scored by their two largest c, the top_groups
    best stay; experts are the `top` largest c among them, ties to the lowest
    index; weights are scale p / sum p (renormalize) or scale p.  Logits of
    -inf mask an expert: places that no expert is left for hold expert -1,
    weight 0, slot -1.  With the row order, experts, offsets, rows and slots
    are views of one allocation, which lives as long as any of them does (keep
    experts.clone() for a backward pass to free the others)."""
    def check():
        d = _route_desc(logits, top, score, groups, top_groups, renormalize, scale)
        _need(bias is None or (isinstance(bias, torch.Tensor) and bias.dtype == torch.float32
                               and bias.device == logits.device and tuple(bias.shape) == (d.E,)
                               and bias.is_contiguous()),
              f"bias must be a contiguous fp32 [{d.E}] tensor on {logits.device}")
        _need(logits.is_cuda, "logits must be a CUDA tensor")
        return d, lib.expert_order_workspace_bytes(d.T, d.top, d.E)

    d, nws = _checked(("route", _sig(logits), top, score, _sig(bias), groups, top_groups, bool(renormalize), scale), check)
    T = d.T
    weights = logits.new_empty((T, top), dtype=torch.float32)
    if not order:
        experts = logits.new_empty((T, top), dtype=torch.int32)
        _run(lib.expert_route, "expert_route", logits, logits.data_ptr(), _ptr(bias), weights.data_ptr(),
             experts.data_ptr(), None, None, None, ctypes.byref(d), None, 0)
        return ExpertRoute(weights, experts, None, None, None)
    ws = _order_ws(workspace, nws, logits)
    # one allocation for the four int32 outputs (7.2 -> 6.0 us of a call's host time)
    n = T * top
    experts, slots, rows, offsets = logits.new_empty((3 * n + d.E + 1,), dtype=torch.int32).split_with_sizes(
        (n, n, n, d.E + 1))
    experts, slots = experts.view(T, top), slots.view(T, top)
    po = offsets.data_ptr()           # no token: rows and slots are empty and may have no address
    _run(lib.expert_route, "expert_route", logits, logits.data_ptr(), _ptr(bias), weights.data_ptr(),
         experts.data_ptr(), po, rows.data_ptr() or po, slots.data_ptr() or po, ctypes.byref(d), _ptr(ws), nws)
    return ExpertRoute(weights, experts, offsets, rows, slots)


def expert_sort(experts, n_experts, workspace=None):
    """(offsets, rows, slots) of experts int32 [T, top] chosen elsewhere, as
    expert_route gives them; values outside [0, n_experts) are no expert."""
    _need(isinstance(experts, torch.Tensor) and experts.dim() == 2, "experts must be a 2-D int32 tensor")
    T, top = experts.shape
    dev = experts.device
    _index("experts", experts, (T, top), dev)
    _need(top >= 1 and n_experts >= 1, "at least one expert")
    _need(experts.is_cuda, "experts must be a CUDA tensor")
    nws = lib.expert_order_workspace_bytes(T, top, n_experts)
    ws = _order_ws(workspace, nws, experts)
    offsets = experts.new_empty((n_experts + 1,))
    rows = experts.new_empty((T * top,))
    slots = experts.new_empty((T, top))
    _run(lib.expert_sort, "expert_sort", experts, _ptr(experts), T, top, n_experts, _ptr(offsets), _ptr(rows),
         _ptr(slots), _ptr(ws), nws)
    return offsets, rows, slots


def expert_route_backward(grad_weights, logits, experts, score="softmax", renormalize=True, scale=1.0):
    """The gradient of the logits ([T, E], their type) from that of
    expert_route's weights (fp32 [T, top]), for the same logits, options and
    the experts it chose."""
    def check():
        _need(isinstance(experts, torch.Tensor) and experts.dim() == 2, "experts must be a 2-D int32 tensor")
        d = _route_desc(logits, experts.shape[1], score, 1, 1, renormalize, scale)
        dev = logits.device
        _index("experts", experts, (d.T, d.top), dev)
        _need(isinstance(grad_weights, torch.Tensor) and grad_weights.dtype == torch.float32
              and grad_weights.device == dev and tuple(grad_weights.shape) == (d.T, d.top)
              and grad_weights.is_contiguous(), f"grad_weights must be a contiguous fp32 {(d.T, d.top)} tensor on {dev}")
        _need(logits.is_cuda, "logits must be a CUDA tensor")
        return d

    d = _checked(("route backward", _sig(grad_weights), _sig(logits), _sig(experts), score, bool(renormalize), scale),
                 check)
    grad = logits.new_empty((d.T, d.E))
    _run(lib.expert_route_backward, "expert_route_backward", logits, grad_weights.data_ptr(), logits.data_ptr(),
         experts.data_ptr(), grad.data_ptr(), ctypes.byref(d))
    return grad


def _combine_args(y, weights, slots, T):
    _need(isinstance(y, torch.Tensor), "y must be a tensor")
    dev = y.device
    _rows_ok("y", y, torch.bfloat16, dev)
    _need(isinstance(slots, torch.Tensor) and slots.dim() == 2 and slots.shape[1] >= 1, "slots must be int32 [T, top]")
    _need(T is None or slots.shape[0] == T, "slots and the other operands disagree on the tokens")
    _index("slots", slots, slots.shape, dev)
    _need(isinstance(weights, torch.Tensor) and weights.dtype == torch.float32 and weights.device == dev
          and weights.shape == slots.shape and weights.is_contiguous(),
          f"weights must be a contiguous fp32 {tuple(slots.shape)} tensor on {dev}")
    return dev


def expert_combine(y, weights, slots, residual=None, out=None):
    """out[t] = residual[t] + sum_j weights[t, j] y[slots[t, j]] in bf16 [T, H]
    (fp32 sums, one rounding): y bf16 [R, H] the experts' rows, weights and
    slots of expert_route; residual bf16 [T, H], which may be out itself."""
    def check():
        dev = _combine_args(y, weights, slots, None)
        want = (slots.shape[0], y.shape[1])
        for name, t in (("residual", residual), ("out", out)):
            if t is not None:
                _rows_ok(name, t, torch.bfloat16, dev)
                _need(tuple(t.shape) == want, f"{name} must have shape {want}")
        _need(y.is_cuda, "y must be a CUDA tensor")
        return (_ld(y), 0 if residual is None else _ld(residual), want[1] if out is None else _ld(out)), want

    (ldy, ldr, ldo), want = _checked(("combine", _sig(y), _sig(weights), _sig(slots), _sig(residual), _sig(out)), check)
    if out is None:
        out = y.new_empty(want)
    _run(lib.expert_combine, "expert_combine", y, y.data_ptr(), y.shape[0], ldy, weights.data_ptr(), slots.data_ptr(),
         want[0], slots.shape[1], want[1], _ptr(residual), ldr, out.data_ptr(), ldo)
    return out


def expert_combine_backward(grad_out, y, weights, slots, grad_y=None):
    """(grad_y bf16 [R, H], grad_weights fp32 [T, top]) of expert_combine from
    grad_out bf16 [T, H] (which is the residual's gradient as it is).  Rows of
    grad_y that no slot names are left as they were (undefined in one
    allocated here); the slots must be distinct, as expert_route's are."""
    def check():
        _need(isinstance(grad_out, torch.Tensor) and grad_out.dim() == 2, "grad_out must be a 2-D bf16 tensor")
        dev = _combine_args(y, weights, slots, grad_out.shape[0])
        R, H = y.shape
        _rows_ok("grad_out", grad_out, torch.bfloat16, dev)
        _need(grad_out.shape[1] == H, f"grad_out must have shape {(slots.shape[0], H)}")
        if grad_y is not None:
            _rows_ok("grad_y", grad_y, torch.bfloat16, dev)
            _need(tuple(grad_y.shape) == (R, H), f"grad_y must have shape {(R, H)}")
        _need(y.is_cuda, "y must be a CUDA tensor")
        return _ld(grad_out), _ld(y), H if grad_y is None else _ld(grad_y)

    ldg, ldy, ldgy = _checked(("combine backward", _sig(grad_out), _sig(y), _sig(weights), _sig(slots), _sig(grad_y)),
                              check)
    (T, top), (R, H) = slots.shape, y.shape
    if grad_y is None:
        grad_y = y.new_empty((R, H))
    grad_weights = weights.new_empty((T, top))
    _run(lib.expert_combine_backward, "expert_combine_backward", y, grad_out.data_ptr(), ldg, y.data_ptr(), R, ldy,
         weights.data_ptr(), slots.data_ptr(), T, top, H, grad_y.data_ptr(), ldgy, grad_weights.data_ptr())
    return grad_y, grad_weights


# ---------------------------------------------------------------------------
# The norm before the products
# ---------------------------------------------------------------------------

RmsNorm = collections.namedtuple("RmsNorm", "out scale normed h rstd")


def _like(name, t, shape, dt, dev):
    """An optional output: 2-D rows of dtype dt and shape `shape` on dev."""
    if t is not None:
        _rows_ok(name, t, dt, dev)
        _need(tuple(t.shape) == tuple(shape), f"{name} must have shape {tuple(shape)}")


def _new_like(x, dtype=None):
    """A contiguous tensor of x's shape on its device."""
    return x.new_empty(x.shape, dtype=dtype)


def _norm_weight(weight, H, dev):
    _need(isinstance(weight, torch.Tensor) and weight.dtype in (torch.bfloat16, torch.float32) and weight.device == dev
          and tuple(weight.shape) == (H,) and weight.is_contiguous(),
          f"weight must be a contiguous bf16 or fp32 [{H}] tensor on {dev}")


def rms_norm(x, weight, residual=None, output="bf16", eps=1e-6, weight_offset=0.0, normed=False, rstd=False, out=None,
             scale=None, h=None):
    """RMS norm of x (bf16 [R, H]), the residual (bf16 [R, H]) added first:
    h = bf16(x + residual), y = h / sqrt(mean(h^2) + eps) * (weight +
    weight_offset), weight bf16 or fp32 [H]; as RmsNorm(out, scale, normed, h,
    rstd).

    output "bf16": out = bf16(y), scale None.  "e4m3_row": out the E4M3 codes
    of y (uint8 [R, H]) and scale fp32 [R], "e4m3_block128": scale fp32
    [ceil(H/128), R], one per 128 elements of a row: the activations of
    gemm_scaled and gemm_grouped in these formats (y is rounded once, to the
    codes); H % 16 == 0.  normed (True, or a bf16 [R, H] tensor to write to)
    asks for bf16(y) beside the codes; False and None do not.  h is the new
    residual stream, None without a residual; it may be written over x or the
    residual (h=x, h=residual), and so may a bf16 out or normed.  rstd=True
    keeps fp32 [R] 1 / sqrt(..) for rms_norm_backward."""
    def check():
        _need(isinstance(x, torch.Tensor) and x.dim() == 2, "x must be a 2-D bf16 tensor")
        dev = x.device
        R, H = x.shape
        _rows_ok("x", x, torch.bfloat16, dev)
        _need(isinstance(output, str) and output in _NORM, f"unknown output {output}")
        _need(isinstance(eps, (int, float)) and math.isfinite(eps) and eps >= 0, "eps must be a finite number, not below 0")
        _need(isinstance(weight_offset, (int, float)) and math.isfinite(weight_offset), "weight_offset must be a finite number")
        _need(H >= 1, "rows must hold at least one element")
        _norm_weight(weight, H, dev)
        coded = output != "bf16"
        _need(not coded or H % 16 == 0, "rows of codes must be a multiple of 16 elements")
        _need(coded or not given and not normed, "a bf16 output is normed itself")
        _need(coded or scale is None, "a bf16 output has no scale")
        if residual is not None:
            _like("residual", residual, (R, H), torch.bfloat16, dev)
        _need(h is None or residual is not None, "h is an output of the residual's addition")
        _like("h", h, (R, H), torch.bfloat16, dev)
        if isinstance(normed, torch.Tensor):
            _like("normed", normed, (R, H), torch.bfloat16, dev)
        _like("out", out, (R, H), torch.uint8 if coded else torch.bfloat16, dev)
        _need(not coded or out is None or _ld(out) % 16 == 0 and out.data_ptr() % 16 == 0,
              "rows of codes must be 16-byte aligned")
        want = (R,) if output == "e4m3_row" else ((H + 127) // 128, R)
        _need(scale is None or isinstance(scale, torch.Tensor) and scale.dtype == torch.float32 and scale.device == dev
              and tuple(scale.shape) == want and scale.is_contiguous(),
              f"scale must be a contiguous fp32 {want} tensor on {dev}")
        _need(x.is_cuda, "x must be a CUDA tensor")
        n = out if not coded else normed if isinstance(normed, torch.Tensor) else None
        d = NormDesc(R, H, _ld(x), H if residual is None else _ld(residual), H if h is None else _ld(h),
                     H if n is None else _ld(n), H if not coded or out is None else _ld(out), eps, weight_offset,
                     int(weight.dtype == torch.float32), _NORM[output], 0)
        return d, coded, want

    given = isinstance(normed, torch.Tensor)
    # (types beside the numbers: 0.5 equals what is refused, a Fraction for one)
    d, coded, want = _checked(("norm", _sig(x), _sig(weight), _sig(residual), output, eps, type(eps), weight_offset,
                               type(weight_offset), _sig(normed) if given else bool(normed), _sig(out), _sig(scale), _sig(h)),
                              check)
    # (empty_like takes 1.2 us of host time where new_empty takes 1.8; on a
    # contiguous tensor both are contiguous)
    like = torch.empty_like if x.is_contiguous() else _new_like
    if h is None and residual is not None:
        h = like(x)
    if coded:
        if out is None:
            out = like(x, dtype=torch.uint8)
        if scale is None:
            scale = x.new_empty(want, dtype=torch.float32)
        n = normed if given else like(x) if normed else None
    else:
        n = out = like(x) if out is None else out
    r = x.new_empty((d.R,), dtype=torch.float32) if rstd else None
    if d.R > 0:
        _run(lib.rms_norm, "rms_norm", x, x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(h), _ptr(n),
             out.data_ptr() if coded else None, _ptr(scale), _ptr(r), ctypes.byref(d))
    return RmsNorm(out, scale, n, h, r)


def norm_workspace(R: int, H: int, device="cuda"):
    """A device workspace for rms_norm_backward on [R, H], or None when it
    needs none."""
    n = lib.rms_norm_backward_workspace_bytes(R, H)
    return torch.empty((n,), dtype=torch.uint8, device=device) if n > 0 else None


def rms_norm_backward(grad_out, h, weight, rstd, grad_residual=None, weight_offset=0.0, grad_x=None, grad_weight=True,
                      workspace=None):
    """(grad_x bf16 [R, H], grad_weight fp32 [H]) of rms_norm's y from grad_out
    bf16 [R, H] (quantization passes gradients straight through), with the h
    and rstd that it left (h: x itself where there was no residual).  grad_x is
    the gradient of x and of the residual alike; grad_residual, the gradient
    that reaches h past the norm, is added to it.  grad_x may be written over
    grad_out, h or grad_residual.  grad_weight=False leaves the weight's
    gradient out (None)."""
    def check():
        _need(isinstance(grad_out, torch.Tensor) and grad_out.dim() == 2, "grad_out must be a 2-D bf16 tensor")
        dev = grad_out.device
        R, H = grad_out.shape
        _rows_ok("grad_out", grad_out, torch.bfloat16, dev)
        _need(H >= 1, "rows must hold at least one element")
        _need(isinstance(h, torch.Tensor), "h must be a tensor")
        _like("h", h, (R, H), torch.bfloat16, dev)
        _like("grad_residual", grad_residual, (R, H), torch.bfloat16, dev)
        _like("grad_x", grad_x, (R, H), torch.bfloat16, dev)
        _norm_weight(weight, H, dev)
        _need(isinstance(rstd, torch.Tensor) and rstd.dtype == torch.float32 and rstd.device == dev
              and tuple(rstd.shape) == (R,) and rstd.is_contiguous(), f"rstd must be a contiguous fp32 [{R}] tensor on {dev}")
        _need(isinstance(weight_offset, (int, float)) and math.isfinite(weight_offset), "weight_offset must be a finite number")
        _need(isinstance(grad_weight, bool), "grad_weight must be True or False")
        _need(grad_out.is_cuda, "grad_out must be a CUDA tensor")
        d = NormGradDesc(R, H, _ld(grad_out), _ld(h), H if grad_residual is None else _ld(grad_residual),
                         H if grad_x is None else _ld(grad_x), weight_offset, int(weight.dtype == torch.float32))
        return d, lib.rms_norm_backward_workspace_bytes(R, H) if grad_weight else 0

    d, nws = _checked(("norm backward", _sig(grad_out), _sig(h), _sig(weight), _sig(rstd), _sig(grad_residual),
                       weight_offset, type(weight_offset), _sig(grad_x), grad_weight, type(grad_weight)), check)
    if grad_x is None:
        grad_x = (torch.empty_like if grad_out.is_contiguous() else _new_like)(grad_out)
    ws = _order_ws(workspace, nws, grad_out)
    gw = grad_out.new_empty((d.H,), dtype=torch.float32) if grad_weight else None
    if d.R > 0 or grad_weight:
        _run(lib.rms_norm_backward, "rms_norm_backward", grad_out, grad_out.data_ptr(), h.data_ptr(), _ptr(grad_residual),
             weight.data_ptr(), rstd.data_ptr(), grad_x.data_ptr(), _ptr(gw), ctypes.byref(d), _ptr(ws), nws)
    return grad_x, gw


# ---------------------------------------------------------------------------
# The norm over all gradients of a step, and clipping
# ---------------------------------------------------------------------------

_GRAD_TYPE = {torch.float32: 0, torch.bfloat16: 1}


_dtype_of = operator.attrgetter("dtype")


def _gradient_fields(name, ts):
    """Addresses, elements and types of a list of tensors, and its first
    tensor.  Every check reads one property of all tensors (a list of 200 takes
    a third of the time that it takes with a tensor's checks side by side)."""
    T = torch.Tensor
    _need(all([issubclass(t, T) for t in set(map(type, ts))]), f"every {name} must be a tensor")
    kinds = list(map(_GRAD_TYPE.get, map(_dtype_of, ts)))
    _need(None not in kinds and all(map(T.is_contiguous, ts)), f"every {name} must be a contiguous fp32 or bf16 tensor")
    dev, index = ts[0].device, set(map(T.get_device, ts))
    _need(len(index) == 1 and (index != {-1} or all([t.device == dev for t in ts])), f"every {name} must be on {dev}")
    return list(map(T.data_ptr, ts)), list(map(T.numel, ts)), kinds, ts[0]


def _gradient_list(grads, out):
    """The C ABI's list (src, dst, elements, bf16) of the tensors and the
    first of them; None stands for a parameter without a gradient."""
    _need(isinstance(grads, (list, tuple)), "gradients must be a list or tuple of tensors")
    _need(out is None or isinstance(out, (list, tuple)) and len(out) == len(grads), "out must hold a tensor for each gradient")
    if any([g is None for g in grads]):
        if out is not None:
            _need(all([(g is None) == (o is None) for g, o in zip(grads, out)]), "an output is None where its gradient is")
            out = [o for o in out if o is not None]
        grads = [g for g in grads if g is not None]
    _need(len(grads) > 0, "at least one gradient")
    src, n, kinds, first = _gradient_fields("gradient", grads)
    dst = src
    if out is not None:
        dst, m, okinds, ofirst = _gradient_fields("output", out)
        _need(m == n and okinds == kinds and ofirst.device == first.device,
              f"outputs must have their gradients' elements and types, on {first.device}")
    _need(first.is_cuda, "gradients must be CUDA tensors")
    return array.array("q", itertools.chain.from_iterable(zip(src, dst, n, kinds))), first


def _gradients(fn, what, grads, out, workspace, *more):
    rows, first = _gradient_list(grads, out)
    p, n = rows.buffer_info()[0], len(rows) // 4
    nws = lib.gradient_workspace_bytes(p, n)
    ws = _order_ws(workspace, max(nws, 16), first)
    norm = first.new_empty((1,), dtype=torch.float32)
    _run(fn, what, first, p, n, *more, norm.data_ptr(), ws.data_ptr(), nws)
    return norm


def gradient_norm(grads, workspace=None):
    """The 2-norm over all elements of all tensors of the list `grads` (fp32 or
    bf16, contiguous, on one device; None entries are left out), fp32 [1] on
    that device.  64-bit sums."""
    return _gradients(lib.gradient_norm, "gradient_norm", grads, None, workspace)


def clip_gradients(grads, max_norm, out=None, workspace=None):
    """Scales the tensors of the list `grads` in place (or into the tensors of
    the list `out`, of the same types and numbers of elements) by max_norm / norm where their
    norm, as gradient_norm gives it, is over max_norm; returns the norm before,
    fp32 [1] on their device.  Where a gradient is NaN or infinite, and the
    norm with it, the gradients stay as they are.  (Finite gradients whose norm
    is past fp32 return infinity too, and are scaled.)  The tensors must not
    share memory."""
    _need(isinstance(max_norm, (int, float)) and math.isfinite(max_norm) and max_norm >= 0,
          "max_norm must be a finite number, not below 0")
    return _gradients(lib.clip_gradients, "clip_gradients", grads, out, workspace, float(max_norm))


def route_cost(bm, bn, per_unit, factor, M, N, batch, units) -> float:
    c = RouteCandidate(bm, bn, per_unit, factor)
    return lib.spg_route_cost(ctypes.byref(c), M, N, batch, units)


def route_select(cands, M, N, batch, units) -> int:
    arr = (RouteCandidate * len(cands))(*[RouteCandidate(*c) for c in cands])
    return lib.spg_route_select(arr, len(cands), M, N, batch, units)


# ---- measurement probes (not steps of the method) ------------------------
PROBE_MFMA_FLOPS = {0: 131072, 1: 32768}     # per MFMA: E4M3 32x32x64, f16 32x32x16


def probe_mfma(kind: int, iters: int, workgroups: int, device="cuda"):
    """Enqueue the MFMA-only probe on the current stream; returns (sink,
    clocks) device tensors (see spg_probe_mfma) and the flops it performs."""
    sink = torch.empty((workgroups * 256,), dtype=torch.float32, device=device)
    clocks = torch.zeros((4,), dtype=torch.int64, device=device)
    _check(lib.spg_probe_mfma(kind, iters, workgroups, _ptr(sink), _ptr(clocks), _stream(sink)), "spg_probe_mfma")
    return sink, clocks, workgroups * 4 * iters * 4 * PROBE_MFMA_FLOPS[kind]


def probe_fp4_rounding(device="cuda") -> dict:
    """Compare the E2M1 conversion instruction with the library's encoder on
    every non-NaN binary32 input (see spg_probe_fp4_rounding)."""
    res = torch.empty((34,), dtype=torch.int32, device=device)
    _check(lib.spg_probe_fp4_rounding(_ptr(res), _stream(res)), "spg_probe_fp4_rounding")
    h = res.cpu().numpy().view("uint32")
    n = int(min(h[1], 16))
    return {"differences": int(h[0]), "examples": [(int(h[2 + 2 * k]), int(h[3 + 2 * k])) for k in range(n)]}


def probe_read(buf: torch.Tensor, workgroups: int):
    """Enqueue the HBM read probe over the bytes of contiguous `buf` on the
    current stream; returns the sink (one XOR-folded word per thread)."""
    _need(buf.is_contiguous(), "probe_read: buf must be contiguous")
    sink = torch.empty((workgroups * 256,), dtype=torch.int32, device=buf.device)
    nbytes = buf.numel() * buf.element_size()
    _check(lib.spg_probe_read(_ptr(buf), nbytes, workgroups, _ptr(sink), _stream(buf)), "spg_probe_read")
    return sink

