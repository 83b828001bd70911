"""Thin Python binding of libcubic.so (the CubicQuant dequant-GEMM for gfx950).

Argument marshalling only: every function takes torch tensors, checks their
dtype, device and contiguity, allocates outputs (and workspaces) with torch, and
calls the C function of the same name on torch's current HIP stream. All the
arithmetic runs in the library's HIP kernels; there is no CPU fallback, and a
missing library raises immediately.

Weight layout (see include/cubic.h): ``codes`` uint8 [N][K*bits/8] bit stream,
``scales`` float32 [N][K/group], ``shapes`` int16 [N][K/group][2] holding the
fp16 bit patterns of (a, b).
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

__all__ = [
    "CubicError", "CubicWeight", "library_path", "load_library",
    "cubic_code_bytes", "cubic_storage_bytes", "cubic_pack", "cubic_unpack",
    "cubic_dequant", "cubic_encode", "cubic_fit", "cubic_gemm_a16", "cubic_gemm_a16_workspace_bytes",
    "act_quant_int8_per_token", "cubic_gemm_a8", "cubic_linear_mode", "cubic_linear_workspace_bytes",
    "cubic_linear", "MODE_A16", "MODE_A8", "cubic_moe_workspace_bytes", "cubic_moe_grouped_gemm",
    "cubic_moe_grouped_gemm_static_max_bytes", "cubic_moe_grouped_gemm_static",
    "cubic_moe_mlp_workspace_bytes", "cubic_moe_mlp", "EXPORTED_SYMBOLS", "cubic_moe_grouped_gemm_a8",
    "cubic_moe_mlp_a8_workspace_bytes", "cubic_moe_mlp_a8",
    "DTYPE_F32", "DTYPE_BF16", "DTYPE_F16",
    "cubic_moe_topk", "cubic_moe_layer_workspace_bytes", "cubic_moe_layer", "SCORE_SOFTMAX", "SCORE_SIGMOID",
    "Int8Weight", "cubic_gemm_w8a8", "cubic_linear_w8a8_workspace_bytes", "cubic_linear_w8a8",
    "Fp8Weight", "cubic_quant_fp8", "cubic_gemm_fp8_workspace_bytes", "cubic_gemm_fp8",
    "cubic_linear_fp8_workspace_bytes", "cubic_linear_fp8",
    "ACT_SILU", "ACT_GELU_TANH", "cubic_gated_ff_workspace_bytes", "cubic_gated_ff",
    "cubic_gated_ff_backward_workspace_bytes", "cubic_gated_ff_backward",
    "cubic_gated_ff_fp8_workspace_bytes", "cubic_gated_ff_fp8",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
EXPORTED_SYMBOLS = [
    "cubic_code_bytes", "cubic_storage_bytes", "cubic_status_string", "cubic_version",
    "cubic_pack", "cubic_unpack", "cubic_dequant", "cubic_encode", "cubic_fit", "cubic_gemm_a16_workspace_bytes",
    "cubic_gemm_a16", "act_quant_int8_per_token", "cubic_gemm_a8", "cubic_linear_mode",
    "cubic_linear_workspace_bytes", "cubic_linear", "cubic_moe_workspace_bytes",
    "cubic_moe_grouped_gemm", "cubic_moe_grouped_gemm_static_max_bytes", "cubic_moe_grouped_gemm_static",
    "cubic_moe_mlp_workspace_bytes", "cubic_moe_mlp",
    "cubic_gemm_a16_ex", "act_quant_int8_per_token_ex", "cubic_gemm_a8_ex", "cubic_moe_grouped_gemm_ex",
    "cubic_moe_grouped_gemm_a8", "cubic_moe_mlp_a8_workspace_bytes", "cubic_moe_mlp_a8",
    "cubic_moe_topk", "cubic_moe_layer_workspace_bytes", "cubic_moe_layer",
    "cubic_gemm_w8a8", "cubic_linear_w8a8_workspace_bytes", "cubic_linear_w8a8",
    "cubic_quant_fp8", "cubic_gemm_fp8_workspace_bytes", "cubic_gemm_fp8",
    "cubic_linear_fp8_workspace_bytes", "cubic_linear_fp8",
    "cubic_gated_ff_workspace_bytes", "cubic_gated_ff",
    "cubic_gated_ff_backward_workspace_bytes", "cubic_gated_ff_backward",
    "cubic_gated_ff_fp8_workspace_bytes", "cubic_gated_ff_fp8",
]
MODE_A16, MODE_A8 = 0, 1          # cubic_linear_mode results
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
ACT_SILU, ACT_GELU_TANH = 0, 1


class CubicError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {_status_string(status)} ({status})")
        self.status = status


class _CWeight(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("shapes", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("bits", ctypes.c_int32), ("group", ctypes.c_int32)]


class _CWeightI8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64)]


class _CWeightFp8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64)]


class _CRouter(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("logits_dtype", ctypes.c_int32),
                ("E", ctypes.c_int32), ("topk", ctypes.c_int32), ("score", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float)]


def library_path() -> str:
    return os.environ.get("CUBIC_LIBRARY", os.path.join(_PKG, "lib", "libcubic.so"))


_lib = None


def load_library():
    """Load libcubic.so (built by dequant_gemm_amd.build); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libcubic.so not found at {path}; run `python -m dequant_gemm_amd.build`")
    lib = ctypes.CDLL(path)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    wp = ctypes.POINTER(_CWeight)
    rp = ctypes.POINTER(_CRouter)
    ip = ctypes.POINTER(_CWeightI8)
    fp = ctypes.POINTER(_CWeightFp8)
    sigs = {
        "cubic_code_bytes": (sz, [i64, i64, i32]),
        "cubic_storage_bytes": (sz, [i64, i64, i32, i32]),
        "cubic_status_string": (ctypes.c_char_p, [i32]),
        "cubic_version": (ctypes.c_char_p, []),
        "cubic_pack": (i32, [vp, i64, i64, i32, vp, vp]),
        "cubic_unpack": (i32, [vp, i64, i64, i32, vp, vp]),
        "cubic_dequant": (i32, [wp, vp, vp]),
        "cubic_encode": (i32, [vp, i64, i64, i32, i32, vp, vp, vp, vp]),
        "cubic_fit": (i32, [vp, i64, i64, i32, i32, vp, vp, vp, vp, vp]),
        "cubic_gemm_a16_workspace_bytes": (sz, [i64, i64]),
        "cubic_gemm_a16": (i32, [vp, i64, wp, vp, vp, sz, vp]),
        "act_quant_int8_per_token": (i32, [vp, i64, i64, vp, vp, vp]),
        "cubic_gemm_a8": (i32, [vp, vp, i64, wp, vp, vp]),
        "cubic_linear_mode": (i32, [i64, i64, i64, i32, i32]),
        "cubic_linear_workspace_bytes": (sz, [i64, i64]),
        "cubic_linear": (i32, [vp, i64, wp, vp, vp, sz, vp]),
        "cubic_moe_workspace_bytes": (sz, [i64, i32, i32]),
        "cubic_moe_grouped_gemm": (i32, [vp, i64, vp, i32, wp, i32, vp, vp, sz, vp]),
        "cubic_moe_grouped_gemm_static_max_bytes": (sz, []),
        "cubic_gemm_a16_ex": (i32, [vp, i32, i64, wp, vp, i32, vp, sz, vp]),
        "act_quant_int8_per_token_ex": (i32, [vp, i32, i64, i64, vp, vp, vp]),
        "cubic_gemm_a8_ex": (i32, [vp, vp, i64, wp, vp, i32, vp]),
        "cubic_moe_grouped_gemm_ex": (i32, [vp, i32, i64, vp, i32, wp, i32, vp, i32, vp, sz, vp]),
        "cubic_moe_grouped_gemm_static": (i32, [vp, i64, vp, i32, wp, i32, vp, vp]),
        "cubic_moe_grouped_gemm_a8": (i32, [vp, vp, i64, vp, i32, wp, i32, vp, i32, vp, sz, vp]),
        "cubic_moe_mlp_workspace_bytes": (sz, [i64, i32, i32, i64, i64]),
        "cubic_moe_mlp": (i32, [vp, i64, vp, vp, i32, wp, wp, i32, vp, vp, sz, vp]),
        "cubic_moe_mlp_a8_workspace_bytes": (sz, [i64, i32, i32, i64, i64]),
        "cubic_moe_mlp_a8": (i32, [vp, i64, vp, vp, i32, wp, wp, i32, vp, vp, sz, vp]),
        "cubic_moe_topk": (i32, [rp, i64, vp, vp, vp]),
        "cubic_moe_layer_workspace_bytes": (sz, [i64, i32, i32, i64, i64]),
        "cubic_moe_layer": (i32, [vp, i64, rp, wp, wp, vp, i32, vp, vp, vp, sz, vp]),
        "cubic_gemm_w8a8": (i32, [vp, vp, i64, ip, vp, vp, i32, vp]),
        "cubic_linear_w8a8_workspace_bytes": (sz, [i64, i64]),
        "cubic_linear_w8a8": (i32, [vp, i32, i64, ip, vp, vp, i32, vp, sz, vp]),
        "cubic_quant_fp8": (i32, [vp, i32, i64, i64, i32, vp, vp, vp]),
        "cubic_gemm_fp8_workspace_bytes": (sz, [i64, i64, i64]),
        "cubic_gemm_fp8": (i32, [vp, vp, i64, fp, vp, vp, i32, vp, sz, vp]),
        "cubic_linear_fp8_workspace_bytes": (sz, [i64, i64, i64]),
        "cubic_linear_fp8": (i32, [vp, i32, i64, fp, vp, vp, i32, vp, sz, vp]),
        "cubic_gated_ff_workspace_bytes": (sz, [i64, i64, i64]),
        "cubic_gated_ff": (i32, [vp, vp, i32, i64, i64, i64, i32, vp, vp, vp, sz, vp]),
        "cubic_gated_ff_backward_workspace_bytes": (sz, [i64, i64, i64]),
        "cubic_gated_ff_backward": (i32, [vp, vp, vp, vp, i32, i64, i64, i64, i32, vp, vp, vp, sz, vp]),
        "cubic_gated_ff_fp8_workspace_bytes": (sz, [i64, i64, i64]),
        "cubic_gated_ff_fp8": (i32, [vp, i32, i64, fp, i32, vp, i32, vp, sz, vp]),
    }
    for name, (res, args) in sigs.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _status_string(status: int) -> str:
    try:
        return load_library().cubic_status_string(status).decode()
    except Exception:  # pragma: no cover
        return "status"


def _check(status: int, what: str):
    if status != 0:
        raise CubicError(status, what)


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _need(t: torch.Tensor, dtype, name: str):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


@dataclass
class CubicWeight:
    """Device buffers of one Cubic weight (or of E experts back to back)."""
    codes: torch.Tensor     # uint8, N*K*bits/8 bytes per matrix
    scales: torch.Tensor    # float32, N*K/group per matrix
    shapes: torch.Tensor    # int16 (fp16 bit patterns), 2*N*K/group per matrix
    N: int
    K: int
    bits: int
    group: int

    def c_struct(self) -> _CWeight:
        _need(self.codes, torch.uint8, "codes")
        _need(self.scales, torch.float32, "scales")
        _need(self.shapes, torch.int16, "shapes")
        return _CWeight(self.codes.data_ptr(), self.scales.data_ptr(), self.shapes.data_ptr(),
                        self.N, self.K, self.bits, self.group)


def cubic_code_bytes(N: int, K: int, bits: int) -> int:
    return int(load_library().cubic_code_bytes(N, K, bits))


def cubic_storage_bytes(N: int, K: int, bits: int, group: int) -> int:
    return int(load_library().cubic_storage_bytes(N, K, bits, group))


def cubic_pack(codes: torch.Tensor, bits: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """int8 codes [N][K] -> uint8 bit stream [N][K*bits/8]."""
    _need(codes, torch.int8, "codes")
    N, K = codes.shape
    if out is None:
        out = torch.empty((N, K * bits // 8), dtype=torch.uint8, device=codes.device)
    _check(load_library().cubic_pack(_ptr(codes), N, K, bits, _ptr(out), _stream(codes)), "cubic_pack")
    return out


def cubic_unpack(packed: torch.Tensor, N: int, K: int, bits: int,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    _need(packed, torch.uint8, "packed")
    if out is None:
        out = torch.empty((N, K), dtype=torch.int8, device=packed.device)
    _check(load_library().cubic_unpack(_ptr(packed), N, K, bits, _ptr(out), _stream(packed)),
           "cubic_unpack")
    return out


def cubic_dequant(w: CubicWeight, out: torch.Tensor | None = None) -> torch.Tensor:
    cw = w.c_struct()
    if out is None:
        out = torch.empty((w.N, w.K), dtype=torch.float32, device=w.codes.device)
    _check(load_library().cubic_dequant(ctypes.byref(cw), _ptr(out), _stream(w.codes)),
           "cubic_dequant")
    return out


def cubic_encode(w: torch.Tensor, scales: torch.Tensor, shapes: torch.Tensor, bits: int, group: int,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """fp32 weights [N][K] -> int8 codes [N][K] of the nearest levels (pack with cubic_pack)."""
    _need(w, torch.float32, "w")
    N, K = w.shape
    if out is None:
        out = torch.empty((N, K), dtype=torch.int8, device=w.device)
    _check(load_library().cubic_encode(_ptr(w), N, K, bits, group, _ptr(scales), _ptr(shapes), _ptr(out),
                                        _stream(w)), "cubic_encode")
    return out


def cubic_fit(w: torch.Tensor, bits: int, group: int, with_loss: bool = False):
    """Fit every group of fp32 weights w [N][K]: returns (codes int8 [N][K], scales
    fp32 [N][K/group], shapes int16 [N][K/group][2] holding fp16 a, b bits), plus the
    per-group loss (fp32) when with_loss."""
    _need(w, torch.float32, "w")
    N, K = w.shape
    G = K // group if group > 0 else 0
    codes = torch.empty((N, K), dtype=torch.int8, device=w.device)
    scales = torch.empty((N, G), dtype=torch.float32, device=w.device)
    shapes = torch.empty((N, G, 2), dtype=torch.int16, device=w.device)
    loss = torch.empty((N, G), dtype=torch.float32, device=w.device) if with_loss else None
    _check(load_library().cubic_fit(_ptr(w), N, K, bits, group, _ptr(codes), _ptr(scales), _ptr(shapes),
                                    _ptr(loss) if loss is not None else None, _stream(w)), "cubic_fit")
    return (codes, scales, shapes, loss) if with_loss else (codes, scales, shapes)


def cubic_gemm_a16_workspace_bytes(M: int, K: int) -> int:
    return int(load_library().cubic_gemm_a16_workspace_bytes(M, K))


DTYPE_F32, DTYPE_BF16, DTYPE_F16 = 0, 1, 2          # element types of the _ex entry points
_DT_IN = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}
_DT_OUT = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}


def _in_dtype(x: torch.Tensor, name: str) -> int:
    if x.dtype not in _DT_IN:
        raise TypeError(f"{name}: expected bfloat16 or float16, got {x.dtype}")
    _need(x, x.dtype, name)
    return _DT_IN[x.dtype]


def _out_dtype(out_dtype) -> int:
    if out_dtype not in _DT_OUT:
        raise TypeError(f"out_dtype: expected float32 or bfloat16, got {out_dtype}")
    return _DT_OUT[out_dtype]


def cubic_gemm_a16(x: torch.Tensor, w: CubicWeight, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, out_dtype=torch.float32) -> torch.Tensor:
    """y[M][N] = x[M][K] * W^T; x bf16 (cubic_gemm_a16) or fp16, y fp32 or bf16
    (cubic_gemm_a16_ex)."""
    xd, yd = _in_dtype(x, "x"), _out_dtype(out_dtype)
    M = x.shape[0]
    cw = w.c_struct()
    if out is None:
        out = torch.empty((M, w.N), dtype=out_dtype, device=x.device)
    elif out.dtype != out_dtype:
        raise TypeError(f"out: expected {out_dtype}, got {out.dtype}")
    need = cubic_gemm_a16_workspace_bytes(M, w.K)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_bytes = workspace.numel() if workspace is not None else 0
    lib = load_library()
    if xd == DTYPE_BF16 and yd == DTYPE_F32:
        st = lib.cubic_gemm_a16(_ptr(x), M, ctypes.byref(cw), _ptr(out), _ptr(workspace), ws_bytes, _stream(x))
    else:
        st = lib.cubic_gemm_a16_ex(_ptr(x), xd, M, ctypes.byref(cw), _ptr(out), yd, _ptr(workspace), ws_bytes,
                                   _stream(x))
    _check(st, "cubic_gemm_a16")
    return out


def act_quant_int8_per_token(x: torch.Tensor, xq: torch.Tensor | None = None,
                             x_scale: torch.Tensor | None = None):
    """bf16 or fp16 [M][K] -> (int8 [M][K], fp32 [M])."""
    xd = _in_dtype(x, "x")
    M, K = x.shape
    if xq is None:
        xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if x_scale is None:
        x_scale = torch.empty((M,), dtype=torch.float32, device=x.device)
    lib = load_library()
    if xd == DTYPE_BF16:
        st = lib.act_quant_int8_per_token(_ptr(x), M, K, _ptr(xq), _ptr(x_scale), _stream(x))
    else:
        st = lib.act_quant_int8_per_token_ex(_ptr(x), xd, M, K, _ptr(xq), _ptr(x_scale), _stream(x))
    _check(st, "act_quant_int8_per_token")
    return xq, x_scale


def cubic_gemm_a8(xq: torch.Tensor, x_scale: torch.Tensor, w: CubicWeight,
                  out: torch.Tensor | None = None, out_dtype=torch.float32) -> torch.Tensor:
    _need(xq, torch.int8, "xq")
    _need(x_scale, torch.float32, "x_scale")
    yd = _out_dtype(out_dtype)
    M = xq.shape[0]
    cw = w.c_struct()
    if out is None:
        out = torch.empty((M, w.N), dtype=out_dtype, device=xq.device)
    elif out.dtype != out_dtype:
        raise TypeError(f"out: expected {out_dtype}, got {out.dtype}")
    lib = load_library()
    if yd == DTYPE_F32:
        st = lib.cubic_gemm_a8(_ptr(xq), _ptr(x_scale), M, ctypes.byref(cw), _ptr(out), _stream(xq))
    else:
        st = lib.cubic_gemm_a8_ex(_ptr(xq), _ptr(x_scale), M, ctypes.byref(cw), _ptr(out), yd, _stream(xq))
    _check(st, "cubic_gemm_a8")
    return out


def cubic_linear_mode(M: int, N: int, K: int, bits: int, group: int) -> int:
    """MODE_A16 or MODE_A8: the activation mode cubic_linear takes for this shape."""
    return int(load_library().cubic_linear_mode(M, N, K, bits, group))


def cubic_linear_workspace_bytes(M: int, K: int) -> int:
    return int(load_library().cubic_linear_workspace_bytes(M, K))


def cubic_linear(x: torch.Tensor, w: CubicWeight, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[M][N] (fp32) from bf16 x[M][K] in the mode of cubic_linear_mode (A16, or
    the per-token INT8 quantiser followed by the A8 product)."""
    _need(x, torch.bfloat16, "x")
    M = x.shape[0]
    cw = w.c_struct()
    if out is None:
        out = torch.empty((M, w.N), dtype=torch.float32, device=x.device)
    need = cubic_linear_workspace_bytes(M, w.K)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_bytes = workspace.numel() if workspace is not None else 0
    _check(load_library().cubic_linear(_ptr(x), M, ctypes.byref(cw), _ptr(out), _ptr(workspace),
                                        ws_bytes, _stream(x)), "cubic_linear")
    return out


def cubic_moe_workspace_bytes(T: int, topk: int, E: int) -> int:
    return int(load_library().cubic_moe_workspace_bytes(T, topk, E))


def cubic_moe_grouped_gemm(x: torch.Tensor, topk_ids: torch.Tensor, experts: CubicWeight, E: int,
                           out: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, out_dtype=torch.float32) -> torch.Tensor:
    """y[T][topk][N]: each (token, slot) pair times its expert's weights; x bf16 or
    fp16, y fp32 or bf16."""
    xd, yd = _in_dtype(x, "x"), _out_dtype(out_dtype)
    _need(topk_ids, torch.int32, "topk_ids")
    T, topk = topk_ids.shape
    cw = experts.c_struct()
    if out is None:
        out = torch.empty((T, topk, experts.N), dtype=out_dtype, device=x.device)
    elif out.dtype != out_dtype:
        raise TypeError(f"out: expected {out_dtype}, got {out.dtype}")
    need = cubic_moe_workspace_bytes(T, topk, E)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    lib = load_library()
    if xd == DTYPE_BF16 and yd == DTYPE_F32:
        st = lib.cubic_moe_grouped_gemm(_ptr(x), T, _ptr(topk_ids), topk, ctypes.byref(cw), E, _ptr(out),
                                        _ptr(workspace), workspace.numel(), _stream(x))
    else:
        st = lib.cubic_moe_grouped_gemm_ex(_ptr(x), xd, T, _ptr(topk_ids), topk, ctypes.byref(cw), E, _ptr(out),
                                           yd, _ptr(workspace), workspace.numel(), _stream(x))
    _check(st, "cubic_moe_grouped_gemm")
    return out


def cubic_moe_grouped_gemm_a8(xq: torch.Tensor, x_scale: torch.Tensor, topk_ids: torch.Tensor,
                              experts: CubicWeight, E: int, out: torch.Tensor | None = None,
                              workspace: torch.Tensor | None = None, out_dtype=torch.float32) -> torch.Tensor:
    """y[T][topk][N]: each (token, slot) pair's Dynamic A8 product with its expert;
    xq int8 [T][K] and x_scale fp32 [T] from act_quant_int8_per_token."""
    _need(xq, torch.int8, "xq")
    _need(x_scale, torch.float32, "x_scale")
    _need(topk_ids, torch.int32, "topk_ids")
    yd = _out_dtype(out_dtype)
    T, topk = topk_ids.shape
    cw = experts.c_struct()
    if out is None:
        out = torch.empty((T, topk, experts.N), dtype=out_dtype, device=xq.device)
    elif out.dtype != out_dtype:
        raise TypeError(f"out: expected {out_dtype}, got {out.dtype}")
    if workspace is None:
        workspace = torch.empty(cubic_moe_workspace_bytes(T, topk, E), dtype=torch.uint8, device=xq.device)
    _check(load_library().cubic_moe_grouped_gemm_a8(_ptr(xq), _ptr(x_scale), T, _ptr(topk_ids), topk,
                                                    ctypes.byref(cw), E, _ptr(out), yd, _ptr(workspace),
                                                    workspace.numel(), _stream(xq)),
           "cubic_moe_grouped_gemm_a8")
    return out


def cubic_moe_grouped_gemm_static_max_bytes() -> int:
    return int(load_library().cubic_moe_grouped_gemm_static_max_bytes())


def cubic_moe_grouped_gemm_static(x: torch.Tensor, topk_ids: torch.Tensor, experts: CubicWeight, E: int,
                                  out: torch.Tensor | None = None) -> torch.Tensor:
    """cubic_moe_grouped_gemm with the library's per-device routing scratch (no workspace)."""
    _need(x, torch.bfloat16, "x")
    _need(topk_ids, torch.int32, "topk_ids")
    T, topk = topk_ids.shape
    cw = experts.c_struct()
    if out is None:
        out = torch.empty((T, topk, experts.N), dtype=torch.float32, device=x.device)
    _check(load_library().cubic_moe_grouped_gemm_static(_ptr(x), T, _ptr(topk_ids), topk, ctypes.byref(cw),
                                                        E, _ptr(out), _stream(x)),
           "cubic_moe_grouped_gemm_static")
    return out


def cubic_moe_mlp_workspace_bytes(T: int, topk: int, E: int, H: int, I: int) -> int:
    return int(load_library().cubic_moe_mlp_workspace_bytes(T, topk, E, H, I))


def cubic_moe_mlp(x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                  gate_up: CubicWeight, down: CubicWeight, E: int, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[T][H] (fp32): sum_j w[t][j] * (bf16(SiLU(gate) * up) of token t through expert
    topk_ids[t][j]'s gate_up) through that expert's down projection."""
    _need(x, torch.bfloat16, "x")
    _need(topk_ids, torch.int32, "topk_ids")
    _need(topk_weights, torch.float32, "topk_weights")
    T, topk = topk_ids.shape
    if out is None:
        out = torch.empty((T, down.N), dtype=torch.float32, device=x.device)
    need = cubic_moe_mlp_workspace_bytes(T, topk, E, gate_up.K, down.K)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    gu, dn = gate_up.c_struct(), down.c_struct()
    _check(load_library().cubic_moe_mlp(_ptr(x), T, _ptr(topk_ids), _ptr(topk_weights), topk,
                                        ctypes.byref(gu), ctypes.byref(dn), E, _ptr(out), _ptr(workspace),
                                        workspace.numel(), _stream(x)), "cubic_moe_mlp")
    return out


def cubic_moe_mlp_a8_workspace_bytes(T: int, topk: int, E: int, H: int, I: int) -> int:
    return int(load_library().cubic_moe_mlp_a8_workspace_bytes(T, topk, E, H, I))


def cubic_moe_mlp_a8(x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                     gate_up: CubicWeight, down: CubicWeight, E: int, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None) -> torch.Tensor:
    """cubic_moe_mlp in the Dynamic A8 mode: the token rows and the intermediate h
    rows are quantised per row to int8 before their grouped products."""
    _need(x, torch.bfloat16, "x")
    _need(topk_ids, torch.int32, "topk_ids")
    _need(topk_weights, torch.float32, "topk_weights")
    T, topk = topk_ids.shape
    if out is None:
        out = torch.empty((T, down.N), dtype=torch.float32, device=x.device)
    need = cubic_moe_mlp_a8_workspace_bytes(T, topk, E, gate_up.K, down.K)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    gu, dn = gate_up.c_struct(), down.c_struct()
    _check(load_library().cubic_moe_mlp_a8(_ptr(x), T, _ptr(topk_ids), _ptr(topk_weights), topk,
                                           ctypes.byref(gu), ctypes.byref(dn), E, _ptr(out), _ptr(workspace),
                                           workspace.numel(), _stream(x)), "cubic_moe_mlp_a8")
    return out


_SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID, SCORE_SOFTMAX: SCORE_SOFTMAX,
           SCORE_SIGMOID: SCORE_SIGMOID}
_DT_LOGITS = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}


# The calls below are short on the device (a few microseconds), so their checks are kept short too: one
# pass over each tensor, integers for pointers, and the raw handle of the current stream.


def _arg(t: torch.Tensor, dtype, index: int, name: str) -> int:
    """Address of a contiguous tensor of this dtype on device `index`."""
    if t.dtype != dtype or t.get_device() != index or not t.is_contiguous():
        _need(t, dtype, name)
        raise ValueError(f"{name}: expected a tensor on cuda:{index}, got {t.device}")
    return t.data_ptr()


def _first(t: torch.Tensor, name: str) -> int:
    """Device index of the argument that the others follow."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name}: must be a device tensor")
    return index


def _call(index: int, f, *args) -> int:
    """f(*args, current stream of device `index`), with that device current."""
    if index == torch.cuda.current_device():
        return f(*args, torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(index):
        return f(*args, torch._C._cuda_getCurrentRawStream(index))


def _result(out, shape, dtype, index: int, name="out"):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=index)
    _arg(out, dtype, index, name)
    if tuple(out.shape) != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(out.shape)}")
    return out


def _router(logits: torch.Tensor, index: int, topk: int, score, bias, renormalize: bool, scale: float) -> _CRouter:
    dtype = logits.dtype
    if dtype not in _DT_LOGITS:
        raise TypeError(f"logits: expected float32, bfloat16 or float16, got {dtype}")
    address = _arg(logits, dtype, index, "logits")
    if logits.dim() != 2:
        raise ValueError("logits: expected [T][E]")
    if score not in _SCORES:
        raise ValueError(f"score: expected 'softmax' or 'sigmoid', got {score!r}")
    E = logits.shape[1]
    at = None
    if bias is not None:
        at = _arg(bias, torch.float32, index, "bias")
        if bias.numel() != E:
            raise ValueError(f"bias: expected {E} values, got {bias.numel()}")
    return _CRouter(address, at, _DT_LOGITS[dtype], E, topk, _SCORES[score], 1 if renormalize else 0, scale)


def cubic_moe_topk(logits: torch.Tensor, topk: int, score="softmax", bias: torch.Tensor | None = None,
                   renormalize: bool = True, scale: float = 1.0, topk_ids: torch.Tensor | None = None,
                   topk_weights: torch.Tensor | None = None):
    """The router: logits [T][E] (fp32, bf16 or fp16) -> (ids int32 [T][topk], weights fp32 [T][topk]).
    Experts are taken by score + bias (ties to the lowest index) and weighted by their scores,
    renormalised over the taken ones and times scale; masked slots get id -1 and weight 0."""
    if logits.dtype not in _DT_LOGITS:
        raise TypeError(f"logits: expected float32, bfloat16 or float16, got {logits.dtype}")
    index = _first(logits, "logits")
    r = _router(logits, index, topk, score, bias, renormalize, scale)
    T = logits.shape[0]
    topk_ids = _result(topk_ids, (T, topk), torch.int32, index, "topk_ids")
    topk_weights = _result(topk_weights, (T, topk), torch.float32, index, "topk_weights")
    _check(_call(index, load_library().cubic_moe_topk, ctypes.byref(r), T, topk_ids.data_ptr(),
                 topk_weights.data_ptr()), "cubic_moe_topk")
    return topk_ids, topk_weights


def cubic_moe_layer_workspace_bytes(T: int, topk: int, E: int, H: int, I: int) -> int:
    return int(load_library().cubic_moe_layer_workspace_bytes(T, topk, E, H, I))


def _expert_args(w: CubicWeight, E: int, index: int, name: str) -> _CWeight:
    """The descriptor of E back-to-back experts, every buffer of at least their size."""
    groups = w.N * (w.K // w.group) if w.group > 0 else 0
    c = _CWeight(_arg(w.codes, torch.uint8, index, name), _arg(w.scales, torch.float32, index, name),
                 _arg(w.shapes, torch.int16, index, name), w.N, w.K, w.bits, w.group)
    if (w.codes.numel() < E * (w.N * w.K * w.bits // 8) or w.scales.numel() < E * groups
            or w.shapes.numel() < 2 * E * groups):
        raise ValueError(f"{name}: smaller than {E} experts of [{w.N}][{w.K}]")
    return c


def cubic_moe_layer(x: torch.Tensor, logits: torch.Tensor, gate_up: CubicWeight, down: CubicWeight, E: int, topk: int,
                    score="softmax", bias: torch.Tensor | None = None, renormalize: bool = True, scale: float = 1.0,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    out_dtype=torch.bfloat16):
    """The whole routed-expert layer: x bf16 [T][H] and router logits [T][E] ->
    (y [T][H] bf16 or fp32, ids int32 [T][topk], weights fp32 [T][topk]). Routing as in
    cubic_moe_topk, experts as in cubic_moe_mlp."""
    yd = _out_dtype(out_dtype)
    index = _first(x, "x")
    xa = _arg(x, torch.bfloat16, index, "x")
    r = _router(logits, index, topk, score, bias, renormalize, scale)
    T, H = logits.shape[0], gate_up.K
    if tuple(x.shape) != (T, H):
        raise ValueError(f"x: expected [{T}][{H}], got {tuple(x.shape)}")
    if r.E != E:
        raise ValueError(f"logits: expected {E} experts, got {r.E}")
    gu, dn = _expert_args(gate_up, E, index, "gate_up"), _expert_args(down, E, index, "down")
    out = _result(out, (T, H), out_dtype, index)
    ids = torch.empty((T, topk), dtype=torch.int32, device=index)
    weights = torch.empty((T, topk), dtype=torch.float32, device=index)
    if workspace is None:
        n = cubic_moe_layer_workspace_bytes(T, topk, E, H, down.K)
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=index)
    wa = _arg(workspace, torch.uint8, index, "workspace")
    _check(_call(index, load_library().cubic_moe_layer, xa, T, ctypes.byref(r), ctypes.byref(gu), ctypes.byref(dn),
                 out.data_ptr(), yd, ids.data_ptr(), weights.data_ptr(), wa, workspace.numel()), "cubic_moe_layer")
    return out, ids, weights


@dataclass
class Int8Weight:
    """A dense int8 weight with one scale per output channel (act_quant_int8_per_token of its rows)."""
    codes: torch.Tensor     # int8 [N][K]
    scales: torch.Tensor    # float32 [N]


def _w8a8_args(x: torch.Tensor, w: Int8Weight, bias, out, out_dtype, index: int, name: str):
    """(descriptor, bias address, output code, output) after the checks that both calls share."""
    yd = _out_dtype(out_dtype)
    codes, scales = w.codes, w.scales
    if codes.dim() != 2 or scales.shape != codes.shape[:1]:
        raise ValueError("Int8Weight: expected codes [N][K] and scales [N]")
    N, K = codes.shape
    cw = _CWeightI8(_arg(codes, torch.int8, index, "codes"), _arg(scales, torch.float32, index, "scales"), N, K)
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"{name}: expected [M][{K}], got {tuple(x.shape)}")
    ba = None
    if bias is not None:
        ba = _arg(bias, torch.float32, index, "bias")
        if bias.numel() != N:
            raise ValueError(f"bias: expected {N} values, got {bias.numel()}")
    return cw, ba, yd, _result(out, (x.shape[0], N), out_dtype, index)


def cubic_gemm_w8a8(xq: torch.Tensor, x_scale: torch.Tensor, w: Int8Weight, bias: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, out_dtype=torch.float32) -> torch.Tensor:
    """y[M][N] = (xq int8 [M][K] times the int8 weight, exact in int32) * w.scales[n] * x_scale[m]
    (+ bias[n]); y fp32 or bf16."""
    index = _first(xq, "xq")
    xa, sa = _arg(xq, torch.int8, index, "xq"), _arg(x_scale, torch.float32, index, "x_scale")
    cw, ba, yd, out = _w8a8_args(xq, w, bias, out, out_dtype, index, "xq")
    M = xq.shape[0]
    if x_scale.numel() != M:
        raise ValueError(f"x_scale: expected {M} values, got {x_scale.numel()}")
    _check(_call(index, load_library().cubic_gemm_w8a8, xa, sa, M, ctypes.byref(cw), ba, out.data_ptr(), yd),
           "cubic_gemm_w8a8")
    return out


def cubic_linear_w8a8_workspace_bytes(M: int, K: int) -> int:
    return int(load_library().cubic_linear_w8a8_workspace_bytes(M, K))


def cubic_linear_w8a8(x: torch.Tensor, w: Int8Weight, bias: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      out_dtype=torch.float32) -> torch.Tensor:
    """cubic_gemm_w8a8 of bf16 or fp16 rows x [M][K], quantised per row on the way (scale
    amax * fp32(1 / 127), as torch's x.abs().amax(-1) / 127 on the device)."""
    if x.dtype not in _DT_IN:
        raise TypeError(f"x: expected bfloat16 or float16, got {x.dtype}")
    index = _first(x, "x")
    xa = _arg(x, x.dtype, index, "x")
    cw, ba, yd, out = _w8a8_args(x, w, bias, out, out_dtype, index, "x")
    M = x.shape[0]
    lib = load_library()
    if workspace is None:
        n = lib.cubic_linear_w8a8_workspace_bytes(M, cw.K)
        workspace = torch.empty(n, dtype=torch.uint8, device=index) if n else None
    wa, n = (None, 0) if workspace is None else (_arg(workspace, torch.uint8, index, "workspace"), workspace.numel())
    _check(_call(index, lib.cubic_linear_w8a8, xa, _DT_IN[x.dtype], M, ctypes.byref(cw), ba, out.data_ptr(), yd, wa, n),
           "cubic_linear_w8a8")
    return out


@dataclass
class Fp8Weight:
    """A dense e4m3 weight with one scale per block of 128 x 128 (cubic_quant_fp8 with block_rows=128)."""
    codes: torch.Tensor     # float8_e4m3fn [N][K]
    scales: torch.Tensor    # float32 [ceil(N / 128)][ceil(K / 128)]


_DT_DENSE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_ACTS = {"silu": ACT_SILU, "gelu_tanh": ACT_GELU_TANH, ACT_SILU: ACT_SILU, ACT_GELU_TANH: ACT_GELU_TANH}


def _dense_dtype(dtype, name: str, floats: dict) -> int:
    if dtype not in floats:
        raise TypeError(f"{name}: expected one of {', '.join(str(d) for d in floats)}, got {dtype}")
    return floats[dtype]


def _act(act) -> int:
    if act not in _ACTS:
        raise ValueError(f"act: expected 'silu' or 'gelu_tanh', got {act!r}")
    return _ACTS[act]


def _dense_out(out, like: torch.Tensor, shape, dtype, index: int, name="out"):
    """out, checked, or a new tensor (new_empty takes less host time than torch.empty)."""
    return like.new_empty(shape, dtype=dtype) if out is None else _result(out, shape, dtype, index, name)


def _scratch(workspace, need: int, index: int):
    """(tensor to keep, address, bytes) of the caller's workspace or a new one."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=index)
    return workspace, _arg(workspace, torch.uint8, index, "workspace"), workspace.numel()


def _fp8_weight(w: Fp8Weight, index: int) -> _CWeightFp8:
    if w.codes.dim() != 2 or tuple(w.scales.shape) != (-(-w.codes.shape[0] // 128), -(-w.codes.shape[1] // 128)):
        raise ValueError("Fp8Weight: expected codes [N][K] and scales [ceil(N / 128)][ceil(K / 128)]")
    return _CWeightFp8(_arg(w.codes, torch.float8_e4m3fn, index, "codes"), _arg(w.scales, torch.float32, index, "scales"),
                       *w.codes.shape)


def _fp8_args(x: torch.Tensor, w: Fp8Weight, bias, out, out_dtype, index: int, name: str):
    """(descriptor, bias address, output code, output) after the checks that both calls share."""
    yd = _dense_dtype(out_dtype, "out_dtype", _DT_DENSE)
    cw = _fp8_weight(w, index)
    if x.dim() != 2 or x.shape[1] != cw.K:
        raise ValueError(f"{name}: expected [M][{cw.K}], got {tuple(x.shape)}")
    ba = None
    if bias is not None:
        ba = _arg(bias, torch.float32, index, "bias")
        if bias.numel() != cw.N:
            raise ValueError(f"bias: expected {cw.N} values, got {bias.numel()}")
    return cw, ba, yd, _dense_out(out, x, (x.shape[0], cw.N), out_dtype, index)


def cubic_quant_fp8(x: torch.Tensor, block_rows: int = 1, xq: torch.Tensor | None = None,
                    scales: torch.Tensor | None = None):
    """x bf16 or fp16 [M][K] -> (e4m3 codes [M][K], fp32 scales [ceil(M / block_rows)][ceil(K / 128)]),
    block_rows 1 (activations) or 128 (weights)."""
    if x.dim() != 2 or block_rows <= 0:
        raise ValueError(f"x: expected [M][K] and a positive block_rows, got {tuple(x.shape)} and {block_rows}")
    xd = _dense_dtype(x.dtype, "x", _DT_IN)
    index = _first(x, "x")
    xa = _arg(x, x.dtype, index, "x")
    M, K = x.shape
    xq = _dense_out(xq, x, (M, K), torch.float8_e4m3fn, index, "xq")
    scales = _dense_out(scales, x, (-(-M // block_rows), -(-K // 128)), torch.float32, index, "scales")
    _check(_call(index, load_library().cubic_quant_fp8, xa, xd, M, K, block_rows, xq.data_ptr(), scales.data_ptr()),
           "cubic_quant_fp8")
    return xq, scales


def cubic_gemm_fp8_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load_library().cubic_gemm_fp8_workspace_bytes(M, N, K))


def cubic_gemm_fp8(xq: torch.Tensor, x_scale: torch.Tensor, w: Fp8Weight, bias: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   out_dtype=torch.float32) -> torch.Tensor:
    """y[M][N] of e4m3 rows xq [M][K] with scales [M][ceil(K / 128)] and the block-scaled weight (+ bias[n]);
    y fp32, bf16 or fp16."""
    index = _first(xq, "xq")
    xa, sa = _arg(xq, torch.float8_e4m3fn, index, "xq"), _arg(x_scale, torch.float32, index, "x_scale")
    cw, ba, yd, out = _fp8_args(xq, w, bias, out, out_dtype, index, "xq")
    M = xq.shape[0]
    if tuple(x_scale.shape) != (M, -(-cw.K // 128)):
        raise ValueError(f"x_scale: expected [{M}][{-(-cw.K // 128)}], got {tuple(x_scale.shape)}")
    lib = load_library()
    workspace, wa, n = _scratch(workspace, lib.cubic_gemm_fp8_workspace_bytes(M, cw.N, cw.K), index)
    _check(_call(index, lib.cubic_gemm_fp8, xa, sa, M, ctypes.byref(cw), ba, out.data_ptr(), yd, wa, n), "cubic_gemm_fp8")
    return out


def cubic_linear_fp8_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load_library().cubic_linear_fp8_workspace_bytes(M, N, K))


def cubic_linear_fp8(x: torch.Tensor, w: Fp8Weight, bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, out_dtype=torch.float32) -> torch.Tensor:
    """cubic_gemm_fp8 of bf16 or fp16 rows x [M][K], quantised per 128 channels on the way (cubic_quant_fp8)."""
    xd = _dense_dtype(x.dtype, "x", _DT_IN)
    index = _first(x, "x")
    xa = _arg(x, x.dtype, index, "x")
    cw, ba, yd, out = _fp8_args(x, w, bias, out, out_dtype, index, "x")
    M = x.shape[0]
    lib = load_library()
    workspace, wa, n = _scratch(workspace, lib.cubic_linear_fp8_workspace_bytes(M, cw.N, cw.K), index)
    _check(_call(index, lib.cubic_linear_fp8, xa, xd, M, ctypes.byref(cw), ba, out.data_ptr(), yd, wa, n), "cubic_linear_fp8")
    return out


def _ff_args(x: torch.Tensor, w: torch.Tensor, index: int):
    """(x, w addresses, dtype code, M, H, I) of a block over 16-bit weights [2 I][H]."""
    xd = _dense_dtype(x.dtype, "x", _DT_IN)
    if x.dim() != 2 or w.dim() != 2 or w.shape[0] % 2 != 0 or w.shape[1] != x.shape[1]:
        raise ValueError(f"expected x [M][H] and w [2 I][H], got {tuple(x.shape)} and {tuple(w.shape)}")
    return _arg(x, x.dtype, index, "x"), _arg(w, x.dtype, index, "w"), xd, x.shape[0], x.shape[1], w.shape[0] // 2


def cubic_gated_ff_workspace_bytes(M: int, H: int, I: int) -> int:
    return int(load_library().cubic_gated_ff_workspace_bytes(M, H, I))


def cubic_gated_ff(x: torch.Tensor, w: torch.Tensor, act="silu", save_pre: bool = False, out: torch.Tensor | None = None,
                   pre: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """h [M][I] = act(x Wg^T) * (x Wu^T) for x [M][H] and w [2 I][H] (gate rows, then up rows), bf16 or fp16.
    With save_pre or a tensor for it, (h, pre): pre fp32 [M][2 I] is what the backward pass takes.
    No graph is recorded, so inputs that require a gradient are refused while one would be (as in
    torch's out= forms): the forward and backward methods of a torch.autograd.Function call this and
    cubic_gated_ff_backward."""
    if (x.requires_grad or w.requires_grad) and torch.is_grad_enabled():
        raise RuntimeError("cubic_gated_ff records no graph, but an input requires a gradient: call it under torch.no_grad(), "
                           "or in a torch.autograd.Function with cubic_gated_ff_backward")
    index = _first(x, "x")
    xa, wa, xd, M, H, I = _ff_args(x, w, index)
    kind = _act(act)
    out = _dense_out(out, x, (M, I), x.dtype, index)
    if save_pre or pre is not None:
        pre = _dense_out(pre, x, (M, 2 * I), torch.float32, index, "pre")
    lib = load_library()
    workspace, sa, n = _scratch(workspace, lib.cubic_gated_ff_workspace_bytes(M, H, I), index)
    _check(_call(index, lib.cubic_gated_ff, xa, wa, xd, M, H, I, kind, out.data_ptr(), None if pre is None else pre.data_ptr(),
                 sa, n), "cubic_gated_ff")
    return out if pre is None else (out, pre)


def cubic_gated_ff_backward_workspace_bytes(M: int, H: int, I: int) -> int:
    return int(load_library().cubic_gated_ff_backward_workspace_bytes(M, H, I))


def cubic_gated_ff_backward(dh: torch.Tensor, x: torch.Tensor, w: torch.Tensor, pre: torch.Tensor, act="silu",
                            need_dx: bool = True, need_dw: bool = True, dx: torch.Tensor | None = None,
                            dw: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """(dx [M][H], dw [2 I][H]) of cubic_gated_ff from dh [M][I] and the forward's pre; None for what is not needed."""
    index = _first(x, "x")
    xa, wa, xd, M, H, I = _ff_args(x, w, index)
    kind = _act(act)
    da, pa = _arg(dh, x.dtype, index, "dh"), _arg(pre, torch.float32, index, "pre")
    if tuple(dh.shape) != (M, I) or tuple(pre.shape) != (M, 2 * I):
        raise ValueError(f"expected dh [{M}][{I}] and pre [{M}][{2 * I}], got {tuple(dh.shape)} and {tuple(pre.shape)}")
    dx = _dense_out(dx, x, (M, H), x.dtype, index, "dx") if need_dx else None
    dw = _dense_out(dw, x, (2 * I, H), x.dtype, index, "dw") if need_dw else None
    lib = load_library()
    workspace, sa, n = _scratch(workspace, lib.cubic_gated_ff_backward_workspace_bytes(M, H, I), index)
    _check(_call(index, lib.cubic_gated_ff_backward, da, xa, wa, pa, xd, M, H, I, kind, None if dx is None else dx.data_ptr(),
                 None if dw is None else dw.data_ptr(), sa, n), "cubic_gated_ff_backward")
    return dx, dw


def cubic_gated_ff_fp8_workspace_bytes(M: int, H: int, I: int) -> int:
    return int(load_library().cubic_gated_ff_fp8_workspace_bytes(M, H, I))


def cubic_gated_ff_fp8(x: torch.Tensor, w: Fp8Weight, act="silu", out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, out_dtype=torch.bfloat16) -> torch.Tensor:
    """cubic_gated_ff over a block-scaled e4m3 weight [2 I][H] (I a multiple of 128), the activations quantised
    on the way; h bf16 or fp16."""
    xd, hd = _dense_dtype(x.dtype, "x", _DT_IN), _dense_dtype(out_dtype, "out_dtype", _DT_IN)
    index = _first(x, "x")
    xa = _arg(x, x.dtype, index, "x")
    cw = _fp8_weight(w, index)
    if x.dim() != 2 or x.shape[1] != cw.K or cw.N % 2 != 0:
        raise ValueError(f"expected x [M][H] and a weight [2 I][H], got {tuple(x.shape)} and [{cw.N}][{cw.K}]")
    kind = _act(act)
    M, I = x.shape[0], cw.N // 2
    out = _dense_out(out, x, (M, I), out_dtype, index)
    lib = load_library()
    workspace, sa, n = _scratch(workspace, lib.cubic_gated_ff_fp8_workspace_bytes(M, cw.K, I), index)
    _check(_call(index, lib.cubic_gated_ff_fp8, xa, xd, M, ctypes.byref(cw), kind, out.data_ptr(), hd, sa, n),
           "cubic_gated_ff_fp8")
    return out
