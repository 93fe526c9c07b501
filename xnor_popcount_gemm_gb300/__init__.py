"""Python binding of libbt, the binarized linear / conv2d forward for GB300.

Argument marshalling only: every step of the forward runs in the CUDA
kernels of ``_build/libbt.so`` (built from ``csrc/`` by ``build.py``). The
functions keep the C names of ``include/bt.h`` and take torch CUDA tensors;
torch supplies device memory and the current stream. A non-OK status raises
``BtError``. If the library has not been built, importing this package raises:
there is no fallback.
"""
from __future__ import annotations

import array
import ctypes
import functools
import math
import operator
import os
import struct

import torch

from . import build as _build

__all__ = [
    "BtError", "lib_path", "BT_F32", "BT_BF16", "BT_F16", "BT_I32", "BT_PACKED", "BT_PACKED_IM2COL",
    "BT_CODE_BITS", "BT_CODE_E4M3", "BT_CODE_E2M1", "BT_LAYOUT_ROWS", "BT_LAYOUT_NCHW_TO_NHWC",
    "BT_ALGO_AUTO", "BT_ALGO_POPC", "BT_ALGO_TC_E4M3", "BT_ALGO_TC_E2M1", "BT_ALGO_TUNE", "BT_OP_LINEAR",
    "BT_OP_CONV2D", "bt_version", "bt_status_string", "bt_packed_row_bytes", "bt_pack_sign",
    "bt_binary_linear_workspace", "bt_binary_linear", "bt_binary_conv2d_workspace",
    "bt_binary_conv2d", "bt_plan", "bt_device_status", "conv2d_out_size", "bt_binary_linear_noalloc",
    "bt_binary_linear_noalloc_max_bytes", "bt_pack_im2col", "bt_conv2d_single_pass", "bt_tune_linear",
    "bt_tune_reset", "bt_tune_conv2d", "bt_conv2d_plan_info", "bt_set_wait_timeout", "bt_binary_linear_dscale_init",
    "bt_binary_conv2d_dscale_init", "bt_distill_topk", "bt_distill_topk_backward", "bt_distill_topk_step",
    "AdapterPlan", "bt_adapter_plan", "bt_adapter_plan_bytes", "bt_adapter_linear", "bt_adapter_linear_workspace",
    "bt_adapter_linear_backward", "bt_adapter_linear_backward_workspace",
    "MxRows", "bt_mx_row_bytes", "bt_mx_scale_bytes", "bt_mx_quantize", "bt_mx_dequantize", "bt_mx_linear",
    "bt_mx_linear_workspace", "bt_mx_transpose", "bt_mx_linear_backward", "bt_mx_linear_backward_workspace",
    "bt_rms_norm", "bt_rms_norm_backward", "bt_rms_norm_backward_workspace", "bt_clip_grads",
    "bt_clip_grads_workspace",
]

BT_OK, BT_ERR_INVALID_ARG, BT_ERR_UNSUPPORTED, BT_ERR_ALIGNMENT = 0, -1, -2, -3
BT_ERR_WORKSPACE, BT_ERR_CUDA, BT_ERR_TIMEOUT = -4, -5, -6
BT_F32, BT_BF16, BT_F16, BT_I32, BT_PACKED, BT_PACKED_IM2COL = 0, 1, 2, 3, 4, 5
BT_CODE_BITS, BT_CODE_E4M3, BT_CODE_E2M1 = 0, 1, 2
BT_LAYOUT_ROWS, BT_LAYOUT_NCHW_TO_NHWC = 0, 1
BT_ALGO_AUTO, BT_ALGO_POPC, BT_ALGO_TC_E4M3, BT_ALGO_TC_E2M1, BT_ALGO_TUNE = 0, 1, 2, 3, 4
BT_OP_LINEAR, BT_OP_CONV2D = 0, 1

_DT = {torch.float32: BT_F32, torch.bfloat16: BT_BF16, torch.float16: BT_F16, torch.int32: BT_I32}
_TORCH = {BT_F32: torch.float32, BT_BF16: torch.bfloat16, BT_F16: torch.float16, BT_I32: torch.int32}

lib_path = _build.LIB
if not os.path.exists(lib_path):
    raise ImportError(f"libbt.so is not built ({lib_path}); run xnor_popcount_gemm_gb300.build.build()")

_lib = ctypes.CDLL(lib_path)
_i64, _p, _f, _i, _sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_int, ctypes.c_size_t


def _sig(name, res, args):
    fn = getattr(_lib, name)
    fn.restype = res
    fn.argtypes = args
    return fn


_c_version = _sig("bt_version", _i, [])
_c_status_string = _sig("bt_status_string", ctypes.c_char_p, [_i])
_c_row_bytes = _sig("bt_packed_row_bytes", _i64, [_i64, _i])
_c_pack = _sig("bt_pack_sign", _i, [_p, _i, _i, _i64, _i64, _i64, _i64, _p, _i64, _i, _p, _p])
_c_lin_ws = _sig("bt_binary_linear_workspace", _sz, [_i64, _i64, _i, _i])
_c_lin = _sig("bt_binary_linear", _i, [_p, _i, _p, _i, _i64, _i64, _i64, _f, _f, _p, _i64, _p, _i, _i,
                                       _p, _sz, _p])
_c_conv_ws = _sig("bt_binary_conv2d_workspace", _sz, [_i64, _i64, _i64, _i64, _i, _i, _i, _i, _i, _i])
_c_conv = _sig("bt_binary_conv2d", _i, [_p, _i, _p, _i, _i64, _i64, _i64, _i64, _i64, _i, _i, _i, _i,
                                        _f, _f, _p, _i64, _p, _i, _i, _p, _sz, _p])
_c_lin_noalloc = _sig("bt_binary_linear_noalloc", _i, [_p, _i, _p, _i, _i64, _i64, _i64, _f, _f, _p, _i64,
                                                      _p, _i, _i, _p])
_c_noalloc_max = _sig("bt_binary_linear_noalloc_max_bytes", _sz, [])
_c_pack_im2col = _sig("bt_pack_im2col", _i, [_p, _i, _i64, _i64, _i64, _i64, _i, _i, _i, _i, _p, _i64, _i, _p, _p])
_c_single_pass = _sig("bt_conv2d_single_pass", _i, [_i64, _i64, _i64, _i64, _i, _i, _i, _i, _i, _i])
_c_bwd_ld = _sig("bt_backward_weight_ld", _i64, [_i64])
_c_sign_t = _sig("bt_sign_transpose", _i, [_p, _i, _i64, _i64, _i64, _p, _p])
_c_bwd_ws = _sig("bt_binary_linear_backward_workspace", _sz, [_i64, _i64, _i64, _i])
_c_bwd = _sig("bt_binary_linear_backward", _i, [_p, _i, _p, _i64, _p, _i64, _i64, _i64, _f, _f, _p, _p, _p, _i,
                                                _p, _sz, _p])
_c_cbwd_ws = _sig("bt_binary_conv2d_backward_workspace", _sz, [_i64, _i64, _i64, _i64, _i64, _i, _i, _i, _i, _i, _i])
_c_cbwd_impl = _sig("bt_conv2d_backward_implicit", _i, [_i64, _i64, _i64, _i64, _i64, _i, _i, _i, _i])
_c_cbwd = _sig("bt_binary_conv2d_backward", _i, [_p, _i, _p, _i64, _p, _i64, _i64, _i64, _i64, _i64, _i, _i, _i, _i,
                                                 _f, _f, _p, _p, _p, _i, _p, _sz, _p])
_c_scale_init = _sig("bt_scale_init", _i, [_p, _i, _i64, _f, _i, _p, _p])
_c_lin_ds = _sig("bt_binary_linear_dscale", _i, [_p, _i, _p, _i, _i64, _i64, _i64, _p, _p, _i64, _p, _i, _i,
                                                _p, _sz, _p])
_c_conv_ds = _sig("bt_binary_conv2d_dscale", _i, [_p, _i, _p, _i, _i64, _i64, _i64, _i64, _i64, _i, _i, _i, _i,
                                                 _p, _p, _i64, _p, _i, _i, _p, _sz, _p])
_c_lin_dsi = _sig("bt_binary_linear_dscale_init", _i, [_p, _i, _p, _i, _i64, _i64, _i64, _p, _f, _i, _p, _i64, _p,
                                                      _i, _i, _p, _sz, _p])
_c_conv_dsi = _sig("bt_binary_conv2d_dscale_init", _i, [_p, _i, _p, _i, _i64, _i64, _i64, _i64, _i64, _i, _i, _i,
                                                       _i, _p, _f, _i, _p, _i64, _p, _i, _i, _p, _sz, _p])
_c_w8_ws = _sig("bt_w8a8_conv2d_workspace", _sz, [_i64, _i64, _i64, _i64, _i64, _i, _i, _i, _i])
_c_w8 = _sig("bt_w8a8_conv2d", _i, [_p, _i, _p, _i, _i64, _i64, _i64, _i64, _i64, _i, _i, _i, _i, _i, _p, _i, _p,
                                    _sz, _p])
_c_distill = _sig("bt_distill_topk", _i, [_p, _i, _i64, _i64, _i64, _p, _i, _p, _i, _i64, _p, _f, _p, _p, _p])
_c_distill_bwd = _sig("bt_distill_topk_backward", _i, [_p, _p, _i, _i64, _i64, _i64, _p, _i, _p, _i, _i64, _p, _p, _f,
                                                      _p, _i64, _p])
_c_distill_step = _sig("bt_distill_topk_step", _i, [_p, _p, _i, _i64, _i64, _i64, _p, _i, _p, _i, _i64, _p, _f, _p,
                                                   _p, _p, _i64, _p])


class AdapterPlanInfo(ctypes.Structure):
    """bt_adapter_plan_info: what bt_adapter_plan says of a batch."""
    _fields_ = [("tokens", _i64), ("adapters", _i64)] + [(n, ctypes.c_int32) for n in (
        "used", "most_tokens", "without", "tiles", "small_tiles", "small_most", "parts", "slots")]


_pinfo = ctypes.POINTER(AdapterPlanInfo)
_c_aplan_bytes = _sig("bt_adapter_plan_bytes", _sz, [_i64, _i64])
_c_aplan = _sig("bt_adapter_plan", _i, [_p, _i64, _i64, _p, _sz, _pinfo])
_c_alin_ws = _sig("bt_adapter_linear_workspace", _sz, [_i64, _i64, _i64, _i64, _pinfo])
_c_alin = _sig("bt_adapter_linear", _i, [_p, _i, _i64, _p, _p, _p, _p, _pinfo, _i64, _i64, _i64, _i64, _p, _i, _i64,
                                         _p, _i, _i64, _p, _p, _sz, _p])
_c_abwd_ws = _sig("bt_adapter_linear_backward_workspace", _sz, [_i64, _i64, _i64, _i64, _pinfo])
_c_abwd = _sig("bt_adapter_linear_backward", _i, [_p, _i64, _p, _i64, _p, _p, _p, _p, _p, _pinfo, _i64, _i64, _i64,
                                                 _i64, _p, _i64, _p, _i64, _p, _p, _p, _sz, _p])
_c_mx_rb = _sig("bt_mx_row_bytes", _i64, [_i64, _i])
_c_mx_sb = _sig("bt_mx_scale_bytes", _sz, [_i64, _i64, _i])
_c_mx_q = _sig("bt_mx_quantize", _i, [_p, _i, _i64, _i64, _i64, _i, _p, _p, _p])
_c_mx_dq = _sig("bt_mx_dequantize", _i, [_p, _p, _i64, _i64, _i, _p, _i, _i64, _p])
_c_mx_lin_ws = _sig("bt_mx_linear_workspace", _sz, [_i64, _i64, _i64, _i, _i])
_c_mx_lin = _sig("bt_mx_linear", _i, [_p, _i, _i64, _p, _p, _p, _i, _i64, _i64, _i64, _p, _i, _i64, _p, _sz, _p])
_c_mx_t = _sig("bt_mx_transpose", _i, [_p, _p, _i64, _i64, _i, _i64, _p, _p])
_c_mx_bwd_ws = _sig("bt_mx_linear_backward_workspace", _sz, [_i64, _i64])
_c_mx_bwd = _sig("bt_mx_linear_backward", _i, [_p, _i64, _p, _i64, _i64, _i64, _i64, _p, _i, _p, _sz, _p])
_c_rms = _sig("bt_rms_norm", _i, [_p, _i, _i64, _p, _i64, _p, _i, _i64, _i64, ctypes.c_double, _p, _i64, _p, _i64, _i, _p,
                                  _p, _p])
_c_rms_bwd_ws = _sig("bt_rms_norm_backward_workspace", _sz, [_i64, _i64])
_c_rms_bwd = _sig("bt_rms_norm_backward", _i, [_p, _i, _i64, _p, _i64, _p, _i, _i64, _i64, ctypes.c_double, _p, _i64, _p,
                                               _i64, _p, _p, _sz, _p])
_c_clip_ws = _sig("bt_clip_grads_workspace", _sz, [_i64])
_c_clip = _sig("bt_clip_grads", _i, [_p, _p, _p, _i64, _f, _f, _p, _p, _sz, _p])
_c_plan = _sig("bt_plan", _i, [_i, _i64, _i64, _i64, ctypes.POINTER(_i), ctypes.POINTER(_i)])


class TuneResult(ctypes.Structure):
    """bt_tune_result: what bt_tune_linear measured and kept."""
    _fields_ = [("code", _i), ("pair", _i), ("bn", _i), ("slices_per_stage", _i), ("epilogue_warps", _i),
                ("candidates", _i), ("us", _f), ("us_model", _f)]


_c_tune = _sig("bt_tune_linear", _i, [_p, _i, _p, _i, _i64, _i64, _i64, _f, _f, _p, _i64, _p, _i, _p, _sz, _i, _p,
                                      ctypes.POINTER(TuneResult)])
_c_tune_reset = _sig("bt_tune_reset", None, [])


class TuneConvResult(ctypes.Structure):
    """bt_tune_conv_result: what bt_tune_conv2d measured and kept."""
    _fields_ = [("code", _i), ("pair", _i), ("weights_resident", _i), ("pixel_stages", _i), ("fused", _i),
                ("candidates", _i), ("us", _f), ("us_model", _f), ("band_split", _i)]


_c_tune_conv = _sig("bt_tune_conv2d", _i, [_p, _i, _p, _i, _i64, _i64, _i64, _i64, _i64, _i, _i, _i, _i, _f, _f, _p,
                                           _i64, _p, _i, _p, _sz, _i, _p, ctypes.POINTER(TuneConvResult)])
_c_status = _sig("bt_device_status", _i, [_p])
_c_wait = _sig("bt_set_wait_timeout", _i, [ctypes.c_uint64])

#: every symbol include/bt.h declares
EXPORTED = ["bt_version", "bt_status_string", "bt_packed_row_bytes", "bt_pack_sign",
            "bt_binary_linear_workspace", "bt_binary_linear", "bt_binary_conv2d_workspace",
            "bt_binary_conv2d", "bt_plan", "bt_device_status", "bt_binary_linear_noalloc",
            "bt_binary_linear_noalloc_max_bytes", "bt_pack_im2col", "bt_conv2d_single_pass", "bt_tune_linear",
            "bt_tune_reset", "bt_tune_conv2d", "bt_conv2d_plan_info",
            "bt_backward_weight_ld", "bt_sign_transpose", "bt_binary_linear_backward_workspace",
            "bt_binary_linear_backward", "bt_binary_conv2d_backward_workspace", "bt_conv2d_backward_implicit",
            "bt_binary_conv2d_backward",
            "bt_scale_init", "bt_binary_linear_dscale", "bt_binary_conv2d_dscale", "bt_w8a8_conv2d_workspace",
            "bt_w8a8_conv2d", "bt_set_wait_timeout", "bt_binary_linear_dscale_init", "bt_binary_conv2d_dscale_init",
            "bt_distill_topk", "bt_distill_topk_backward", "bt_distill_topk_step", "bt_adapter_plan_bytes",
            "bt_adapter_plan", "bt_adapter_linear_workspace", "bt_adapter_linear",
            "bt_adapter_linear_backward_workspace", "bt_adapter_linear_backward",
            "bt_mx_row_bytes", "bt_mx_scale_bytes", "bt_mx_quantize", "bt_mx_dequantize", "bt_mx_linear_workspace",
            "bt_mx_linear", "bt_mx_transpose", "bt_mx_linear_backward_workspace", "bt_mx_linear_backward", "bt_rms_norm",
            "bt_rms_norm_backward_workspace", "bt_rms_norm_backward", "bt_clip_grads_workspace", "bt_clip_grads"]


class BtError(RuntimeError):
    def __init__(self, status: int):
        super().__init__(bt_status_string(status))
        self.status = status


def _check(st: int) -> None:
    if st != BT_OK:
        raise BtError(st)


def _stream(stream=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def bt_version() -> int:
    return int(_c_version())


def bt_status_string(status: int) -> str:
    return _c_status_string(status).decode()


def bt_packed_row_bytes(k: int, code: int) -> int:
    return int(_c_row_bytes(k, code))


def conv2d_out_size(h: int, k: int, s: int, p: int, d: int) -> int:
    return (h + 2 * p - d * (k - 1) - 1) // s + 1


def _contig(t: torch.Tensor, name: str) -> None:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def bt_pack_sign(x: torch.Tensor, code: int, layout: int = BT_LAYOUT_ROWS, bias=None,
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Shift + sign + pack. ROWS: x [R, K] -> uint8 [R, row_bytes(K)];
    NCHW_TO_NHWC: x [B, C, H, W] -> uint8 [B, H, W, row_bytes(C)]."""
    _contig(x, "x")
    if layout == BT_LAYOUT_ROWS:
        if x.dim() != 2:
            raise ValueError("ROWS layout wants a 2-D x")
        d = (x.shape[0], x.shape[1], 1, 1)
        shape = (x.shape[0], bt_packed_row_bytes(x.shape[1], code))
    else:
        if x.dim() != 4:
            raise ValueError("NCHW_TO_NHWC layout wants a 4-D x")
        d = tuple(x.shape)
        shape = (x.shape[0], x.shape[2], x.shape[3], bt_packed_row_bytes(x.shape[1], code))
    if out is None:
        out = torch.empty(shape, dtype=torch.uint8, device=x.device)
    blen = 0 if bias is None else bias.numel()
    _check(_c_pack(_ptr(x), _DT[x.dtype], layout, *d, _ptr(bias), blen, code, _ptr(out), _stream(stream)))
    return out


def bt_pack_im2col(x: torch.Tensor, code: int, kernel_size: int, stride: int, padding: int, dilation: int,
                   bias=None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Shift + sign + pack + unfold of NCHW x [B, C, H, W]: the im2col rows
    uint8 [B*Ho*Wo, k*k*row_bytes(C)] a tensor-core conv contracts."""
    _contig(x, "x")
    if x.dim() != 4:
        raise ValueError("bt_pack_im2col wants a 4-D x")
    B, C, H, W = x.shape
    Ho = conv2d_out_size(H, kernel_size, stride, padding, dilation)
    Wo = conv2d_out_size(W, kernel_size, stride, padding, dilation)
    if out is None:
        out = torch.empty((B * max(Ho, 0) * max(Wo, 0), kernel_size * kernel_size * bt_packed_row_bytes(C, code)),
                          dtype=torch.uint8, device=x.device)
    blen = 0 if bias is None else bias.numel()
    _check(_c_pack_im2col(_ptr(x), _DT[x.dtype], B, C, H, W, kernel_size, stride, padding, dilation, _ptr(bias),
                          blen, code, _ptr(out), _stream(stream)))
    return out


def bt_conv2d_single_pass(B: int, C: int, H: int, W: int, kernel_size: int, stride: int, padding: int,
                          dilation: int, x_dtype: int, code: int) -> int:
    """How bt_binary_conv2d splits its work on float x: 2 one kernel from x,
    1 one-pass im2col rows + contraction, 0 NHWC pack + contraction."""
    return int(_c_single_pass(B, C, H, W, kernel_size, stride, padding, dilation, x_dtype, code))


def bt_backward_weight_ld(N: int) -> int:
    return int(_c_bwd_ld(N))


def bt_sign_transpose(w: torch.Tensor, ld: int | None = None, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """torch.sign of w [R, C], transposed to bf16 [C, ld] (zeros past R):
    the weight operand of bt_binary_linear_backward (ld defaults to
    bt_backward_weight_ld(R))."""
    _contig(w, "w")
    if w.dim() != 2:
        raise ValueError("bt_sign_transpose wants a 2-D w")
    R, C = w.shape
    ld = bt_backward_weight_ld(R) if ld is None else ld
    if out is None:
        out = torch.empty((C, ld), dtype=torch.bfloat16, device=w.device)
    _check(_c_sign_t(_ptr(w), _DT[w.dtype], R, C, ld, _ptr(out), _stream(stream)))
    return out


def bt_binary_linear_backward_workspace(M: int, N: int, K: int, want_grad_weight: bool = True) -> int:
    return int(_c_bwd_ws(M, N, K, 1 if want_grad_weight else 0))


def bt_binary_linear_backward(x: torch.Tensor, wst: torch.Tensor | None, g: torch.Tensor, scale_a: float,
                              scale_w: float, grad_input: bool = True, grad_weight_dtype=torch.bfloat16,
                              grad_x: torch.Tensor | None = None, grad_scale_a: torch.Tensor | None = None,
                              grad_w: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                              stream=None):
    """Straight-through backward of the binary linear layer for upstream
    gradient g [M, N] (bf16) and forward input x [M, K] (bf16 or f32):
    returns (grad_x [M, K] bf16, grad_scale_a (device float tensor),
    grad_w [N, K]); grad_x / grad_scale_a are None unless grad_input,
    grad_w is None when grad_weight_dtype is None. wst is
    bt_sign_transpose(W)."""
    _contig(x, "x")
    _contig(g, "g")
    M, K = x.shape
    N = g.shape[1]
    if g.shape[0] != M:
        raise ValueError("g and x disagree on M")
    if grad_input:
        if wst is None:
            raise ValueError("grad_input needs wst = bt_sign_transpose(W)")
        _contig(wst, "wst")
        if grad_x is None:
            grad_x = torch.empty((M, K), dtype=torch.bfloat16, device=x.device)
        if grad_scale_a is None:
            grad_scale_a = torch.empty((), dtype=torch.float32, device=x.device)
    else:
        grad_x = grad_scale_a = None
    if grad_weight_dtype is not None and grad_w is None:
        grad_w = torch.empty((N, K), dtype=grad_weight_dtype, device=x.device)
    elif grad_weight_dtype is None:
        grad_w = None
    ws = _workspace(bt_binary_linear_backward_workspace(M, N, K, grad_w is not None), x.device, workspace)
    ldw = wst.shape[1] if (grad_input and wst is not None) else 0
    _check(_c_bwd(_ptr(x), _DT[x.dtype], _ptr(wst) if grad_input else None, ldw, _ptr(g), M, N, K, scale_a,
                  scale_w, _ptr(grad_x), _ptr(grad_scale_a), _ptr(grad_w),
                  _DT[grad_w.dtype] if grad_w is not None else BT_BF16, _ptr(ws),
                  0 if ws is None else ws.numel(), _stream(stream)))
    return grad_x, grad_scale_a, grad_w


def bt_binary_conv2d_backward_workspace(B: int, C: int, H: int, W: int, O: int, kernel_size: int, stride: int,
                                        padding: int, dilation: int, want_grad_input: bool = True,
                                        want_grad_weight: bool = True) -> int:
    return int(_c_cbwd_ws(B, C, H, W, O, kernel_size, stride, padding, dilation, 1 if want_grad_input else 0,
                          1 if want_grad_weight else 0))


def bt_conv2d_backward_implicit(B: int, C: int, H: int, W: int, O: int, kernel_size: int, stride: int, padding: int,
                                dilation: int) -> bool:
    """Whether bt_binary_conv2d_backward computes grad_x of this geometry as
    one implicit GEMM (else the tap matrix and gather route)."""
    return bool(_c_cbwd_impl(B, C, H, W, O, kernel_size, stride, padding, dilation))


def bt_binary_conv2d_backward(x: torch.Tensor, wst: torch.Tensor | None, g: torch.Tensor, O: int, kernel_size: int,
                              stride: int, padding: int, dilation: int, scale_a: float, scale_w: float,
                              grad_input: bool = True, grad_weight_dtype=torch.bfloat16,
                              grad_x: torch.Tensor | None = None, grad_scale_a: torch.Tensor | None = None,
                              grad_w: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                              stream=None):
    """Straight-through backward of the binary conv2d layer: x [B, C, H, W]
    (bf16 or f32), g [B, O, Ho, Wo] bf16, wst = bt_sign_transpose(w.view(O,
    -1)). Returns (grad_x [B, C, H, W] bf16, grad_scale_a (device float
    tensor), grad_w [O, C, k, k]), as bt_binary_linear_backward does."""
    _contig(x, "x")
    _contig(g, "g")
    B, C, H, W = x.shape
    k = kernel_size
    if grad_input:
        if wst is None:
            raise ValueError("grad_input needs wst = bt_sign_transpose(w.view(O, -1))")
        _contig(wst, "wst")
        if grad_x is None:
            grad_x = torch.empty((B, C, H, W), dtype=torch.bfloat16, device=x.device)
        if grad_scale_a is None:
            grad_scale_a = torch.empty((), dtype=torch.float32, device=x.device)
    else:
        grad_x = grad_scale_a = None
    if grad_weight_dtype is not None and grad_w is None:
        grad_w = torch.empty((O, C, k, k), dtype=grad_weight_dtype, device=x.device)
    elif grad_weight_dtype is None:
        grad_w = None
    ws = _workspace(bt_binary_conv2d_backward_workspace(B, C, H, W, O, k, stride, padding, dilation,
                                                        grad_x is not None, grad_w is not None), x.device, workspace)
    ldw = wst.shape[1] if (grad_input and wst is not None) else 0
    _check(_c_cbwd(_ptr(x), _DT[x.dtype], _ptr(wst) if grad_input else None, ldw, _ptr(g), B, C, H, W, O, k, stride,
                   padding, dilation, scale_a, scale_w, _ptr(grad_x), _ptr(grad_scale_a), _ptr(grad_w),
                   _DT[grad_w.dtype] if grad_w is not None else BT_BF16, _ptr(ws), 0 if ws is None else ws.numel(),
                   _stream(stream)))
    return grad_x, grad_scale_a, grad_w


def bt_binary_linear_workspace(M: int, K: int, x_dtype: int, code: int) -> int:
    return int(_c_lin_ws(M, K, x_dtype, code))


def bt_binary_conv2d_workspace(B: int, C: int, H: int, W: int, kernel_size: int, stride: int,
                               padding: int, dilation: int, x_dtype: int, code: int) -> int:
    return int(_c_conv_ws(B, C, H, W, kernel_size, stride, padding, dilation, x_dtype, code))


def _workspace(nbytes: int, device, ws):
    if nbytes == 0:
        return None
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws


def bt_binary_linear(x: torch.Tensor, weight: torch.Tensor, w_code: int, K: int, scale_a: float,
                     scale_w: float, bias_a=None, out_dtype=None, algo: int = BT_ALGO_AUTO,
                     x_packed: bool = False, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = cast(fp32(dot * fp32(scale_a*scale_w))) for x [M, K] (or packed rows)
    and a packed weight [N, row_bytes(K)]. Passing a device float tensor
    {scale_a, scale_w} as scale_a (scale_w ignored) reads the scales on the
    device (bt_binary_linear_dscale)."""
    _contig(x, "x")
    _contig(weight, "weight")
    M, N = x.shape[0], weight.shape[0]
    xt = BT_PACKED if x_packed else _DT[x.dtype]
    if out_dtype is None:
        out_dtype = x.dtype if not x_packed else torch.float32
    ot = _DT[out_dtype]
    if out is None:
        out = torch.empty((M, N), dtype=_TORCH[ot], device=x.device)
    ws = _workspace(bt_binary_linear_workspace(M, K, xt, w_code), x.device, workspace)
    blen = 0 if bias_a is None else bias_a.numel()
    if isinstance(scale_a, torch.Tensor):
        # device scales: scale_a is a device float tensor holding {scale_a, scale_w}
        _contig(scale_a, "scales")
        _check(_c_lin_ds(_ptr(x), xt, _ptr(weight), w_code, M, N, K, _ptr(scale_a), _ptr(bias_a), blen,
                         _ptr(out), ot, algo, _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))
        return out
    _check(_c_lin(_ptr(x), xt, _ptr(weight), w_code, M, N, K, scale_a, scale_w, _ptr(bias_a), blen,
                  _ptr(out), ot, algo, _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))
    return out


def bt_binary_conv2d(x: torch.Tensor, weight: torch.Tensor, w_code: int, C: int, kernel_size: int,
                     stride: int, padding: int, dilation: int, scale_a: float, scale_w: float,
                     bias_a=None, out_dtype=None, algo: int = BT_ALGO_AUTO, x_packed: bool = False,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None, x_im2col_hw: tuple | None = None) -> torch.Tensor:
    """NCHW x [B, C, H, W] (or packed NHWC [B, H, W, row_bytes(C)]) with a
    packed weight [O, k, k, row_bytes(C)] -> NCHW [B, O, Ho, Wo]. With
    x_im2col_hw = (B, H, W), x is the rows bt_pack_im2col wrote for an input
    of that batch and size."""
    _contig(x, "x")
    _contig(weight, "weight")
    if x_im2col_hw is not None:
        B, H, W = x_im2col_hw
        xt = BT_PACKED_IM2COL
    elif x_packed:
        B, H, W = x.shape[0], x.shape[1], x.shape[2]
        xt = BT_PACKED
    else:
        B, C2, H, W = x.shape
        if C2 != C:
            raise ValueError("C does not match x")
        xt = _DT[x.dtype]
    O = weight.shape[0]
    if out_dtype is None:
        out_dtype = x.dtype if xt not in (BT_PACKED, BT_PACKED_IM2COL) else torch.float32
    ot = _DT[out_dtype]
    Ho = conv2d_out_size(H, kernel_size, stride, padding, dilation)
    Wo = conv2d_out_size(W, kernel_size, stride, padding, dilation)
    if out is None:
        out = torch.empty((B, O, max(Ho, 0), max(Wo, 0)), dtype=_TORCH[ot], device=x.device)
    ws = _workspace(bt_binary_conv2d_workspace(B, C, H, W, kernel_size, stride, padding, dilation, xt, w_code),
                    x.device, workspace)
    blen = 0 if bias_a is None else bias_a.numel()
    if isinstance(scale_a, torch.Tensor):
        # device scales: scale_a is a device float tensor holding {scale_a, scale_w}
        _contig(scale_a, "scales")
        _check(_c_conv_ds(_ptr(x), xt, _ptr(weight), w_code, B, C, H, W, O, kernel_size, stride, padding,
                          dilation, _ptr(scale_a), _ptr(bias_a), blen, _ptr(out), ot, algo, _ptr(ws),
                          0 if ws is None else ws.numel(), _stream(stream)))
        return out
    _check(_c_conv(_ptr(x), xt, _ptr(weight), w_code, B, C, H, W, O, kernel_size, stride, padding,
                   dilation, scale_a, scale_w, _ptr(bias_a), blen, _ptr(out), ot, algo, _ptr(ws),
                   0 if ws is None else ws.numel(), _stream(stream)))
    return out


def bt_binary_linear_dscale_init(x: torch.Tensor, weight: torch.Tensor, w_code: int, K: int, scales: torch.Tensor,
                                 factor: float = 2.0, scale_dtype=None, bias_a=None, out_dtype=None,
                                 algo: int = BT_ALGO_AUTO, out: torch.Tensor | None = None,
                                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """A layer's first forward: scales[0] = (factor * mean|x|) in x's dtype,
    then scale_dtype (x's dtype by default), computed from the read of x that
    packs it; then the forward with alpha = fp32(scales[0] * scales[1])."""
    _contig(x, "x")
    _contig(weight, "weight")
    _contig(scales, "scales")
    M, N = x.shape[0], weight.shape[0]
    xt = _DT[x.dtype]
    st = _DT[scale_dtype if scale_dtype is not None else x.dtype]
    ot = _DT[out_dtype if out_dtype is not None else x.dtype]
    if out is None:
        out = torch.empty((M, N), dtype=_TORCH[ot], device=x.device)
    ws = _workspace(bt_binary_linear_workspace(M, K, xt, w_code), x.device, workspace)
    blen = 0 if bias_a is None else bias_a.numel()
    _check(_c_lin_dsi(_ptr(x), xt, _ptr(weight), w_code, M, N, K, _ptr(scales), factor, st, _ptr(bias_a), blen,
                      _ptr(out), ot, algo, _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))
    return out


def bt_binary_conv2d_dscale_init(x: torch.Tensor, weight: torch.Tensor, w_code: int, kernel_size: int, stride: int,
                                 padding: int, dilation: int, scales: torch.Tensor, factor: float = 2.0,
                                 scale_dtype=None, bias_a=None, out_dtype=None, algo: int = BT_ALGO_AUTO,
                                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                                 stream=None) -> torch.Tensor:
    """The conv2d form of bt_binary_linear_dscale_init (NCHW x, packed weight
    [O, k, k, row_bytes(C)], NCHW out)."""
    _contig(x, "x")
    _contig(weight, "weight")
    _contig(scales, "scales")
    B, C, H, W = x.shape
    O = weight.shape[0]
    xt = _DT[x.dtype]
    st = _DT[scale_dtype if scale_dtype is not None else x.dtype]
    ot = _DT[out_dtype if out_dtype is not None else x.dtype]
    Ho = conv2d_out_size(H, kernel_size, stride, padding, dilation)
    Wo = conv2d_out_size(W, kernel_size, stride, padding, dilation)
    if out is None:
        out = torch.empty((B, O, max(Ho, 0), max(Wo, 0)), dtype=_TORCH[ot], device=x.device)
    ws = _workspace(bt_binary_conv2d_workspace(B, C, H, W, kernel_size, stride, padding, dilation, xt, w_code),
                    x.device, workspace)
    blen = 0 if bias_a is None else bias_a.numel()
    _check(_c_conv_dsi(_ptr(x), xt, _ptr(weight), w_code, B, C, H, W, O, kernel_size, stride, padding, dilation,
                       _ptr(scales), factor, st, _ptr(bias_a), blen, _ptr(out), ot, algo, _ptr(ws),
                       0 if ws is None else ws.numel(), _stream(stream)))
    return out


def bt_w8a8_conv2d_workspace(B: int, C: int, H: int, W: int, O: int, kernel_size: int, stride: int, padding: int,
                             dilation: int) -> int:
    return int(_c_w8_ws(B, C, H, W, O, kernel_size, stride, padding, dilation))


def bt_w8a8_conv2d(x: torch.Tensor, w: torch.Tensor, stride: int, padding: int, dilation: int, smooth: bool = False,
                   out_dtype=torch.float32, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """W8A8 im2col + gemm convolution of NCHW x with OIHW w (f32 or bf16),
    optionally with SmoothQuant; NCHW out in out_dtype (f32 or bf16)."""
    _contig(x, "x")
    _contig(w, "w")
    B, C, H, W = x.shape
    O, _, k, _ = w.shape
    Ho, Wo = conv2d_out_size(H, k, stride, padding, dilation), conv2d_out_size(W, k, stride, padding, dilation)
    if out is None:
        out = torch.empty((B, O, max(Ho, 0), max(Wo, 0)), dtype=out_dtype, device=x.device)
    ws = _workspace(bt_w8a8_conv2d_workspace(B, C, H, W, O, k, stride, padding, dilation), x.device, workspace)
    _check(_c_w8(_ptr(x), _DT[x.dtype], _ptr(w), _DT[w.dtype], B, C, H, W, O, k, stride, padding, dilation,
                 1 if smooth else 0, _ptr(out), _DT[out.dtype], _ptr(ws), 0 if ws is None else ws.numel(),
                 _stream(stream)))
    return out


def bt_scale_init(x: torch.Tensor, factor: float = 2.0, scale_dtype=None, out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """(factor * x.abs().mean()).to(scale_dtype) computed on the device into a
    one-element float tensor (scale_dtype defaults to x's dtype)."""
    _contig(x, "x")
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=x.device)
    st = _DT[x.dtype if scale_dtype is None else scale_dtype]
    _check(_c_scale_init(_ptr(x), _DT[x.dtype], x.numel(), factor, st, _ptr(out), _stream(stream)))
    return out


_ID_BYTES = {torch.int32: 4, torch.int64: 8}


_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _on_device_of(name: str, at: int):
    """Runs the call with the device of its operand `name` (the at-th argument) current: launches, workspace sizes and
    kernel attributes belong to the current device."""
    def wrap(fn):
        @functools.wraps(fn)
        def call(*args, **kw):
            t = args[at] if at < len(args) else kw.get(name)
            if type(t) is AdapterPlan:
                t = t.buffer
            elif type(t) is MxRows:
                t = t._tensors()[0]
            device = t.get_device() if isinstance(t, torch.Tensor) else -1
            if device < 0 or device == _current_device():
                return fn(*args, **kw)
            with torch.cuda.device(device):
                return fn(*args, **kw)
        return call
    return wrap


def _same_device(first, stream, *tensors) -> None:
    at = first.get_device()
    for t in tensors:
        if t is not None and t.get_device() != at:
            raise ValueError(f"operands must be on one device, {first.device} by the first: one is on {t.device}")
    if stream is not None and stream.device != first.device:
        raise ValueError(f"stream must be one of {first.device}, where the first operand is")


def _scratch(workspace, need: int, device, stream):
    """A workspace of need bytes: the one given, where it holds them."""
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        if workspace.numel() * workspace.element_size() >= need:
            return workspace
    return _empty((need,), torch.uint8, device, stream) if need else None


def _on_stream(stream, device) -> int:
    """The raw stream of a call: the one given, or the device's current one."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """A tensor of the caching allocator that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _written(*given) -> None:
    """Tells autograd which tensors of the caller's a call has written (in place or not; None: not the caller's): a graph
    that holds one for its backward refuses to go on with other values."""
    given = [t for t in given if t is not None]
    if given:
        torch.autograd.graph.increment_version(given)


def _dense(t, name: str, shape: tuple, dtype) -> None:
    if t.shape != shape or t.dtype != dtype or not t.is_cuda:
        raise ValueError(f"{name} must be a {dtype} CUDA tensor of shape {list(shape)}")
    _contig(t, name)


def _distill_args(logits, ids, top, teacher_lse, stream, *others):
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be [T, V] with elements of a row next to each other")
    T, V = logits.shape
    if ids.dim() != 2 or ids.shape[0] != T or top.shape != ids.shape:
        raise ValueError("ids and top must both be [T, S]")
    if ids.dtype not in _ID_BYTES:
        raise ValueError("ids must be int32 or int64")
    _contig(ids, "ids")
    _contig(top, "top")
    if teacher_lse is not None:
        _dense(teacher_lse, "teacher_lse", (T,), torch.float32)
    _same_device(logits, stream, ids, top, teacher_lse, *others)
    return T, V, (logits.stride(0) if T > 1 else max(V, logits.stride(0)))


def _distill_grad(logits, grad, T, V, stream):
    if grad is None:
        grad = _empty((T, V), logits.dtype, logits.device, stream)
    elif not grad.is_cuda or grad.shape != logits.shape or grad.dtype != logits.dtype or (V > 1 and grad.stride(1) != 1):
        raise ValueError("grad must be a CUDA tensor of the logits' shape and dtype, with elements of a row next to each other")
    return grad, (grad.stride(0) if T > 1 else max(V, grad.stride(0)))


@_on_device_of("logits", 0)
def bt_distill_topk(logits: torch.Tensor, ids: torch.Tensor, top: torch.Tensor, teacher_lse: torch.Tensor | None = None,
                    temperature: float = 1.0, loss: torch.Tensor | None = None, stats: torch.Tensor | None = None,
                    stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Distillation loss of every row of logits [T, V] against a teacher's top
    logits (top [T, S] at the vocabulary entries ids [T, S], -1 for an empty
    slot): (loss [T], stats [T, 2]), both float. teacher_lse [T], the
    teacher's log-sum-exp of its logits / temperature, counts the teacher's
    remaining probability as one more outcome; without it the teacher is
    normalized over its slots."""
    T, V, ld = _distill_args(logits, ids, top, teacher_lse, stream, loss, stats)
    given = loss, stats
    if loss is None:
        loss = _empty((T,), torch.float32, logits.device, stream)
    else:
        _dense(loss, "loss", (T,), torch.float32)
    if stats is None:
        stats = _empty((T, 2), torch.float32, logits.device, stream)
    else:
        _dense(stats, "stats", (T, 2), torch.float32)
    _check(_c_distill(_ptr(logits), _DT[logits.dtype], T, V, ld, _ptr(ids), _ID_BYTES[ids.dtype], _ptr(top),
                      _DT[top.dtype], ids.shape[1], _ptr(teacher_lse), temperature, _ptr(loss), _ptr(stats),
                      _on_stream(stream, logits.device)))
    _written(*given)
    return loss, stats


@_on_device_of("logits", 1)
def bt_distill_topk_backward(grad_loss: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, top: torch.Tensor,
                             stats: torch.Tensor, teacher_lse: torch.Tensor | None = None, temperature: float = 1.0,
                             grad: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient [T, V] (the logits' dtype) of bt_distill_topk's loss for
    grad_loss [T] and the forward's stats, for teachers whose probabilities
    sum to one: with top in 16 bits, a teacher_lse below logsumexp(top /
    temperature) is to be raised to it. grad may be the logits."""
    T, V, ld = _distill_args(logits, ids, top, teacher_lse, stream, grad_loss, stats, grad)
    given = grad
    _dense(grad_loss, "grad_loss", (T,), torch.float32)
    _dense(stats, "stats", (T, 2), torch.float32)
    grad, ldg = _distill_grad(logits, grad, T, V, stream)
    _check(_c_distill_bwd(_ptr(grad_loss), _ptr(logits), _DT[logits.dtype], T, V, ld, _ptr(ids), _ID_BYTES[ids.dtype],
                          _ptr(top), _DT[top.dtype], ids.shape[1], _ptr(stats), _ptr(teacher_lse), temperature,
                          _ptr(grad), ldg, _on_stream(stream, logits.device)))
    _written(given)
    return grad


@_on_device_of("logits", 1)
def bt_distill_topk_step(grad_loss: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, top: torch.Tensor,
                         teacher_lse: torch.Tensor | None = None, temperature: float = 1.0,
                         loss: torch.Tensor | None = None, grad: torch.Tensor | None = None,
                         stats: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Loss [T] and gradient [T, V] in one kernel (few rows are read once, many
    twice, the second time out of L2), for an upstream
    gradient grad_loss [T] known beforehand. grad may be the logits."""
    T, V, ld = _distill_args(logits, ids, top, teacher_lse, stream, grad_loss, loss, grad, stats)
    given = loss, grad, stats
    _dense(grad_loss, "grad_loss", (T,), torch.float32)
    if loss is None:
        loss = _empty((T,), torch.float32, logits.device, stream)
    else:
        _dense(loss, "loss", (T,), torch.float32)
    if stats is not None:
        _dense(stats, "stats", (T, 2), torch.float32)
    grad, ldg = _distill_grad(logits, grad, T, V, stream)
    _check(_c_distill_step(_ptr(grad_loss), _ptr(logits), _DT[logits.dtype], T, V, ld, _ptr(ids),
                           _ID_BYTES[ids.dtype], _ptr(top), _DT[top.dtype], ids.shape[1], _ptr(teacher_lse),
                           temperature, _ptr(loss), _ptr(stats), _ptr(grad), ldg, _on_stream(stream, logits.device)))
    _written(*given)
    return loss, grad


class AdapterPlan:
    """The adapters of a batch's tokens, sorted for bt_adapter_linear and its
    backward: `buffer` on the device, `info` on the host. One plan serves every
    projection the batch goes through."""

    def __init__(self, buffer: torch.Tensor, info: AdapterPlanInfo):
        self.buffer, self.info = buffer, info
        self.tokens, self.adapters = info.tokens, info.adapters
        self._ref = ctypes.byref(info)

    def __repr__(self) -> str:
        return "AdapterPlan(%s)" % ", ".join(f"{f}={getattr(self.info, f)}" for f, _ in AdapterPlanInfo._fields_)


def bt_adapter_plan_bytes(T: int, L: int) -> int:
    return int(_c_aplan_bytes(T, L))


def bt_adapter_plan(adapter_ids, num_adapters: int, device="cuda", stream=None) -> AdapterPlan:
    """Plan of a batch from the adapter of every token (a sequence of ints or
    a CPU tensor; -1 for a token without one), copied to the device on the
    stream."""
    ids = torch.as_tensor(adapter_ids) if len(adapter_ids) else torch.empty(0, dtype=torch.int32)
    if ids.dim() != 1 or ids.is_cuda or ids.is_floating_point() or ids.dtype == torch.bool:
        raise ValueError("adapter_ids must be a 1-D sequence or CPU tensor of integers")
    if ids.dtype != torch.int32:
        if ids.numel() and (int(ids.min()) < -1 or int(ids.max()) >= num_adapters):
            raise BtError(BT_ERR_INVALID_ARG)
        ids = ids.to(torch.int32)
    ids = ids.contiguous()
    T = ids.numel()
    if stream is not None and torch.device(device) not in (torch.device("cuda"), stream.device):
        raise ValueError(f"stream must be one of {device}")
    host = torch.empty(max(bt_adapter_plan_bytes(T, num_adapters) // 4, 1), dtype=torch.int32,
                       pin_memory=torch.device(device).type == "cuda")
    info = AdapterPlanInfo()
    _check(_c_aplan(_ptr(ids), T, num_adapters, _ptr(host), host.numel() * 4, ctypes.byref(info)))
    if stream is None:
        return AdapterPlan(host.to(device, non_blocking=True), info)
    with torch.cuda.stream(stream):
        return AdapterPlan(host.to(device, non_blocking=True), info)


_F32, _BF16, _F16 = (torch.float32,), (torch.bfloat16,), (torch.float16,)
_HALVES = {torch.bfloat16: _BF16 + _F32, torch.float16: _F16 + _F32}


def _rows(t: torch.Tensor, name: str, T: int, C: int, dtypes) -> int:
    """Elements from one row of a [T, C] operand to the next."""
    if t.shape != (T, C) or t.dtype not in dtypes or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor of shape {[T, C]} and type {' or '.join(map(str, dtypes))}")
    ld, one = t.stride()
    if one != 1 and C > 1:
        raise ValueError(f"{name} must have the elements of a row next to each other")
    return ld if T > 1 else max(C, ld)


def _adapter_args(x, a, b, scale, plan, stream, *others):
    if x.dim() != 2 or a.dim() != 3 or b.dim() != 3:
        raise ValueError("x must be [T, K], a [L, R, K] and b [L, N, R]")
    T, K = x.shape
    L, R, _ = a.shape
    N = b.shape[1]
    dt = x.dtype
    if dt not in _HALVES:
        raise ValueError("x must be bfloat16 or float16")
    if a.shape != (L, R, K) or b.shape != (L, N, R) or a.dtype != dt or b.dtype != dt or not (a.is_cuda and b.is_cuda):
        raise ValueError("a [L, R, K] and b [L, N, R] must be CUDA tensors of x's type that agree with x and with each other")
    if not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("a and b must be contiguous")
    if scale.shape != (L,):
        raise ValueError("scale must be [L]")
    _dense(scale, "scale", (L,), torch.float32)
    if type(plan) is not AdapterPlan or plan.tokens != T or plan.adapters != L or not plan.buffer.is_cuda:
        raise ValueError("plan must be bt_adapter_plan of these tokens and adapters, on the device")
    _same_device(x, stream, a, b, scale, plan.buffer, *others)
    return T, K, N, R


@_on_device_of("plan", 4)
def bt_adapter_linear_workspace(T: int, K: int, N: int, R: int, plan: AdapterPlan) -> int:
    return int(_c_alin_ws(T, K, N, R, plan._ref))


@_on_device_of("x", 0)
def bt_adapter_linear(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, scale: torch.Tensor, plan: AdapterPlan,
                      base: torch.Tensor | None = None, out_dtype=None, u: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """base [T, N] plus scale[i] * b[i] (a[i] x_t) for the adapter i of every
    token of x [T, K] (bf16 or f16), a [L, R, K], b [L, N, R]: out [T, N] in
    out_dtype (base's type, else x's). out may be base. u [T, R] (float), if
    given, receives a[i] x_t for the backward."""
    T, K, N, R = _adapter_args(x, a, b, scale, plan, stream, base, u, out, workspace)
    given = u, out
    dt = x.dtype
    ldx = _rows(x, "x", T, K, (dt,))
    if base is None:
        pbase, base_type, ldb = None, BT_F32, 0
    else:
        ldb = _rows(base, "base", T, N, _HALVES[dt])
        pbase, base_type = base.data_ptr(), _DT[base.dtype]
    if out is None:
        out = _empty((T, N), out_dtype if out_dtype is not None else dt if base is None else base.dtype, x.device, stream)
    ldo = _rows(out, "out", T, N, _HALVES[dt] if out_dtype is None else (out_dtype,))
    if u is not None:
        _dense(u, "u", (T, R), torch.float32)
    need = _c_alin_ws(T, K, N, R, plan._ref)
    workspace = _scratch(workspace, need, x.device, stream)
    _check(_c_alin(x.data_ptr(), _DT[dt], ldx, a.data_ptr(), b.data_ptr(), scale.data_ptr(), plan.buffer.data_ptr(),
                   plan._ref, T, K, N, R, pbase, base_type, ldb, out.data_ptr(), _DT[out.dtype], ldo,
                   None if u is None else u.data_ptr(), None if workspace is None else workspace.data_ptr(), need,
                   _on_stream(stream, x.device)))
    _written(*given)
    return out


@_on_device_of("plan", 4)
def bt_adapter_linear_backward_workspace(T: int, K: int, N: int, R: int, plan: AdapterPlan) -> int:
    return int(_c_abwd_ws(T, K, N, R, plan._ref))


@_on_device_of("x", 0)
def bt_adapter_linear_backward(x: torch.Tensor, g: torch.Tensor, u: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                               scale: torch.Tensor, plan: AdapterPlan, grad_base: torch.Tensor | None = None,
                               grad_x: torch.Tensor | None = None, grad_a: torch.Tensor | None = None,
                               grad_b: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradients of bt_adapter_linear for g [T, N] (bf16, the gradient of its
    result), its input x and its u: (grad_x [T, K] bf16, grad_a [L, R, K],
    grad_b [L, N, R], both float). grad_base [T, K], the projection's own
    input gradient, is added to grad_x, which may be grad_base itself."""
    T, K, N, R = _adapter_args(x, a, b, scale, plan, stream, g, u, grad_base, grad_x, grad_a, grad_b, workspace)
    given = grad_x, grad_a, grad_b
    ldx, ldg = _rows(x, "x", T, K, _BF16), _rows(g, "g", T, N, _BF16)
    _dense(u, "u", (T, R), torch.float32)
    ldgb = 0 if grad_base is None else _rows(grad_base, "grad_base", T, K, _BF16)
    if grad_x is None:
        grad_x = _empty((T, K), torch.bfloat16, x.device, stream)
    ldgx = _rows(grad_x, "grad_x", T, K, _BF16)
    if grad_a is None:
        grad_a = _empty(a.shape, torch.float32, x.device, stream)
    else:
        _dense(grad_a, "grad_a", tuple(a.shape), torch.float32)
    if grad_b is None:
        grad_b = _empty(b.shape, torch.float32, x.device, stream)
    else:
        _dense(grad_b, "grad_b", tuple(b.shape), torch.float32)
    need = _c_abwd_ws(T, K, N, R, plan._ref)
    workspace = _scratch(workspace, need, x.device, stream)
    _check(_c_abwd(_ptr(x), ldx, _ptr(g), ldg, _ptr(u), _ptr(a), _ptr(b), _ptr(scale), _ptr(plan.buffer), plan._ref, T,
                   K, N, R, _ptr(grad_base), ldgb, _ptr(grad_x), ldgx, _ptr(grad_a), _ptr(grad_b), _ptr(workspace), need,
                   _on_stream(stream, x.device)))
    _written(*given)
    return grad_x, grad_a, grad_b


class MxRows:
    """A microscaled operand [R, K]: `codes` uint8 [R, bt_mx_row_bytes(K, code)] and `scales` uint8
    [bt_mx_scale_bytes(R, K, code)] on the device, `code` BT_CODE_E4M3 or BT_CODE_E2M1."""

    __slots__ = ("K", "code", "_rows", "_row", "_codes", "_scales", "_buffer")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, K: int, code: int):
        row = bt_mx_row_bytes(K, code)
        if row == 0:
            raise ValueError("code must be BT_CODE_E4M3 or BT_CODE_E2M1 and K in [1, 2^24)")
        if codes.dim() != 2 or codes.shape[1] != row or codes.dtype != torch.uint8 or not codes.is_cuda:
            raise ValueError(f"codes must be a uint8 CUDA tensor of shape [R, {row}]")
        _contig(codes, "codes")
        _dense(scales, "scales", (bt_mx_scale_bytes(codes.shape[0], K, code),), torch.uint8)
        self._codes, self._scales, self._buffer, self.K, self.code = codes, scales, None, K, code
        self._rows, self._row = codes.shape[0], row

    @classmethod
    def _new(cls, R: int, K: int, code: int, device, stream) -> "MxRows":
        """One of the library's own: codes, then scales, in one allocation."""
        if code not in (BT_CODE_E4M3, BT_CODE_E2M1) or not 1 <= K < 1 << 24:
            raise BtError(BT_ERR_INVALID_ARG)
        q = cls.__new__(cls)
        q.K, q.code, q._rows = K, code, R
        q._row = row = (K + 255) // 256 * 128 if code == BT_CODE_E2M1 else (K + 127) // 128 * 128
        q._codes = q._scales = None
        # 512 bytes of scales for 128 rows and 128 values of K
        q._buffer = _empty((R * row + (R + 127) // 128 * (row * (8 if code == BT_CODE_E2M1 else 4)),), torch.uint8, device, stream)
        return q

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            self._codes = self._buffer[:self._rows * self._row].view(self._rows, self._row)
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            self._scales = self._buffer[self._rows * self._row:]
        return self._scales

    @property
    def shape(self) -> tuple[int, int]:
        return self._rows, self.K

    @property
    def device(self) -> torch.device:
        return self._tensors()[0].device

    def _tensors(self):
        """What holds its memory."""
        return (self._codes, self._scales) if self._buffer is None else (self._buffer,)

    def _pointers(self):
        if self._buffer is None:
            return self._codes.data_ptr(), self._scales.data_ptr()
        p = self._buffer.data_ptr()
        return p, p + self._rows * self._row

    def __repr__(self) -> str:
        return f"MxRows({list(self.shape)}, {'E4M3' if self.code == BT_CODE_E4M3 else 'E2M1'}, {self.device})"


def bt_mx_row_bytes(K: int, code: int) -> int:
    return int(_c_mx_rb(K, code))


def bt_mx_scale_bytes(R: int, K: int, code: int) -> int:
    return int(_c_mx_sb(R, K, code))


_FLOATS = (torch.float32, torch.bfloat16, torch.float16)


def _float_rows(t: torch.Tensor, name: str, dtypes=_FLOATS):
    """A 2-D operand's elements from one row to the next, its rows and its columns."""
    if t.dim() != 2 or t.dtype not in dtypes or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D CUDA tensor of type {' or '.join(map(str, dtypes))}")
    T, C = t.shape
    ld, one = t.stride()
    if one != 1 and C > 1:
        raise ValueError(f"{name} must have the elements of a row next to each other")
    return (ld if T > 1 else max(C, ld)), T, C


def _mx(q, name: str):
    if type(q) is not MxRows:
        raise ValueError(f"{name} must be MxRows")
    return q


@_on_device_of("x", 0)
def bt_mx_quantize(x: torch.Tensor, code: int, out: MxRows | None = None, stream=None) -> MxRows:
    """x [R, K] in blocks of 32 along K that share a power of two, as E4M3 or E2M1 values."""
    ld, R, K = _float_rows(x, "x")
    given = out
    if out is not None:
        if _mx(out, "out").shape != (R, K) or out.code != code:
            raise ValueError("out must be MxRows of x's shape and the code")
        _same_device(x, stream, *out._tensors())
    else:
        _same_device(x, stream)
        out = MxRows._new(R, K, code, x.device, stream)
    _check(_c_mx_q(x.data_ptr(), _DT[x.dtype], ld, R, K, code, *out._pointers(), _on_stream(stream, x.device)))
    if given is not None:
        _written(*given._tensors())
    return out


@_on_device_of("q", 0)
def bt_mx_dequantize(q: MxRows, out_dtype=torch.float32, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values [R, K] of an operand in out_dtype."""
    R, K = _mx(q, "q").shape
    first, *others = q._tensors()
    _same_device(first, stream, *others, out)
    given = out
    if out is None and out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype must be {' or '.join(map(str, _FLOATS))}")
    if out is None:
        out = _empty((R, K), out_dtype, first.device, stream)
    ldo = _rows(out, "out", R, K, _FLOATS)
    _check(_c_mx_dq(*q._pointers(), R, K, q.code, out.data_ptr(), _DT[out.dtype], ldo, _on_stream(stream, first.device)))
    _written(given)
    return out


def bt_mx_linear_workspace(M: int, N: int, K: int, x_dtype: int, code: int) -> int:
    return int(_c_mx_lin_ws(M, N, K, x_dtype, code))


@_on_device_of("x", 0)
def bt_mx_linear(x, w: MxRows, out_dtype=None, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """out [M, N] = x w^T for a weight operand w [N, K] and x [M, K]: a float tensor (quantised to w's code by the
    call) or MxRows in w's code. out_dtype: x's type, bfloat16 for MxRows."""
    N, K = _mx(w, "w").shape
    code = w.code
    if out_dtype is not None and out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype must be {' or '.join(map(str, _FLOATS))}")
    if type(x) is MxRows:
        if x.code != code or x.K != K:
            raise ValueError("x and w must agree on K and the code")
        M, xt, ldx, dt = x._rows, BT_PACKED, K, torch.bfloat16
        first, *others = x._tensors()
        xp, xs = x._pointers()
    else:
        ldx, M, columns = _float_rows(x, "x")
        if columns != K:
            raise ValueError("x and w must agree on K")
        dt, first, others, xp, xs = x.dtype, x, (), x.data_ptr(), None
        xt = _DT[dt]
    _same_device(first, stream, *others, *w._tensors(), out, workspace)
    device, given = first.device, out
    if out is None:
        out = _empty((M, N), dt if out_dtype is None else out_dtype, device, stream)
    ldo = _rows(out, "out", M, N, _FLOATS if out_dtype is None else (out_dtype,))
    call = (xp, xt, ldx, xs, *w._pointers(), code, M, N, K, out.data_ptr(), _DT[out.dtype], ldo)
    raw = _on_stream(stream, device)
    if M <= 16 and workspace is None:
        # few rows need no workspace: the query costs a microsecond of a call's sixteen
        status = _c_mx_lin(*call, None, 0, raw)
        if status != BT_ERR_WORKSPACE:
            _check(status)
            _written(given)
            return out
    need = _c_mx_lin_ws(M, N, K, xt, code)
    workspace = _scratch(workspace, need, device, stream)
    _check(_c_mx_lin(*call, None if workspace is None else workspace.data_ptr(), need, raw))
    _written(given)
    return out


@_on_device_of("w", 0)
def bt_mx_transpose(w: MxRows, ld: int | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """An operand w [N, K] as bf16 [K, ld], transposed, zeros past N: the weight of bt_mx_linear_backward
    (ld defaults to bt_backward_weight_ld(N))."""
    N, K = _mx(w, "w").shape
    ld = bt_backward_weight_ld(N) if ld is None else ld
    first, *others = w._tensors()
    _same_device(first, stream, *others, out)
    given = out
    if out is None:
        out = _empty((K, ld), torch.bfloat16, first.device, stream)
    else:
        _dense(out, "out", (K, ld), torch.bfloat16)
    _check(_c_mx_t(*w._pointers(), N, K, w.code, ld, out.data_ptr(), _on_stream(stream, first.device)))
    _written(given)
    return out


def bt_mx_linear_backward_workspace(M: int, N: int) -> int:
    return int(_c_mx_bwd_ws(M, N))


@_on_device_of("g", 0)
def bt_mx_linear_backward(g: torch.Tensor, wt: torch.Tensor, out_dtype=torch.bfloat16, grad_x: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The input gradient [M, K] of bt_mx_linear for the upstream gradient g [M, N] (bf16), wt = bt_mx_transpose(w)."""
    ldg, M, N = _float_rows(g, "g", _BF16)
    if wt.dim() != 2 or wt.dtype != torch.bfloat16 or not wt.is_cuda or wt.shape[1] < N:
        raise ValueError("wt must be bt_mx_transpose(w) for g's N columns")
    _contig(wt, "wt")
    K, ldw = wt.shape
    _same_device(g, stream, wt, grad_x, workspace)
    given = grad_x
    if (out_dtype if grad_x is None else grad_x.dtype) not in (torch.bfloat16, torch.float32):
        raise ValueError("grad_x must be bfloat16 or float32")
    if grad_x is None:
        grad_x = _empty((M, K), out_dtype, g.device, stream)
    _dense(grad_x, "grad_x", (M, K), grad_x.dtype)
    need = 0 if ldg % 8 == 0 and N % 8 == 0 and g.data_ptr() % 16 == 0 else _c_mx_bwd_ws(M, N)
    workspace = _scratch(workspace, need, g.device, stream)
    _check(_c_mx_bwd(g.data_ptr(), ldg, wt.data_ptr(), ldw, M, N, K, grad_x.data_ptr(), _DT[grad_x.dtype],
                     None if workspace is None else workspace.data_ptr(), need, _on_stream(stream, g.device)))
    _written(given)
    return grad_x


def _norm_weight(weight, N: int, dtype) -> int:
    if weight is None:
        return BT_F32
    t = weight.dtype
    if t not in (dtype, torch.float32) or weight.shape != (N,) or not weight.is_cuda or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous CUDA tensor of shape {[N]} and of x's type or float32")
    return _DT[t]


@_on_device_of("x", 0)
def bt_rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6,
                residual: torch.Tensor | None = None, want_out: bool = True, code: int | None = None,
                sum: torch.Tensor | None = None, out: torch.Tensor | None = None, q: MxRows | None = None, stream=None):
    """h = x + residual (in x's type), y = h * weight / sqrt(mean(h^2) + eps) along the rows of x [T, N]: returns
    (y, h, codes). y is None unless want_out; h (which may be written over x or residual: sum) None without a
    residual; codes, y as MxRows in `code`, None without a code."""
    ldx, T, N = _float_rows(x, "x")
    dt = (x.dtype,)
    if q is not None:
        if _mx(q, "q").shape != (T, N) or (code is not None and q.code != code):
            raise ValueError("q must be MxRows of x's shape and the code")
        code = q.code
    if out is not None and not want_out:
        raise ValueError("out is given and not wanted")
    if sum is not None and residual is None:
        raise ValueError("sum needs a residual")
    given = sum, out, *(() if q is None else q._tensors())
    _same_device(x, stream, weight, residual, *given)
    wt = _norm_weight(weight, N, x.dtype)
    ldr = lds = ldo = 0
    if residual is not None:
        ldr = _rows(residual, "residual", T, N, dt)
        if sum is None:
            sum = _empty((T, N), x.dtype, x.device, stream)
        lds = _rows(sum, "sum", T, N, dt)
    if want_out:
        if out is None:
            out = _empty((T, N), x.dtype, x.device, stream)
        ldo = _rows(out, "out", T, N, dt)
    if code is not None and q is None:
        q = MxRows._new(T, N, code, x.device, stream)
    codes, scales = (None, None) if q is None else q._pointers()
    _check(_c_rms(x.data_ptr(), _DT[x.dtype], ldx, _ptr(residual), ldr, _ptr(weight), wt, T, N, eps, _ptr(sum), lds, _ptr(out),
                  ldo, 0 if q is None else code, codes, scales, _on_stream(stream, x.device)))
    _written(*given)
    return out, sum, q


def bt_rms_norm_backward_workspace(T: int, N: int) -> int:
    return int(_c_rms_bwd_ws(T, N))


@_on_device_of("g", 0)
def bt_rms_norm_backward(g: torch.Tensor, h: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6,
                         grad_sum: torch.Tensor | None = None, want_grad_weight: bool = True,
                         grad_x: torch.Tensor | None = None, grad_weight: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, stream=None):
    """Gradients of bt_rms_norm for the upstream gradient g [T, N] of y, h what was normed (its sum, or x) and grad_sum
    the gradient of h that comes along the residual stream: (grad_x [T, N], of x and of the residual alike,
    grad_weight [N] float, None unless wanted)."""
    ldg, T, N = _float_rows(g, "g")
    dt = (g.dtype,)
    ldh = _rows(h, "h", T, N, dt)
    _same_device(g, stream, h, weight, grad_sum, grad_x, grad_weight, workspace)
    given = grad_x, grad_weight
    wt = _norm_weight(weight, N, g.dtype)
    ldgs = 0 if grad_sum is None else _rows(grad_sum, "grad_sum", T, N, dt)
    if grad_x is None:
        grad_x = _empty((T, N), g.dtype, g.device, stream)
    ldgx = _rows(grad_x, "grad_x", T, N, dt)
    if grad_weight is not None:
        if not want_grad_weight:
            raise ValueError("grad_weight is given and not wanted")
        _dense(grad_weight, "grad_weight", (N,), torch.float32)
    elif want_grad_weight:
        grad_weight = _empty((N,), torch.float32, g.device, stream)
    need = _c_rms_bwd_ws(T, N)
    workspace = _scratch(workspace, need, g.device, stream)
    _check(_c_rms_bwd(g.data_ptr(), _DT[g.dtype], ldg, h.data_ptr(), ldh, _ptr(weight), wt, T, N, eps, _ptr(grad_sum), ldgs,
                      grad_x.data_ptr(), ldgx, _ptr(grad_weight), _ptr(workspace), need, _on_stream(stream, g.device)))
    _written(*given)
    return grad_x, grad_weight


def bt_clip_grads_workspace(count: int) -> int:
    return int(_c_clip_ws(count))


_dtype_of = operator.attrgetter("dtype")


def bt_clip_grads(grads, max_norm: float, eps: float = 1e-6, norm: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The norm of all of grads (contiguous CUDA tensors, float32, bfloat16 or float16) as a device float, and each of them
    times min(1, max_norm / (norm + eps)), in place. max_norm = inf: the norm alone."""
    grads = list(grads)
    if not grads or not all(issubclass(t, torch.Tensor) for t in set(map(type, grads))):
        raise ValueError("grads must be tensors, one at least")
    return _clip_grads(grads[0], grads, max_norm, eps, norm, workspace, stream)


@_on_device_of("first", 0)
def _clip_grads(first, grads, max_norm, eps, norm, workspace, stream):
    # (maps, sets and arrays: hundreds of tensors are looked at before a launch of microseconds)
    n = len(grads)
    dtypes = list(map(_dtype_of, grads))
    kinds = set(dtypes)
    if not kinds.issubset(_FLOATS) or not first.is_cuda:
        raise ValueError("grads must be CUDA tensors of float32, bfloat16 or float16")
    _same_device(first, stream, norm, workspace)
    if set(map(torch.Tensor.get_device, grads)) != {first.get_device()}:
        raise ValueError(f"grads must be on one device, {first.device} by the first")
    if not all(map(torch.Tensor.is_contiguous, grads)):
        raise ValueError("grads must be contiguous")
    given = norm
    if norm is None:
        norm = _empty((), torch.float32, first.device, stream)
    else:
        _dense(norm, "norm", (), torch.float32)
    need = _c_clip_ws(n)
    workspace = _scratch(workspace, need, first.device, stream)
    pointers = struct.pack(f"{n}Q", *map(torch.Tensor.data_ptr, grads))
    numels = struct.pack(f"{n}q", *map(torch.Tensor.numel, grads))
    types = array.array("i", map(_DT.__getitem__, dtypes)) if len(kinds) > 1 else array.array("i", (_DT[first.dtype],)) * n
    _check(_c_clip(pointers, numels, types.buffer_info()[0], n, max_norm, eps, norm.data_ptr(), _ptr(workspace), need,
                   _on_stream(stream, first.device)))
    # (while the GPU is at work)
    _written(given)
    if max_norm < math.inf:
        torch.autograd.graph.increment_version(grads)
    return norm


def bt_binary_linear_noalloc_max_bytes() -> int:
    return int(_c_noalloc_max())


def bt_binary_linear_noalloc(x: torch.Tensor, weight: torch.Tensor, w_code: int, K: int, scale_a: float,
                             scale_w: float, bias_a=None, out_dtype=None, algo: int = BT_ALGO_AUTO,
                             x_packed: bool = False, out: torch.Tensor | None = None,
                             stream=None) -> torch.Tensor:
    """bt_binary_linear without a workspace: for callers that cannot allocate
    device memory (the packed activations go to the library's fixed scratch
    array). Only `out`, if not given, is allocated here, by torch."""
    _contig(x, "x")
    _contig(weight, "weight")
    M, N = x.shape[0], weight.shape[0]
    xt = BT_PACKED if x_packed else _DT[x.dtype]
    if out_dtype is None:
        out_dtype = x.dtype if not x_packed else torch.float32
    ot = _DT[out_dtype]
    if out is None:
        out = torch.empty((M, N), dtype=_TORCH[ot], device=x.device)
    blen = 0 if bias_a is None else bias_a.numel()
    _check(_c_lin_noalloc(_ptr(x), xt, _ptr(weight), w_code, M, N, K, scale_a, scale_w, _ptr(bias_a), blen,
                          _ptr(out), ot, algo, _stream(stream)))
    return out


def bt_plan(op: int, M: int, N: int, K: int) -> tuple[int, int]:
    """The (code, algo) the library runs fastest for this problem size."""
    code, algo = _i(0), _i(0)
    _check(_c_plan(op, M, N, K, ctypes.byref(code), ctypes.byref(algo)))
    return code.value, algo.value


def bt_tune_linear(x: torch.Tensor, weight: torch.Tensor, w_code: int, K: int, scale_a: float, scale_w: float,
                   bias_a=None, out_dtype=None, x_packed: bool = False, reps: int = 10,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Time this linear forward in every candidate launch shape and keep the
    fastest for later bt_binary_linear calls of the same size; returns the
    bt_tune_result fields as a dict."""
    _contig(x, "x")
    _contig(weight, "weight")
    M, N = x.shape[0], weight.shape[0]
    xt = BT_PACKED if x_packed else _DT[x.dtype]
    if out_dtype is None:
        out_dtype = x.dtype if not x_packed else torch.float32
    ot = _DT[out_dtype]
    if out is None:
        out = torch.empty((M, N), dtype=_TORCH[ot], device=x.device)
    ws = _workspace(bt_binary_linear_workspace(M, K, xt, w_code), x.device, workspace)
    blen = 0 if bias_a is None else bias_a.numel()
    res = TuneResult()
    _check(_c_tune(_ptr(x), xt, _ptr(weight), w_code, M, N, K, scale_a, scale_w, _ptr(bias_a), blen, _ptr(out), ot,
                   _ptr(ws), 0 if ws is None else ws.numel(), reps, _stream(stream), ctypes.byref(res)))
    return {f: getattr(res, f) for f, _ in TuneResult._fields_}


def bt_tune_conv2d(x: torch.Tensor, weight: torch.Tensor, w_code: int, C: int, kernel_size: int, stride: int,
                   padding: int, dilation: int, scale_a: float, scale_w: float, bias_a=None, out_dtype=None,
                   x_packed: bool = False, reps: int = 10, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Time this convolution in every candidate plan and keep the fastest for
    later bt_binary_conv2d calls of the same geometry; returns the
    bt_tune_conv_result fields as a dict."""
    _contig(x, "x")
    _contig(weight, "weight")
    if x_packed:
        B, H, W = x.shape[0], x.shape[1], x.shape[2]
        xt = BT_PACKED
    else:
        B, C2, H, W = x.shape
        if C2 != C:
            raise ValueError("C does not match x")
        xt = _DT[x.dtype]
    O = weight.shape[0]
    if out_dtype is None:
        out_dtype = x.dtype if not x_packed else torch.float32
    ot = _DT[out_dtype]
    Ho = conv2d_out_size(H, kernel_size, stride, padding, dilation)
    Wo = conv2d_out_size(W, kernel_size, stride, padding, dilation)
    if out is None:
        out = torch.empty((B, O, max(Ho, 0), max(Wo, 0)), dtype=_TORCH[ot], device=x.device)
    ws = _workspace(bt_binary_conv2d_workspace(B, C, H, W, kernel_size, stride, padding, dilation, xt, w_code),
                    x.device, workspace)
    blen = 0 if bias_a is None else bias_a.numel()
    res = TuneConvResult()
    _check(_c_tune_conv(_ptr(x), xt, _ptr(weight), w_code, B, C, H, W, O, kernel_size, stride, padding, dilation,
                        scale_a, scale_w, _ptr(bias_a), blen, _ptr(out), ot, _ptr(ws), 0 if ws is None else ws.numel(),
                        reps, _stream(stream), ctypes.byref(res)))
    return {f: getattr(res, f) for f, _ in TuneConvResult._fields_}


class ConvPlanInfo(ctypes.Structure):
    """bt_conv_plan_info: the tiling of the implicit-im2col convolution."""
    _fields_ = [(n, _i) for n in ("implicit", "pair", "weights_resident", "pixel_stages", "bands", "band_rows",
                                  "cta_rows", "row_width", "tile_n", "cta_n", "staged_rows", "phases",
                                  "max_tap_shift", "tiles", "smem_bytes")]


_c_plan_info = _sig("bt_conv2d_plan_info", _i, [_i64, _i64, _i64, _i64, _i64, _i, _i, _i, _i, _i, _i, _i, _i, _i,
                                               ctypes.POINTER(ConvPlanInfo)])


def bt_conv2d_plan_info(B: int, C: int, H: int, W: int, O: int, kernel_size: int, stride: int, padding: int,
                        dilation: int, code: int, out_dtype=torch.float32, sms: int = 152, pair: int = -1,
                        split: int = 1) -> dict:
    """The tiling the implicit-im2col convolution takes for this geometry
    (host only): the bt_conv_plan_info fields as a dict."""
    info = ConvPlanInfo()
    _check(_c_plan_info(B, C, H, W, O, kernel_size, stride, padding, dilation, code, _DT[out_dtype], sms, pair,
                        split, ctypes.byref(info)))
    return {f: getattr(info, f) for f, _ in ConvPlanInfo._fields_}


def bt_tune_reset() -> None:
    """Forget every launch shape, plan and code bt_tune_linear / bt_tune_conv2d kept."""
    _c_tune_reset()


def bt_set_wait_timeout(ns: int) -> None:
    """Limit (ns) of the tensor-core kernels' bounded waits for later launches;
    0 restores the default (2 s)."""
    _check(_c_wait(ns))


def bt_device_status(stream=None) -> int:
    """Synchronize the stream; return (and clear) the device error status."""
    return int(_c_status(_stream(stream)))
