"""ctypes binding of libmoe_b200.so: the C entry points under the same names.

Argument marshalling only. Tensors are passed as their device addresses,
shapes as ints, the stream as torch's current CUDA stream unless given. Every
step of the layer runs in the library's CUDA kernels; there is no fallback:
if the library is missing or cannot load, importing this module raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re
from typing import Optional

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_b200.so")
HEADER_PATH = os.path.join(os.path.dirname(PKG), "include", "moe_b200.h")

MOE_OK = 0
STATUS = {0: "MOE_OK", 1: "MOE_ERR_NULL", 2: "MOE_ERR_INVALID", 3: "MOE_ERR_UNSUPPORTED",
          4: "MOE_ERR_WORKSPACE", 5: "MOE_ERR_ALIGN", 6: "MOE_ERR_CUDA", 7: "MOE_ERR_DEVICE"}
MOE_F32, MOE_BF16 = 0, 1
MOE_ACT_GELU, MOE_ACT_SWIGLU = 0, 1
MOE_LAYER_GATHER_IN_GEMM, MOE_LAYER_BINNED, MOE_LAYER_Z_LOSS, MOE_LAYER_COMBINE_IN_GEMM = 1, 2, 4, 8
MOE_LAYER_MXFP4 = 32
DEVERR_EXPERT_RANGE, DEVERR_ROW_RANGE, DEVERR_TIMEOUT = 1, 2, 4
_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str = ""):
        super().__init__(f"{fn} -> {STATUS.get(status, status)} {msg}".strip())
        self.status = status


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"libmoe_b200.so is not built ({path}); run "
                          "`python mixture_experts_routing_route_b200/build.py`")
    return ctypes.CDLL(path)


_lib = load_library()

c_void_p, c_int, c_int64, c_size_t = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
c_double, c_uint32 = ctypes.c_double, ctypes.c_uint32


class MoeLayerC(ctypes.Structure):
    _fields_ = [("d", c_int), ("E", c_int), ("k", c_int), ("F", c_int), ("dtype", c_int),
                ("act", c_int), ("capacity_factor", c_double), ("w_router", c_void_p),
                ("router_bias", c_void_p), ("w1", c_void_p), ("w3", c_void_p), ("w2", c_void_p),
                ("flags", c_int), ("x_router", c_void_p), ("logit_noise", c_void_p),
                ("router_temperature", ctypes.c_float), ("w1_scales", c_void_p),
                ("w3_scales", c_void_p), ("w2_scales", c_void_p)]


class MoeViewsC(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in ("topk_idx", "topk_w", "aux_loss", "z_loss", "counts", "bins",
                                        "kept_counts", "seg_offsets", "sorted_slot",
                                        "slot_to_row", "row_slot", "drop_mask", "x_perm", "h",
                                        "y_perm")] + [("rows_max", c_int64), ("capacity", c_int64),
                                                     ("x_perm_scales", c_void_p), ("h_scales", c_void_p)]


_SIGS = {
    "moe_status_string": (ctypes.c_char_p, [c_int]),
    "moe_workspace_init": (c_int, [c_void_p, c_size_t, c_void_p]),
    "moe_workspace_set_wait_limit": (c_int, [c_void_p, c_size_t, c_uint32, c_void_p]),
    "moe_kernel_launches": (ctypes.c_uint64, []),
    "moe_get_device_error": (c_int, [c_void_p, c_void_p, ctypes.POINTER(c_uint32), c_int]),
    "moe_capacity": (c_int64, [c_double, c_int, c_int, c_int]),
    "moe_rows_max": (c_int64, [c_int, c_int, c_int, c_int64]),
    "moe_route_workspace_size": (c_size_t, [c_int, c_int, c_int]),
    "moe_route": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int,
                          c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                          c_void_p]),
    "moe_permute_workspace_size": (c_size_t, [c_int, c_int, c_int]),
    "moe_permute": (c_int, [c_void_p, c_int, c_int, c_int, c_int64] + [c_void_p] * 8
                    + [c_void_p, c_size_t, c_void_p]),
    "moe_permute_noalloc": (c_int, [c_void_p, c_int, c_int, c_int, c_int64] + [c_void_p] * 9
                            + [c_void_p]),
    "moe_route_train": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, ctypes.c_float, c_int, c_int,
                                c_int, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p,
                                c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "moe_route_backward_workspace_size": (c_size_t, [c_int, c_int, c_int]),
    "moe_route_backward": (c_int, [c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int] + [c_void_p] * 5
                           + [ctypes.c_float] * 3 + [c_void_p] * 4 + [c_size_t, c_void_p]),
    "moe_router_jitter": (c_int, [c_void_p, c_int, c_int, c_int, ctypes.c_float, ctypes.c_uint64,
                                  c_void_p, c_void_p]),
    "moe_router_noise": (c_int, [c_int, c_int, ctypes.c_float, ctypes.c_uint64, c_void_p, c_void_p]),
    "moe_permute_binned": (c_int, [c_void_p, c_int, c_int, c_int, c_int64] + [c_void_p] * 8
                           + [c_void_p, c_size_t, c_void_p]),
    "moe_rows_max_binned": (c_int64, [c_int, c_int, c_int, c_int64]),
    "moe_gather": (c_int, [c_void_p, c_int, c_int, c_int, c_int, c_void_p, c_void_p, c_int,
                           c_int64, c_void_p, c_void_p, c_size_t, c_void_p]),
    "moe_expert_ffn": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int64,
                               c_int, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p,
                               c_size_t, c_void_p]),
    "moe_combine": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int64,
                            c_void_p, c_void_p, c_size_t, c_void_p]),
    "moe_combine_backward": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int,
                                     c_int, c_int64, c_void_p, c_void_p, c_void_p, c_size_t,
                                     c_void_p]),
    "moe_gather_backward": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int,
                                    c_int64, c_void_p, c_void_p, c_size_t, c_void_p]),
    "moe_mxfp4_weight_scales_size": (c_size_t, [c_int, c_int, c_int]),
    "moe_mxfp4_row_scales_size": (c_size_t, [c_int64, c_int, c_int]),
    "moe_mxfp4_quantize_weights": (c_int, [c_void_p, c_int, c_int, c_int, c_int, c_void_p,
                                           c_void_p, c_void_p]),
    "moe_mxfp4_dequantize_weights": (c_int, [c_void_p, c_void_p, c_int, c_int, c_int, c_int,
                                             c_void_p, c_void_p]),
    "moe_gather_mxfp4": (c_int, [c_void_p, c_int, c_int, c_int, c_int, c_void_p, c_void_p, c_int,
                                 c_int64, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "moe_mxfp4_dequantize_rows": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_int64, c_int,
                                          c_int, c_void_p, c_void_p, c_size_t, c_void_p]),
    "moe_expert_ffn_mxfp4_workspace_size": (c_size_t, [c_int64, c_int, c_int, c_int]),
    "moe_expert_ffn_mxfp4": (c_int, [c_void_p] * 8 + [c_int, c_int64, c_int, c_int, c_int]
                             + [c_void_p] * 5 + [c_size_t, c_void_p]),
    "moe_ep_send_plan": (c_int, [c_void_p, c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p,
                                 c_size_t, c_void_p]),
    "moe_ep_recv_plan": (c_int, [c_void_p, c_int, c_int, c_int64, c_void_p, c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "moe_forward_workspace_size": (c_size_t, [ctypes.POINTER(MoeLayerC), c_int]),
    "moe_forward_host_workspace_size": (c_size_t, [ctypes.POINTER(MoeLayerC), c_int]),
    "moe_forward": (c_int, [ctypes.POINTER(MoeLayerC), c_void_p, c_int, c_void_p, c_void_p,
                            c_void_p, c_size_t, c_void_p, c_void_p]),
    "moe_forward_views": (c_int, [ctypes.POINTER(MoeLayerC), c_int, c_void_p, c_size_t,
                                  ctypes.POINTER(MoeViewsC)]),
    "moe_forward_host": (c_int, [ctypes.POINTER(MoeLayerC), c_void_p, c_int, c_void_p, c_void_p,
                                 c_void_p, c_size_t, c_void_p]),
}

for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


def header_functions(path: str = HEADER_PATH):
    """Names of the functions include/moe_b200.h declares."""
    with open(path) as f:
        text = f.read()
    return sorted(set(re.findall(r"^MOE_API\s+[\w\s\*]*?\b(moe_\w+)\s*\(", text, flags=re.M)))


# ---------------------------------------------------------------- marshalling
def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    return t.data_ptr()


# The current stream's handle without building a torch.cuda.Stream (3 us of a
# 9 us call); the public way where this torch has no such function.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int:
    if stream is None:
        if torch.cuda.is_initialized():
            return _raw_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _on_gpu(*tensors):
    """The addresses of tensors (None: NULL). Refuses a tensor that is not on the
    current device (its kernels and streams are the current device's), or not
    contiguous; _addr checks type and size too."""
    current = None
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        d = t.get_device()
        if d != current:
            if current is None and d >= 0:
                current = _current_device()
            if d != current:
                raise ValueError(f"tensor on {t.device}, not on the current CUDA device")
        if not t.is_contiguous():
            raise ValueError(f"tensor of shape {tuple(t.shape)} and strides {t.stride()} is not contiguous")
        out.append(t.data_ptr())
    return out


_capture_info = None


def _capture_id(handle: int) -> int:
    """The capture into a graph that a stream is part of, 0 for none."""
    global _capture_info
    if _capture_info is None:
        _capture_info = ctypes.CDLL("libcuda.so.1").cuStreamGetCaptureInfo_v2
        _capture_info.argtypes = [c_void_p, ctypes.POINTER(c_int), ctypes.POINTER(ctypes.c_uint64)] + [c_void_p] * 3
    status, which = c_int(0), ctypes.c_uint64(0)
    # the error is that of the legacy stream while others capture: not part of it
    if _capture_info(handle, status, which, None, None, None) != 0 or status.value == 0:
        return 0
    return which.value


def _device_of(t: torch.Tensor) -> int:
    """The current device, which t has to be on."""
    d = t.get_device()
    if d < 0 or d != _current_device():
        _on_gpu(t)
    return d


# One call per operand, all checks in one expression, and the wrappers look up
# the dtype's code and the current stream without a call of their own: a small
# call's time is the host's (a loop over (tensor, dtype, n) took 0.4 us of 7).
def _addr(t: Optional[torch.Tensor], dtype: torch.dtype, n: int, device: int) -> Optional[int]:
    """The address of t (None: NULL), which the library takes for n values of
    dtype on this device, the current one. Refuses what it would misread or
    what is too short for it. torch.uint8 stands for any type of one byte."""
    if t is None:
        return None
    if t.get_device() == device and t.dtype is dtype and t.numel() >= n and t.is_contiguous():
        return t.data_ptr()
    address, = _on_gpu(t)
    if t.dtype is not dtype and not (dtype is torch.uint8 and t.dtype.itemsize == 1):
        raise ValueError(f"tensor of {t.dtype} where {dtype} is read or written")
    if t.numel() < n:
        raise ValueError(f"tensor of shape {tuple(t.shape)} where {n} values are read or written")
    return address


def _host_addr(t: Optional[torch.Tensor], dtype: torch.dtype, n: int) -> Optional[int]:
    """_addr for a host buffer."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{t.dtype} tensor of shape {tuple(t.shape)} and strides {t.stride()} where {n} contiguous "
                         f"values of {dtype} are read or written")
    return t.data_ptr()


def _check(fn: str, st: int):
    if st != MOE_OK:
        raise MoeError(fn, st, _lib.moe_status_string(st).decode())


class _Codes(dict):
    def __missing__(self, t):
        raise ValueError(f"unsupported dtype {t}")


_CODES = _Codes({torch.bfloat16: MOE_BF16, torch.float32: MOE_F32})
_DTYPES = {code: t for t, code in _CODES.items()}


def dtype_code(t: torch.dtype) -> int:
    return _CODES[t]


def status_string(st: int) -> str:
    return _lib.moe_status_string(st).decode()


def moe_kernel_launches() -> int:
    """Kernels the library has launched so far in this process."""
    return int(_lib.moe_kernel_launches())


def moe_capacity(cf: float, T: int, k: int, E: int) -> int:
    return _lib.moe_capacity(float(cf), T, k, E)


def moe_rows_max(T: int, k: int, E: int, capacity: int) -> int:
    return _lib.moe_rows_max(T, k, E, capacity)


def moe_rows_max_binned(T: int, k: int, E: int, capacity: int) -> int:
    return _lib.moe_rows_max_binned(T, k, E, capacity)


def moe_route_workspace_size(T, d, E) -> int:
    return _lib.moe_route_workspace_size(T, d, E)


def moe_permute_workspace_size(T, k, E) -> int:
    return _lib.moe_permute_workspace_size(T, k, E)


def moe_workspace_init(ws: torch.Tensor, stream=None):
    _check("moe_workspace_init", _lib.moe_workspace_init(_ptr(ws), ws.numel(), _stream(stream)))


def moe_workspace_set_wait_limit(ws: torch.Tensor, limit_us: int, stream=None):
    _check("moe_workspace_set_wait_limit",
           _lib.moe_workspace_set_wait_limit(_ptr(ws), ws.numel(), int(limit_us), _stream(stream)))


def moe_get_device_error(ws: torch.Tensor, stream=None, clear: bool = True) -> int:
    bits = c_uint32(0)
    st = _lib.moe_get_device_error(_ptr(ws), _stream(stream), ctypes.byref(bits), int(clear))
    if st not in (MOE_OK, 7):
        _check("moe_get_device_error", st)
    return bits.value


def moe_route(x, w_router, bias, T, d, E, k, topk_idx, topk_w, aux_loss, logits, probs, ws,
              stream=None):
    _check("moe_route", _lib.moe_route(
        _ptr(x), _ptr(w_router), _ptr(bias), dtype_code(x.dtype), T, d, E, k, _ptr(topk_idx),
        _ptr(topk_w), _ptr(aux_loss), _ptr(logits), _ptr(probs), _ptr(ws), ws.numel(),
        _stream(stream)))


def moe_route_train(x, w_router, bias, logit_noise, T, d, E, k, topk_idx, topk_w, aux_loss, z_loss,
                    logits, probs, ws, stream=None, temperature=1.0):
    _check("moe_route_train", _lib.moe_route_train(
        _ptr(x), _ptr(w_router), _ptr(bias), _ptr(logit_noise), float(temperature),
        dtype_code(x.dtype), T, d, E, k,
        _ptr(topk_idx), _ptr(topk_w), _ptr(aux_loss), _ptr(z_loss), _ptr(logits), _ptr(probs),
        _ptr(ws), ws.numel(), _stream(stream)))


def moe_route_backward_workspace_size(T, d, E) -> int:
    return _lib.moe_route_backward_workspace_size(T, d, E)


def moe_route_backward(x, w_router, T, d, E, k, probs, logits, topk_idx, topk_w, d_topk_w, d_aux, d_z,
                       temperature, d_logits, dx, d_wg, ws, stream=None, dtype=None):
    dt = dtype_code(x.dtype) if x is not None else dtype
    _check("moe_route_backward", _lib.moe_route_backward(
        _ptr(x), _ptr(w_router), dt, T, d, E, k, _ptr(probs), _ptr(logits), _ptr(topk_idx),
        _ptr(topk_w), _ptr(d_topk_w), float(d_aux), float(d_z), float(temperature), _ptr(d_logits),
        _ptr(dx), _ptr(d_wg), _ptr(ws), ws.numel(), _stream(stream)))


def moe_router_jitter(x, T, d, eps, seed, x_out, stream=None):
    _check("moe_router_jitter", _lib.moe_router_jitter(
        _ptr(x), dtype_code(x.dtype), T, d, float(eps), int(seed), _ptr(x_out), _stream(stream)))


def moe_router_noise(T, E, std, seed, noise_out, stream=None):
    _check("moe_router_noise", _lib.moe_router_noise(T, E, float(std), int(seed), _ptr(noise_out),
                                                     _stream(stream)))


def moe_permute(topk_idx, T, k, E, capacity, counts, bins, sorted_slot, slot_to_row, row_slot,
                drop_mask, kept_counts, seg_offsets, ws, stream=None):
    _check("moe_permute", _lib.moe_permute(
        _ptr(topk_idx), T, k, E, int(capacity), _ptr(counts), _ptr(bins), _ptr(sorted_slot),
        _ptr(slot_to_row), _ptr(row_slot), _ptr(drop_mask), _ptr(kept_counts), _ptr(seg_offsets),
        _ptr(ws), ws.numel(), _stream(stream)))


def moe_permute_binned(topk_idx, T, k, E, capacity, counts, bins, sorted_slot, slot_to_row,
                       row_slot, drop_mask, kept_counts, seg_offsets, ws, stream=None):
    _check("moe_permute_binned", _lib.moe_permute_binned(
        _ptr(topk_idx), T, k, E, int(capacity), _ptr(counts), _ptr(bins), _ptr(sorted_slot),
        _ptr(slot_to_row), _ptr(row_slot), _ptr(drop_mask), _ptr(kept_counts), _ptr(seg_offsets),
        _ptr(ws), ws.numel(), _stream(stream)))


def moe_permute_noalloc(topk_idx, T, k, E, capacity, counts, bins, sorted_slot, slot_to_row,
                        row_slot, drop_mask, kept_counts, seg_offsets, device_error=None,
                        stream=None):
    _check("moe_permute_noalloc", _lib.moe_permute_noalloc(
        _ptr(topk_idx), T, k, E, int(capacity), _ptr(counts), _ptr(bins), _ptr(sorted_slot),
        _ptr(slot_to_row), _ptr(row_slot), _ptr(drop_mask), _ptr(kept_counts), _ptr(seg_offsets),
        _ptr(device_error), _stream(stream)))


def moe_gather(x, T, d, k, row_slot, seg_offsets, E, rows_max, x_perm, ws, stream=None):
    _check("moe_gather", _lib.moe_gather(
        _ptr(x), dtype_code(x.dtype), T, d, k, _ptr(row_slot), _ptr(seg_offsets), E,
        int(rows_max), _ptr(x_perm), _ptr(ws), ws.numel(), _stream(stream)))


def moe_expert_ffn(x_perm, w1, w3, w2, act, rows_max, d, F, E, seg_offsets, h, y_perm, ws,
                   stream=None):
    _check("moe_expert_ffn", _lib.moe_expert_ffn(
        _ptr(x_perm), _ptr(w1), _ptr(w3), _ptr(w2), dtype_code(w1.dtype), act, int(rows_max), d,
        F, E, _ptr(seg_offsets), _ptr(h), _ptr(y_perm), _ptr(ws), ws.numel(), _stream(stream)))


def moe_combine(y_perm, topk_w, slot_to_row, T, d, k, rows_max, out, ws, stream=None):
    _check("moe_combine", _lib.moe_combine(
        _ptr(y_perm), _ptr(topk_w), _ptr(slot_to_row), dtype_code(out.dtype), T, d, k,
        int(rows_max), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))


def moe_combine_backward(d_out, y_perm, topk_w, slot_to_row, T, d, k, rows_max, d_y_perm, d_topk_w,
                         ws, stream=None):
    rows_max = int(rows_max)
    dev, dt, slots, row_values = _device_of(d_out), d_out.dtype, T * k, rows_max * d
    st = _lib.moe_combine_backward(
        _addr(d_out, dt, T * d, dev), _addr(y_perm, dt, row_values, dev), _addr(topk_w, _F32, slots, dev),
        _addr(slot_to_row, _I32, slots, dev), _CODES[dt], T, d, k, rows_max,
        _addr(d_y_perm, dt, row_values, dev), _addr(d_topk_w, _F32, slots, dev), _addr(ws, ws.dtype, 0, dev),
        ws.numel(), _raw_stream(dev) if stream is None else _stream(stream))
    if st != MOE_OK:
        _check("moe_combine_backward", st)


def moe_gather_backward(d_x_perm, slot_to_row, dx_in, T, d, k, rows_max, dx, ws, stream=None):
    rows_max = int(rows_max)
    dev, dt = _device_of(dx), dx.dtype
    st = _lib.moe_gather_backward(
        _addr(d_x_perm, dt, rows_max * d, dev), _addr(slot_to_row, _I32, T * k, dev),
        _addr(dx_in, dt, T * d, dev), _CODES[dt], T, d, k, rows_max, _addr(dx, dt, T * d, dev),
        _addr(ws, ws.dtype, 0, dev), ws.numel(), _raw_stream(dev) if stream is None else _stream(stream))
    if st != MOE_OK:
        _check("moe_gather_backward", st)


def moe_mxfp4_weight_scales_size(E: int, K: int, N: int) -> int:
    return _lib.moe_mxfp4_weight_scales_size(E, K, N)


def moe_mxfp4_row_scales_size(rows_max: int, E: int, K: int) -> int:
    return _lib.moe_mxfp4_row_scales_size(int(rows_max), E, K)


def moe_mxfp4_quantize_weights(w, E, K, N, codes, scales, stream=None):
    dev = _device_of(w)
    st = _lib.moe_mxfp4_quantize_weights(
        _addr(w, w.dtype, E * K * N, dev), _CODES[w.dtype], E, K, N, _addr(codes, _U8, E * N * K // 2, dev),
        _addr(scales, _U8, moe_mxfp4_weight_scales_size(E, K, N), dev),
        _raw_stream(dev) if stream is None else _stream(stream))
    if st != MOE_OK:
        _check("moe_mxfp4_quantize_weights", st)


def moe_mxfp4_dequantize_weights(codes, scales, E, K, N, w, stream=None):
    dev = _device_of(w)
    st = _lib.moe_mxfp4_dequantize_weights(
        _addr(codes, _U8, E * N * K // 2, dev), _addr(scales, _U8, moe_mxfp4_weight_scales_size(E, K, N), dev),
        _CODES[w.dtype], E, K, N, _addr(w, w.dtype, E * K * N, dev),
        _raw_stream(dev) if stream is None else _stream(stream))
    if st != MOE_OK:
        _check("moe_mxfp4_dequantize_weights", st)


def moe_gather_mxfp4(x, T, d, k, slot_to_row, seg_offsets, E, rows_max, codes, scales, ws,
                     stream=None):
    rows_max = int(rows_max)
    dev, dt = _device_of(x), x.dtype
    st = _lib.moe_gather_mxfp4(
        _addr(x, dt, T * d, dev), _CODES[dt], T, d, k, _addr(slot_to_row, _I32, T * k, dev),
        _addr(seg_offsets, _I32, E + 1, dev), E, rows_max, _addr(codes, _U8, rows_max * d // 2, dev),
        _addr(scales, _U8, (rows_max // 128 + E) * (d // 128) * 512, dev), _addr(ws, ws.dtype, 0, dev), ws.numel(),
        _raw_stream(dev) if stream is None else _stream(stream))
    if st != MOE_OK:
        _check("moe_gather_mxfp4", st)


def moe_mxfp4_dequantize_rows(codes, scales, seg_offsets, E, rows_max, K, out, ws, stream=None):
    rows_max = int(rows_max)
    dev, dt = _device_of(out), out.dtype
    st = _lib.moe_mxfp4_dequantize_rows(
        _addr(codes, _U8, rows_max * K // 2, dev), _addr(scales, _U8, (rows_max // 128 + E) * (K // 128) * 512, dev),
        _addr(seg_offsets, _I32, E + 1, dev), E, rows_max, K, _CODES[dt],
        _addr(out, dt, rows_max * K, dev), _addr(ws, ws.dtype, 0, dev), ws.numel(),
        _raw_stream(dev) if stream is None else _stream(stream))
    if st != MOE_OK:
        _check("moe_mxfp4_dequantize_rows", st)


def moe_expert_ffn_mxfp4_workspace_size(rows_max: int, d: int, F: int, E: int) -> int:
    return _lib.moe_expert_ffn_mxfp4_workspace_size(int(rows_max), d, F, E)


def moe_expert_ffn_mxfp4(x_codes, x_scales, w1, w1_scales, w3, w3_scales, w2, w2_scales, act,
                         rows_max, d, F, E, seg_offsets, h_codes, h_scales, y_perm, ws, stream=None):
    rows_max = int(rows_max)
    dev = _device_of(y_perm)
    matrix, matrix_scales = E * d * F // 2, moe_mxfp4_weight_scales_size(E, d, F)  # the same for [E, F, d]
    groups = rows_max // 128 + E
    if act != MOE_ACT_SWIGLU:
        w3 = w3_scales = None
    st = _lib.moe_expert_ffn_mxfp4(
        _addr(x_codes, _U8, rows_max * d // 2, dev), _addr(x_scales, _U8, groups * (d // 128) * 512, dev),
        _addr(w1, _U8, matrix, dev), _addr(w1_scales, _U8, matrix_scales, dev), _addr(w3, _U8, matrix, dev),
        _addr(w3_scales, _U8, matrix_scales, dev), _addr(w2, _U8, matrix, dev),
        _addr(w2_scales, _U8, matrix_scales, dev), act, rows_max, d, F, E, _addr(seg_offsets, _I32, E + 1, dev),
        _addr(h_codes, _U8, rows_max * F // 2, dev), _addr(h_scales, _U8, groups * (F // 128) * 512, dev),
        _addr(y_perm, torch.bfloat16, rows_max * d, dev), _addr(ws, ws.dtype, 0, dev), ws.numel(),
        _raw_stream(dev) if stream is None else _stream(stream))
    if st != MOE_OK:
        _check("moe_expert_ffn_mxfp4", st)


def moe_ep_send_plan(kept_counts, seg_offsets, E, world, send_rows, send_offsets, ws, stream=None):
    _check("moe_ep_send_plan", _lib.moe_ep_send_plan(
        _ptr(kept_counts), _ptr(seg_offsets), E, world, _ptr(send_rows), _ptr(send_offsets), _ptr(ws),
        ws.numel(), _stream(stream)))


def moe_ep_recv_plan(recv_counts, world, experts_per_rank, rows_cap, recv_rows, recv_offsets, local_seg,
                     local_to_recv, recv_to_local, ws, stream=None):
    _check("moe_ep_recv_plan", _lib.moe_ep_recv_plan(
        _ptr(recv_counts), world, experts_per_rank, int(rows_cap), _ptr(recv_rows), _ptr(recv_offsets),
        _ptr(local_seg), _ptr(local_to_recv), _ptr(recv_to_local), _ptr(ws), ws.numel(), _stream(stream)))


def layer_struct(d, E, k, F, dtype, act, cf, w_router, bias, w1, w3, w2, flags=0,
                 router_temperature=1.0, scales=(None, None, None)) -> MoeLayerC:
    """scales: those of w1, w3 and w2 (MOE_LAYER_MXFP4)."""
    return MoeLayerC(d, E, k, F, dtype, act, float(cf), _ptr(w_router), _ptr(bias), _ptr(w1),
                     _ptr(w3), _ptr(w2), int(flags), None, None, float(router_temperature),
                     *map(_ptr, scales))


def quantize_expert_weights(w: torch.Tensor, stream=None):
    """Expert weights [E, K, N] (bf16 or fp32, on the GPU) as MXFP4: codes [E, N, K / 2] and scales."""
    E, K, N = w.shape
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    # the copy and the allocations too belong to the stream that the kernel runs on
    with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
        codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device=w.device)
        scales = torch.empty(moe_mxfp4_weight_scales_size(E, K, N), dtype=torch.uint8, device=w.device)
        moe_mxfp4_quantize_weights(w.contiguous(), E, K, N, codes, scales, stream)
    return codes, scales


def moe_forward_workspace_size(layer: MoeLayerC, T: int) -> int:
    return _lib.moe_forward_workspace_size(ctypes.byref(layer), T)


def moe_forward_host_workspace_size(layer: MoeLayerC, T: int) -> int:
    return _lib.moe_forward_host_workspace_size(ctypes.byref(layer), T)


def moe_forward(layer: MoeLayerC, x, T, out, aux_loss, ws, stream=None, events=None):
    ev = None
    if events is not None:
        # torch creates a CUDA event lazily, on its first record(): record once
        # so that the handle exists (the library then re-records it in place).
        for e in events:
            if e is not None and e.cuda_event == 0:
                e.record(torch.cuda.current_stream() if stream is None else stream)
        arr = (c_void_p * 7)(*[e.cuda_event if e is not None else None for e in events])
        ev = ctypes.cast(arr, c_void_p)
    # (a dtype that is neither is the library's to refuse)
    dev, dt = _device_of(ws), _DTYPES.get(layer.dtype, x.dtype)
    st = _lib.moe_forward(
        ctypes.byref(layer), _addr(x, dt, T * layer.d, dev), T, _addr(out, dt, T * layer.d, dev),
        _addr(aux_loss, _F32, 1, dev), _addr(ws, ws.dtype, 0, dev), ws.numel(),
        _raw_stream(dev) if stream is None else _stream(stream), ev)
    if st != MOE_OK:
        _check("moe_forward", st)


def moe_forward_views(layer: MoeLayerC, T: int, ws) -> MoeViewsC:
    v = MoeViewsC()
    _check("moe_forward_views", _lib.moe_forward_views(ctypes.byref(layer), T, _ptr(ws),
                                                       ws.numel(), ctypes.byref(v)))
    return v


def moe_forward_host(layer: MoeLayerC, x_host, T, out_host, aux_host, ws, stream=None):
    dev, dt = _device_of(ws), _DTYPES.get(layer.dtype, x_host.dtype)
    st = _lib.moe_forward_host(
        ctypes.byref(layer), _host_addr(x_host, dt, T * layer.d), T, _host_addr(out_host, dt, T * layer.d),
        _host_addr(aux_host, _F32, 1), _addr(ws, ws.dtype, 0, dev), ws.numel(),
        _raw_stream(dev) if stream is None else _stream(stream))
    if st != MOE_OK:
        _check("moe_forward_host", st)
