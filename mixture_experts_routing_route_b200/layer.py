"""MoeLayer: a user-facing handle around the C ABI's whole-layer forward.

Holds the layer's device weights and a workspace (device memory allocated by
torch: plumbing only), fills the C layer struct, and calls moe_forward /
moe_forward_host. Intermediates of the last forward can be read as torch views
of the workspace.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _abi as abi


class MoeLayer:
    def __init__(self, w_router: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor,
                 w3: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                 k: int = 2, act: str = "swiglu", capacity_factor: float = 0.0,
                 gather_in_gemm: bool = False, binned: bool = False, z_loss: bool = False,
                 combine_in_gemm: bool = False, router_temperature: float = 1.0,
                 mxfp4: bool = False):
        if not w1.is_cuda:
            raise ValueError("weights must be CUDA tensors")
        self.E, self.d, self.F = w1.shape
        shapes = {"w_router": (w_router, (self.d, self.E)), "w2": (w2, (self.E, self.F, self.d))}
        if w3 is not None and act == "swiglu":
            shapes["w3"] = w3, (self.E, self.d, self.F)
        for name, (w, shape) in shapes.items():
            if tuple(w.shape) != shape:
                raise ValueError(f"{name} of shape {tuple(w.shape)}, not {shape} as w1 has it")
            if w.device != w1.device:
                raise ValueError(f"{name} on {w.device}, w1 on {w1.device}")
            if not mxfp4 and w.dtype != w1.dtype:
                raise ValueError(f"{name} is {w.dtype}, w1 {w1.dtype}")
        self.k = k
        self.dtype = w1.dtype
        self.act = abi.MOE_ACT_SWIGLU if act == "swiglu" else abi.MOE_ACT_GELU
        self.cf = float(capacity_factor)
        self.w_router = w_router.contiguous()
        self.bias = None if bias is None else bias.to(device=w1.device, dtype=torch.float32).contiguous()
        # mxfp4: the experts in microscaled 4-bit floating point
        # (MOE_LAYER_MXFP4); the weights given (bf16 or fp32) are quantised here
        # and only their codes and scales are kept. x and out are bf16.
        self.mxfp4 = mxfp4
        if mxfp4:
            if w_router.dtype != torch.bfloat16:
                raise ValueError("w_router must be bf16 with mxfp4 experts")
            self.dtype = torch.bfloat16
            self.w1, s1 = abi.quantize_expert_weights(w1)
            self.w3, s3 = (None, None) if w3 is None else abi.quantize_expert_weights(w3)
            self.w2, s2 = abi.quantize_expert_weights(w2)
            self.scales = (s1, s3, s2)
            # forward may be called on any stream: all of the layer's tensors
            # are complete from here on
            torch.cuda.current_stream().synchronize()
        else:
            self.w1 = w1.contiguous()
            self.w3 = None if w3 is None else w3.contiguous()
            self.w2 = w2.contiguous()
            self.scales = (None, None, None)
        # gather_in_gemm: the up projection gathers x rows itself (bf16; see
        # MOE_LAYER_GATHER_IN_GEMM in include/moe_b200.h)
        # binned: the [E, C, hs] bucket layout (MOE_LAYER_BINNED); with
        # capacity_factor <= 0 the bin size is the call's largest expert count
        # combine_in_gemm: k = 1, bf16: the down projection scales its rows by
        # the top-k weight and writes out (MOE_LAYER_COMBINE_IN_GEMM)
        flags = (abi.MOE_LAYER_GATHER_IN_GEMM if gather_in_gemm else 0) | \
            (abi.MOE_LAYER_BINNED if binned else 0) | (abi.MOE_LAYER_Z_LOSS if z_loss else 0) | \
            (abi.MOE_LAYER_COMBINE_IN_GEMM if combine_in_gemm else 0) | \
            (abi.MOE_LAYER_MXFP4 if mxfp4 else 0)
        # router_temperature: the router softmax sees logits / tau (training
        # variant; moe_route_train in include/moe_b200.h)
        self.c = abi.layer_struct(self.d, self.E, k, self.F, abi.dtype_code(self.dtype), self.act,
                                  self.cf, self.w_router, self.bias, self.w1, self.w3, self.w2,
                                  flags, router_temperature, self.scales)
        # (T, host_io, slot, stream handle), whether captured into a graph: the capture's id, workspace
        self._ws = {}
        self._last = {}  # (T, host_io, slot): the last call's

    def workspace(self, T: int, host_io: bool = False, stream=None, slot: int = 0) -> torch.Tensor:
        """The device workspace of the last call with T tokens and this slot,
        or (stream given) the one that calls on `stream` use. Calls on two
        streams may run at the same time, so every stream has its own, and
        calls that are captured into a graph have one in the graph's memory,
        which every replay initialises (there is nothing to read in it before
        the first); `slot` keeps more of them apart."""
        if stream is None and (T, host_io, slot) in self._last:
            return self._last[T, host_io, slot]
        return self._workspace(T, host_io, stream, slot)

    def _workspace(self, T: int, host_io: bool, stream, slot: int) -> torch.Tensor:
        handle = abi._stream(stream)
        key = T, host_io, slot, handle
        if stream is not None or torch.cuda.is_current_stream_capturing():
            capture = abi._capture_id(handle)
        else:
            capture = 0
        made_in, ws = self._ws.get((key, capture != 0), (0, None))
        if ws is None or made_in != capture:
            n = (abi.moe_forward_host_workspace_size(self.c, T) if host_io
                 else abi.moe_forward_workspace_size(self.c, T))
            if stream is not None and not isinstance(stream, torch.Stream):
                stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
            # allocated and initialised on the stream that uses it
            with torch.cuda.stream(stream):
                ws = torch.empty(max(n, 256), dtype=torch.uint8, device=self.w1.device)
                abi.moe_workspace_init(ws)
            self._ws[key, capture != 0] = capture, ws
        return ws

    def _tokens(self, x: torch.Tensor) -> int:
        T = x.shape[0]
        if x.numel() != T * self.d:
            raise ValueError(f"x of shape {tuple(x.shape)}, not [T, {self.d}]")
        return T

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None,
                aux: Optional[torch.Tensor] = None, stream=None, events=None,
                x_router: Optional[torch.Tensor] = None,
                logit_noise: Optional[torch.Tensor] = None):
        """x_router: the router's own input (e.g. moe_router_jitter of x);
        logit_noise: [T, E] fp32 added to the gate logits (training variants).
        x, x_router and out have the layer's dtype, aux is fp32; tensors of
        another type, shorter or strided raise ValueError. Threads that call
        one layer at the same time call it on different streams."""
        T = self._tokens(x)
        c = self.c
        if x_router is not None or logit_noise is not None:
            # a struct of this call's: another thread's may read the layer's
            c, dev = abi.MoeLayerC.from_buffer_copy(c), abi._device_of(x)
            c.x_router = abi._addr(x_router, self.dtype, T * self.d, dev)
            c.logit_noise = abi._addr(logit_noise, torch.float32, T * self.E, dev)
        if out is None:
            out = torch.empty(T, self.d, dtype=self.dtype, device=x.device)
        if aux is None:
            aux = torch.empty(1, dtype=torch.float32, device=x.device)
        ws = self._last[T, False, 0] = self._workspace(T, False, stream, 0)
        abi.moe_forward(c, x, T, out, aux, ws, stream, events)
        return out, aux

    __call__ = forward

    def forward_host(self, x_host: torch.Tensor, out_host: torch.Tensor, aux_host: torch.Tensor,
                     stream=None, slot: int = 0):
        """Pinned host x in, pinned host out and aux back, all asynchronous on
        `stream`. Calls with different `slot`s use different workspaces on one
        stream too (double-buffered serving)."""
        T = self._tokens(x_host)
        ws = self._last[T, True, slot] = self._workspace(T, True, stream, slot)
        abi.moe_forward_host(self.c, x_host, T, out_host, aux_host, ws, stream)

    def device_error(self, T: int, stream=None) -> int:
        return abi.moe_get_device_error(self.workspace(T, stream=stream), stream)

    def views(self, T: int, stream=None) -> dict:
        """Torch views of the intermediates that the last forward of T tokens
        (on `stream`, if given) left in its workspace."""
        ws = self.workspace(T, stream=stream)
        v = abi.moe_forward_views(self.c, T, ws)
        base = ws.data_ptr()
        R = v.rows_max
        S = T * self.k

        def view(ptr, n, dt, shape):
            es = torch.empty(0, dtype=dt).element_size()
            off = ptr - base
            return ws[off:off + n * es].view(dt).view(*shape)

        def scales(ptr, K):
            n = abi.moe_mxfp4_row_scales_size(R, self.E, K)
            return view(ptr, n, torch.uint8, (n,)) if self.mxfp4 else None

        return {
            "topk_idx": view(v.topk_idx, S, torch.int32, (T, self.k)),
            "topk_w": view(v.topk_w, S, torch.float32, (T, self.k)),
            "aux": view(v.aux_loss, 1, torch.float32, (1,)),
            "z_loss": view(v.z_loss, 1, torch.float32, (1,)),
            "counts": view(v.counts, self.E, torch.int32, (self.E,)),
            "bins": view(v.bins, self.E, torch.int32, (self.E,)),
            "kept_counts": view(v.kept_counts, self.E, torch.int32, (self.E,)),
            "seg_offsets": view(v.seg_offsets, self.E + 1, torch.int32, (self.E + 1,)),
            "sorted_slot": view(v.sorted_slot, S, torch.int32, (S,)),
            "slot_to_row": view(v.slot_to_row, S, torch.int32, (S,)),
            "row_slot": view(v.row_slot, R, torch.int32, (R,)),
            "drop": view(v.drop_mask, S, torch.uint8, (S,)),
            # no x_perm when the up projection gathers x rows itself
            # (mxfp4: x_perm and h are the rows' codes, two to a byte)
            "x_perm": (view(v.x_perm, R * self.d // 2, torch.uint8, (R, self.d // 2)) if self.mxfp4 else
                       view(v.x_perm, R * self.d, self.dtype, (R, self.d)) if v.x_perm else None),
            "h": (view(v.h, R * self.F // 2, torch.uint8, (R, self.F // 2)) if self.mxfp4 else
                  view(v.h, R * self.F, self.dtype, (R, self.F))),
            "x_perm_scales": scales(v.x_perm_scales, self.d),
            "h_scales": scales(v.h_scales, self.F),
            # no y_perm when the down projection writes the output itself
            "y_perm": view(v.y_perm, R * self.d, self.dtype, (R, self.d)) if v.y_perm else None,
            "rows_max": R,
            "capacity": v.capacity,
        }
