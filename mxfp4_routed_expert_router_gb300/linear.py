"""A linear layer with 4-bit or BF16 weights held by the library.

torch is used only for device memory and streams; the products run in
libmoe_gb300.so through ``binding``.
"""
from __future__ import annotations

import threading
from typing import Optional

import torch

from . import binding as B

FORMATS = {"mxfp4": B.MOE_W_MXFP4, "bf16": B.MOE_W_BF16, "int4g32": B.MOE_W_INT4G32}

KEPT_WORKSPACE = 32 << 20  # largest workspace that stays with its stream


class _Workspaces(threading.local):
    """(device, stream) -> bytes that the calls on that stream share; a thread has its own, as a call's launches may
    lie between those of another thread's."""

    def __init__(self):
        self.of = {}


_workspaces = _Workspaces()


def stream_workspace(n: int, device: torch.device) -> torch.Tensor:
    """At least n bytes for a call on torch's current stream.  Up to KEPT_WORKSPACE they stay with the stream for its
    next call, which comes after this one there (an allocation between two launches costs as much as a launch).  A
    captured call gets bytes of its graph's own, as a replay may run on another stream."""
    if n > KEPT_WORKSPACE or torch.cuda.is_current_stream_capturing():
        return torch.empty(n, dtype=torch.uint8, device=device)
    key = (device.index, B._current_stream())
    ws = _workspaces.of.get(key)
    if ws is None or ws.numel() < n:
        ws = _workspaces.of[key] = torch.empty(n, dtype=torch.uint8, device=device)
    return ws


class QuantLinear:
    """y = x W^T for a weight W [N, K] in one of the library's formats.

    * "mxfp4": codes uint8 [N, K/2], scales uint8 (E8M0) [N, K/32]
    * "int4g32": codes uint8 [N, K/2], scales float16 [N, K/32], zeros uint8 [N, K/32] or None (all 8)
    * "bf16": codes bfloat16 [N, K]

    The library keeps its own copy: the tensors given here may be freed.
    """

    def __init__(self, fmt: str, codes: torch.Tensor, scales: Optional[torch.Tensor] = None,
                 zeros: Optional[torch.Tensor] = None, stream=None):
        self.handle = None
        if fmt not in FORMATS:
            raise B.MoeError(B.MOE_EINVAL, f"unknown weight format {fmt!r}")
        if codes.dim() != 2:
            raise B.MoeError(B.MOE_EINVAL, "codes: a [N, K] or [N, K/2] matrix is needed")
        self.fmt = fmt
        self.N, self.K = codes.shape[0], codes.shape[1] * (1 if fmt == "bf16" else 2)
        want = {"mxfp4": (torch.uint8, torch.uint8), "int4g32": (torch.uint8, torch.float16),
                "bf16": (torch.bfloat16, None)}[fmt]
        self._dense("codes", codes, want[0], codes.shape)
        if want[1] is not None:
            if scales is None:
                raise B.MoeError(B.MOE_EINVAL, f"{fmt} weights have scales")
            self._dense("scales", scales, want[1], (self.N, self.K // 32))
        if fmt == "int4g32" and zeros is not None:
            self._dense("zeros", zeros, torch.uint8, (self.N, self.K // 32))
        self.device = codes.device
        self.handle = B.moe_linear_load(self.N, self.K, FORMATS[fmt], codes, scales, zeros, stream)
        self._no_ws = 0  # the largest T that needs no workspace
        while B.moe_linear_workspace_bytes(self.handle, self._no_ws + 1) == 0 and self._no_ws < 64:
            self._no_ws += 1

    @staticmethod
    def _dense(name, t, dtype, shape):
        if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise B.MoeError(B.MOE_EINVAL, f"{name}: a dense {dtype} tensor of shape {tuple(shape)} is needed, "
                                           f"not {t.dtype} {tuple(t.shape)}")

    def forward(self, x: torch.Tensor, x_scales: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                accumulate: bool = False, stream=None) -> torch.Tensor:
        """x: bfloat16 [T, K], or float8_e4m3fn [T, K] with x_scales uint8 [T, K/32] (MXFP8 rows).
        out: float32 (the default) or bfloat16 [T, N]; accumulate adds to a float32 out."""
        if x.dim() != 2 or x.shape[1] != self.K:
            raise B.MoeError(B.MOE_EINVAL, f"x: shape {tuple(x.shape)} where [T, {self.K}] is needed")
        T = x.shape[0]
        if out is None:
            if accumulate:
                raise B.MoeError(B.MOE_EINVAL, "accumulate needs an out to add to")
        elif tuple(out.shape) != (T, self.N):
            raise B.MoeError(B.MOE_EINVAL, f"out: shape {tuple(out.shape)} where ({T}, {self.N}) is needed")
        n = 0
        if T > self._no_ws and not (self.fmt == "bf16" and x.dtype == torch.bfloat16):  # (these rows go in as they are)
            n = B.moe_linear_workspace_bytes(self.handle, T)
        ws = None
        if n or out is None:
            # On the call's own stream: calls on several streams, and captured calls, then stay apart.
            if stream is None:
                out, ws = self._allocate(T, n, out)
            else:
                on = torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream
                with torch.cuda.stream(on):
                    out, ws = self._allocate(T, n, out)
        B.moe_linear_forward(self.handle, x, x_scales, out, accumulate, ws, n, stream)
        return out

    def _allocate(self, T: int, n: int, out):
        if out is None:
            out = torch.empty((T, self.N), dtype=torch.float32, device=self.device)
        return out, stream_workspace(n, self.device) if n else None

    def sync(self, stream=None):
        B.moe_linear_sync_status(self.handle, stream)

    def free(self):
        if self.handle:
            B.moe_linear_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass
