"""Thin ctypes binding of libmoe_gb300.so (declared in include/moe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  Functions keep the C names; tensors are torch tensors (device memory)
or raw integer device addresses.  A non-OK status raises MoeError carrying the
status and the library's message.  Importing this module fails loudly when the
library has not been built -- there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_gb300.so")

MOE_OK, MOE_EINVAL, MOE_EDIMS, MOE_ESCALE, MOE_ENOMEM, MOE_ECUDA, MOE_EWORKSPACE, MOE_EDEVICE = range(8)
STATUS_NAMES = ["MOE_OK", "MOE_EINVAL", "MOE_EDIMS", "MOE_ESCALE", "MOE_ENOMEM", "MOE_ECUDA", "MOE_EWORKSPACE",
                "MOE_EDEVICE"]
MOE_W_MXFP4, MOE_W_BF16, MOE_W_INT4G32 = 0, 1, 2
MOE_ROWS_BF16, MOE_ROWS_F32, MOE_ROWS_MXFP8 = 0, 1, 2
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_GROUP_MAX, MOE_GROUP_TOP2 = 0, 1

# every symbol include/moe.h declares
EXPORTED = ("moe_load_weights", "moe_workspace_bytes", "moe_forward", "moe_forward_routed", "moe_set_expert_range",
            "moe_route_sigmoid", "moe_dense_sliced_forward", "moe_sync_status", "moe_profile_enable",
            "moe_profile_read", "moe_route_static", "moe_route_static_status", "moe_graph_create",
            "moe_graph_launch", "moe_graph_free", "moe_debug_expire_next_wait", "moe_last_error", "moe_free",
            "moe_add_rmsnorm", "moe_route_grouped", "moe_linear_load", "moe_linear_workspace_bytes",
            "moe_linear_forward", "moe_linear_sync_status", "moe_linear_free")
STAGES = ("routing", "grouping", "gate_up", "down", "combine", "layer")


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES[status] if 0 <= status < 8 else status}: {message}")
        self.status = status


class MoeConfig(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int), ("inter", ctypes.c_int), ("n_experts", ctypes.c_int),
                ("n_shared", ctypes.c_int), ("k_max", ctypes.c_int), ("n_slices", ctypes.c_int),
                ("fmt", ctypes.c_int)]


class MoeMx(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p)]


class MoeHostIO(ctypes.Structure):
    _fields_ = [("x_host", ctypes.c_void_p), ("logits_host", ctypes.c_void_p), ("ids_host", ctypes.c_void_p),
                ("w_host", ctypes.c_void_p), ("out_host", ctypes.c_void_p)]


class MoeRoutingOut(ctypes.Structure):
    _fields_ = [("topk_ids", ctypes.c_void_p), ("topk_w", ctypes.c_void_p), ("expert_offsets", ctypes.c_void_p),
                ("sorted_slot", ctypes.c_void_p), ("slot_pos", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m mxfp4_routed_expert_router_gb300.build`"
                          " (or __graft_entry__.build())")
    L = ctypes.CDLL(LIB_PATH)
    vp, ci, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.moe_load_weights.argtypes = [ctypes.POINTER(MoeConfig), ctypes.POINTER(MoeMx), ctypes.POINTER(MoeMx), vp,
                                   ctypes.POINTER(vp)]
    L.moe_load_weights.restype = ci
    L.moe_workspace_bytes.argtypes = [vp, ci, ci]
    L.moe_workspace_bytes.restype = sz
    L.moe_forward.argtypes = [vp, vp, vp, ci, ci, vp, ci, vp, sz, ctypes.POINTER(MoeRoutingOut), vp]
    L.moe_forward.restype = ci
    L.moe_forward_routed.argtypes = [vp, vp, vp, vp, ci, ci, vp, ci, vp, sz, ctypes.POINTER(MoeRoutingOut), vp]
    L.moe_forward_routed.restype = ci
    L.moe_set_expert_range.argtypes = [vp, ci, ci]
    L.moe_set_expert_range.restype = ci
    L.moe_route_sigmoid.argtypes = [vp, vp, ci, ci, ci, ctypes.c_float, vp, vp, vp]
    L.moe_route_sigmoid.restype = ci
    L.moe_graph_create.argtypes = [vp, vp, vp, vp, vp, ci, ci, vp, ci, vp, sz, ctypes.POINTER(MoeHostIO),
                                   ctypes.POINTER(vp)]
    L.moe_graph_create.restype = ci
    L.moe_graph_launch.argtypes = [vp, vp]
    L.moe_graph_launch.restype = ci
    L.moe_graph_free.argtypes = [vp]
    L.moe_graph_free.restype = None
    L.moe_dense_sliced_forward.argtypes = [vp, vp, ci, vp, ci, vp, sz, vp]
    L.moe_dense_sliced_forward.restype = ci
    L.moe_sync_status.argtypes = [vp, vp]
    L.moe_sync_status.restype = ci
    L.moe_profile_enable.argtypes = [vp, ci]
    L.moe_profile_enable.restype = ci
    L.moe_profile_read.argtypes = [vp, ctypes.POINTER(ctypes.c_float), ci]
    L.moe_profile_read.restype = ci
    L.moe_route_static.argtypes = [vp, ci, ci, ci, vp, vp, vp, vp, vp, vp]
    L.moe_route_static.restype = ci
    L.moe_route_static_status.argtypes = [vp]
    L.moe_route_static_status.restype = ci
    L.moe_debug_expire_next_wait.argtypes = [vp, ci]
    L.moe_debug_expire_next_wait.restype = ci
    ll, cf = ctypes.c_longlong, ctypes.c_float
    L.moe_add_rmsnorm.argtypes = [vp, ci, ll, vp, ci, ll, vp, ci, cf, ci, ci, vp, ll, vp, ll, vp, ll, vp, vp]
    L.moe_add_rmsnorm.restype = ci
    L.moe_route_grouped.argtypes = [vp, vp, ci, ci, ci, ci, ci, ci, ci, ci, cf, vp, vp, vp]
    L.moe_route_grouped.restype = ci
    L.moe_linear_load.argtypes = [ci, ci, ci, ctypes.POINTER(MoeMx), vp, ctypes.POINTER(vp)]
    L.moe_linear_load.restype = ci
    L.moe_linear_workspace_bytes.argtypes = [vp, ci]
    L.moe_linear_workspace_bytes.restype = sz
    L.moe_linear_forward.argtypes = [vp, vp, ci, ll, vp, ci, vp, ci, ll, ci, vp, sz, vp]
    L.moe_linear_forward.restype = ci
    L.moe_linear_sync_status.argtypes = [vp, vp]
    L.moe_linear_sync_status.restype = ci
    L.moe_linear_free.argtypes = [vp]
    L.moe_linear_free.restype = None
    L.moe_last_error.argtypes = []
    L.moe_last_error.restype = ctypes.c_char_p
    L.moe_free.argtypes = [vp]
    L.moe_free.restype = None
    return L


lib = _load()


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _current_stream() -> int:
    """torch's current stream on the current device, as a cudaStream_t (without building a torch.cuda.Stream: that
    costs as much as a launch)."""
    global _current_stream
    import torch
    try:
        raw, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        raw(device())
    except AttributeError:
        def current():
            return torch.cuda.current_stream().cuda_stream
    else:
        def current():
            return raw(device())
    _current_stream = current
    return current()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int):
    if status != MOE_OK:
        raise MoeError(status, moe_last_error())


def moe_last_error() -> str:
    return lib.moe_last_error().decode()


def moe_load_weights(cfg: MoeConfig, gate_up: Sequence[Tuple], down: Sequence[Tuple], stream=None) -> int:
    """Copy weights into the library; gate_up / down are sequences of
    (codes, scales_or_None) or, for INT4G32, (codes, scales, zeros_or_None)."""
    def mx(m):
        return MoeMx(_ptr(m[0]), _ptr(m[1]), _ptr(m[2]) if len(m) > 2 else None)

    gu = (MoeMx * max(1, len(gate_up)))(*[mx(m) for m in gate_up])
    dn = (MoeMx * max(1, len(down)))(*[mx(m) for m in down])
    h = ctypes.c_void_p()
    _check(lib.moe_load_weights(ctypes.byref(cfg), gu, dn, _stream(stream), ctypes.byref(h)))
    return h.value


def moe_workspace_bytes(handle: int, T: int, k: int) -> int:
    return int(lib.moe_workspace_bytes(handle, T, k))


def moe_forward(handle: int, x_bf16, router_logits, T: int, k: int, out_fp32, accumulate: bool, workspace,
                ws_bytes: int, routing: Optional[MoeRoutingOut] = None, stream=None) -> None:
    _check(lib.moe_forward(handle, _ptr(x_bf16), _ptr(router_logits), T, k, _ptr(out_fp32), int(bool(accumulate)),
                           _ptr(workspace), ws_bytes, ctypes.byref(routing) if routing is not None else None,
                           _stream(stream)))


def moe_forward_routed(handle: int, x_bf16, topk_ids, topk_w, T: int, k: int, out_fp32, accumulate: bool, workspace,
                       ws_bytes: int, routing: Optional[MoeRoutingOut] = None, stream=None) -> None:
    _check(lib.moe_forward_routed(handle, _ptr(x_bf16), _ptr(topk_ids), _ptr(topk_w), T, k, _ptr(out_fp32),
                                  int(bool(accumulate)), _ptr(workspace), ws_bytes,
                                  ctypes.byref(routing) if routing is not None else None, _stream(stream)))


def moe_set_expert_range(handle: int, expert_base: int, n_experts_total: int) -> None:
    _check(lib.moe_set_expert_range(handle, int(expert_base), int(n_experts_total)))


def moe_route_sigmoid(router_logits, bias, T: int, E: int, k: int, routed_scale: float, topk_ids, topk_w,
                      stream=None) -> None:
    _check(lib.moe_route_sigmoid(_ptr(router_logits), _ptr(bias), T, E, k, float(routed_scale), _ptr(topk_ids),
                                 _ptr(topk_w), _stream(stream)))


def moe_graph_create(handle: int, x_bf16, router_logits, topk_ids, topk_w, T: int, k: int, out_fp32,
                     accumulate: bool, workspace, ws_bytes: int, x_host=None, logits_host=None, ids_host=None,
                     w_host=None, out_host=None) -> int:
    """Capture one forward call into a CUDA graph; the *_host buffers (pinned host memory, optional) add the
    step's input and output copies to the graph."""
    io = MoeHostIO(_ptr(x_host), _ptr(logits_host), _ptr(ids_host), _ptr(w_host), _ptr(out_host))
    any_io = any(v is not None for v in (x_host, logits_host, ids_host, w_host, out_host))
    g = ctypes.c_void_p()
    _check(lib.moe_graph_create(handle, _ptr(x_bf16), _ptr(router_logits), _ptr(topk_ids), _ptr(topk_w), T, k,
                                _ptr(out_fp32), int(bool(accumulate)), _ptr(workspace), ws_bytes,
                                ctypes.byref(io) if any_io else None, ctypes.byref(g)))
    return g.value


def moe_graph_launch(graph: int, stream=None) -> None:
    _check(lib.moe_graph_launch(graph, _stream(stream)))


def moe_graph_free(graph: int) -> None:
    lib.moe_graph_free(graph)


def moe_dense_sliced_forward(handle: int, x_bf16, T: int, out_fp32, accumulate: bool, workspace, ws_bytes: int,
                             stream=None) -> None:
    _check(lib.moe_dense_sliced_forward(handle, _ptr(x_bf16), T, _ptr(out_fp32), int(bool(accumulate)),
                                        _ptr(workspace), ws_bytes, _stream(stream)))


def moe_sync_status(handle: int, stream=None) -> None:
    _check(lib.moe_sync_status(handle, _stream(stream)))


def moe_profile_enable(handle: int, enable: bool = True) -> None:
    _check(lib.moe_profile_enable(handle, int(bool(enable))))


def moe_profile_read(handle: int) -> dict:
    """Stage durations (ms) of the most recent profiled forward call."""
    buf = (ctypes.c_float * len(STAGES))()
    n = lib.moe_profile_read(handle, buf, len(STAGES))
    if n < 0:
        raise MoeError(MOE_EINVAL, "no profiled call")
    return {STAGES[i]: float(buf[i]) for i in range(n)}


def moe_route_static(router_logits, T: int, E: int, k: int, topk_ids, topk_w, expert_offsets, sorted_slot,
                     slot_pos, stream=None) -> None:
    """Routing and grouping with the library's fixed scratch; allocates nothing (see include/moe.h)."""
    _check(lib.moe_route_static(_ptr(router_logits), T, E, k, _ptr(topk_ids), _ptr(topk_w), _ptr(expert_offsets),
                                _ptr(sorted_slot), _ptr(slot_pos), _stream(stream)))


def moe_route_static_status(stream=None) -> None:
    """Raise MoeError(MOE_EDEVICE) if the most recent moe_route_static call on this device flagged a device error."""
    _check(lib.moe_route_static_status(_stream(stream)))


def moe_debug_expire_next_wait(handle: int, limit_us: int) -> None:
    """Test hook: the next single-kernel launch on this handle lets its completion wait expire (include/moe.h)."""
    _check(lib.moe_debug_expire_next_wait(handle, int(limit_us)))


def moe_free(handle: int) -> None:
    lib.moe_free(handle)


_ROW_TYPES = {}


def _row_type(dtype) -> int:
    """The row type of a torch dtype, -1 for one that has none."""
    if not _ROW_TYPES:
        import torch
        _ROW_TYPES.update({torch.bfloat16: MOE_ROWS_BF16, torch.float32: MOE_ROWS_F32,
                           torch.float8_e4m3fn: MOE_ROWS_MXFP8})
    return _ROW_TYPES.get(dtype, -1)


def _rows(t, name: str, shape):
    """Address, row type and row stride (elements) of a tensor of rows of that shape, (None, 0, 0) for None."""
    if t is None:
        return None, 0, 0
    if t.shape != shape:
        raise MoeError(MOE_EINVAL, f"{name}: shape {tuple(t.shape)} where {tuple(shape)} is needed")
    ty = _ROW_TYPES.get(t.dtype, -1)
    if ty < 0 and (ty := _row_type(t.dtype)) < 0:
        raise MoeError(MOE_EINVAL, f"{name}: rows are bfloat16, float32 or float8_e4m3fn, not {t.dtype}")
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise MoeError(MOE_EINVAL, f"{name}: the values of a row must lie side by side")
    return t.data_ptr(), ty, (ld if shape[0] > 1 else shape[1])


def moe_add_rmsnorm(residual, delta, gain, eps: float, sum=None, y=None, q=None, q_scales=None, stream=None) -> None:
    """s = residual + delta, the RMS norm of s times gain as BF16 rows (y) and MXFP8 rows (q, q_scales); see
    include/moe.h.  residual, delta and sum are bfloat16 or float32 [T, H] tensors, y bfloat16, q float8_e4m3fn,
    q_scales uint8 [T, H/32]; delta, gain and any output may be None, and sum may be residual itself."""
    shape = residual.shape
    if len(shape) != 2:
        raise MoeError(MOE_EINVAL, "residual: a [T, H] tensor is needed")
    T, H = shape
    r, rt, rld = _rows(residual, "residual", shape)
    d, dt, dld = _rows(delta, "delta", shape)
    s, sty, sld = _rows(sum, "sum", shape)
    yp, yt, yld = _rows(y, "y", shape)
    qp, qt, qld = _rows(q, "q", shape)
    if sty != rt and s is not None:
        raise MoeError(MOE_EINVAL, "sum: the residual's type is needed")
    if yt != MOE_ROWS_BF16 or (qt != MOE_ROWS_MXFP8 and qp is not None):
        raise MoeError(MOE_EINVAL, "y is bfloat16 and q float8_e4m3fn")
    g = gt = 0
    if gain is not None:
        if gain.shape != (H,) or not gain.is_contiguous():
            raise MoeError(MOE_EINVAL, f"gain: a dense vector of {H} values is needed")
        g, gt = gain.data_ptr(), _row_type(gain.dtype)
    qs = None
    if q_scales is not None:
        if q_scales.shape != (T, H // 32) or not q_scales.is_contiguous() or q_scales.element_size() != 1:
            raise MoeError(MOE_EINVAL, f"q_scales: a dense uint8 [{T}, {H // 32}] tensor is needed")
        qs = q_scales.data_ptr()
    status = lib.moe_add_rmsnorm(r, rt, rld, d, dt, dld, g, gt, eps, T, H, s, sld, yp, yld, qp, qld, qs,
                                 _stream(stream))
    if status:
        _check(status)


_DTYPES = []  # torch.float32, torch.int32: filled by the first call that needs them


def _dtypes():
    if not _DTYPES:
        import torch
        _DTYPES.extend((torch.float32, torch.int32))
    return _DTYPES


def _dense(t, name: str, dtype, rows: int, cols: int):
    """Address of a dense tensor of `rows` rows (or more, or flat) of `cols` values; None and plain addresses pass."""
    if t is None or isinstance(t, int):
        return t
    if t.dtype is not dtype or not t.is_contiguous() or t.numel() < rows * cols or (
            t.dim() > 1 and t.size(-1) != cols):
        raise MoeError(MOE_EINVAL, f"{name}: a dense {dtype} tensor [{rows}, {cols}] is needed, not {t.dtype} "
                                   f"{tuple(t.shape)}")
    return t.data_ptr()


def moe_route_grouped(router_logits, bias, T: int, E: int, k: int, n_groups: int, k_groups: int, score: int,
                      group_score: int, renormalize: bool, scale: float, topk_ids, topk_w, stream=None) -> None:
    """Group-limited routing (see include/moe.h); the outputs feed moe_forward_routed.  router_logits float32 [T, E],
    bias float32 [E] or None, topk_ids int32 and topk_w float32 [T, k], all dense; longer buffers may be given."""
    f32, i32 = _DTYPES or _dtypes()
    status = lib.moe_route_grouped(_dense(router_logits, "router_logits", f32, T, E), _dense(bias, "bias", f32, 1, E),
                                   T, E, k, n_groups, k_groups, score, group_score, bool(renormalize), scale,
                                   _dense(topk_ids, "topk_ids", i32, T, k), _dense(topk_w, "topk_w", f32, T, k),
                                   _stream(stream))
    if status:
        _check(status)


def moe_linear_load(N: int, K: int, fmt: int, codes, scales=None, zeros=None, stream=None) -> int:
    """Copy a [N, K] weight (formats and layouts of moe_load_weights) into the library; returns its handle."""
    h = ctypes.c_void_p()
    _check(lib.moe_linear_load(N, K, fmt, ctypes.byref(MoeMx(_ptr(codes), _ptr(scales), _ptr(zeros))),
                               _stream(stream), ctypes.byref(h)))
    return h.value


def moe_linear_workspace_bytes(handle: int, T: int) -> int:
    return int(lib.moe_linear_workspace_bytes(handle, T))


def moe_linear_forward(handle: int, x, x_scales, y, accumulate: bool = False, workspace=None, ws_bytes: int = 0,
                       stream=None) -> None:
    """y = x W^T (see include/moe.h): x is bfloat16 [T, K], or float8_e4m3fn [T, K] with x_scales uint8 [T, K/32];
    y is float32 or bfloat16 [T, N]."""
    if x.dim() != 2 or y.dim() != 2 or x.shape[0] != y.shape[0]:
        raise MoeError(MOE_EINVAL, f"x {tuple(x.shape)} and y {tuple(y.shape)}: [T, K] and [T, N] are needed")
    xp, xt, xld = _rows(x, "x", x.shape)
    yp, yt, yld = _rows(y, "y", y.shape)
    if x_scales is not None and not isinstance(x_scales, int) and (
            x_scales.shape != (x.shape[0], x.shape[1] // 32) or x_scales.element_size() != 1 or
            not x_scales.is_contiguous()):
        raise MoeError(MOE_EINVAL, f"x_scales: dense bytes [{x.shape[0]}, {x.shape[1] // 32}] are needed, not "
                                   f"{x_scales.dtype} {tuple(x_scales.shape)}")
    status = lib.moe_linear_forward(handle, xp, xt, xld, _ptr(x_scales), x.shape[0], yp, yt, yld, bool(accumulate),
                                    _ptr(workspace), ws_bytes, _stream(stream))
    if status:
        _check(status)


def moe_linear_sync_status(handle: int, stream=None) -> None:
    _check(lib.moe_linear_sync_status(handle, _stream(stream)))


def moe_linear_free(handle: int) -> None:
    lib.moe_linear_free(handle)


def routing_out(topk_ids=None, topk_w=None, expert_offsets=None, sorted_slot=None, slot_pos=None) -> MoeRoutingOut:
    return MoeRoutingOut(_ptr(topk_ids), _ptr(topk_w), _ptr(expert_offsets), _ptr(sorted_slot), _ptr(slot_pos))
