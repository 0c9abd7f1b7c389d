"""Python binding of the B200 routed MoE FFN forward library (``libmoe_b200.so``).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels, enqueued on the current torch CUDA stream.  torch provides device
memory (outputs, workspace) and streams.  There is no CPU fallback: if the
library is missing or no CUDA device is present, calls raise.

The entry points mirror the C ABI in ``include/moe_b200.h``:
``moe_route``, ``moe_route_from_logits``, ``moe_permute``, ``moe_expert_ffn``,
``moe_combine``, ``moe_forward``, ``moe_quantize_int4``, the 8-bit integer experts (``moe_quantize_int8``,
``moe_permute_int8``, ``moe_expert_ffn_int8``), the gradients of the grouping and of the combine
(``moe_permute_backward``, ``moe_combine_backward``), plus ``moe_workspace_size``, ``moe_capacity``,
``moe_get_status``.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_b200.so")

ACT_SWIGLU, ACT_GEGLU = 0, 1
WFMT_BF16, WFMT_INT4_G128, WFMT_INT8 = 0, 1, 2
DTYPE_CODE = {torch.bfloat16: 0, torch.float32: 1}
FLAG_SINGLE_CTA_GEMM = 1
STATUS = {0: "MOE_OK", 1: "MOE_INVALID_ARGUMENT", 2: "MOE_UNSUPPORTED_SHAPE", 3: "MOE_WORKSPACE_TOO_SMALL",
          4: "MOE_CUDA_ERROR", 5: "MOE_DEVICE_TIMEOUT"}

EXPORTED = ["moe_grouped_rows", "moe_capacity", "moe_workspace_size", "moe_route", "moe_route_from_logits",
            "moe_permute", "moe_expert_ffn", "moe_combine", "moe_forward", "moe_quantize_int4", "moe_get_status",
            "moe_set_wait_limit_ns", "moe_selftest_wait_timeout", "moe_launch_count", "moe_status_string",
            "moe_permute_noalloc", "moe_transpose_experts", "moe_backward_workspace_size", "moe_backward_x",
            "moe_backward", "moe_route_tree_workspace_size", "moe_route_tree", "moe_quantize_int8",
            "moe_permute_int8", "moe_expert_ffn_int8_workspace_size", "moe_expert_ffn_int8", "moe_combine_backward",
            "moe_permute_backward"]


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {STATUS.get(code, code)}")
        self.code = code


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("H", ctypes.c_int32), ("H_s", ctypes.c_int32), ("capacity", ctypes.c_int32),
                ("act", ctypes.c_int32), ("wfmt", ctypes.c_int32), ("renorm", ctypes.c_int32),
                ("flags", ctypes.c_int32)]

    def __init__(self, T, d, E, k, H, H_s=0, capacity=0, act=ACT_SWIGLU, wfmt=WFMT_BF16, renorm=1, flags=0):
        super().__init__(T, d, E, k, H, H_s, capacity, act, wfmt, renorm, flags)

    @property
    def R(self) -> int:
        return self.E * self.capacity if self.capacity > 0 else self.T * self.k

    def __repr__(self):
        return "MoeShape(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


_lib = None
_P = ctypes.c_void_p


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library (built by ``__graft_entry__.build()``); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} is missing (run __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    S = ctypes.POINTER(MoeShape)
    i32, i64, u64, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t
    sig = {
        "moe_grouped_rows": (i64, [S]),
        "moe_capacity": (ctypes.c_int, [i64, i32, i32, ctypes.c_double, ctypes.POINTER(i32)]),
        "moe_workspace_size": (ctypes.c_int, [S, ctypes.POINTER(sz)]),
        "moe_route": (ctypes.c_int, [S, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, sz, _P]),
        "moe_route_from_logits": (ctypes.c_int, [S, _P, _P, _P, _P, _P, _P, _P, _P, sz, _P]),
        "moe_permute": (ctypes.c_int, [S, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, sz, _P]),
        "moe_expert_ffn": (ctypes.c_int, [S, i32, i32, i64, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
        "moe_combine": (ctypes.c_int, [S, _P, _P, _P, _P, _P, _P]),
        "moe_forward": (ctypes.c_int, [S] + [_P] * 20 + [sz, _P, _P]),
        "moe_quantize_int4": (ctypes.c_int, [_P, i64, i32, _P, _P, _P]),
        "moe_get_status": (ctypes.c_int, [_P, ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_uint32)]),
        "moe_set_wait_limit_ns": (ctypes.c_int, [u64]),
        "moe_selftest_wait_timeout": (ctypes.c_int, [_P]),
        "moe_launch_count": (u64, []),
        "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "moe_permute_noalloc": (ctypes.c_int, [S, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
        "moe_transpose_experts": (ctypes.c_int, [_P, i64, i32, i32, _P, _P]),
        "moe_backward_workspace_size": (ctypes.c_int, [S, ctypes.POINTER(sz)]),
        "moe_backward_x": (ctypes.c_int, [S] + [_P] * 10 + [ctypes.c_float, _P, _P, sz, _P]),
        "moe_backward": (ctypes.c_int, [S] + [_P] * 10 + [ctypes.c_float] + [_P] * 7 + [sz, _P, _P]),
        "moe_route_tree_workspace_size": (ctypes.c_int, [S, i32, i32, ctypes.POINTER(sz)]),
        "moe_route_tree": (ctypes.c_int, [S, i32, i32] + [_P] * 8 + [sz, _P]),
        "moe_quantize_int8": (ctypes.c_int, [_P, i32, i64, i32, _P, _P, _P]),
        "moe_permute_int8": (ctypes.c_int, [S] + [_P] * 11 + [sz, _P]),
        "moe_expert_ffn_int8_workspace_size": (ctypes.c_int, [S, i32, i64, ctypes.POINTER(sz)]),
        "moe_expert_ffn_int8": (ctypes.c_int, [S, i32, i32, i64] + [_P] * 10 + [sz, _P]),
        "moe_combine_backward": (ctypes.c_int, [S] + [_P] * 8),
        "moe_permute_backward": (ctypes.c_int, [S, _P, i32, _P, _P, _P, i32, _P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _L():
    return _lib if _lib is not None else load()


def _check(code: int, where: str):
    if code != 0:
        raise MoeError(code, where)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return t.data_ptr()


# The current stream's handle without a Stream object around it (0.1 us a call instead of 3.2), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# torch.cuda.current_device and is_current_stream_capturing without their checks that CUDA is up (0.3 us a call).
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(_device())
    return torch.cuda.current_stream().cuda_stream


def _want(t, dtype, shape, name):
    if t is None:
        raise ValueError(f"{name}: missing")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _holds(t, dtype, n, name, more=True):
    """t holds the n values that are read or written from its first on (more: it may hold others behind them)."""
    if t is None:
        raise ValueError(f"{name}: missing")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.numel() < n or (t.numel() > n and not more):
        raise ValueError(f"{name}: expected {'at least ' if more else ''}{n} values, got shape {tuple(t.shape)}")


_HERE_CTX = contextlib.nullcontext()


def _on(stream, *tensors):
    """Context of a call on these tensors (the first is not None): their one device current, and `stream` (or that
    device's current stream) the one that outputs and scratch are allocated for."""
    first = tensors[0]
    index = first.get_device()
    if index < 0:
        raise ValueError("device tensor expected")
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on {first.device} and {t.device}")
    if stream is None and index == _device():
        return _HERE_CTX
    dev = first.device
    if stream is not None and stream.device != dev:
        raise ValueError(f"stream of {stream.device}, tensors on {dev}")
    ctx = contextlib.ExitStack()
    ctx.enter_context(torch.cuda.device(dev))
    if stream is not None:
        ctx.enter_context(torch.cuda.stream(stream))
    return ctx


def _given(stream):
    """Context in which `stream` is the current one (None: as it is)."""
    return _HERE_CTX if stream is None else torch.cuda.stream(stream)


class _Held(threading.local):
    """The scratch that workspace() keeps: device index -> (stream handle, buffer), one of each host thread."""

    def __init__(self):
        self.of = {}


_held = _Held()


def moe_workspace_size(shape: MoeShape) -> int:
    n = ctypes.c_size_t(0)
    _check(_L().moe_workspace_size(ctypes.byref(shape), ctypes.byref(n)), "moe_workspace_size")
    return int(n.value)


def workspace(shape: MoeShape, device=None) -> torch.Tensor:
    """A device buffer of moe_workspace_size(shape) bytes, for calls on the device's current stream.  Between calls of one
    host thread on one stream it is kept and grown on demand.  A call on another stream, from another thread or under
    graph capture gets a buffer of its own, allocated for that stream (or by the graph): scratch is never shared by
    calls that may overlap."""
    index = torch.device(device).index if device is not None else None
    if index is None or index == _device():
        return _scratch(shape)
    with torch.cuda.device(index):
        return _scratch(shape)


def _scratch(shape: MoeShape, stream=None) -> torch.Tensor:
    """workspace() on the current device, for a call on `stream` (None: the current one)."""
    if stream is not None:
        with _given(stream):
            return _scratch(shape)
    need, index = max(moe_workspace_size(shape), 256), _device()
    if _capturing():
        return torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", index))
    handle = _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream
    held = _held.of.get(index)
    if held is None or held[0] != handle or held[1].numel() < need:
        held = (handle, torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", index)))
        _held.of[index] = held
    return held[1]


def moe_capacity(T: int, k: int, E: int, factor: float) -> int:
    c = ctypes.c_int32(0)
    _check(_L().moe_capacity(T, k, E, float(factor), ctypes.byref(c)), "moe_capacity")
    return int(c.value)


def moe_route(shape: MoeShape, x, w_router, bias=None, *, logits=False, aux=False, ws=None, stream=None):
    T, d, E, k = shape.T, shape.d, shape.E, shape.k
    _want(x, torch.bfloat16, (T, d), "x")
    _want(w_router, torch.float32, (E, d), "w_router")
    with _on(None, x, w_router, bias, ws):
        dev = x.device
        out = dict(topk_idx=torch.empty(T, k, dtype=torch.int32, device=dev),
                   topk_w=torch.empty(T, k, dtype=torch.float32, device=dev),
                   counts=torch.empty(E, dtype=torch.int32, device=dev))
        if logits:
            out["logits"] = torch.empty(T, E, dtype=torch.float32, device=dev)
        if aux:
            out["aux_f"] = torch.empty(E, dtype=torch.float32, device=dev)
            out["aux_p"] = torch.empty(E, dtype=torch.float32, device=dev)
            out["aux"] = torch.empty(1, dtype=torch.float32, device=dev)
        ws = ws if ws is not None else _scratch(shape, stream)
        rc = _L().moe_route(ctypes.byref(shape), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(out.get("logits")),
                            _ptr(out["topk_idx"]), _ptr(out["topk_w"]), _ptr(out["counts"]), _ptr(out.get("aux_f")),
                            _ptr(out.get("aux_p")), _ptr(out.get("aux")), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "moe_route")
    return out


def moe_route_from_logits(shape: MoeShape, logits, *, aux=False, ws=None, stream=None):
    T, E, k = shape.T, shape.E, shape.k
    _want(logits, torch.float32, (T, E), "logits")
    with _on(None, logits, ws):
        dev = logits.device
        out = dict(topk_idx=torch.empty(T, k, dtype=torch.int32, device=dev),
                   topk_w=torch.empty(T, k, dtype=torch.float32, device=dev),
                   counts=torch.empty(E, dtype=torch.int32, device=dev))
        if aux:
            out["aux_f"] = torch.empty(E, dtype=torch.float32, device=dev)
            out["aux_p"] = torch.empty(E, dtype=torch.float32, device=dev)
            out["aux"] = torch.empty(1, dtype=torch.float32, device=dev)
        ws = ws if ws is not None else _scratch(shape, stream)
        rc = _L().moe_route_from_logits(ctypes.byref(shape), _ptr(logits), _ptr(out["topk_idx"]), _ptr(out["topk_w"]),
                                        _ptr(out["counts"]), _ptr(out.get("aux_f")), _ptr(out.get("aux_p")),
                                        _ptr(out.get("aux")), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "moe_route_from_logits")
    return out


def permute_outputs(shape: MoeShape, device):
    """Output buffers of moe_permute: row_src = -1 and x_perm = 0 in the rows the call leaves unfilled."""
    T, d, E, k, R = shape.T, shape.d, shape.E, shape.k, shape.R
    return dict(slot_pos=torch.empty(T, k, dtype=torch.int32, device=device),
                drop_mask=torch.empty(T, k, dtype=torch.uint8, device=device),
                counts=torch.empty(E, dtype=torch.int32, device=device),
                kept=torch.empty(E, dtype=torch.int32, device=device),
                offsets=torch.empty(E + 1, dtype=torch.int32, device=device),
                row_src=torch.full((R,), -1, dtype=torch.int32, device=device),
                x_perm=torch.zeros(R, d, dtype=torch.bfloat16, device=device))


def moe_permute(shape: MoeShape, x, topk_idx, *, ws=None, stream=None, out=None):
    """Grouping by expert.  `out` (from permute_outputs) reuses buffers: rows this call leaves unfilled keep
    what they held, and nothing is allocated or filled here."""
    T, d, E, k = shape.T, shape.d, shape.E, shape.k
    _want(x, torch.bfloat16, (T, d), "x")
    _want(topk_idx, torch.int32, (T, k), "topk_idx")
    with _on(stream, x, topk_idx, ws, None if out is None else out["x_perm"]):
        if out is None:
            out = permute_outputs(shape, x.device)
        else:
            _want(out["x_perm"], torch.bfloat16, (shape.R, d), "out['x_perm']")
            _want(out["row_src"], torch.int32, (shape.R,), "out['row_src']")
            _want(out["slot_pos"], torch.int32, (T, k), "out['slot_pos']")
        ws = ws if ws is not None else _scratch(shape)
        rc = _L().moe_permute(ctypes.byref(shape), _ptr(x), _ptr(topk_idx), _ptr(out["slot_pos"]),
                              _ptr(out["drop_mask"]), _ptr(out["counts"]), _ptr(out["kept"]), _ptr(out["offsets"]),
                              _ptr(out["row_src"]), _ptr(out["x_perm"]), _ptr(ws), ws.numel(), _stream())
    _check(rc, "moe_permute")
    return out


def moe_permute_noalloc(shape: MoeShape, x, topk_idx, *, stream=None):
    """moe_permute without a workspace: the library's fixed scratch array is used instead.

    For callers that cannot allocate device scratch; the outputs here are still
    torch tensors.  Calls that overlap on the GPU race on the shared scratch.
    """
    T, d, E, k = shape.T, shape.d, shape.E, shape.k
    _want(x, torch.bfloat16, (T, d), "x")
    _want(topk_idx, torch.int32, (T, k), "topk_idx")
    dev = x.device
    R = shape.R
    out = dict(slot_pos=torch.empty(T, k, dtype=torch.int32, device=dev),
               drop_mask=torch.empty(T, k, dtype=torch.uint8, device=dev),
               counts=torch.empty(E, dtype=torch.int32, device=dev),
               kept=torch.empty(E, dtype=torch.int32, device=dev),
               offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
               row_src=torch.full((R,), -1, dtype=torch.int32, device=dev),
               x_perm=torch.zeros(R, d, dtype=torch.bfloat16, device=dev))
    rc = _L().moe_permute_noalloc(ctypes.byref(shape), _ptr(x), _ptr(topk_idx), _ptr(out["slot_pos"]),
                                  _ptr(out["drop_mask"]), _ptr(out["counts"]), _ptr(out["kept"]),
                                  _ptr(out["offsets"]), _ptr(out["row_src"]), _ptr(out["x_perm"]), _stream(stream))
    _check(rc, "moe_permute_noalloc")
    return out


def moe_expert_ffn(shape: MoeShape, x_grouped, w13, w2, *, hidden=None, group_start=None, group_rows=None,
                   s13=None, s2=None, h=None, y=None, want_h=True, stream=None):
    """Grouped gated expert FFN.  Returns (h, y); with ``want_h=False`` (bf16 experts of hidden 128 or 256) h
    stays on chip in the fused kernel and None is returned in its place.  INT8 experts: the rows are quantised
    (moe_quantize_int8) and go through moe_expert_ffn_int8; h is None."""
    hidden = shape.H if hidden is None else hidden
    if shape.wfmt == WFMT_INT8:
        if h is not None:
            raise ValueError("moe_expert_ffn: INT8 experts return no h")
        _want(x_grouped, torch.bfloat16, (x_grouped.shape[0], shape.d), "x_grouped")
        _want_experts(shape, hidden, w13, s13, w2, s2)
        xq, xs = moe_quantize_int8(x_grouped, stream=stream)
        return None, moe_expert_ffn_int8(shape, xq, xs, w13, s13, w2, s2, hidden=hidden, group_start=group_start,
                                         group_rows=group_rows, y=y, stream=stream)
    R = x_grouped.shape[0]
    n_groups = w13.shape[0]
    dev = x_grouped.device
    if h is None and want_h:
        h = torch.empty(R, hidden, dtype=torch.bfloat16, device=dev)
    if y is None:
        y = torch.empty(R, shape.d, dtype=torch.bfloat16, device=dev)
    rc = _L().moe_expert_ffn(ctypes.byref(shape), n_groups, hidden, R, _ptr(x_grouped), _ptr(group_start),
                             _ptr(group_rows), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2), _ptr(h), _ptr(y),
                             _stream(stream))
    _check(rc, "moe_expert_ffn")
    return h, y


def moe_combine(shape: MoeShape, y_perm, slot_pos, topk_w, y_shared=None, *, out=None, stream=None):
    """Weighted top-k reduction back to token order: out [T, d] bf16.  y_perm, slot_pos, topk_w and ``out`` may be larger
    buffers or have other leading dimensions ([E, capacity, d], flat): their first R d, T k, T k and T d values count."""
    T, d, k = shape.T, shape.d, shape.k
    _holds(y_perm, torch.bfloat16, shape.R * d, "y_perm")
    _holds(slot_pos, torch.int32, T * k, "slot_pos")
    _holds(topk_w, torch.float32, T * k, "topk_w")
    if y_shared is not None:
        _holds(y_shared, torch.bfloat16, T * d, "y_shared", more=False)
    if out is not None:
        _holds(out, torch.bfloat16, T * d, "out")
    with _on(stream, y_perm, slot_pos, topk_w, y_shared, out):
        if out is None:
            out = torch.empty(T, d, dtype=torch.bfloat16, device=y_perm.device)
        rc = _L().moe_combine(ctypes.byref(shape), _ptr(y_perm), _ptr(slot_pos), _ptr(topk_w), _ptr(y_shared),
                              _ptr(out), _stream())
    _check(rc, "moe_combine")
    return out


def moe_forward(shape: MoeShape, x, w_router, w13, w2, *, bias=None, s13=None, s2=None, w13_sh=None, s13_sh=None,
                w2_sh=None, s2_sh=None, out=None, routing=False, aux=False, ws=None, stream=None, side_stream=None):
    """The whole layer.  Returns ``out`` [T, d] bf16, or a dict with routing outputs when asked.
    ``side_stream`` (a torch.cuda.Stream) lets a bf16 or INT8 shared expert overlap the routing and routed experts."""
    T, d, E, k = shape.T, shape.d, shape.E, shape.k
    _want(x, torch.bfloat16, (T, d), "x")
    if shape.wfmt == WFMT_INT8:
        _want_experts(shape, shape.H, w13, s13, w2, s2, n=E)
        if shape.H_s:
            _want_experts(shape, shape.H_s, w13_sh, s13_sh, w2_sh, s2_sh, n=1, sfx="_sh")
    with _on(None, x, w_router, bias, w13, s13, w2, s2, w13_sh, s13_sh, w2_sh, s2_sh, out, ws):
        dev = x.device
        if out is None:
            out = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
        r = {}
        if routing:
            r = dict(topk_idx=torch.empty(T, k, dtype=torch.int32, device=dev),
                     topk_w=torch.empty(T, k, dtype=torch.float32, device=dev),
                     counts=torch.empty(E, dtype=torch.int32, device=dev),
                     drop_mask=torch.empty(T, k, dtype=torch.uint8, device=dev))
        if aux:
            r.update(aux_f=torch.empty(E, dtype=torch.float32, device=dev),
                     aux_p=torch.empty(E, dtype=torch.float32, device=dev),
                     aux=torch.empty(1, dtype=torch.float32, device=dev))
        ws = ws if ws is not None else _scratch(shape, stream)
        rc = _L().moe_forward(ctypes.byref(shape), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(w13), _ptr(s13), _ptr(w2),
                              _ptr(s2), _ptr(w13_sh), _ptr(s13_sh), _ptr(w2_sh), _ptr(s2_sh), _ptr(out),
                              _ptr(r.get("topk_idx")), _ptr(r.get("topk_w")), _ptr(r.get("counts")),
                              _ptr(r.get("drop_mask")), _ptr(r.get("aux_f")), _ptr(r.get("aux_p")), _ptr(r.get("aux")),
                              _ptr(ws), ws.numel(), _stream(stream),
                              ctypes.c_void_p(side_stream.cuda_stream) if side_stream is not None else None)
    _check(rc, "moe_forward")
    if r:
        r["out"] = out
        return r
    return out


def moe_transpose_experts(w, *, out=None, stream=None):
    """[n, rows, cols] bf16 -> [n, cols, rows] bf16 (the transposed expert weights moe_backward_x takes)."""
    n, rows, cols = w.shape
    _want(w, torch.bfloat16, (n, rows, cols), "w")
    if out is None:
        out = torch.empty(n, cols, rows, dtype=torch.bfloat16, device=w.device)
    _check(_L().moe_transpose_experts(_ptr(w), n, rows, cols, _ptr(out), _stream(stream)), "moe_transpose_experts")
    return out


def _backward(shape, x, w_router, w13, w2, dout, bias, w13t, w2t, w13_sh, w2_sh, w13t_sh, w2t_sh, aux_coef, ws,
              stream, weights, side_stream=None):
    T, d, E, H, Hs = shape.T, shape.d, shape.E, shape.H, shape.H_s
    _want(x, torch.bfloat16, (T, d), "x")
    _want(dout, torch.bfloat16, (T, d), "dout")
    with _given(stream):   # scratch and transposed copies live for this call on its stream
        w13t = w13t if w13t is not None else moe_transpose_experts(w13)
        w2t = w2t if w2t is not None else moe_transpose_experts(w2)
        if Hs:
            w13t_sh = w13t_sh if w13t_sh is not None else moe_transpose_experts(w13_sh)
            w2t_sh = w2t_sh if w2t_sh is not None else moe_transpose_experts(w2_sh)
        if ws is None:
            n = ctypes.c_size_t(0)
            _check(_L().moe_backward_workspace_size(ctypes.byref(shape), ctypes.byref(n)), "moe_backward_workspace_size")
            ws = torch.empty(int(n.value), dtype=torch.uint8, device=x.device)
    f32 = dict(dtype=torch.float32, device=x.device)
    g = dict(dx=torch.empty(T, d, **f32))
    head = [ctypes.byref(shape), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(w13), _ptr(w13t), _ptr(w2t),
            _ptr(w13_sh), _ptr(w13t_sh), _ptr(w2t_sh), _ptr(dout), float(aux_coef), _ptr(g["dx"])]
    tail = [_ptr(ws), ws.numel(), _stream(stream)]
    if not weights:
        _check(_L().moe_backward_x(*head, *tail), "moe_backward_x")
        return g
    g.update(dw13=torch.empty(E, 2 * H, d, **f32), dw2=torch.empty(E, d, H, **f32),
             dw13_sh=torch.empty(1, 2 * Hs, d, **f32) if Hs else None,
             dw2_sh=torch.empty(1, d, Hs, **f32) if Hs else None, dw_router=torch.empty(E, d, **f32))
    side = ctypes.c_void_p(side_stream.cuda_stream) if side_stream is not None else None
    _check(_L().moe_backward(*head, _ptr(g["dw13"]), _ptr(g["dw2"]), _ptr(g["dw13_sh"]), _ptr(g["dw2_sh"]),
                             _ptr(g["dw_router"]), *tail, side), "moe_backward")
    return g


def moe_backward_x(shape: MoeShape, x, w_router, w13, w2, dout, *, bias=None, w13t=None, w2t=None, w13_sh=None,
                   w2_sh=None, w13t_sh=None, w2t_sh=None, aux_coef=0.0, ws=None, stream=None):
    """Input gradient dL/dx [T, d] fp32 of L = sum(dout * out) + aux_coef * aux (bf16 experts).  The transposed
    weights are made here when not given (moe_transpose_experts); the down projections enter only transposed."""
    return _backward(shape, x, w_router, w13, w2, dout, bias, w13t, w2t, w13_sh, w2_sh, w13t_sh, w2t_sh, aux_coef,
                     ws, stream, False)["dx"]


def moe_backward(shape: MoeShape, x, w_router, w13, w2, dout, *, bias=None, w13t=None, w2t=None, w13_sh=None,
                 w2_sh=None, w13t_sh=None, w2t_sh=None, aux_coef=0.0, ws=None, stream=None, side_stream=None):
    """All gradients of L = sum(dout * out) + aux_coef * aux: a dict of fp32 tensors dx [T, d], dw13 [E, 2H, d],
    dw2 [E, d, H], dw13_sh [1, 2H_s, d] and dw2_sh [1, d, H_s] (None without a shared expert), dw_router [E, d].
    ``side_stream`` (a torch.cuda.Stream) lets the shared expert's chain overlap the routed one."""
    return _backward(shape, x, w_router, w13, w2, dout, bias, w13t, w2t, w13_sh, w2_sh, w13t_sh, w2t_sh, aux_coef,
                     ws, stream, True, side_stream)


def moe_route_tree(shape: MoeShape, branch: int, levels: int, x, w_tree, bias_tree=None, *, counts=False,
                   logits=False, ws=None, stream=None):
    """Hierarchical router over E = branch**levels experts (shape.E).  w_tree [levels * branch, d] fp32 stacks
    the levels' routers.  Returns dict(topk_idx [T, k] int32, topk_w [T, k] fp32, counts [E] int32 or None,
    level_logits [T, levels * branch] fp32 or None)."""
    T, d, E, k = shape.T, shape.d, shape.E, shape.k
    n = branch * levels
    _want(x, torch.bfloat16, (T, d), "x")
    _want(w_tree, torch.float32, (n, d), "w_tree")
    if bias_tree is not None:
        _want(bias_tree, torch.float32, (n,), "bias_tree")
    dev = x.device
    if ws is None:
        nb = ctypes.c_size_t(0)
        _check(_L().moe_route_tree_workspace_size(ctypes.byref(shape), branch, levels, ctypes.byref(nb)),
               "moe_route_tree_workspace_size")
        with _given(stream):
            ws = torch.empty(int(nb.value), dtype=torch.uint8, device=dev)
    out = dict(topk_idx=torch.empty(T, k, dtype=torch.int32, device=dev),
               topk_w=torch.empty(T, k, dtype=torch.float32, device=dev),
               counts=torch.empty(E, dtype=torch.int32, device=dev) if counts else None,
               level_logits=torch.empty(T, n, dtype=torch.float32, device=dev) if logits else None)
    rc = _L().moe_route_tree(ctypes.byref(shape), branch, levels, _ptr(x), _ptr(w_tree), _ptr(bias_tree),
                             _ptr(out["topk_idx"]), _ptr(out["topk_w"]), _ptr(out["counts"]),
                             _ptr(out["level_logits"]), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "moe_route_tree")
    return out


def moe_quantize_int4(w, *, q=None, scales=None, stream=None):
    """w [..., K] fp32 -> (q [..., K/2] uint8, scales [..., K/128] bf16)."""
    K = w.shape[-1]
    rows = w.numel() // K
    if q is None:
        q = torch.empty(*w.shape[:-1], K // 2, dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty(*w.shape[:-1], K // 128, dtype=torch.bfloat16, device=w.device)
    rc = _L().moe_quantize_int4(_ptr(w), rows, K, _ptr(q), _ptr(scales), _stream(stream))
    _check(rc, "moe_quantize_int4")
    return q, scales


def moe_quantize_int8(x, *, q=None, scales=None, stream=None):
    """x [..., K] bf16 or fp32 -> (q [..., K] int8, scales [...] fp32): one scale per row, x ~ q * scale."""
    if x.dtype not in DTYPE_CODE:
        raise TypeError(f"x: expected torch.bfloat16 or torch.float32, got {x.dtype}")
    if x.dim() < 1:
        raise ValueError("x: expected at least one dimension")
    K = x.shape[-1]
    rows = x.numel() // K if K else 0
    with _on(stream, x, q, scales):
        if q is None:
            q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
        if scales is None:
            scales = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        _want(q, torch.int8, x.shape, "q")
        _want(scales, torch.float32, x.shape[:-1], "scales")
        _check(_L().moe_quantize_int8(_ptr(x), DTYPE_CODE[x.dtype], rows, K, _ptr(q), _ptr(scales), _stream()),
               "moe_quantize_int8")
    return q, scales


def moe_permute_int8(shape: MoeShape, x, topk_idx, *, full=False, ws=None, stream=None):
    """moe_permute with the rows quantised on the way: a dict with slot_pos, kept, offsets, xq_perm [R, d] int8 and
    xs_perm [R] fp32; with ``full`` also drop_mask, counts and row_src (-1 in rows that no token fills).  With a
    capacity, the rows behind an expert's kept ones hold nothing in particular."""
    T, d, E, k = shape.T, shape.d, shape.E, shape.k
    _want(x, torch.bfloat16, (T, d), "x")
    _want(topk_idx, torch.int32, (T, k), "topk_idx")
    dev, R = x.device, shape.R
    with _on(stream, x, topk_idx, ws):
        i32 = dict(dtype=torch.int32, device=dev)
        out = dict(slot_pos=torch.empty_like(topk_idx), kept=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
                   xq_perm=torch.empty(R, d, dtype=torch.int8, device=dev),
                   xs_perm=torch.empty(R, dtype=torch.float32, device=dev))
        if full:
            out.update(drop_mask=torch.empty(T, k, dtype=torch.uint8, device=dev), counts=torch.empty(E, **i32),
                       row_src=torch.full((R,), -1, **i32))
        if ws is None:
            ws = torch.empty(moe_workspace_size(shape), dtype=torch.uint8, device=dev)
        rc = _L().moe_permute_int8(ctypes.byref(shape), _ptr(x), _ptr(topk_idx), _ptr(out["slot_pos"]),
                                   _ptr(out.get("drop_mask")), _ptr(out.get("counts")), _ptr(out["kept"]),
                                   _ptr(out["offsets"]), _ptr(out.get("row_src")), _ptr(out["xq_perm"]),
                                   _ptr(out["xs_perm"]), _ptr(ws), ws.numel(), _stream())
        _check(rc, "moe_permute_int8")
    return out


def _want_experts(shape, hidden, w13, s13, w2, s2, n=None, sfx=""):
    """INT8 weights and scales of n experts (None: as many as w13 holds) of this hidden width."""
    if n is None and w13 is not None:
        n = w13.shape[0]
    for t, name, dtype, dims in ((w13, "w13", torch.int8, (n, 2 * hidden, shape.d)), (s13, "s13", torch.float32, (n, 2 * hidden)),
                                 (w2, "w2", torch.int8, (n, shape.d, hidden)), (s2, "s2", torch.float32, (n, shape.d))):
        _want(t, dtype, dims, name + sfx)


def moe_expert_ffn_int8(shape: MoeShape, xq, xs, w13, s13, w2, s2, *, hidden=None, group_start=None,
                        group_rows=None, y=None, ws=None, stream=None):
    """Grouped gated expert FFN in 8-bit integers (shape.wfmt == WFMT_INT8): xq [R, d] int8 with one scale a row
    xs [R], w13 [n, 2 hidden, d] and w2 [n, d, hidden] int8 with one scale an output channel.  Returns y [R, d]
    bf16; rows outside every group are not written."""
    hidden = shape.H if hidden is None else hidden
    _want_experts(shape, hidden, w13, s13, w2, s2)
    n, R, d = w13.shape[0], xq.shape[0] if xq is not None else 0, shape.d
    _want(xq, torch.int8, (R, d), "xq")
    _want(xs, torch.float32, (R,), "xs")
    for t, name in ((group_start, "group_start"), (group_rows, "group_rows")):
        if t is not None and (t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] < n):
            raise ValueError(f"{name}: expected at least {n} int32 values")
    with _on(stream, xq, xs, w13, s13, w2, s2, group_start, group_rows, y, ws):
        if y is None:
            y = torch.empty(R, d, dtype=torch.bfloat16, device=xq.device)
        _want(y, torch.bfloat16, (R, d), "y")
        if ws is None:
            nb = ctypes.c_size_t(0)
            _check(_L().moe_expert_ffn_int8_workspace_size(ctypes.byref(shape), hidden, R, ctypes.byref(nb)),
                   "moe_expert_ffn_int8_workspace_size")
            ws = torch.empty(int(nb.value), dtype=torch.uint8, device=xq.device)
        rc = _L().moe_expert_ffn_int8(ctypes.byref(shape), n, hidden, R, _ptr(xq), _ptr(xs), _ptr(group_start),
                                      _ptr(group_rows), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2), _ptr(y), _ptr(ws),
                                      ws.numel(), _stream())
        _check(rc, "moe_expert_ffn_int8")
    return y


def moe_combine_backward(shape: MoeShape, dout, y_perm, slot_pos, topk_w, *, kept=None, want_dw=True, want_dy=True,
                         stream=None):
    """Gradient of moe_combine: dict(dy_perm [R, d] bf16, dtopk_w [T, k] fp32), None for one that is not wanted; that
    of y_shared is dout.  With a capacity and ``kept`` (of moe_permute), rows that no token fills come back zero;
    without ``kept`` they hold nothing in particular."""
    if not (want_dw or want_dy):
        raise ValueError("moe_combine_backward: neither want_dw nor want_dy")
    T, d, k, R = shape.T, shape.d, shape.k, shape.R
    _want(dout, torch.bfloat16, (T, d), "dout")
    _want(y_perm, torch.bfloat16, (R, d), "y_perm")
    _want(slot_pos, torch.int32, (T, k), "slot_pos")
    _want(topk_w, torch.float32, (T, k), "topk_w")
    if kept is not None:
        _want(kept, torch.int32, (shape.E,), "kept")
    with _on(stream, dout, y_perm, slot_pos, topk_w, kept):
        dy = torch.empty_like(y_perm) if want_dy else None
        dw = torch.empty_like(topk_w) if want_dw else None
        rc = _L().moe_combine_backward(ctypes.byref(shape), _ptr(dout), _ptr(y_perm), _ptr(slot_pos), _ptr(topk_w),
                                       _ptr(kept) if want_dy and shape.capacity > 0 else None, _ptr(dy), _ptr(dw),
                                       _stream())
        _check(rc, "moe_combine_backward")
    return dict(dy_perm=dy, dtopk_w=dw)


def moe_permute_backward(shape: MoeShape, dx_perm, slot_pos, *, add=None, dtype=torch.float32, out=None,
                         stream=None):
    """Gradient of moe_permute's row moves: dx [T, d] (dtype bf16 or fp32) = the sum of each token's kept rows of
    dx_perm [R, d] (bf16 or fp32), plus ``add`` [T, d] of that dtype when given.  ``out`` may be ``add``."""
    T, d, R = shape.T, shape.d, shape.R
    if dx_perm is None:
        raise ValueError("dx_perm: missing")
    if dx_perm.dtype not in DTYPE_CODE or dtype not in DTYPE_CODE:
        raise TypeError(f"dx_perm, dtype: expected torch.bfloat16 or torch.float32, got {dx_perm.dtype}, {dtype}")
    _want(dx_perm, dx_perm.dtype, (R, d), "dx_perm")
    _want(slot_pos, torch.int32, (T, shape.k), "slot_pos")
    if add is not None:
        _want(add, dtype, (T, d), "add")
    with _on(stream, dx_perm, slot_pos, add, out):
        if out is None:
            out = torch.empty(T, d, dtype=dtype, device=dx_perm.device)
        _want(out, dtype, (T, d), "out")
        rc = _L().moe_permute_backward(ctypes.byref(shape), _ptr(dx_perm), DTYPE_CODE[dx_perm.dtype],
                                       _ptr(slot_pos), _ptr(add), _ptr(out), DTYPE_CODE[dtype], _stream())
        _check(rc, "moe_permute_backward")
    return out


def moe_get_status(stream=None):
    st, site = ctypes.c_int32(0), ctypes.c_uint32(0)
    _check(_L().moe_get_status(_stream(stream), ctypes.byref(st), ctypes.byref(site)), "moe_get_status")
    return int(st.value), int(site.value)


def moe_launch_count() -> int:
    return int(_L().moe_launch_count())
