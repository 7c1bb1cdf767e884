"""ctypes binding of include/moe_ops.h, the operators around the layer: routing
from logits, layer and RMS norm, the dense product with an epilogue, gradient
clipping.

As in _binding: argument marshalling only, every function forwards to the
library's function of the same name and returns its moe_status; tensors may be
torch tensors, raw addresses or None.  The descriptors (route_desc, norm_desc,
linear_desc) are plain C structs that a caller makes once per shape and passes
to every call.
"""
from __future__ import annotations

import ctypes

from . import _binding as _b
from ._binding import _nbytes, _stream

MOE_F16 = 5
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_NORM_LAYER, MOE_NORM_RMS = 0, 1
MOE_ACT_NONE, MOE_ACT_RELU, MOE_ACT_SILU, MOE_ACT_GELU, MOE_ACT_GELU_TANH = range(5)
MOE_CLIP_L2, MOE_CLIP_MAX = 0, 1

_DTYPES = {"f32": _b.MOE_F32, "bf16": _b.MOE_BF16, "f16": MOE_F16}
_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
_NORMS = {"layer": MOE_NORM_LAYER, "rms": MOE_NORM_RMS}
_ACTS = {"none": MOE_ACT_NONE, "relu": MOE_ACT_RELU, "silu": MOE_ACT_SILU, "gelu": MOE_ACT_GELU,
         "gelu_tanh": MOE_ACT_GELU_TANH}
_CLIPS = {"l2": MOE_CLIP_L2, "max": MOE_CLIP_MAX}

EXPORTED_OPS = (
    "moe_route",
    "moe_route_backward",
    "moe_norm",
    "moe_norm_backward_workspace_size",
    "moe_norm_backward",
    "moe_linear_workspace_size",
    "moe_linear",
    "moe_linear_backward_workspace_size",
    "moe_linear_backward",
    "moe_clip_grads_workspace_size",
    "moe_clip_grads",
)


class moe_route_desc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("keep_groups", ctypes.c_int32), ("group_top", ctypes.c_int32), ("score", ctypes.c_int),
                ("renorm", ctypes.c_int32), ("scale", ctypes.c_float), ("dtype", ctypes.c_int)]


class moe_norm_desc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("kind", ctypes.c_int), ("eps", ctypes.c_float),
                ("dtype", ctypes.c_int)]


class moe_linear_desc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("act", ctypes.c_int),
                ("dtype", ctypes.c_int), ("y_out", ctypes.c_int)]


class moe_grad_tensor(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int)]


_ready = None


def _lib() -> ctypes.CDLL:
    """The library with the operators' signatures set; raises MoeLibraryMissing
    if it was not built."""
    global _ready
    L = _b.lib()
    if _ready is not L:
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        pr, pn = ctypes.POINTER(moe_route_desc), ctypes.POINTER(moe_norm_desc)
        pl, pg = ctypes.POINTER(moe_linear_desc), ctypes.POINTER(moe_grad_tensor)
        L.moe_route.argtypes = [pr, vp, vp, vp, vp, vp]
        L.moe_route_backward.argtypes = [pr, vp, vp, vp, vp, vp]
        L.moe_norm.argtypes = [pn] + [vp] * 7
        L.moe_norm_backward_workspace_size.argtypes = [pn]
        L.moe_norm_backward.argtypes = [pn] + [vp] * 9 + [sz, vp]
        L.moe_linear_workspace_size.argtypes = [pl]
        L.moe_linear.argtypes = [pl] + [vp] * 7 + [sz, vp]
        L.moe_linear_backward_workspace_size.argtypes = [pl]
        L.moe_linear_backward.argtypes = [pl] + [vp] * 8 + [sz, vp]
        L.moe_clip_grads_workspace_size.argtypes = [pg, i32]
        L.moe_clip_grads.argtypes = [pg, i32, ctypes.c_int, ctypes.c_float, vp, vp, sz, vp]
        for f in EXPORTED_OPS:
            getattr(L, f).restype = sz if f.endswith("_size") else ctypes.c_int
        _ready = L
    return L


def _ptr(t):
    try:
        return t.data_ptr()
    except AttributeError:  # an address, or None
        return t


def route_desc(T: int, E: int, k: int, groups: int = 1, keep_groups: int | None = None, group_top: int = 1,
               score: str = "sigmoid", renorm: bool = True, scale: float = 1.0, dtype: str = "f32") -> moe_route_desc:
    return moe_route_desc(T, E, k, groups, groups if keep_groups is None else keep_groups, group_top, _SCORES[score],
                          int(renorm), scale, _DTYPES[dtype])


def norm_desc(T: int, H: int, kind: str = "layer", eps: float = 1e-6, dtype: str = "bf16") -> moe_norm_desc:
    return moe_norm_desc(T, H, _NORMS[kind], eps, _DTYPES[dtype])


def linear_desc(M: int, N: int, K: int, act: str = "none", dtype: str = "bf16",
                y_out: str | None = None) -> moe_linear_desc:
    return moe_linear_desc(M, N, K, _ACTS[act], _DTYPES[dtype], _DTYPES[dtype if y_out is None else y_out])


def moe_route(d: moe_route_desc, logits, bias, idx, w, stream=None) -> int:
    return _lib().moe_route(ctypes.byref(d), _ptr(logits), _ptr(bias), _ptr(idx), _ptr(w), _stream(stream))


def moe_route_backward(d: moe_route_desc, logits, idx, dw, dlogits, stream=None) -> int:
    return _lib().moe_route_backward(ctypes.byref(d), _ptr(logits), _ptr(idx), _ptr(dw), _ptr(dlogits),
                                     _stream(stream))


def moe_norm(d: moe_norm_desc, x, gamma, beta, y, mean=None, rstd=None, stream=None) -> int:
    return _lib().moe_norm(ctypes.byref(d), _ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(mean), _ptr(rstd),
                           _stream(stream))


def moe_norm_backward_workspace_size(d: moe_norm_desc) -> int:
    return int(_lib().moe_norm_backward_workspace_size(ctypes.byref(d)))


def _ws_bytes(ws, ws_bytes) -> int:
    if ws_bytes is not None:
        return ws_bytes
    return 0 if ws is None else _nbytes(ws)


def moe_norm_backward(d: moe_norm_desc, dy, x, gamma, mean, rstd, dx, dgamma, dbeta, ws, ws_bytes=None,
                      stream=None) -> int:
    return _lib().moe_norm_backward(ctypes.byref(d), _ptr(dy), _ptr(x), _ptr(gamma), _ptr(mean), _ptr(rstd), _ptr(dx),
                                    _ptr(dgamma), _ptr(dbeta), _ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream))


def moe_linear_workspace_size(d: moe_linear_desc) -> int:
    return int(_lib().moe_linear_workspace_size(ctypes.byref(d)))


def moe_linear(d: moe_linear_desc, x, weight, bias, residual, pre, y, ws=None, ws_bytes=None, stream=None) -> int:
    return _lib().moe_linear(ctypes.byref(d), _ptr(x), _ptr(weight), _ptr(bias), _ptr(residual), _ptr(pre), _ptr(y),
                             _ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream))


def moe_linear_backward_workspace_size(d: moe_linear_desc) -> int:
    return int(_lib().moe_linear_backward_workspace_size(ctypes.byref(d)))


def moe_linear_backward(d: moe_linear_desc, dy, pre, x, weight, dx, dweight, dbias, ws, ws_bytes=None,
                        stream=None) -> int:
    return _lib().moe_linear_backward(ctypes.byref(d), _ptr(dy), _ptr(pre), _ptr(x), _ptr(weight), _ptr(dx),
                                      _ptr(dweight), _ptr(dbias), _ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream))


class GradList:
    """The host array of moe_clip_grads: what to read and what to write.  It
    holds the tensors whose addresses it carries."""

    def __init__(self, grads, out):
        self.tensors = (list(grads), list(out))
        if len(self.tensors[0]) != len(self.tensors[1]):
            raise ValueError("one output for each gradient")
        self.count = len(self.tensors[0])
        self.array = (moe_grad_tensor * max(1, self.count))()
        for slot, g, o in zip(self.array, *self.tensors):
            if g.dtype != o.dtype or g.numel() != o.numel():
                raise ValueError("a gradient and its output have the same type and number of elements")
            if not (g.is_contiguous() and o.is_contiguous()):
                raise ValueError("gradients are contiguous")
            slot.in_, slot.out, slot.n, slot.dtype = g.data_ptr(), o.data_ptr(), g.numel(), _torch_dtype(g.dtype)


def _torch_dtype(dt) -> int:
    import torch

    codes = {torch.float32: _b.MOE_F32, torch.bfloat16: _b.MOE_BF16, torch.float16: MOE_F16}
    if dt not in codes:
        raise ValueError(f"gradients are float32, bfloat16 or float16, not {dt}")
    return codes[dt]


def tensor_list(grads, out=None) -> GradList:
    """GradList of torch tensors; without `out` they are clipped in place."""
    grads = list(grads)
    return GradList(grads, grads if out is None else out)


def moe_clip_grads_workspace_size(grads: GradList) -> int:
    return int(_lib().moe_clip_grads_workspace_size(grads.array, grads.count))


def moe_clip_grads(grads: GradList, kind: str, max_norm: float, norm_out, ws, ws_bytes=None, stream=None) -> int:
    return _lib().moe_clip_grads(grads.array, grads.count, _CLIPS[kind], max_norm, _ptr(norm_out), _ptr(ws),
                                 _ws_bytes(ws, ws_bytes), _stream(stream))
