"""Python binding of libsketchattn.so (include/sketch_attn.h).

Argument marshalling only: PyTorch supplies device memory and the current
stream; every step of SA and STCA runs in the library's CUDA kernels.  There
is no CPU fallback: if the library is missing or a call fails, an exception
is raised.

Entry points keep the C names: ``sa_forward``, ``sa_backward``,
``stca_forward``, ``stca_forward_full``, ``stca_fuse`` and the others of the header (plus the
workspace queries); ``AdamWTensors`` describes the tensors of ``sa_adamw_step``.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Sequence

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsketchattn.so")

SA_F32, SA_BF16 = 0, 1
_STATUS = {0: "SA_OK", 1: "SA_ERR_INVALID_ARG", 2: "SA_ERR_UNSUPPORTED", 3: "SA_ERR_CUDA",
           4: "SA_ERR_TIMEOUT", 5: "SA_ERR_WORKSPACE"}

# Symbols include/sketch_attn.h declares.
EXPORTS = ("sa_version", "sa_last_error", "sa_poll_device_status", "sa_forward_workspace",
           "sa_forward", "sa_backward_workspace", "sa_backward", "stca_forward_workspace",
           "stca_forward", "stca_fuse", "sa_launch_count", "sa_profile", "sa_profile_read",
           "sa_forward_noalloc", "sa_refine_workspace", "sa_refine_forward",
           "sa_forward_tokenwise_workspace", "sa_forward_tokenwise", "sa_backward_accumulate",
           "stca_forward_full_workspace", "stca_forward_full", "stca_backward_full_workspace",
           "stca_backward_full", "sa_gather_events", "sa_gather_events_fused",
           "sa_gather_events_fused_workspace", "sa_measure_exp2_rate", "sa_selftest_bounded_wait",
           "sa_refine_backward_workspace", "sa_refine_backward", "sa_backward_tokenwise_workspace",
           "sa_backward_tokenwise", "sa_gather_events_backward_workspace", "sa_gather_events_backward",
           "sa_adamw_step", "sa_selftest_unsorted_events")


class SAError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {_STATUS.get(status, status)}: {msg}")
        self.status = status


class StcaLayerC(ctypes.Structure):
    _fields_ = [("W_Q", ctypes.c_void_p), ("W_K", ctypes.c_void_p),
                ("W_V", ctypes.c_void_p), ("W_O", ctypes.c_void_p)]


STCA_FFN_KEYS = ("hist_W1", "hist_W3", "hist_W2", "q_W1", "q_W3", "q_W2")


class StcaFullLayerC(ctypes.Structure):
    _fields_ = [("attn", StcaLayerC)] + [(k, ctypes.c_void_p) for k in STCA_FFN_KEYS]


STCA_GRAD_KEYS = ("dW_Q", "dW_K", "dW_V", "dW_O", "hist_dW1", "hist_dW3", "hist_dW2", "q_dW1", "q_dW3", "q_dW2")


class StcaFullLayerGradC(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in STCA_GRAD_KEYS]


class RefineLayerC(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("W_Q", "W_K", "ln1_g", "ln1_b", "W1", "W3", "W2",
                                               "ln2_g", "ln2_b")]


REFINE_GRAD_KEYS = ("dW_Q", "dW_K", "dln1_g", "dln1_b", "dW1", "dW3", "dW2", "dln2_g", "dln2_b")


class RefineLayerGradC(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in REFINE_GRAD_KEYS]


SA_STATE_F32, SA_STATE_8BIT = 0, 1
ADAMW_BLOCK = 128        # values per scale of an 8-bit state


class AdamWTensorC(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("grad_dtype", ctypes.c_int),
                ("state", ctypes.c_int), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("param_bf16", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("weight_decay", ctypes.c_float)]


class AdamWConfigC(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64), ("step_dev", ctypes.c_void_p),
                ("lr_dev", ctypes.c_void_p), ("grad_scale_dev", ctypes.c_void_p)]


_lib = None

_vp, _i, _i64, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


def load(path: Optional[str] = None):
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m sketch_attention_b200.build`")
    lib = ctypes.CDLL(path)
    lib.sa_version.restype = _i
    lib.sa_last_error.restype = ctypes.c_char_p
    lib.sa_poll_device_status.restype = _i
    lib.sa_poll_device_status.argtypes = [_vp]
    lib.sa_forward_workspace.restype = _sz
    lib.sa_forward_workspace.argtypes = [_i, _i64, _i, _i, _i]
    lib.sa_forward.restype = _i
    lib.sa_forward.argtypes = [_vp, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _f,
                               _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.sa_backward_workspace.restype = _sz
    lib.sa_backward_workspace.argtypes = [_i, _i64, _i, _i, _i]
    lib.sa_backward.restype = _i
    lib.sa_backward.argtypes = [_vp, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _f,
                                _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.sa_backward_accumulate.restype = _i
    lib.sa_backward_accumulate.argtypes = lib.sa_backward.argtypes
    lib.stca_forward_workspace.restype = _sz
    lib.stca_forward_workspace.argtypes = [_i, _i64, _i, _i, _i, _i]
    lib.stca_forward.restype = _i
    lib.stca_forward.argtypes = [_vp, _i, _vp, _vp, _i, _vp, _i64, _vp, _vp, _vp, _vp,
                                 _i, _i, _i, _i, ctypes.POINTER(StcaLayerC), _vp, _vp, _sz, _vp]
    lib.stca_forward_full_workspace.restype = _sz
    lib.stca_forward_full_workspace.argtypes = [_i, _i64, _i64, _i, _i, _i, _i]
    lib.stca_forward_full.restype = _i
    lib.stca_forward_full.argtypes = [_vp, _i, _vp, _vp, _i, _vp, _i64, _vp, _vp, _vp, _vp,
                                      _i, _i, _i, _i, ctypes.POINTER(StcaFullLayerC), _vp, _vp, _sz, _vp]
    lib.stca_backward_full_workspace.restype = _sz
    lib.stca_backward_full_workspace.argtypes = [_i, _vp, _vp, _vp, _i, _i, _i, _i, _i]
    lib.stca_backward_full.restype = _i
    lib.stca_backward_full.argtypes = [_vp, _i, _vp, _vp, _i, _vp, _i64, _vp, _vp, _vp, _vp,
                                       _i, _i, _i, _i, ctypes.POINTER(StcaFullLayerC), _vp, _vp, _vp,
                                       ctypes.POINTER(StcaFullLayerGradC), _vp, _sz, _vp]
    lib.sa_selftest_bounded_wait.restype = _i
    lib.sa_selftest_bounded_wait.argtypes = [ctypes.c_longlong, _vp]
    lib.sa_measure_exp2_rate.restype = _i
    lib.sa_measure_exp2_rate.argtypes = [_i, ctypes.POINTER(ctypes.c_double), _vp]
    lib.sa_gather_events.restype = _i
    lib.sa_gather_events.argtypes = [_vp, _i64, _vp, _i, _vp, _vp, _i64, _i, _vp, _vp]
    lib.sa_gather_events_fused_workspace.restype = _sz
    lib.sa_gather_events_fused_workspace.argtypes = [_i, _i, _i]
    lib.sa_gather_events_fused.restype = _i
    lib.sa_gather_events_fused.argtypes = [_vp, _i64, _vp, _i, _vp, _vp, _i64, _i, _vp, _vp, _vp, _i, _vp, _vp,
                                           _sz, _vp]
    lib.stca_fuse.restype = _i
    lib.stca_fuse.argtypes = [_vp, _vp, _vp, _vp, _i64, _i, _vp, _vp]
    lib.sa_forward_noalloc.restype = _i
    lib.sa_forward_noalloc.argtypes = [_vp, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _f,
                                       _vp, _vp, _vp, _vp, _vp, _vp]
    lib.sa_forward_tokenwise_workspace.restype = _sz
    lib.sa_forward_tokenwise_workspace.argtypes = [_i, _i64, _i, _i, _i]
    lib.sa_forward_tokenwise.restype = _i
    lib.sa_forward_tokenwise.argtypes = [_vp, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _f,
                                         _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.sa_refine_workspace.restype = _sz
    lib.sa_refine_workspace.argtypes = [_i, _i64, _i, _i, _i]
    lib.sa_refine_forward.restype = _i
    lib.sa_refine_forward.argtypes = [_vp, _i, _vp, _vp, _i, _i, _i, _vp, _i,
                                      ctypes.POINTER(RefineLayerC), _f, _vp, _vp, _sz, _vp]
    lib.sa_refine_backward_workspace.restype = _sz
    lib.sa_refine_backward_workspace.argtypes = [_i, _i64, _i, _i, _i, _i]
    lib.sa_refine_backward.restype = _i
    lib.sa_refine_backward.argtypes = [_vp, _i, _vp, _vp, _i, _i, _i, _vp, _i, ctypes.POINTER(RefineLayerC), _f,
                                       _vp, _vp, _vp, ctypes.POINTER(RefineLayerGradC), _vp, _sz, _vp]
    lib.sa_backward_tokenwise_workspace.restype = _sz
    lib.sa_backward_tokenwise_workspace.argtypes = [_i, _i64, _i, _i, _i]
    lib.sa_backward_tokenwise.restype = _i
    lib.sa_backward_tokenwise.argtypes = [_vp, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _f, _vp, _vp,
                                          _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.sa_gather_events_backward_workspace.restype = _sz
    lib.sa_gather_events_backward_workspace.argtypes = [_i64, _i64, _i, _i]
    lib.sa_gather_events_backward.restype = _i
    lib.sa_gather_events_backward.argtypes = [_vp, _vp, _i64, _vp, _i, _i64, _i, _i, _vp, _vp, _vp, _sz, _vp]
    lib.sa_selftest_unsorted_events.restype = _i
    lib.sa_selftest_unsorted_events.argtypes = [_vp, _vp, _vp, _i64, _i64, _i, _i, _vp, _vp, _vp, _sz, _vp]
    lib.sa_adamw_step.restype = _i
    lib.sa_adamw_step.argtypes = [ctypes.POINTER(AdamWTensorC), _i, ctypes.POINTER(AdamWConfigC), _vp]
    lib.sa_launch_count.restype = ctypes.c_longlong
    lib.sa_profile.restype = _i
    lib.sa_profile.argtypes = [_i]
    lib.sa_profile_read.restype = _i
    lib.sa_profile_read.argtypes = [_i, ctypes.c_char_p, _i, ctypes.POINTER(ctypes.c_double),
                                    ctypes.POINTER(ctypes.c_longlong)]
    _lib = lib
    return lib


def _check(fn: str, status: int):
    if status != 0:
        raise SAError(fn, status, load().sa_last_error().decode())


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SA_F32
    if t.dtype == torch.bfloat16:
        return SA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _host_i64(a) -> np.ndarray:
    if isinstance(a, torch.Tensor):
        a = a.cpu().numpy()
    return np.ascontiguousarray(np.asarray(a, dtype=np.int64))


def _hp(a: np.ndarray):
    return a.ctypes.data_as(ctypes.c_void_p)


def _dev_i64(host: np.ndarray, device, given: Optional[torch.Tensor]) -> torch.Tensor:
    if given is not None:
        return given
    return torch.from_numpy(host).to(device, non_blocking=False)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def _need(name: str, t: torch.Tensor, dtype, shape, device):
    """t is a contiguous CUDA tensor of that dtype, shape and device."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous() and t.is_cuda:
        return t
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, not on {device}")


_SAME_PLACE = contextlib.nullcontext()
# torch.cuda.current_stream builds a Stream object, as long as two kernel launches take
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _at(device, stream):
    """Runs a call on its tensors' device and on `stream`: buffers allocated inside belong to that
    stream, so the allocator hands them out again only behind the call's kernels."""
    if stream is None:
        return _SAME_PLACE if device.index == torch.cuda.current_device() else torch.cuda.device(device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


def _raw_stream(device, stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _current_raw_stream(device.index)


def _used_on(stream, *ts):
    """Tensors of the caller that a call on `stream` uses: the allocator keeps their memory until that
    work is done, although the caller may drop them as soon as the call returns."""
    if stream is not None:
        for t in ts:
            if t is not None:
                t.record_stream(stream)


def _workspace(given: Optional[torch.Tensor], size: int, device) -> torch.Tensor:
    """The caller's workspace if it is large enough, else a new one (at least one byte)."""
    if given is None:
        return torch.empty(size or 1, dtype=torch.uint8, device=device)
    if not given.is_cuda or not given.is_contiguous() or given.device != device:
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return given if given.nbytes >= size else torch.empty(size, dtype=torch.uint8, device=device)


# --------------------------------------------------------------------------
def sa_forward_workspace(B: int, n_total: int, k: int, d: int, dtype: int) -> int:
    return int(load().sa_forward_workspace(B, n_total, k, d, dtype))


def sa_forward(X: torch.Tensor, offsets, P, W_Q, W_K, W_V, eps: float = 1e-6, *,
               offsets_dev: Optional[torch.Tensor] = None, want_H: bool = False,
               want_bf16: bool = False, want_lse: bool = False, out: Optional[dict] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Sketches of a ragged batch.  Returns {"S", "mass"[, "H"][, "S_bf16"][, "lse"]}."""
    lib = load()
    _need_cuda(X, P, W_Q, W_K, W_V)
    off = _host_i64(offsets)
    B = len(off) - 1
    k, d = P.shape
    dev = X.device
    dt = _dtype_code(X)
    o = dict(out or {})
    S = o.get("S") if o.get("S") is not None else torch.empty(B, k, d, device=dev)
    mass = o.get("mass") if o.get("mass") is not None else torch.empty(B, k, device=dev)
    H = o.get("H") if o.get("H") is not None else (torch.empty(B, k, d, device=dev) if want_H else None)
    Sb = o.get("S_bf16") if o.get("S_bf16") is not None else (
        torch.empty(B, k, d, device=dev, dtype=torch.bfloat16) if want_bf16 else None)
    lse = o.get("lse") if o.get("lse") is not None else (
        torch.empty(max(int(off[-1]), 1), device=dev) if want_lse else None)
    ws_bytes = lib.sa_forward_workspace(B, int(off[-1]), k, d, dt)
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    offd = _dev_i64(off, dev, offsets_dev)
    st = lib.sa_forward(_p(X), dt, _hp(off), _p(offd), B, k, d, _p(P), _p(W_Q), _p(W_K), _p(W_V),
                        float(eps), _p(S), _p(mass), _p(H), _p(Sb), _p(lse), _p(workspace),
                        workspace.numel(), _stream(stream))
    _check("sa_forward", st)
    res = {"S": S, "mass": mass}
    if H is not None:
        res["H"] = H
    if Sb is not None:
        res["S_bf16"] = Sb
    if lse is not None:
        res["lse"] = lse
    return res


def sa_forward_tokenwise_workspace(B: int, n_total: int, k: int, d: int, x_dtype: int) -> int:
    return int(load().sa_forward_tokenwise_workspace(B, n_total, k, d, x_dtype))


def sa_forward_tokenwise(X: torch.Tensor, offsets, P, W_Q, W_K, W_V, eps: float = 1e-6, *,
                         offsets_dev: Optional[torch.Tensor] = None, want_H: bool = False,
                         want_bf16: bool = False, out: Optional[dict] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """The token-wise normalisation variant (softmax over each prototype's tokens).
    Returns {"S", "mass"[, "H"][, "S_bf16"]}."""
    lib = load()
    _need_cuda(X, P, W_Q, W_K, W_V)
    off = _host_i64(offsets)
    B = len(off) - 1
    k, d = P.shape
    dev = X.device
    dt = _dtype_code(X)
    o = dict(out or {})
    S = o.get("S") if o.get("S") is not None else torch.empty(B, k, d, device=dev)
    mass = o.get("mass") if o.get("mass") is not None else torch.empty(B, k, device=dev)
    H = o.get("H") if o.get("H") is not None else (torch.empty(B, k, d, device=dev) if want_H else None)
    Sb = o.get("S_bf16") if o.get("S_bf16") is not None else (
        torch.empty(B, k, d, device=dev, dtype=torch.bfloat16) if want_bf16 else None)
    ws_bytes = lib.sa_forward_tokenwise_workspace(B, int(off[-1]), k, d, dt)
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    offd = _dev_i64(off, dev, offsets_dev)
    st = lib.sa_forward_tokenwise(_p(X), dt, _hp(off), _p(offd), B, k, d, _p(P), _p(W_Q), _p(W_K),
                                  _p(W_V), float(eps), _p(S), _p(mass), _p(H), _p(Sb),
                                  _p(workspace), workspace.numel(), _stream(stream))
    _check("sa_forward_tokenwise", st)
    res = {"S": S, "mass": mass}
    if H is not None:
        res["H"] = H
    if Sb is not None:
        res["S_bf16"] = Sb
    return res


def sa_backward_tokenwise_workspace(B: int, n_total: int, k: int, d: int, x_dtype: int) -> int:
    return int(load().sa_backward_tokenwise_workspace(B, n_total, k, d, x_dtype))


def sa_backward_tokenwise(X: torch.Tensor, offsets, P, W_Q, W_K, W_V, eps: float, H, dS, *,
                          offsets_dev: Optional[torch.Tensor] = None, out: Optional[dict] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients {"dX", "dP", "dW_Q", "dW_K", "dW_V"} of <dS, S> through sa_forward_tokenwise,
    given its H; dX is bf16, the others fp32.  ``out`` may supply any of these buffers.  dP, dW_Q and
    dW_K are fp32-grade for the H that is given; sa_forward_tokenwise's own H is 1e-3 to 5e-3 off, and
    with it they are 4e-4 (logits of a standard deviation of 1) to 1e-2 (of 8) off the exact forward's,
    dW_V as much as H."""
    lib = load()
    off = _host_i64(offsets)
    B, n = len(off) - 1, int(off[-1])
    k, d = P.shape
    dev, f32 = X.device, torch.float32
    _need("X", X, torch.bfloat16, (n, d), dev)
    _need("P", P, f32, (k, d), dev)
    _need("W_Q", W_Q, f32, (d, d), dev)
    _need("W_K", W_K, f32, (d, d), dev)
    _need("W_V", W_V, f32, (d, d), dev)
    _need("H", H, f32, (B, k, d), dev)
    _need("dS", dS, f32, (B, k, d), dev)
    if offsets_dev is not None:
        _need("offsets_dev", offsets_dev, torch.int64, (B + 1,), dev)
    with _at(dev, stream):
        res = {}
        for name, like in (("dX", X), ("dP", P), ("dW_Q", W_Q), ("dW_K", W_K), ("dW_V", W_V)):
            t = out.get(name) if out else None
            res[name] = torch.empty_like(like) if t is None else _need(name, t, like.dtype, like.shape, dev)
        ws = _workspace(workspace, lib.sa_backward_tokenwise_workspace(B, n, k, d, SA_BF16), dev)
        offd = _dev_i64(off, dev, offsets_dev)
        st = lib.sa_backward_tokenwise(X.data_ptr(), SA_BF16, off.ctypes.data, offd.data_ptr(), B, k, d, P.data_ptr(),
                                       W_Q.data_ptr(), W_K.data_ptr(), W_V.data_ptr(), eps, H.data_ptr(), dS.data_ptr(),
                                       *(t.data_ptr() for t in res.values()), ws.data_ptr(), ws.nbytes,
                                       _raw_stream(dev, stream))
        _check("sa_backward_tokenwise", st)
    _used_on(stream, X, P, W_Q, W_K, W_V, H, dS, offsets_dev, workspace, *res.values())
    return res


def sa_forward_noalloc(X: torch.Tensor, offsets, P, W_Q, W_K, W_V, eps: float = 1e-6, *,
                       offsets_dev: torch.Tensor, out: dict, stream=None) -> dict:
    """sa_forward without a workspace, for callers that cannot allocate device
    memory: every buffer is the caller's (``out`` holds preallocated "S" and
    "mass", optionally "H", "S_bf16", "lse"; ``offsets_dev`` is a device copy of
    the offsets), and the library's fixed scratch array stands in for the
    workspace.  This wrapper allocates nothing on the device."""
    lib = load()
    _need_cuda(X, P, W_Q, W_K, W_V, offsets_dev)
    off = _host_i64(offsets)
    B = len(off) - 1
    k, d = P.shape
    o = {n: out.get(n) for n in ("S", "mass", "H", "S_bf16", "lse")}
    _need_cuda(*[t for t in o.values() if t is not None])
    st = lib.sa_forward_noalloc(_p(X), _dtype_code(X), _hp(off), _p(offsets_dev), B, k, d, _p(P),
                                _p(W_Q), _p(W_K), _p(W_V), float(eps), _p(o["S"]), _p(o["mass"]),
                                _p(o["H"]), _p(o["S_bf16"]), _p(o["lse"]), _stream(stream))
    _check("sa_forward_noalloc", st)
    return {n: t for n, t in o.items() if t is not None}


def sa_backward_workspace(B: int, n_total: int, k: int, d: int, dtype: int) -> int:
    return int(load().sa_backward_workspace(B, n_total, k, d, dtype))


def sa_backward(X: torch.Tensor, offsets, P, W_Q, W_K, W_V, eps: float, H, mass, dS,
                dmass=None, lse=None, *, offsets_dev: Optional[torch.Tensor] = None,
                out: Optional[dict] = None, workspace: Optional[torch.Tensor] = None,
                stream=None, accumulate: bool = False) -> dict:
    """Gradients {"dX", "dP", "dW_Q", "dW_K", "dW_V"} of <dS, S> + <dmass, mass>.
    With ``accumulate`` the weight gradients are added into out's dP, dW_Q, dW_K,
    dW_V (sa_backward_accumulate), e.g. one call per group of users."""
    lib = load()
    _need_cuda(X, P, W_Q, W_K, W_V, H, mass, dS, dmass, lse)
    off = _host_i64(offsets)
    B = len(off) - 1
    k, d = P.shape
    dev = X.device
    dt = _dtype_code(X)
    o = dict(out or {})
    dX = o.get("dX") if o.get("dX") is not None else torch.empty_like(X)
    dP = o.get("dP") if o.get("dP") is not None else torch.empty(k, d, device=dev)
    dWQ = o.get("dW_Q") if o.get("dW_Q") is not None else torch.empty(d, d, device=dev)
    dWK = o.get("dW_K") if o.get("dW_K") is not None else torch.empty(d, d, device=dev)
    dWV = o.get("dW_V") if o.get("dW_V") is not None else torch.empty(d, d, device=dev)
    ws_bytes = lib.sa_backward_workspace(B, int(off[-1]), k, d, dt)
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    offd = _dev_i64(off, dev, offsets_dev)
    if accumulate and any(o.get(n) is None for n in ("dP", "dW_Q", "dW_K", "dW_V")):
        raise ValueError("accumulate needs out with dP, dW_Q, dW_K and dW_V")
    fn = lib.sa_backward_accumulate if accumulate else lib.sa_backward
    st = fn(_p(X), dt, _hp(off), _p(offd), B, k, d, _p(P), _p(W_Q), _p(W_K), _p(W_V),
            float(eps), _p(H), _p(mass), _p(dS), _p(dmass), _p(lse), _p(dX), _p(dP), _p(dWQ),
            _p(dWK), _p(dWV), _p(workspace), workspace.numel(), _stream(stream))
    _check("sa_backward_accumulate" if accumulate else "sa_backward", st)
    return {"dX": dX, "dP": dP, "dW_Q": dWQ, "dW_K": dWK, "dW_V": dWV}


def stca_forward_workspace(B: int, C_total: int, D: int, heads: int, d_h: int, dtype: int) -> int:
    return int(load().stca_forward_workspace(B, C_total, D, heads, d_h, dtype))


def stca_forward(q: torch.Tensor, cand_offsets, kv: torch.Tensor, kv_begin, kv_end,
                 layers: Sequence[dict], heads: int, d_h: int, *,
                 cand_offsets_dev=None, kv_begin_dev=None, kv_end_dev=None,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """One STCA branch.  ``layers``: dicts with W_Q, W_K, W_V [heads, D, d_h] and
    W_O [heads*d_h, D] or None (fp32 CUDA tensors).  Returns out [C_total, D] fp32."""
    lib = load()
    _need_cuda(q, kv)
    dt = _dtype_code(q)
    if kv.dtype != q.dtype:
        raise TypeError("q and kv must have the same dtype")
    cand = _host_i64(cand_offsets)
    kb, ke = _host_i64(kv_begin), _host_i64(kv_end)
    B = len(cand) - 1
    D = q.shape[1]
    dev = q.device
    C = int(cand[-1])
    res = out if out is not None else torch.empty(C, D, device=dev)
    arr = (StcaLayerC * len(layers))()
    for i, L in enumerate(layers):
        _need_cuda(L["W_Q"], L["W_K"], L["W_V"], L.get("W_O"))
        arr[i].W_Q = L["W_Q"].data_ptr()
        arr[i].W_K = L["W_K"].data_ptr()
        arr[i].W_V = L["W_V"].data_ptr()
        arr[i].W_O = L["W_O"].data_ptr() if L.get("W_O") is not None else None
    ws_bytes = lib.stca_forward_workspace(B, C, D, heads, d_h, dt)
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    cd = _dev_i64(cand, dev, cand_offsets_dev)
    kbd = _dev_i64(kb, dev, kv_begin_dev)
    ked = _dev_i64(ke, dev, kv_end_dev)
    st = lib.stca_forward(_p(q), dt, _hp(cand), _p(cd), B, _p(kv), kv.shape[0], _hp(kb), _hp(ke),
                          _p(kbd), _p(ked), D, heads, d_h, len(layers), arr, _p(res),
                          _p(workspace), workspace.numel(), _stream(stream))
    _check("stca_forward", st)
    return res


def stca_forward_full_workspace(B: int, C_total: int, kv_total: int, D: int, heads: int, d_h: int,
                                dtype: int) -> int:
    return int(load().stca_forward_full_workspace(B, C_total, kv_total, D, heads, d_h, dtype))


def stca_forward_full(q: torch.Tensor, cand_offsets, kv: torch.Tensor, kv_begin, kv_end,
                      layers: Sequence[dict], heads: int, d_h: int, *,
                      cand_offsets_dev=None, kv_begin_dev=None, kv_end_dev=None,
                      out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """One STCA branch of full layers (the attention layer plus the history- and
    query-side SwiGLU FFNs).  ``layers``: dicts as for stca_forward plus, each
    optional (absent or None = no such FFN), hist_W1, hist_W3 [D, 2D], hist_W2
    [2D, D], q_W1, q_W3 [D, 2D], q_W2 [2D, D] (fp32 CUDA tensors).  Returns
    out [C_total, D] fp32."""
    lib = load()
    _need_cuda(q, kv)
    dt = _dtype_code(q)
    if kv.dtype != q.dtype:
        raise TypeError("q and kv must have the same dtype")
    cand = _host_i64(cand_offsets)
    kb, ke = _host_i64(kv_begin), _host_i64(kv_end)
    B = len(cand) - 1
    D = q.shape[1]
    dev = q.device
    C = int(cand[-1])
    kv_total = int((ke - kb).sum()) if B else 0
    res = out if out is not None else torch.empty(C, D, device=dev)
    arr = (StcaFullLayerC * len(layers))()
    for i, L in enumerate(layers):
        _need_cuda(L["W_Q"], L["W_K"], L["W_V"], L.get("W_O"), *(L.get(k) for k in STCA_FFN_KEYS))
        arr[i].attn.W_Q = L["W_Q"].data_ptr()
        arr[i].attn.W_K = L["W_K"].data_ptr()
        arr[i].attn.W_V = L["W_V"].data_ptr()
        arr[i].attn.W_O = L["W_O"].data_ptr() if L.get("W_O") is not None else None
        for k in STCA_FFN_KEYS:
            setattr(arr[i], k, L[k].data_ptr() if L.get(k) is not None else None)
    ws_bytes = lib.stca_forward_full_workspace(B, C, kv_total, D, heads, d_h, dt)
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    cd = _dev_i64(cand, dev, cand_offsets_dev)
    kbd = _dev_i64(kb, dev, kv_begin_dev)
    ked = _dev_i64(ke, dev, kv_end_dev)
    st = lib.stca_forward_full(_p(q), dt, _hp(cand), _p(cd), B, _p(kv), kv.shape[0], _hp(kb), _hp(ke),
                               _p(kbd), _p(ked), D, heads, d_h, len(layers), arr, _p(res),
                               _p(workspace), workspace.numel(), _stream(stream))
    _check("stca_forward_full", st)
    return res


def selftest_bounded_wait(budget_cycles: int = 2_000_000, stream=None) -> None:
    """Launch a kernel whose only wait cannot complete (bounded to ~budget_cycles);
    the next poll_device_status() raises SAError with SA_ERR_TIMEOUT."""
    _check("sa_selftest_bounded_wait", load().sa_selftest_bounded_wait(budget_cycles, _stream(stream)))


def selftest_unsorted_events(pairs: torch.Tensor, dX: torch.Tensor, action_ids: torch.Tensor, vocab: int,
                             n_actions: int) -> dict:
    """The sums of sa_gather_events_backward over a given list ``pairs`` [n, 2] (int32 words: item id,
    event) in place of the sort's; fp32 dX."""
    lib = load()
    n, d = dX.shape
    dev = dX.device
    _need("dX", dX, torch.float32, (n, d), dev)
    _need("pairs", pairs, torch.int32, (n, 2), dev)
    _need("action_ids", action_ids, torch.uint8, (n,), dev)
    with _at(dev, None):
        res = {"d_item": torch.empty(vocab, d, dtype=torch.float32, device=dev),
               "d_action": torch.empty(n_actions, d, dtype=torch.float32, device=dev)}
        ws = _workspace(None, lib.sa_gather_events_backward_workspace(n, vocab, n_actions, d), dev)
        st = lib.sa_selftest_unsorted_events(pairs.data_ptr(), dX.data_ptr(), action_ids.data_ptr(), n, vocab, n_actions, d,
                                             res["d_item"].data_ptr(), res["d_action"].data_ptr(), ws.data_ptr(), ws.nbytes,
                                             _raw_stream(dev, None))
        _check("sa_selftest_unsorted_events", st)
    return res


def measure_exp2_rate(mode: int = 1, stream=None) -> float:
    """Exponentials per second on the current GPU: mode 0 all on the MUFU, mode 1 the
    SA forward kernels' mix (one pair in four on the FMA pipe)."""
    out = ctypes.c_double(0.0)
    _check("sa_measure_exp2_rate", load().sa_measure_exp2_rate(mode, ctypes.byref(out), _stream(stream)))
    return out.value


def sa_gather_events(item_table: torch.Tensor, action_table: torch.Tensor, item_ids: torch.Tensor,
                     action_ids: torch.Tensor, *, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """X[i] = item_table[item_ids[i]] + action_table[action_ids[i]] (bf16 tables and
    output, int32 / uint8 ids, CUDA tensors).  Returns X [n, d] bf16."""
    lib = load()
    _need_cuda(item_table, action_table, item_ids, action_ids)
    if item_table.dtype != torch.bfloat16 or action_table.dtype != torch.bfloat16:
        raise TypeError("the tables must be bf16")
    if item_ids.dtype != torch.int32 or action_ids.dtype != torch.uint8:
        raise TypeError("item_ids must be int32 and action_ids uint8")
    n, d = item_ids.numel(), item_table.shape[1]
    X = out if out is not None else torch.empty(n, d, dtype=torch.bfloat16, device=item_table.device)
    st = lib.sa_gather_events(_p(item_table), item_table.shape[0], _p(action_table), action_table.shape[0],
                              _p(item_ids), _p(action_ids), n, d, _p(X), _stream(stream))
    _check("sa_gather_events", st)
    return X


def sa_gather_events_backward_workspace(n: int, vocab: int, n_actions: int, d: int) -> int:
    return int(load().sa_gather_events_backward_workspace(n, vocab, n_actions, d))


def sa_gather_events_backward(item_ids: torch.Tensor, action_ids: torch.Tensor, dX: torch.Tensor, vocab: int,
                              n_actions: int, *, want_item: bool = True, want_action: bool = True,
                              out: Optional[dict] = None, workspace: Optional[torch.Tensor] = None,
                              stream=None) -> dict:
    """The tables' gradients through sa_gather_events: {"d_item": [vocab, d], "d_action": [n_actions, d]},
    fp32, from dX [n, d] (bf16 or fp32).  ``out`` may supply the buffers."""
    lib = load()
    n, d = dX.shape
    dev = dX.device
    _need("dX", dX, dX.dtype, (n, d), dev)
    _need("item_ids", item_ids, torch.int32, (n,), dev)
    _need("action_ids", action_ids, torch.uint8, (n,), dev)
    with _at(dev, stream):
        res = {}
        for name, want, rows in (("d_item", want_item, vocab), ("d_action", want_action, n_actions)):
            t = out.get(name) if out else None
            if t is not None:
                res[name] = _need(name, t, torch.float32, (rows, d), dev)
            elif want:
                res[name] = torch.empty(rows, d, dtype=torch.float32, device=dev)
        ws = _workspace(workspace, lib.sa_gather_events_backward_workspace(n, vocab, n_actions, d), dev)
        item, action = res.get("d_item"), res.get("d_action")
        st = lib.sa_gather_events_backward(item_ids.data_ptr(), action_ids.data_ptr(), n, dX.data_ptr(),
                                           _dtype_code(dX), vocab, n_actions, d,
                                           None if item is None else item.data_ptr(),
                                           None if action is None else action.data_ptr(), ws.data_ptr(), ws.nbytes,
                                           _raw_stream(dev, stream))
        _check("sa_gather_events_backward", st)
    _used_on(stream, item_ids, action_ids, dX, workspace, *res.values())
    return res


def _refuse_overlaps(spans: list) -> None:
    """ValueError where memory that an AdamW step writes belongs to two arrays of its list.  ``spans``:
    (begin, end, name) of each array, an entry's gradient behind its other arrays."""
    kept, own = [], set()
    for begin, end, name in spans:
        # a gradient that is one of its entry's arrays is read there before it is written, value by value
        if name != "grad" or (begin, end) not in own:
            kept.append((begin, end, name))
        own = set() if name == "grad" else own | {(begin, end)}
    far = {True: (0, 0, ""), False: (0, 0, "")}     # a gradient or not: the span that ends furthest so far
    for span in sorted(kept):
        grad = span[2] == "grad"
        for other_grad in (True, False):
            other = far[other_grad]
            if span[0] < other[1] and not (grad and other_grad):
                raise ValueError(f"{other[2]} and {span[2]} of the list's tensors share memory: an array that the step "
                                 "writes may not be in the list twice, not even in part")
        if span[1] > far[grad][1]:
            far[grad] = span


class AdamWTensors:
    """The tensors of an AdamW step, described once for many steps.  ``tensors``: dicts with
    "param" (fp32), "grad" (fp32 or bf16), "m" and "v" (both fp32, or both float8_e4m3fn with
    "m_scale" and "v_scale", fp32, one value per ADAMW_BLOCK values), all of one size and device;
    optionally "param_bf16" (bf16, receives the rounded parameter) and "weight_decay" (default 0).
    The arrays are held by reference: a step reads and updates them in place.  No array that a step
    writes may be in the list twice or share a part of its memory with another one (two blocks of
    threads would use it at once): ValueError.  Gradients may be shared.  The addresses are taken
    here, once, and the arrays kept alive: a loop that makes new gradient tensors every step (as
    zero_grad(set_to_none=True) does) needs a new list every step, 3.5 to 4.7 us of host time a tensor;
    one that fills the same gradient buffers keeps its list."""

    def __init__(self, tensors: Sequence[dict]):
        self.tensors = [dict(t) for t in tensors]
        self.c = (AdamWTensorC * max(len(self.tensors), 1))()
        self.device = dev = self.tensors[0]["param"].device if self.tensors else None
        f32, f8 = torch.float32, torch.float8_e4m3fn
        width = {f32: 4, torch.bfloat16: 2, f8: 1}
        spans = []                                  # (begin, end, name), an entry's gradient behind its other arrays

        def at(t, name, dtype, size):
            x = t[name]
            if not (x.dtype is dtype and x.numel() == size and x.device == dev and x.is_contiguous() and x.is_cuda):
                _need(name, x if not x.is_contiguous() else x.view(-1), dtype, (size,), dev)
            begin = x.data_ptr()
            if size:
                spans.append((begin, begin + size * width[dtype], name))
            return begin

        for c, t in zip(self.c, self.tensors):
            n = t["param"].numel()
            c.n, c.weight_decay = n, t.get("weight_decay", 0.0)
            c.param = at(t, "param", f32, n)
            if t["m"].dtype is f8:
                blocks = -(-n // ADAMW_BLOCK)
                c.state, c.m, c.v = SA_STATE_8BIT, at(t, "m", f8, n), at(t, "v", f8, n)
                c.m_scale, c.v_scale = at(t, "m_scale", f32, blocks), at(t, "v_scale", f32, blocks)
            else:
                c.state, c.m, c.v = SA_STATE_F32, at(t, "m", f32, n), at(t, "v", f32, n)
            if t.get("param_bf16") is not None:
                c.param_bf16 = at(t, "param_bf16", torch.bfloat16, n)
            c.grad_dtype = _dtype_code(t["grad"])
            c.grad = at(t, "grad", t["grad"].dtype, n)
        order = sorted(spans)
        for a, b in zip(order, order[1:]):
            if a[1] > b[0]:                         # two share memory: look whether they may
                _refuse_overlaps(spans)
                break


def sa_adamw_step(tensors, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, *, step: int = 0,
                  step_dev: Optional[torch.Tensor] = None, lr_dev: Optional[torch.Tensor] = None,
                  grad_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """One AdamW step, in place, over an AdamWTensors, or a list of its dicts, which is checked and
    described anew in every call (62 tensors: 0.22 ms of host time with fp32 states and 0.29 with 8-bit
    ones, where an AdamWTensors takes 0.01).  ``step`` counts from 1; ``step_dev`` (int64), ``lr_dev``
    and ``grad_scale`` (fp32) are optional one-value CUDA tensors read when the step runs (for captured
    steps, clipping and loss scaling)."""
    lib = load()
    if not isinstance(tensors, AdamWTensors):
        tensors = AdamWTensors(tensors)
    dev = tensors.device
    if dev is None:
        return
    scalars = []
    for name, t, dt in (("step_dev", step_dev, torch.int64), ("lr_dev", lr_dev, torch.float32),
                        ("grad_scale", grad_scale, torch.float32)):
        scalars.append(None if t is None else _need(name, t.view(-1), dt, (1,), dev).data_ptr())
    cfg = AdamWConfigC(lr, beta1, beta2, eps, step, *scalars)
    with _at(dev, stream):
        status = lib.sa_adamw_step(tensors.c, len(tensors.tensors), cfg, _raw_stream(dev, stream))
    _check("sa_adamw_step", status)
    if stream is not None:                                   # hundreds of tensors: not for nothing
        _used_on(stream, step_dev, lr_dev, grad_scale, *(x for t in tensors.tensors for x in t.values()
                                                          if isinstance(x, torch.Tensor)))


def sa_gather_events_fused_workspace(n_actions: int, d: int = 128, d_ff: int = 256) -> int:
    return int(load().sa_gather_events_fused_workspace(n_actions, d, d_ff))


def sa_gather_events_fused(item_table: torch.Tensor, action_table: torch.Tensor, item_ids: torch.Tensor,
                           action_ids: torch.Tensor, W1: torch.Tensor, W3: torch.Tensor, W2: torch.Tensor, *,
                           out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """X[i] = e + (SiLU(z W1) * (z W3)) W2 with e = item_table[item_ids[i]],
    z = [e ; action_table[action_ids[i]]] (eq. (20)); bf16 tables and output,
    int32 / uint8 ids, fp32 weights W1, W3 [2d, d_ff], W2 [d_ff, d].  Returns X [n, d]."""
    lib = load()
    _need_cuda(item_table, action_table, item_ids, action_ids, W1, W3, W2)
    if item_table.dtype != torch.bfloat16 or action_table.dtype != torch.bfloat16:
        raise TypeError("the tables must be bf16")
    if item_ids.dtype != torch.int32 or action_ids.dtype != torch.uint8:
        raise TypeError("item_ids must be int32 and action_ids uint8")
    n, d = item_ids.numel(), item_table.shape[1]
    d_ff = W2.shape[0]
    na = action_table.shape[0]
    X = out if out is not None else torch.empty(n, d, dtype=torch.bfloat16, device=item_table.device)
    if workspace is None:
        workspace = torch.empty(max(sa_gather_events_fused_workspace(na, d, d_ff), 16), dtype=torch.uint8,
                                device=item_table.device)
    st = lib.sa_gather_events_fused(_p(item_table), item_table.shape[0], _p(action_table), na, _p(item_ids),
                                    _p(action_ids), n, d, _p(W1), _p(W3), _p(W2), d_ff, _p(X), _p(workspace),
                                    workspace.numel(), _stream(stream))
    _check("sa_gather_events_fused", st)
    return X


def _full_layers_c(layers):
    arr = (StcaFullLayerC * len(layers))()
    for i, L in enumerate(layers):
        _need_cuda(L["W_Q"], L["W_K"], L["W_V"], L.get("W_O"), *(L.get(k) for k in STCA_FFN_KEYS))
        arr[i].attn.W_Q = L["W_Q"].data_ptr()
        arr[i].attn.W_K = L["W_K"].data_ptr()
        arr[i].attn.W_V = L["W_V"].data_ptr()
        arr[i].attn.W_O = L["W_O"].data_ptr() if L.get("W_O") is not None else None
        for k in STCA_FFN_KEYS:
            setattr(arr[i], k, L[k].data_ptr() if L.get(k) is not None else None)
    return arr


def stca_backward_full_workspace(cand_offsets, kv_begin, kv_end, D: int, heads: int, d_h: int,
                                 n_layers: int, dtype: int) -> int:
    cand, kb, ke = _host_i64(cand_offsets), _host_i64(kv_begin), _host_i64(kv_end)
    return int(load().stca_backward_full_workspace(len(cand) - 1, _hp(cand), _hp(kb), _hp(ke), D, heads, d_h,
                                                   n_layers, dtype))


def stca_backward_full(q: torch.Tensor, cand_offsets, kv: torch.Tensor, kv_begin, kv_end,
                       layers: Sequence[dict], heads: int, d_h: int, dout: torch.Tensor, *,
                       cand_offsets_dev=None, kv_begin_dev=None, kv_end_dev=None,
                       out: Optional[dict] = None, workspace: Optional[torch.Tensor] = None,
                       stream=None) -> dict:
    """Backward of stca_forward_full.  ``dout`` [C_total, D] fp32.  Returns {"dq": [C, D],
    "dkv": [kv_rows, D], "layers": [dict of weight gradients per layer]} (fp32; the
    gradient keys are dW_Q, dW_K, dW_V, dW_O and hist_dW1.. / q_dW1.. for the FFNs that
    the layer has).  ``out`` may supply any of these buffers."""
    lib = load()
    _need_cuda(q, kv, dout)
    dt = _dtype_code(q)
    if kv.dtype != q.dtype:
        raise TypeError("q and kv must have the same dtype")
    cand = _host_i64(cand_offsets)
    kb, ke = _host_i64(kv_begin), _host_i64(kv_end)
    B = len(cand) - 1
    D = q.shape[1]
    dev = q.device
    C = int(cand[-1])
    out = dict(out or {})
    dq = out.get("dq") if out.get("dq") is not None else torch.empty(C, D, device=dev)
    dkv = out.get("dkv") if out.get("dkv") is not None else torch.empty(kv.shape[0], D, device=dev)
    lg_out = out.get("layers") or [{} for _ in layers]
    grads = []
    garr = (StcaFullLayerGradC * len(layers))()
    for i, L in enumerate(layers):
        g = {}
        have = {"dW_Q": "W_Q", "dW_K": "W_K", "dW_V": "W_V", "dW_O": "W_O", "hist_dW1": "hist_W1",
                "hist_dW3": "hist_W3", "hist_dW2": "hist_W2", "q_dW1": "q_W1", "q_dW3": "q_W3", "q_dW2": "q_W2"}
        for gk, wk in have.items():
            if L.get(wk) is None:
                continue
            buf = lg_out[i].get(gk) if lg_out[i].get(gk) is not None else torch.empty_like(L[wk])
            _need_cuda(buf)
            g[gk] = buf
            setattr(garr[i], gk, buf.data_ptr())
        grads.append(g)
    arr = _full_layers_c(layers)
    ws_bytes = lib.stca_backward_full_workspace(B, _hp(cand), _hp(kb), _hp(ke), D, heads, d_h, len(layers), dt)
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    cd = _dev_i64(cand, dev, cand_offsets_dev)
    kbd = _dev_i64(kb, dev, kv_begin_dev)
    ked = _dev_i64(ke, dev, kv_end_dev)
    st = lib.stca_backward_full(_p(q), dt, _hp(cand), _p(cd), B, _p(kv), kv.shape[0], _hp(kb), _hp(ke),
                                _p(kbd), _p(ked), D, heads, d_h, len(layers), arr, _p(dout), _p(dq), _p(dkv),
                                garr, _p(workspace), workspace.numel(), _stream(stream))
    _check("stca_backward_full", st)
    return {"dq": dq, "dkv": dkv, "layers": grads}


REFINE_KEYS = ("W_Q", "W_K", "ln1_g", "ln1_b", "W1", "W3", "W2", "ln2_g", "ln2_b")


def sa_refine_workspace(B: int, n_total: int, k: int, d: int, x_dtype: int) -> int:
    return int(load().sa_refine_workspace(B, n_total, k, d, x_dtype))


def sa_refine_forward(X: torch.Tensor, offsets, P0: torch.Tensor, layers: Sequence[dict],
                      ln_eps: float = 1e-5, *, offsets_dev=None, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Stacked SA refinement, len(layers) iterations from the shared prototypes P0
    [k, d].  ``layers``: dicts with W_Q, W_K [d, d], W1, W3 [d, 2d], W2 [2d, d] and
    optional ln1_g, ln1_b, ln2_g, ln2_b [d] (fp32 CUDA tensors).  Returns the
    sketch [B, k, d] fp32."""
    lib = load()
    _need_cuda(X, P0)
    dt = _dtype_code(X)
    off = _host_i64(offsets)
    B = len(off) - 1
    k, d = P0.shape
    dev = X.device
    res = out if out is not None else torch.empty(B, k, d, device=dev)
    arr = (RefineLayerC * len(layers))()
    for i, L in enumerate(layers):
        for key in REFINE_KEYS:
            t = L.get(key)
            _need_cuda(t)
            setattr(arr[i], key, t.data_ptr() if t is not None else None)
    ws_bytes = lib.sa_refine_workspace(B, int(off[-1]), k, d, dt)
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    od = _dev_i64(off, dev, offsets_dev)
    st = lib.sa_refine_forward(_p(X), dt, _hp(off), _p(od), B, k, d, _p(P0), len(layers), arr,
                               ln_eps, _p(res), _p(workspace), workspace.numel(), _stream(stream))
    _check("sa_refine_forward", st)
    return res


def sa_refine_backward_workspace(B: int, n_total: int, k: int, d: int, n_iter: int, dtype: int) -> int:
    return int(load().sa_refine_backward_workspace(B, n_total, k, d, n_iter, dtype))


def sa_refine_backward(X: torch.Tensor, offsets, P0: torch.Tensor, layers: Sequence[dict], dsketch: torch.Tensor,
                       ln_eps: float = 1e-5, *, offsets_dev=None, out: Optional[dict] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of <dsketch, sa_refine_forward(X, offsets, P0, layers)>: returns
    {"dX": [n, d] fp32, "dP0": [k, d] fp32, "layers": [{"dW_Q", "dW_K", "dW1", "dW3", "dW2",
    and "dln1_g", ... for the LayerNorm parameters the layer has}]}."""
    lib = load()
    _need_cuda(X, P0, dsketch)
    dt = _dtype_code(X)
    off = _host_i64(offsets)
    B = len(off) - 1
    k, d = P0.shape
    n = int(off[-1])
    dev = X.device
    o = dict(out or {})
    dX = o.get("dX") if o.get("dX") is not None else torch.empty(max(n, 1), d, device=dev)
    dP0 = o.get("dP0") if o.get("dP0") is not None else torch.empty(k, d, device=dev)
    arr = (RefineLayerC * len(layers))()
    garr = (RefineLayerGradC * len(layers))()
    gl = []
    for i, L in enumerate(layers):
        g = {}
        for key in REFINE_KEYS:
            t = L.get(key)
            _need_cuda(t)
            setattr(arr[i], key, t.data_ptr() if t is not None else None)
            if t is not None:
                g["d" + key] = torch.empty_like(t)
                setattr(garr[i], "d" + key, g["d" + key].data_ptr())
        gl.append(g)
    ws_bytes = lib.sa_refine_backward_workspace(B, n, k, d, len(layers), dt)
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    od = _dev_i64(off, dev, offsets_dev)
    st = lib.sa_refine_backward(_p(X), dt, _hp(off), _p(od), B, k, d, _p(P0), len(layers), arr, ln_eps,
                                _p(dsketch), _p(dX), _p(dP0), garr, _p(workspace), workspace.numel(),
                                _stream(stream))
    _check("sa_refine_backward", st)
    return {"dX": dX[:n], "dP0": dP0, "layers": gl}


def stca_fuse(z_r: torch.Tensor, z_u: torch.Tensor, W_F: torch.Tensor, b_F=None, *,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """[z_r ; z_u] W_F + b_F."""
    lib = load()
    _need_cuda(z_r, z_u, W_F, b_F)
    C, D = z_r.shape
    res = out if out is not None else torch.empty(C, D, device=z_r.device)
    st = lib.stca_fuse(_p(z_r), _p(z_u), _p(W_F), _p(b_F), C, D, _p(res), _stream(stream))
    _check("stca_fuse", st)
    return res


def poll_device_status(stream=None) -> None:
    _check("sa_poll_device_status", load().sa_poll_device_status(_stream(stream)))


# --------------------------------------------------------------------------
# measurement support
def launch_count() -> int:
    """Kernels the library has launched in this process."""
    return int(load().sa_launch_count())


def profile(enable: bool) -> None:
    """Start (clearing) or stop the library's per-kernel event timers."""
    load().sa_profile(1 if enable else 0)


def profile_read() -> dict:
    """{kernel name: (total device ms, launches)} since profile(True)."""
    lib = load()
    out = {}
    buf = ctypes.create_string_buffer(128)
    ms, cnt = ctypes.c_double(), ctypes.c_longlong()
    i = 0
    while lib.sa_profile_read(i, buf, 128, ctypes.byref(ms), ctypes.byref(cnt)):
        out[buf.value.decode()] = (ms.value, cnt.value)
        i += 1
    return out
