"""Python binding of the MI355X (gfx950) rotated W4G128 linear library.

Thin ctypes marshalling over ``libparo.so`` (C ABI in ``include/paro.h``):
torch tensors are passed as device pointers plus the current HIP stream, and
every step of the hot path runs in the library's HIP kernels. There is no
fallback: if the library is missing or no GPU is visible the calls raise.

Names follow the C ABI: ``paro_device_init``, ``paro_rotation_create`` / ``Rotation``,
``paro_rotate``, ``paro_quantize_weights``, ``paro_w4_linear``,
``paro_w4_linear_workspace_size``, ``paro_w4_linear_noalloc``, ``paro_rotation_backward``,
``paro_rotation_backward_workspace_size``, ``paro_layer_loss``,
``paro_layer_loss_workspace_size``, ``paro_w4_linear_act``, ``paro_w4_gated``, their
``..._backward``, ``paro_experts_route`` / ``paro_experts_sort`` / ``Routing``,
``paro_w4_experts_gated``, ``paro_w4_experts_combine``, their ``..._backward``,
``paro_distill_loss``, ``paro_adamw_create`` / ``AdamW``, ``paro_pairs_random``,
``paro_pairs_by_gap``, ``paro_sparsify_angles``.

``stream``: calls that take one run on it (on the current stream without). What
they allocate then belongs to that stream. The caller orders it behind the work
that makes the inputs, and keeps the inputs until it has passed.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Tuple

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libparo.so")

PARO_OK = 0
STATUS = {
    0: "PARO_OK", -1: "PARO_ERR_NULL", -2: "PARO_ERR_SHAPE", -3: "PARO_ERR_PAIRING",
    -4: "PARO_ERR_VALUE", -5: "PARO_ERR_ALIGN", -6: "PARO_ERR_UNSUPPORTED",
    -7: "PARO_ERR_WORKSPACE", -8: "PARO_ERR_HIP",
}

_lib = None


class ParoError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class _Routing(ctypes.Structure):
    """``paro_routing``"""
    _fields_ = [("M", ctypes.c_int64), ("E", ctypes.c_int32), ("k", ctypes.c_int32)] + [
        (name, ctypes.c_void_p) for name in ("ids", "offsets", "order", "place", "weights")]


def load_library() -> ctypes.CDLL:
    """Load libparo.so (built by ``rotated_w4_linear_amd.build``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m rotated_w4_linear_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    c_f64 = ctypes.c_double
    c_i64, c_i32, vp, c_size = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t
    lib.paro_status_string.restype = ctypes.c_char_p
    lib.paro_status_string.argtypes = [ctypes.c_int]
    lib.paro_last_error.restype = ctypes.c_char_p
    lib.paro_last_error.argtypes = []
    lib.paro_device_init.restype = ctypes.c_int
    lib.paro_device_init.argtypes = []
    lib.paro_rotation_create.restype = ctypes.c_int
    lib.paro_rotation_create.argtypes = [c_i64, c_i32, c_i32, vp, vp, vp, ctypes.POINTER(vp)]
    lib.paro_rotation_destroy.restype = None
    lib.paro_rotation_destroy.argtypes = [vp]
    lib.paro_rotation_info.restype = ctypes.c_int
    lib.paro_rotation_info.argtypes = [vp, ctypes.POINTER(c_i64), ctypes.POINTER(c_i32),
                                       ctypes.POINTER(c_i32)]
    lib.paro_rotate.restype = ctypes.c_int
    lib.paro_rotate.argtypes = [vp, vp, vp, c_i64, vp]
    lib.paro_quantize_weights.restype = ctypes.c_int
    lib.paro_quantize_weights.argtypes = [vp, vp, c_i64, c_i64, c_i32, vp, vp, vp, vp]
    lib.paro_w4_linear_workspace_size.restype = c_size
    lib.paro_w4_linear_workspace_size.argtypes = [vp, c_i64, c_i64, c_i64]
    lib.paro_w4_linear.restype = ctypes.c_int
    lib.paro_w4_linear.argtypes = [vp, vp, vp, vp, vp, vp, vp, c_i64, c_i64, c_i64, c_i32, vp,
                                   c_size, vp]
    lib.paro_w4_linear_noalloc.restype = ctypes.c_int
    lib.paro_w4_linear_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, c_i64, c_i64, c_i64, c_i32,
                                           vp]
    lib.paro_rotation_backward_workspace_size.restype = c_size
    lib.paro_rotation_backward_workspace_size.argtypes = [vp, c_i64]
    lib.paro_rotation_backward.restype = ctypes.c_int
    lib.paro_rotation_backward.argtypes = [vp, c_i32, vp, vp, vp, vp, vp, c_i64, vp, c_size, vp]
    lib.paro_layer_loss_workspace_size.restype = c_size
    lib.paro_layer_loss_workspace_size.argtypes = [vp, c_i64, c_i64, c_i64, c_i32]
    lib.paro_layer_loss.restype = ctypes.c_int
    lib.paro_layer_loss.argtypes = [vp, vp, vp, vp, vp, vp, c_i64, c_i64, c_i64, c_i32, vp, vp, vp,
                                    vp, c_size, vp]
    lib.paro_w4_linear_act.restype = ctypes.c_int
    lib.paro_w4_linear_act.argtypes = [vp, vp, vp, vp, vp, vp, vp, c_i32, vp, c_i64, c_i64, c_i64, c_i32, vp,
                                       c_size, vp]
    lib.paro_w4_gated_workspace_size.restype = c_size
    lib.paro_w4_gated_workspace_size.argtypes = [vp, c_i64, c_i64, c_i64]
    lib.paro_w4_gated.restype = ctypes.c_int
    lib.paro_w4_gated.argtypes = [vp, vp, vp, vp, vp, vp, c_i32, vp, c_i64, c_i64, c_i64, c_i32, vp, c_size, vp]
    lib.paro_w4_linear_act_backward_workspace_size.restype = c_size
    lib.paro_w4_linear_act_backward_workspace_size.argtypes = [c_i64, c_i64, c_i64, c_i32]
    lib.paro_w4_gated_backward_workspace_size.restype = c_size
    lib.paro_w4_gated_backward_workspace_size.argtypes = [c_i64, c_i64, c_i64]
    for fn in (lib.paro_w4_linear_act_backward, lib.paro_w4_gated_backward):
        fn.restype = ctypes.c_int
        fn.argtypes = [vp, vp, vp, vp, vp, c_i32, vp, vp, vp, c_i64, c_i64, c_i64, c_i32, vp, c_size, vp]
    rt = ctypes.POINTER(_Routing)
    lib.paro_experts_route_workspace_size.restype = c_size
    lib.paro_experts_route_workspace_size.argtypes = [c_i64, c_i32, c_i32]
    lib.paro_experts_route.restype = ctypes.c_int
    lib.paro_experts_route.argtypes = [vp, c_i32, c_i64, c_i32, c_i32, c_i32, vp, vp, vp, vp, vp, vp, c_size, vp]
    lib.paro_experts_sort.restype = ctypes.c_int
    lib.paro_experts_sort.argtypes = [vp, c_i64, c_i32, c_i32, vp, vp, vp, vp, c_size, vp]
    lib.paro_experts_route_backward.restype = ctypes.c_int
    lib.paro_experts_route_backward.argtypes = [vp, c_i32, c_i64, c_i32, c_i32, c_i32, vp, vp, vp, vp, vp]
    for name in ("gated", "combine", "gated_backward", "combine_backward"):
        size = getattr(lib, f"paro_w4_experts_{name}_workspace_size")
        size.restype = c_size
        size.argtypes = [c_i64, c_i32, c_i32, c_i64, c_i64]
    lib.paro_w4_experts_gated.restype = ctypes.c_int
    lib.paro_w4_experts_gated.argtypes = [rt, vp, vp, vp, vp, vp, c_i32, vp, c_i64, c_i64, c_i32, vp, c_size, vp]
    lib.paro_w4_experts_combine.restype = ctypes.c_int
    lib.paro_w4_experts_combine.argtypes = [rt, vp, vp, vp, vp, vp, vp, vp, c_i64, c_i64, c_i32, vp, c_size, vp]
    lib.paro_w4_experts_gated_backward.restype = ctypes.c_int
    lib.paro_w4_experts_gated_backward.argtypes = [rt, vp, vp, vp, vp, vp, c_i32, vp, vp, vp, c_i64, c_i64, c_i32, vp,
                                                   c_size, vp]
    lib.paro_w4_experts_combine_backward.restype = ctypes.c_int
    lib.paro_w4_experts_combine_backward.argtypes = [rt, vp, vp, vp, vp, vp, vp, vp, vp, c_i64, c_i64, c_i32, vp,
                                                     c_size, vp]
    lib.paro_distill_loss.restype = ctypes.c_int
    lib.paro_distill_loss.argtypes = [vp, c_i32, vp, c_i32, vp, vp, vp, c_i64, c_i64, c_i64, c_f64, c_f64, vp, vp, vp]
    lib.paro_adamw_moments.restype = c_i64
    lib.paro_adamw_moments.argtypes = [c_i32, vp]
    lib.paro_adamw_create.restype = ctypes.c_int
    lib.paro_adamw_create.argtypes = [c_i32, vp, vp, c_i32, vp, c_i32, c_i32, vp, vp, vp, vp, ctypes.POINTER(vp)]
    lib.paro_adamw_destroy.restype = None
    lib.paro_adamw_destroy.argtypes = [vp]
    lib.paro_adamw_step.restype = ctypes.c_int
    lib.paro_adamw_step.argtypes = [vp, c_i64, c_f64, c_f64, c_f64, c_f64, c_f64, vp]
    lib.paro_pairs_random.restype = ctypes.c_int
    lib.paro_pairs_random.argtypes = [c_i64, c_i32, c_i32, ctypes.c_uint64, vp]
    lib.paro_pairs_by_gap.restype = ctypes.c_int
    lib.paro_pairs_by_gap.argtypes = [c_i64, c_i32, c_i32, vp, vp]
    lib.paro_sparsify_angles.restype = ctypes.c_int
    lib.paro_sparsify_angles.argtypes = [c_i64, c_i32, vp, c_i64, vp]
    lib.paro_stream_copy.restype = ctypes.c_int
    lib.paro_stream_copy.argtypes = [vp, vp, c_size, c_i32, vp]
    lib.paro_mfma_loop.restype = ctypes.c_int
    lib.paro_mfma_loop.argtypes = [vp, c_i64, vp, c_i32, c_i32, vp]
    lib.paro_rotation_plan_host.restype = ctypes.c_int
    lib.paro_rotation_plan_host.argtypes = [c_i64, c_i32, c_i32, vp, vp, vp, vp, c_size,
                                            ctypes.POINTER(c_size), ctypes.POINTER(c_i32)]
    _lib = lib
    return lib


def _check(status: int):
    if status != PARO_OK:
        raise ParoError(status, load_library().paro_last_error().decode())


def _host_arrays(pairs, theta, alpha):
    pairs = np.ascontiguousarray(np.asarray(pairs, dtype=np.int32))
    theta = np.ascontiguousarray(np.asarray(theta, dtype=np.float32))
    alpha = np.ascontiguousarray(np.asarray(alpha, dtype=np.float32))
    return pairs, theta, alpha


def _ptr(a: np.ndarray):
    return a.ctypes.data_as(ctypes.c_void_p) if a.size else None


def _stream(stream=None):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


_HERE = contextlib.nullcontext()


def _made_on(stream):
    """Context of a call's allocations. They are filled, used and, once freed, used
    again in the order of the stream that they are made on: the call's own."""
    if stream is None:
        return _HERE
    import torch
    _same_device(stream, torch.cuda.current_device())
    return torch.cuda.stream(stream)


def _same_device(stream, device):
    if stream.device_index != device:
        raise ValueError("stream must belong to the current device")


def _handed_out(stream, *tensors):
    """Tensors that a call on ``stream`` made and returns: the caller may use them on
    the current stream as well, so they are not used again before it has passed."""
    if stream is None:
        return
    import torch
    current = torch.cuda.current_stream()
    if current != stream:
        for t in tensors:
            if t is not None and t.is_cuda:
                t.record_stream(current)


def _given(t, name, shape, device, made):
    """The fp32 output ``t``, of this shape, or a new one (noted in ``made``)."""
    if t is None:
        import torch
        t = torch.empty(shape, dtype=torch.float32, device=device)
        made.append(t)
    elif tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    return t


def _dptr(t, name, dtype=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a ROCm device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def paro_device_init():
    """Per-device set-up of the current device (``paro_device_init``)."""
    _check(load_library().paro_device_init())


class Rotation:
    """``paro_rotation_create`` / ``paro_rotation_destroy`` for one layer's (pairs, theta, alpha)."""

    def __init__(self, pairs, theta, alpha, group: int):
        lib = load_library()
        pairs, theta, alpha = _host_arrays(pairs, theta, alpha)
        self.d = int(alpha.shape[0])
        self.K = int(pairs.shape[0]) if pairs.ndim == 3 else 0
        self.group = int(group)
        h = ctypes.c_void_p()
        _check(lib.paro_rotation_create(self.d, self.group, self.K, _ptr(pairs), _ptr(theta),
                                        _ptr(alpha), ctypes.byref(h)))
        self._h = h

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            load_library().paro_rotation_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


paro_rotation_create = Rotation


def _handle(r: Optional[Rotation]):
    return r.handle if r is not None else None


def paro_rotate(r: Rotation, x, y=None, stream=None):
    """X' = X T^-1 row by row (fp16 [M][d] -> fp16 [M][d]); ``y`` may be ``x``."""
    import torch
    if y is None:
        with _made_on(stream):
            y = torch.empty_like(x)
        _handed_out(stream, y)
    _check(load_library().paro_rotate(r.handle, _dptr(x, "x", torch.float16),
                                      _dptr(y, "y", torch.float16), int(x.shape[0]),
                                      _stream(stream)))
    return y


def paro_quantize_weights(r: Optional[Rotation], w, group: int = 128, stream=None):
    """Q(T W) (or Q(W) when ``r`` is None): returns (qweight u8 [N][d/2], scales fp16, zeros u8)."""
    import torch
    N, d = w.shape
    with _made_on(stream):
        qweight = torch.empty((N, d // 2), dtype=torch.uint8, device=w.device)
        scales = torch.empty((N, d // group), dtype=torch.float16, device=w.device)
        zeros = torch.empty((N, d // group), dtype=torch.uint8, device=w.device)
    _handed_out(stream, qweight, scales, zeros)
    _check(load_library().paro_quantize_weights(
        _handle(r), _dptr(w, "w", torch.float16), N, d, group, _dptr(qweight, "qweight"),
        _dptr(scales, "scales"), _dptr(zeros, "zeros"), _stream(stream)))
    return qweight, scales, zeros


def paro_w4_linear_workspace_size(r: Optional[Rotation], M: int, N: int, d: int) -> int:
    return int(load_library().paro_w4_linear_workspace_size(_handle(r), M, N, d))


def new_workspace(r: Optional[Rotation], M: int, N: int, d: int, device="cuda"):
    """A zero-filled workspace for paro_w4_linear (None when none is needed)."""
    import torch
    need = paro_w4_linear_workspace_size(r, M, N, d)
    return torch.zeros(need, dtype=torch.uint8, device=device) if need else None


def paro_w4_linear(r: Optional[Rotation], x, qweight, scales, zeros, bias=None, y=None,
                   group: int = 128, workspace=None, stream=None):
    """Y = rot(X) dequant(W)^T + b (fp16 [M][N]); rot is the identity when ``r`` is None."""
    import torch
    M, d = x.shape
    N = qweight.shape[0]
    made = []
    with _made_on(stream):
        if y is None:
            y = torch.empty((M, N), dtype=torch.float16, device=x.device)
            made.append(y)
        if workspace is None:
            workspace = new_workspace(r, M, N, d, x.device)
    _handed_out(stream, *made)
    ws_ptr = _dptr(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load_library().paro_w4_linear(
        _handle(r), _dptr(x, "x", torch.float16), _dptr(qweight, "qweight", torch.uint8),
        _dptr(scales, "scales", torch.float16), _dptr(zeros, "zeros", torch.uint8),
        _dptr(bias, "bias", torch.float16) if bias is not None else None,
        _dptr(y, "y", torch.float16), M, N, d, group, ws_ptr, ws_bytes, _stream(stream)))
    return y


def paro_w4_linear_noalloc(r: Optional[Rotation], x, qweight, scales, zeros, y, bias=None,
                           group: int = 128, stream=None):
    """``paro_w4_linear`` on the library's static scratch: ``y`` (fp16 [M][N])
    is written in place and nothing is allocated."""
    import torch
    M, d = x.shape
    N = qweight.shape[0]
    _check(load_library().paro_w4_linear_noalloc(
        _handle(r), _dptr(x, "x", torch.float16), _dptr(qweight, "qweight", torch.uint8),
        _dptr(scales, "scales", torch.float16), _dptr(zeros, "zeros", torch.uint8),
        _dptr(bias, "bias", torch.float16) if bias is not None else None,
        _dptr(y, "y", torch.float16), M, N, d, group, _stream(stream)))
    return y


SIDES = {"activation": 0, "weight": 1}


def paro_rotation_backward_workspace_size(r: Rotation, M: int) -> int:
    return int(load_library().paro_rotation_backward_workspace_size(r.handle, M))


def paro_rotation_backward(r: Rotation, x, gy, side: str = "activation", gx=None,
                           want_gx: bool = True, workspace=None, stream=None, dtheta=None, dalpha=None):
    """Gradients of the transform: returns (gx fp32 [M][d] or None, dtheta fp32
    [K][d/2], dalpha fp32 [d]) for x fp16 [M][d] and gy = dL/d(output) fp32.
    ``gx``, ``dtheta``, ``dalpha`` that are given are overwritten: an ``AdamW``
    reads its gradients where they were when it was made."""
    import torch
    M, d = x.shape
    info_K = r.K
    made = []
    with _made_on(stream):
        if gx is None and want_gx:
            gx = torch.empty((M, d), dtype=torch.float32, device=x.device)
            made.append(gx)
        dtheta = _given(dtheta, "dtheta", (info_K, d // 2), x.device, made)
        dalpha = _given(dalpha, "dalpha", (d,), x.device, made)
        if workspace is None:
            need = paro_rotation_backward_workspace_size(r, M)
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
    _handed_out(stream, *made)
    ws_ptr = _dptr(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load_library().paro_rotation_backward(
        r.handle, SIDES[side], _dptr(x, "x", torch.float16), _dptr(gy, "gy", torch.float32),
        _dptr(gx, "gx", torch.float32) if gx is not None else None,
        _dptr(dtheta, "dtheta", torch.float32) if info_K else None,
        _dptr(dalpha, "dalpha", torch.float32), M, ws_ptr, ws_bytes, _stream(stream)))
    return gx, dtheta, dalpha


def paro_layer_loss(r: Rotation, x, w, qweight, scales, zeros, gradients: bool = True,
                    workspace=None, stream=None, loss=None, dtheta=None, dalpha=None):
    """Layer-wise output loss sum (Y_q - X W^T)^2 (fp32 device scalar) and, with
    ``gradients``, its straight-through dtheta [K][d/2] and dalpha [d]. ``loss``
    [1], ``dtheta``, ``dalpha`` that are given are overwritten: an ``AdamW`` reads
    its gradients where they were when it was made."""
    import torch
    M, d = x.shape
    N = w.shape[0]
    dev_ = x.device
    made = []
    with _made_on(stream):
        loss = _given(loss, "loss", (1,), dev_, made)
        dth = _given(dtheta, "dtheta", (r.K, d // 2), dev_, made) if gradients else None
        dal = _given(dalpha, "dalpha", (d,), dev_, made) if gradients else None
        if workspace is None:
            need = int(load_library().paro_layer_loss_workspace_size(r.handle, M, N, d, int(gradients)))
            workspace = torch.zeros(need, dtype=torch.uint8, device=dev_) if need else None
    _handed_out(stream, *made)
    ws_ptr = _dptr(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load_library().paro_layer_loss(
        r.handle, _dptr(x, "x", torch.float16), _dptr(w, "w", torch.float16),
        _dptr(qweight, "qweight", torch.uint8), _dptr(scales, "scales", torch.float16),
        _dptr(zeros, "zeros", torch.uint8), M, N, d, r.group, _dptr(loss, "loss", torch.float32),
        _dptr(dth, "dtheta", torch.float32) if (gradients and r.K) else None,
        _dptr(dal, "dalpha", torch.float32) if gradients else None, ws_ptr, ws_bytes,
        _stream(stream)))
    return loss, dth, dal


_COUNTERS = 16384  # bytes of the arrival counters that a workspace starts with
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}


def _act(act: str) -> int:
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def _expect(t, name, shape, dtype, device):
    """Address of a contiguous tensor of this shape and type on this device (None: NULL)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    _dptr(t, name, dtype)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be on the current device")


def _raw_stream(stream, device):
    """Handle of ``stream``, or of the device's current stream."""
    if stream is not None:
        _same_device(stream, device)
        return stream.cuda_stream
    import torch
    return torch._C._cuda_getCurrentRawStream(device)


def _workspace(workspace, need, device, current=None):
    """(workspace, its address, its bytes); a zero-filled one of ``need`` bytes where none is given.
    One that is given has to be on the ``current`` device."""
    import torch
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = torch.zeros(need, dtype=torch.uint8, device=device)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor")
    if current is not None and workspace.get_device() != current:
        raise ValueError("workspace must be on the current device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def paro_w4_linear_act(r: Optional[Rotation], x, qweight, scales, zeros, bias=None, residual=None,
                       act: str = "none", y=None, group: int = 128, workspace=None, stream=None):
    """Y = act(rot(X) dequant(W)^T + b) + residual (fp16 [M][N]); ``y`` may be ``residual``.
    The workspace is paro_w4_linear's (``new_workspace``); without a plan 16 KiB do up to 64 tokens."""
    import torch
    M, d = x.shape
    N = qweight.shape[0]
    need = 0
    if workspace is None:
        need = _COUNTERS if r is None and 0 < M <= 64 else paro_w4_linear_workspace_size(r, M, N, d)
    dev, f16, u8 = torch.cuda.current_device(), torch.float16, torch.uint8
    given = y is not None
    with _made_on(stream):
        workspace, ws_ptr, ws_bytes = _workspace(workspace, need, x.device, dev)
        if not given:
            y = x.new_empty((M, N))  # fp16 on dev as x has to be
    if given:
        y_ptr = _expect(y, "y", (M, N), f16, dev)
    else:
        y_ptr = y.data_ptr()
        _handed_out(stream, y)
    _check(load_library().paro_w4_linear_act(
        _handle(r), _expect(x, "x", (M, d), f16, dev), _expect(qweight, "qweight", (N, d // 2), u8, dev),
        _expect(scales, "scales", (N, d // group), f16, dev), _expect(zeros, "zeros", (N, d // group), u8, dev),
        _expect(bias, "bias", (N,), f16, dev), _expect(residual, "residual", (M, N), f16, dev), _act(act),
        y_ptr, M, N, d, group, ws_ptr, ws_bytes, _raw_stream(stream, dev)))
    return y


def paro_w4_gated_workspace_size(r: Optional[Rotation], M: int, N: int, d: int) -> int:
    return int(load_library().paro_w4_gated_workspace_size(_handle(r), M, N, d))


def new_gated_workspace(r: Optional[Rotation], M: int, N: int, d: int, device="cuda"):
    """A zero-filled workspace for paro_w4_gated (None when none is needed)."""
    return _workspace(None, paro_w4_gated_workspace_size(r, M, N, d), device)[0]


def paro_w4_gated(r: Optional[Rotation], x, qweight, scales, zeros, bias=None, act: str = "silu", y=None,
                  group: int = 128, workspace=None, stream=None):
    """Y = act(rot(X) Wg^T + bg) * (rot(X) Wu^T + bu) (fp16 [M][N]) on a weight block of 2 N rows
    (gate, then up: quantize the two weights concatenated along their rows)."""
    import torch
    M, d = x.shape
    N = qweight.shape[0] // 2
    need = 0
    if workspace is None:
        need = _COUNTERS if r is None and 0 < M <= 64 else paro_w4_gated_workspace_size(r, M, N, d)
    dev, f16, u8 = torch.cuda.current_device(), torch.float16, torch.uint8
    given = y is not None
    with _made_on(stream):
        workspace, ws_ptr, ws_bytes = _workspace(workspace, need, x.device, dev)
        if not given:
            y = x.new_empty((M, N))  # fp16 on dev as x has to be
    if given:
        y_ptr = _expect(y, "y", (M, N), f16, dev)
    else:
        y_ptr = y.data_ptr()
        _handed_out(stream, y)
    _check(load_library().paro_w4_gated(
        _handle(r), _expect(x, "x", (M, d), f16, dev), _expect(qweight, "qweight", (2 * N, d // 2), u8, dev),
        _expect(scales, "scales", (2 * N, d // group), f16, dev),
        _expect(zeros, "zeros", (2 * N, d // group), u8, dev), _expect(bias, "bias", (2 * N,), f16, dev), _act(act),
        y_ptr, M, N, d, group, ws_ptr, ws_bytes, _raw_stream(stream, dev)))
    return y


def new_linear_act_backward_workspace(M: int, N: int, d: int, act: str = "none", device="cuda"):
    """A zero-filled workspace for paro_w4_linear_act_backward (None when none is needed)."""
    need = int(load_library().paro_w4_linear_act_backward_workspace_size(M, N, d, _act(act)))
    return _workspace(None, need, device)[0]


def new_gated_backward_workspace(M: int, N: int, d: int, device="cuda"):
    """A zero-filled workspace for paro_w4_gated_backward (None when none is needed)."""
    return _workspace(None, int(load_library().paro_w4_gated_backward_workspace_size(M, N, d)), device)[0]


def _backward(fn, new_workspace_, rows, cols, computes, x, qweight, scales, zeros, dy, bias, act, dz, dx, want_dx,
              group, workspace, stream):
    import torch
    M, N = dy.shape
    d = 2 * qweight.shape[1]
    dev, f16, u8 = torch.cuda.current_device(), torch.float16, torch.uint8
    made = []
    with _made_on(stream):
        if dz is None and computes:
            dz = torch.empty((M, cols), dtype=torch.float16, device=dy.device)
            made.append(dz)
        if dx is None and want_dx:
            dx = torch.empty((M, d), dtype=torch.float16, device=dy.device)
            made.append(dx)
        workspace, ws_ptr, ws_bytes = _workspace(new_workspace_() if workspace is None else workspace, 0, dy.device, dev)
    _handed_out(stream, *made)
    _check(fn(_expect(x, "x", (M, d), f16, dev), _expect(qweight, "qweight", (rows, d // 2), u8, dev),
              _expect(scales, "scales", (rows, d // group), f16, dev),
              _expect(zeros, "zeros", (rows, d // group), u8, dev), _expect(bias, "bias", (rows,), f16, dev),
              _act(act), _expect(dy, "dy", (M, N), f16, dev), _expect(dz, "dz", (M, cols), f16, dev),
              _expect(dx, "dx", (M, d), f16, dev), M, N, d, group, ws_ptr, ws_bytes, _raw_stream(stream, dev)))
    return dx, dz


def paro_w4_linear_act_backward(x, qweight, scales, zeros, dy, bias=None, act: str = "none", dz=None, dx=None,
                                want_dx: bool = True, group: int = 128, workspace=None, stream=None):
    """Gradients of paro_w4_linear_act for the transformed activations ``x`` (X'; may be None without
    activation) and dy = dL/dY: returns (dx fp16 [M][d] or None, dz fp16 [M][N]; without activation, where dZ
    is dy, a copy of dy if ``dz`` is given, else None)."""
    M, N = dy.shape
    return _backward(load_library().paro_w4_linear_act_backward,
                     lambda: new_linear_act_backward_workspace(M, N, 2 * qweight.shape[1], act, dy.device), N, N,
                     act != "none", x, qweight, scales, zeros, dy, bias, act, dz, dx, want_dx, group, workspace,
                     stream)


def paro_w4_gated_backward(x, qweight, scales, zeros, dy, bias=None, act: str = "silu", dz=None, dx=None,
                           want_dx: bool = True, group: int = 128, workspace=None, stream=None):
    """Gradients of paro_w4_gated for the transformed activations ``x`` (X') and dy = dL/dY: returns
    (dx fp16 [M][d] or None, dz fp16 [M][2N]: the gate's columns, then the up projection's)."""
    M, N = dy.shape
    return _backward(load_library().paro_w4_gated_backward,
                     lambda: new_gated_backward_workspace(M, N, 2 * qweight.shape[1], dy.device), 2 * N, 2 * N,
                     True, x, qweight, scales, zeros, dy, bias, act, dz, dx, want_dx, group, workspace, stream)


_TYPES = {}


def _type(t, name) -> int:
    """paro_type of a tensor."""
    if not _TYPES:
        import torch
        _TYPES.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
    if t.dtype not in _TYPES:
        raise TypeError(f"{name} must be fp32, fp16 or bf16, got {t.dtype}")
    return _TYPES[t.dtype]


class Routing:
    """Which experts every token goes to, and the tables that the experts' products read
    (``paro_routing``): ``ids`` int32 and ``weights`` fp32 [M][k], ``offsets`` int32 [E + 1],
    ``order`` and ``place`` int32 [M k]. ``paro_experts_route`` and ``paro_experts_sort`` make it;
    ``weights`` may be None where only paro_w4_experts_gated and its gradient are called."""

    def __init__(self, ids, weights, offsets, order, place):
        import torch
        M, k = ids.shape
        E = offsets.shape[0] - 1
        at, i32, R = ids.get_device(), torch.int32, M * k
        self._tensors = ids, weights, offsets, order, place
        self._set(M, E, k, at, _expect(ids, "ids", (M, k), i32, at), _expect(offsets, "offsets", (E + 1,), i32, at),
                  _expect(order, "order", (R,), i32, at), _expect(place, "place", (R,), i32, at),
                  _expect(weights, "weights", (M, k), torch.float32, at))

    def _set(self, M, E, k, device, *pointers):
        self.M, self.E, self.k, self.device = M, E, k, device
        self._c = _Routing(M, E, k, *pointers)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def _made(cls, table, M, E, k, device, given=None):
        """A routing in one int32 tensor: order, place, offsets, then ids and weights, which may be ``given``
        instead. The tensors are cut out of it when they are asked for."""
        self = cls.__new__(cls)
        self._tensors, self._table, self._given = None, table, given
        R, at = M * k, table.data_ptr()
        if given is None:
            ids = at + 4 * (2 * R + E + 1)
            weights = ids + 4 * R
        else:
            ids, weights = (None if t is None else t.data_ptr() for t in given)
        self._set(M, E, k, device, ids, at + 8 * R, at, at + 4 * R, weights)
        return self

    def _cut(self):
        if self._tensors is None:
            import torch
            R = self.M * self.k
            order, place, offsets, *own = self._table.split_with_sizes(
                [R, R, self.E + 1] + ([R, R] if self._given is None else []))
            ids, weights = self._given or (own[0].view(self.M, self.k),
                                           own[1].view(torch.float32).view(self.M, self.k))
            self._tensors = ids, weights, offsets, order, place
        return self._tensors

    ids = property(lambda self: self._cut()[0])
    weights = property(lambda self: self._cut()[1])
    offsets = property(lambda self: self._cut()[2])
    order = property(lambda self: self._cut()[3])
    place = property(lambda self: self._cut()[4])

    def _on(self, device):
        if self.device != device:
            raise ValueError("routing must be on the current device")
        return self._ref


def _route_workspace(M, E, k, workspace, device, current):
    if workspace is None:
        need = load_library().paro_experts_route_workspace_size(M, E, k)
        if not need:
            return None, None, 0
        import torch
        workspace = torch.empty(need, dtype=torch.uint8, device=device)  # (scratch: nothing has to be zero)
    return _workspace(workspace, 0, device, current)


def new_experts_route_workspace(M: int, E: int, k: int, device="cuda"):
    """A workspace for paro_experts_route and paro_experts_sort (None when none is needed)."""
    return _workspace(None, int(load_library().paro_experts_route_workspace_size(M, E, k)), device)[0]


def paro_experts_route(logits, k: int, normalize: bool = True, workspace=None, stream=None) -> Routing:
    """The ``k`` experts of every token with the largest logits ([M][E], fp32, fp16 or bf16), their softmax
    weights (``normalize``: divided by their sum) and the tables of the routing."""
    import torch
    M, E = logits.shape
    dev = torch.cuda.current_device()
    with _made_on(stream):
        table = torch.empty(4 * M * k + E + 1, dtype=torch.int32, device=logits.device)
        workspace, ws_ptr, ws_bytes = _route_workspace(M, E, k, workspace, logits.device, dev)
    _handed_out(stream, table)
    r = Routing._made(table, M, E, k, dev)
    c = r._c
    _check(load_library().paro_experts_route(
        _expect(logits, "logits", (M, E), logits.dtype, dev), _type(logits, "logits"), M, E, k, int(normalize),
        c.ids, c.weights, c.offsets, c.order, c.place, ws_ptr, ws_bytes, _raw_stream(stream, dev)))
    return r


def paro_experts_sort(ids, E: int, weights=None, workspace=None, stream=None) -> Routing:
    """The routing of given ``ids`` (int32 [M][k]; outside 0 .. E - 1: no expert) and ``weights``."""
    import torch
    M, k = ids.shape
    dev = torch.cuda.current_device()
    at = _expect(ids, "ids", (M, k), torch.int32, dev)
    _expect(weights, "weights", (M, k), torch.float32, dev)
    with _made_on(stream):
        table = torch.empty(2 * M * k + E + 1, dtype=torch.int32, device=ids.device)
        workspace, ws_ptr, ws_bytes = _route_workspace(M, E, k, workspace, ids.device, dev)
    _handed_out(stream, table)
    r = Routing._made(table, M, E, k, dev, (ids, weights))
    c = r._c
    _check(load_library().paro_experts_sort(at, M, E, k, c.offsets, c.order, c.place, ws_ptr, ws_bytes,
                                            _raw_stream(stream, dev)))
    return r


def paro_experts_route_backward(logits, ids, weights, dweights, normalize: bool = True, dlogits=None, stream=None):
    """Gradient at the logits of paro_experts_route ([M][E], their type) for dweights = dL/dweights (fp32 [M][k]);
    ``ids`` and ``weights`` are the forward call's."""
    import torch
    M, E = logits.shape
    k = ids.shape[1]
    dev, f32 = torch.cuda.current_device(), torch.float32
    if dlogits is None:
        with _made_on(stream):
            dlogits = torch.empty_like(logits)
        _handed_out(stream, dlogits)
    _check(load_library().paro_experts_route_backward(
        _expect(logits, "logits", (M, E), logits.dtype, dev), _type(logits, "logits"), M, E, k, int(normalize),
        _expect(ids, "ids", (M, k), torch.int32, dev), _expect(weights, "weights", (M, k), f32, dev),
        _expect(dweights, "dweights", (M, k), f32, dev), _expect(dlogits, "dlogits", (M, E), logits.dtype, dev),
        _raw_stream(stream, dev)))
    return dlogits


def _experts_size(call, M, E, k, N, d) -> int:
    return int(getattr(load_library(), f"paro_w4_experts_{call}_workspace_size")(M, E, k, N, d))


def new_experts_gated_workspace(M: int, E: int, k: int, N: int, d: int, device="cuda"):
    """A workspace for paro_w4_experts_gated (None when none is needed)."""
    return _workspace(None, _experts_size("gated", M, E, k, N, d), device)[0]


def new_experts_combine_workspace(M: int, E: int, k: int, N: int, d: int, device="cuda"):
    """A workspace for paro_w4_experts_combine (None when none is needed)."""
    return _workspace(None, _experts_size("combine", M, E, k, N, d), device)[0]


def new_experts_gated_backward_workspace(M: int, E: int, k: int, N: int, d: int, device="cuda"):
    """A workspace for paro_w4_experts_gated_backward (None when none is needed)."""
    return _workspace(None, _experts_size("gated_backward", M, E, k, N, d), device)[0]


def new_experts_combine_backward_workspace(M: int, E: int, k: int, N: int, d: int, device="cuda"):
    """A workspace for paro_w4_experts_combine_backward (None when none is needed)."""
    return _workspace(None, _experts_size("combine_backward", M, E, k, N, d), device)[0]


def _experts_weights(r, qweight, scales, zeros, bias, P, d, group, dev):
    """Addresses of the weight stack of a routing's experts."""
    import torch
    f16, u8, E = torch.float16, torch.uint8, r.E
    return (_expect(qweight, "qweight", (E, P, d // 2), u8, dev), _expect(scales, "scales", (E, P, d // group), f16, dev),
            _expect(zeros, "zeros", (E, P, d // group), u8, dev), _expect(bias, "bias", (E, P), f16, dev))


def paro_w4_experts_gated(routing: Routing, x, qweight, scales, zeros, bias=None, act: str = "silu", h=None,
                          group: int = 128, workspace=None, stream=None):
    """H = act(x Wg^T + bg) * (x Wu^T + bu) of every (token, expert) pair (fp16 [M k][N], rows in expert order) for the
    transformed activations ``x`` [M][d] and the experts' weight blocks [E][2 N][d / 2] (gate, then up). Rows behind the
    last pair with an expert are 0 in an ``h`` that is made here, and left as they were in one that is given (which
    saves filling it). paro_rotation_backward over h sums all its rows: zero-fill a given one before the call."""
    import torch
    M, d = routing.M, x.shape[1]
    N = qweight.shape[1] // 2
    dev, f16 = torch.cuda.current_device(), torch.float16
    if h is None:
        with _made_on(stream):
            h = torch.zeros((M * routing.k, N), dtype=x.dtype, device=x.device)
        _handed_out(stream, h)
    # (the call needs no workspace)
    workspace, ws_ptr, ws_bytes = _workspace(workspace, 0, x.device, dev)
    _check(load_library().paro_w4_experts_gated(
        routing._on(dev), _expect(x, "x", (M, d), f16, dev),
        *_experts_weights(routing, qweight, scales, zeros, bias, 2 * N, d, group, dev), _act(act),
        _expect(h, "h", (M * routing.k, N), f16, dev), N, d, group, ws_ptr, ws_bytes, _raw_stream(stream, dev)))
    return h


def _scratch(call, r, N, d, workspace, device, current):
    """A call's workspace, given or made (scratch: nothing has to be zero)."""
    if workspace is None:
        need = _experts_size(call, r.M, r.E, r.k, N, d)
        if need:
            import torch
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return _workspace(workspace, 0, device, current)


def paro_w4_experts_combine(routing: Routing, h, qweight, scales, zeros, bias=None, residual=None, y=None,
                            group: int = 128, workspace=None, stream=None):
    """Y = residual + sum over a token's experts of weight (H W^T + b) (fp16 [M][N]) for rows ``h`` [M k][d] in expert
    order and the experts' weights [E][N][d / 2]; ``y`` may be ``residual``."""
    import torch
    M, d = routing.M, h.shape[1]
    N = qweight.shape[1]
    dev, f16 = torch.cuda.current_device(), torch.float16
    made = []
    with _made_on(stream):
        if y is None:
            y = h.new_empty((M, N))
            made.append(y)
        workspace, ws_ptr, ws_bytes = _scratch("combine", routing, N, d, workspace, h.device, dev)
    _handed_out(stream, *made)
    _check(load_library().paro_w4_experts_combine(
        routing._on(dev), _expect(h, "h", (M * routing.k, d), f16, dev),
        *_experts_weights(routing, qweight, scales, zeros, bias, N, d, group, dev),
        _expect(residual, "residual", (M, N), f16, dev), _expect(y, "y", (M, N), f16, dev), N, d, group, ws_ptr,
        ws_bytes, _raw_stream(stream, dev)))
    return y


def paro_w4_experts_gated_backward(routing: Routing, x, qweight, scales, zeros, dh, bias=None, act: str = "silu",
                                   dz=None, dx=None, want_dx: bool = True, group: int = 128, workspace=None,
                                   stream=None):
    """Gradients of paro_w4_experts_gated for dh = dL/dH ([M k][N], by row): returns (dx fp16 [M][d] or None, dz fp16
    [M k][2 N]: the gate's columns, then the up projection's; rows behind the last pair are left as they were, and hold
    anything in a ``dz`` that is made here)."""
    import torch
    M, d = routing.M, x.shape[1]
    N = qweight.shape[1] // 2
    R = M * routing.k
    dev, f16 = torch.cuda.current_device(), torch.float16
    made = []
    with _made_on(stream):
        if dz is None:
            dz = x.new_empty((R, 2 * N))
            made.append(dz)
        if dx is None and want_dx:
            dx = x.new_empty((M, d))
            made.append(dx)
        workspace, ws_ptr, ws_bytes = _scratch("gated_backward", routing, N, d, workspace, x.device, dev) \
            if dx is not None or workspace is not None else (None, None, 0)
    _handed_out(stream, *made)
    _check(load_library().paro_w4_experts_gated_backward(
        routing._on(dev), _expect(x, "x", (M, d), f16, dev),
        *_experts_weights(routing, qweight, scales, zeros, bias, 2 * N, d, group, dev), _act(act),
        _expect(dh, "dh", (R, N), f16, dev), _expect(dz, "dz", (R, 2 * N), f16, dev),
        _expect(dx, "dx", (M, d), f16, dev), N, d, group, ws_ptr, ws_bytes, _raw_stream(stream, dev)))
    return dx, dz


def paro_w4_experts_combine_backward(routing: Routing, h, qweight, scales, zeros, dy, bias=None, dh=None,
                                     dweights=None, group: int = 128, workspace=None, stream=None):
    """Gradients of paro_w4_experts_combine for dy = dL/dY ([M][N]): returns (dh fp16 [M k][d], rows in expert order;
    dweights fp32 [M][k]). Rows behind the last pair with an expert are 0 in a ``dh`` that is made here, and left as
    they were in one that is given: zero-fill that one before the call where paro_rotation_backward sums its rows."""
    import torch
    M, d = routing.M, h.shape[1]
    N = qweight.shape[1]
    R = M * routing.k
    dev, f16 = torch.cuda.current_device(), torch.float16
    made = []
    with _made_on(stream):
        if dh is None:
            dh = torch.zeros((R, d), dtype=h.dtype, device=h.device)
            made.append(dh)
        dweights = _given(dweights, "dweights", (M, routing.k), h.device, made)
        workspace, ws_ptr, ws_bytes = _scratch("combine_backward", routing, N, d, workspace, h.device, dev)
    _handed_out(stream, *made)
    _check(load_library().paro_w4_experts_combine_backward(
        routing._on(dev), _expect(h, "h", (R, d), f16, dev),
        *_experts_weights(routing, qweight, scales, zeros, bias, N, d, group, dev),
        _expect(dy, "dy", (M, N), f16, dev), _expect(dh, "dh", (R, d), f16, dev),
        _expect(dweights, "dweights", (M, routing.k), torch.float32, dev), N, d, group, ws_ptr, ws_bytes,
        _raw_stream(stream, dev)))
    return dh, dweights


def paro_distill_loss(z, values, index, lse=None, row_weight=None, temperature: float = 1.0, grad_scale: float = 1.0,
                      gradients: bool = True, loss=None, dz=None, stream=None):
    """T^2 KL(teacher || student) of each row, from the teacher's top logits ``values`` [M][K] at ``index`` int32 [M][K]
    (-1: no entry) and the student's logits ``z`` [M][V]: returns (loss fp32 [M], grad_scale dL/dz of z's type or None).
    ``lse`` fp32 [M]: log-sum-exp of all the teacher's logits / T, with which the rest of its mass is one more class.
    ``row_weight`` fp32 [M]: rows of weight 0 are left out. ``dz`` may be ``z``."""
    import torch
    M, V = z.shape
    K = values.shape[1]
    dev, f32 = torch.cuda.current_device(), torch.float32
    made = []
    with _made_on(stream):
        loss = _given(loss, "loss", (M,), z.device, made)
        if dz is None and gradients:
            dz = torch.empty_like(z)
            made.append(dz)
    _handed_out(stream, *made)
    _check(load_library().paro_distill_loss(
        _expect(z, "z", (M, V), z.dtype, dev), _type(z, "z"), _expect(values, "values", (M, K), values.dtype, dev),
        _type(values, "values"), _expect(index, "index", (M, K), torch.int32, dev),
        _expect(lse, "lse", (M,), f32, dev), _expect(row_weight, "row_weight", (M,), f32, dev), M, V, K, temperature,
        grad_scale, _expect(loss, "loss", (M,), f32, dev), _expect(dz, "dz", (M, V), z.dtype, dev),
        _raw_stream(stream, dev)))
    return loss, dz


def paro_adamw_moments(sizes) -> int:
    """Values of each moment of tensors of these sizes (each rounded up to 256)."""
    n = np.ascontiguousarray(np.asarray(list(sizes), dtype=np.int64))
    total = int(load_library().paro_adamw_moments(len(n), _ptr(n)))
    if total < 0:
        raise ValueError("bad tensor sizes")
    return total


class AdamW:
    """``paro_adamw_create`` / ``paro_adamw_step``: AdamW over a fixed list of tensors.

    ``params`` and ``grads``: contiguous device tensors, one type each (fp32,
    fp16 or bf16), stepped in place and read where they are; ``m``, ``v`` (and
    for 8-bit moments ``m_scale``, ``v_scale``): the moments, zero-filled ones
    are made (and waited for) when they are not given: fp32, or with
    ``state_bits=8`` e4m3 with fp32 scales (``v`` then holds sqrt(v)).
    """

    def __init__(self, params, grads, m=None, v=None, m_scale=None, v_scale=None, state_bits: int = 32):
        import torch
        params, grads = list(params), list(grads)
        if len(params) != len(grads) or not params:
            raise ValueError("params and grads must be lists of the same length, not empty")
        types = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
        ptype, gtype = params[0].dtype, grads[0].dtype
        if ptype not in types or gtype not in types:
            raise TypeError("params and grads must be fp32, fp16 or bf16")
        total = paro_adamw_moments(p.numel() for p in params)
        if m is not None:
            state_bits = 8 * m.element_size()
        if state_bits not in (32, 8):
            raise ValueError("state_bits must be 32 or 8")
        state = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        self._made = []

        def new(n, t):
            if torch.cuda.is_current_stream_capturing():
                raise ValueError("moments made inside a capture would be zero-filled by every replay: pass them")
            made = torch.zeros(n, dtype=torch.uint8 if t != torch.float32 else t, device=params[0].device).view(t)
            self._made.append(made)
            return made

        self.m = new(total, state) if m is None else m
        self.v = new(total, state) if v is None else v
        self.m_scale, self.v_scale = m_scale, v_scale
        if state_bits == 8:
            self.m_scale = new(total // 256, torch.float32) if m_scale is None else m_scale
            self.v_scale = new(total // 256, torch.float32) if v_scale is None else v_scale
        elif m_scale is not None or v_scale is not None:
            raise ValueError("scales belong to 8-bit moments")
        self.params, self.grads = params, grads  # kept alive: the plan holds their addresses
        n = np.array([p.numel() for p in params], dtype=np.int64)
        self._device = dev = torch.cuda.current_device()
        ptrs = np.array([_expect(p, "a parameter", p.shape, ptype, dev) for p in params], dtype=np.uint64)
        gptrs = np.array([_expect(g, "a gradient", p.shape, gtype, dev) for p, g in zip(params, grads)],
                         dtype=np.uint64)
        scales = [_expect(s, "a scale", (total // 256,), torch.float32, dev) for s in (self.m_scale, self.v_scale)]
        h = ctypes.c_void_p()
        _check(load_library().paro_adamw_create(
            len(n), _ptr(n), _ptr(ptrs), types[ptype], _ptr(gptrs), types[gtype], state_bits,
            _expect(self.m, "m", (total,), state, dev), _expect(self.v, "v", (total,), state, dev), *scales,
            ctypes.byref(h)))
        self._h = h
        self._made_on = torch.cuda.current_stream()
        if self._made:  # zero before the first step, whatever stream that runs on
            self._made_on.synchronize()

    def step(self, step: int, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
             stream=None):
        """Step ``step`` (from 1 on) with the gradients as they are."""
        import torch
        if self._device != torch.cuda.current_device():
            raise ValueError("the tensors must be on the current device")
        at = _raw_stream(stream, self._device)
        _check(load_library().paro_adamw_step(self._h, step, lr, betas[0], betas[1], eps, weight_decay, at))
        if at != self._made_on.cuda_stream:  # the moments made here stay until the step has passed
            for t in self._made:
                t.record_stream(stream if stream is not None else torch.cuda.current_stream())

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            load_library().paro_adamw_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


paro_adamw_create = AdamW


def paro_rotation_plan_host(pairs, theta, alpha, group: int) -> Tuple[np.ndarray, dict]:
    """Host-only schedule image (what paro_rotation_create uploads) and its layout."""
    lib = load_library()
    pairs, theta, alpha = _host_arrays(pairs, theta, alpha)
    d = int(alpha.shape[0])
    K = int(pairs.shape[0]) if pairs.ndim == 3 else 0
    need = ctypes.c_size_t()
    lay = (ctypes.c_int32 * 5)()
    _check(lib.paro_rotation_plan_host(d, group, K, _ptr(pairs), _ptr(theta), _ptr(alpha), None,
                                       0, ctypes.byref(need), lay))
    img = np.zeros(need.value // 4, dtype=np.uint32)
    _check(lib.paro_rotation_plan_host(d, group, K, _ptr(pairs), _ptr(theta), _ptr(alpha),
                                       img.ctypes.data_as(ctypes.c_void_p), need.value,
                                       ctypes.byref(need), lay))
    return img, {"seg_ch": lay[0], "ppl": lay[1], "words": lay[2], "fast": bool(lay[3]),
                 "stages": lay[4]}


def paro_pairs_random(d: int, group: int, K: int, seed: int) -> np.ndarray:
    """Random pairs with de-duplication across stages: int32 [K][d/2][2]."""
    out = np.zeros((K, d // 2, 2), dtype=np.int32)
    _check(load_library().paro_pairs_random(d, group, K, ctypes.c_uint64(seed & (2 ** 64 - 1)),
                                            _ptr(out)))
    return out


def paro_pairs_by_gap(score, group: int, K: int) -> np.ndarray:
    """Pairs of strongly differing channels by per-channel ``score``: int32 [K][d/2][2]."""
    score = np.ascontiguousarray(np.asarray(score, dtype=np.float32))
    d = int(score.shape[0])
    out = np.zeros((K, d // 2, 2), dtype=np.int32)
    _check(load_library().paro_pairs_by_gap(d, group, K, _ptr(score), _ptr(out)))
    return out


def paro_sparsify_angles(theta, n_keep: int) -> np.ndarray:
    """The ``n_keep`` largest-|theta| pairs keep their angle, the rest get 0."""
    theta = np.ascontiguousarray(np.asarray(theta, dtype=np.float32))
    K, half = theta.shape
    out = np.zeros_like(theta)
    _check(load_library().paro_sparsify_angles(2 * half, K, _ptr(theta), int(n_keep), _ptr(out)))
    return out


def paro_stream_copy(src, dst, blocks: int = 8192, stream=None):
    """Plain device copy of ``src`` into ``dst`` (same byte size): the
    measured HBM ceiling the memory-bound kernels are reported against."""
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("src and dst must have the same size")
    _check(load_library().paro_stream_copy(_dptr(src, "src"), _dptr(dst, "dst"), nbytes, int(blocks),
                                           _stream(stream)))
    return dst


def paro_mfma_loop(src, out, blocks: int, iters: int, stream=None):
    """fp16 matrix-core loop on operands read from ``src`` (fp16, a multiple of
    8 elements); ``out`` holds blocks * 256 floats: the measured matrix-core
    ceiling the prefill linear is reported against."""
    import torch
    if src.numel() % 8:
        raise ValueError("src must hold a multiple of 8 elements")
    if out.numel() < int(blocks) * 256:
        raise ValueError("out must hold blocks * 256 floats")
    _check(load_library().paro_mfma_loop(_dptr(src, "src", torch.float16), src.numel(),
                                         _dptr(out, "out", torch.float32), int(blocks), int(iters),
                                         _stream(stream)))
    return out
