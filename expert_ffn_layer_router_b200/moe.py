"""ctypes binding of ``libmoe_b200.so`` (the C ABI declared in ``include/moe_b200.h``).

Argument marshalling only: torch tensors provide device memory and the current CUDA stream;
every step of the layer runs in the library's kernels.  Importing this module fails loudly if
the library has not been built, and every call raises :class:`MoeError` on a non-zero status.
There is no CPU path.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import operator
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_b200.so")

MOE_F32, MOE_BF16 = 0, 1
FLAG_RENORMALIZE, FLAG_ARRIVAL_ORDER, FLAG_GATED, FLAG_ROUTER_PREPARED = 1, 2, 4, 8
MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_DEVICE = 5       # the status word holds an error (moe_get_device_status)
DEV_OK, DEV_TIMEOUT, DEV_BAD_INDEX = 0, 1, 2


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (what, _status_string(status), status))


class Problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("capacity_factor", ctypes.c_float), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class W4(ctypes.Structure):
    """moe_w4: device pointers of 4-bit weights and their group size."""
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p),
                ("group", ctypes.c_int32)]


class Norm(ctypes.Structure):
    """moe_norm: parameters of the layer norm in front of a block, and where its results go."""
    _fields_ = [("gamma", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("y", ctypes.c_void_p), ("mean", ctypes.c_void_p), ("rstd", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libmoe_b200.so is not built (run __graft_entry__.build() or "
                          "python expert_ffn_layer_router_b200/build.py); there is no fallback")
    L = ctypes.CDLL(LIB_PATH)
    P, PW, PN = ctypes.POINTER(Problem), ctypes.POINTER(W4), ctypes.POINTER(Norm)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
    sig = {
        "moe_capacity": [P, ctypes.POINTER(ctypes.c_int64)],
        "moe_workspace_size": [P, ctypes.POINTER(ctypes.c_size_t)],
        "moe_route": [P, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moe_capacity_dispatch": [P, ctypes.c_int64] + [vp] * 8 + [sz, vp],
        "moe_router_logits": [P, vp, vp, vp, vp, vp, sz, vp],
        "moe_prepare_router": [P, vp, vp, sz, vp],
        "moe_dispatch": [P, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moe_expert_ffn": [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moe_combine": [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moe_forward": [P] + [vp] * 15 + [sz, vp],
        "moe_get_device_status": [vp, sz, vp, ctypes.POINTER(ctypes.c_int32)],
        "moe_reset_device_status": [vp, sz, vp],
        "moe_set_stage_events": [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int32],
        "moe_route_static": [P, vp, vp, vp, vp, vp, vp, vp],
        "moe_selftest_wait_timeout": [vp, sz, ctypes.c_int32, vp],
        "moe_quantize_packed": [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp],
        "moe_dequantize_packed": [PW, i32, i32, i32, vp, vp],
        "moe_workspace_size_packed": [P, ctypes.POINTER(ctypes.c_size_t)],
        "moe_expert_ffn_packed": [P, vp, vp, vp, PW, vp, PW, vp, vp, vp, sz, vp],
        "moe_layer_norm": [P, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp],
        "moe_layer_norm_backward": [P] + [vp] * 10 + [sz, vp],
        "moe_balance_loss": [P] + [vp] * 7 + [sz, vp],
        "moe_route_backward": [P] + [vp] * 8 + [sz, vp],
        "moe_forward_block": [P, vp, PN, vp, vp, vp, vp, PW, PW] + [vp] * 10 + [sz, vp],
    }
    for name, args in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    L.moe_status_string.argtypes = [ctypes.c_int]
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_last_launch_count.argtypes = []
    L.moe_last_launch_count.restype = ctypes.c_int32
    return L


_lib = _load()

EXPORTS = ("moe_capacity", "moe_workspace_size", "moe_route", "moe_dispatch", "moe_expert_ffn",
           "moe_combine", "moe_forward", "moe_get_device_status", "moe_reset_device_status",
           "moe_last_launch_count", "moe_status_string", "moe_set_stage_events",
           "moe_route_static", "moe_selftest_wait_timeout", "moe_capacity_dispatch",
           "moe_router_logits", "moe_prepare_router", "moe_quantize_packed", "moe_dequantize_packed",
           "moe_workspace_size_packed", "moe_expert_ffn_packed", "moe_layer_norm",
           "moe_layer_norm_backward", "moe_balance_loss", "moe_route_backward",
           "moe_forward_block")

STAGE_EVENTS = 7
STAGE_NAMES = ("router_logits", "route_topk", "capacity_dispatch", "expert_gemm1",
               "expert_gemm2", "combine")


def lib():
    return _lib


def _status_string(s: int) -> str:
    return _lib.moe_status_string(int(s)).decode()


def _check(status: int, what: str):
    if status != MOE_OK:
        raise MoeError(status, what)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def problem(T, d_model, d_ff, E, k, capacity_factor, dtype, flags=0) -> Problem:
    if isinstance(dtype, str):
        dtype = {"f32": MOE_F32, "bf16": MOE_BF16}[dtype]
    elif isinstance(dtype, torch.dtype):
        dtype = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return Problem(int(T), int(d_model), int(d_ff), int(E), int(k), float(capacity_factor),
                   int(dtype), int(flags))


def moe_capacity(p: Problem) -> int:
    K = ctypes.c_int64()
    _check(_lib.moe_capacity(ctypes.byref(p), ctypes.byref(K)), "moe_capacity")
    return K.value


def moe_workspace_size(p: Problem) -> int:
    n = ctypes.c_size_t()
    _check(_lib.moe_workspace_size(ctypes.byref(p), ctypes.byref(n)), "moe_workspace_size")
    return n.value


def moe_route(p, logits, ids, w, slot, drop, counts, ws, stream=None):
    _check(_lib.moe_route(ctypes.byref(p), _ptr(logits), _ptr(ids), _ptr(w), _ptr(slot),
                          _ptr(drop), _ptr(counts), _ptr(ws), ws.numel() * ws.element_size(),
                          _stream(stream)), "moe_route")


def moe_capacity_dispatch(p, K, ids, w, slot, drop, counts, ws, offsets=None, rowtok=None,
                          stream=None):
    _check(_lib.moe_capacity_dispatch(ctypes.byref(p), int(K), _ptr(ids), _ptr(w), _ptr(slot),
                                      _ptr(drop), _ptr(counts), _ptr(offsets), _ptr(rowtok),
                                      _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "moe_capacity_dispatch")


def moe_prepare_router(p, Wr, ws, stream=None):
    _check(_lib.moe_prepare_router(ctypes.byref(p), _ptr(Wr), _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(stream)),
           "moe_prepare_router")


def moe_router_logits(p, x, Wr, br, logits, ws, stream=None):
    _check(_lib.moe_router_logits(ctypes.byref(p), _ptr(x), _ptr(Wr), _ptr(br), _ptr(logits),
                                  _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "moe_router_logits")


def moe_dispatch(p, ids, slot, offsets, rowtok, ws, x=None, x_perm=None, stream=None):
    _check(_lib.moe_dispatch(ctypes.byref(p), _ptr(ids), _ptr(slot), _ptr(offsets),
                             _ptr(rowtok), _ptr(x), _ptr(x_perm), _ptr(ws),
                             ws.numel() * ws.element_size(), _stream(stream)), "moe_dispatch")


def moe_expert_ffn(p, x, offsets, rowtok, W1, b1, W2, b2, Y, ws, stream=None):
    _check(_lib.moe_expert_ffn(ctypes.byref(p), _ptr(x), _ptr(offsets), _ptr(rowtok), _ptr(W1),
                               _ptr(b1), _ptr(W2), _ptr(b2), _ptr(Y), _ptr(ws),
                               ws.numel() * ws.element_size(), _stream(stream)),
           "moe_expert_ffn")


def moe_combine(p, x, Y, w, ids, slot, offsets, out, ws=None, stream=None):
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_lib.moe_combine(ctypes.byref(p), _ptr(x), _ptr(Y), _ptr(w), _ptr(ids), _ptr(slot),
                            _ptr(offsets), _ptr(out), _ptr(ws), nbytes, _stream(stream)),
           "moe_combine")


def moe_forward(p, x, Wr, br, W1, b1, W2, b2, out, ws, logits_out=None, ids_out=None,
                w_out=None, slot_out=None, drop_out=None, counts_out=None, stream=None):
    _check(_lib.moe_forward(ctypes.byref(p), _ptr(x), _ptr(Wr), _ptr(br), _ptr(W1), _ptr(b1),
                            _ptr(W2), _ptr(b2), _ptr(out), _ptr(logits_out), _ptr(ids_out),
                            _ptr(w_out), _ptr(slot_out), _ptr(drop_out), _ptr(counts_out),
                            _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "moe_forward")


def _at(t):
    """A tensor's address as a plain int (None stays None)."""
    return None if t is None else t.data_ptr()


def _at_stream(stream):
    return stream if isinstance(stream, int) else _stream(stream)


def moe_workspace_size_packed(p: Problem) -> int:
    n = ctypes.c_size_t()
    _check(_lib.moe_workspace_size_packed(ctypes.byref(p), ctypes.byref(n)), "moe_workspace_size_packed")
    return n.value


def moe_quantize_packed(W, E, N, K, group, q, scale, zero=None, stream=None):
    dtype = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}.get(W.dtype, -1)     # (-1: refused)
    _check(_lib.moe_quantize_packed(_at(W), dtype, int(E), int(N), int(K), int(group), _at(q),
                                _at(scale), _at(zero), _at_stream(stream)), "moe_quantize_packed")


def moe_dequantize_packed(w: W4, E, N, K, W, stream=None):
    _check(_lib.moe_dequantize_packed(ctypes.byref(w), int(E), int(N), int(K), _at(W),
                                  _at_stream(stream)), "moe_dequantize_packed")


def _ref(s):
    return None if s is None else ctypes.byref(s)


def moe_expert_ffn_packed(p, x, offsets, rowtok, W1: W4, b1, W2: W4, b2, Y, ws, stream=None):
    _check(_lib.moe_expert_ffn_packed(ctypes.byref(p), _at(x), _at(offsets), _at(rowtok),
                                  _ref(W1), _at(b1), _ref(W2), _at(b2), _at(Y), _at(ws),
                                  ws.numel() * ws.element_size(), _at_stream(stream)),
           "moe_expert_ffn_packed")


def moe_layer_norm(p, x, gamma, beta, eps, y, mean, rstd, stream=None):
    _check(_lib.moe_layer_norm(ctypes.byref(p), _at(x), _at(gamma), _at(beta), float(eps),
                               _at(y), _at(mean), _at(rstd), _at_stream(stream)),
           "moe_layer_norm")


def moe_layer_norm_backward(p, dy, x, gamma, mean, rstd, dx, dgamma, dbeta, ws, dres=None,
                            stream=None):
    _check(_lib.moe_layer_norm_backward(ctypes.byref(p), _at(dy), _at(x), _at(gamma),
                                        _at(mean), _at(rstd), _at(dres), _at(dx),
                                        _at(dgamma), _at(dbeta), _at(ws),
                                        ws.numel() * ws.element_size(), _at_stream(stream)),
           "moe_layer_norm_backward")


def moe_balance_loss(p, logits, ids, losses, counts, probs, ws, mask=None, stream=None):
    _check(_lib.moe_balance_loss(ctypes.byref(p), _at(logits), _at(ids), _at(mask),
                                 _at(losses), _at(counts), _at(probs), _at(ws),
                                 ws.numel() * ws.element_size(), _at_stream(stream)),
           "moe_balance_loss")


def moe_route_backward(p, logits, ids, counts, dlogits, ws, grad_losses=None, grad_w=None,
                       mask=None, stream=None):
    _check(_lib.moe_route_backward(ctypes.byref(p), _at(logits), _at(ids), _at(mask),
                                   _at(counts), _at(grad_losses), _at(grad_w), _at(dlogits),
                                   _at(ws), ws.numel() * ws.element_size(), _at_stream(stream)),
           "moe_route_backward")


def moe_forward_block(p, x, norm, Wr, br, W1, W2, Q1, Q2, b1, b2, out, ws, logits_out=None,
                      ids_out=None, w_out=None, slot_out=None, drop_out=None, counts_out=None,
                      stream=None):
    _check(_lib.moe_forward_block(ctypes.byref(p), _at(x), _ref(norm), _at(Wr), _at(br),
                                  _at(W1), _at(W2), _ref(Q1), _ref(Q2), _at(b1), _at(b2),
                                  _at(out), _at(logits_out), _at(ids_out), _at(w_out),
                                  _at(slot_out), _at(drop_out), _at(counts_out), _at(ws),
                                  ws.numel() * ws.element_size(), _at_stream(stream)),
           "moe_forward_block")


def moe_get_device_status(ws, stream=None) -> int:
    """Status word of ``ws``; ``ws=None``: that of moe_route_static on the current device."""
    code = ctypes.c_int32()
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = _lib.moe_get_device_status(_ptr(ws), nbytes, _stream(stream), ctypes.byref(code))
    if rc not in (MOE_OK, MOE_ERR_DEVICE):
        raise MoeError(rc, "moe_get_device_status")
    return code.value


def moe_reset_device_status(ws, stream=None):
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_lib.moe_reset_device_status(_ptr(ws), nbytes, _stream(stream)),
           "moe_reset_device_status")


def moe_selftest_wait_timeout(ws, limit_us, stream=None):
    _check(_lib.moe_selftest_wait_timeout(_ptr(ws), ws.numel() * ws.element_size(), int(limit_us),
                                          _stream(stream)), "moe_selftest_wait_timeout")


def moe_last_launch_count() -> int:
    return int(_lib.moe_last_launch_count())


def moe_set_stage_events(events):
    """``events``: STAGE_EVENTS torch.cuda.Event objects (or None to turn recording off)."""
    if not events:
        _check(_lib.moe_set_stage_events(None, 0), "moe_set_stage_events")
        return
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(_lib.moe_set_stage_events(arr, len(events)), "moe_set_stage_events")


# ----------------------------------------------------------------------------------------------
# Argument checks and streams of the tensor-level calls below
# ----------------------------------------------------------------------------------------------
def _need(what, name, t, dtype, shape, device):
    """``t`` must be a dense tensor of this type and shape (a tuple) on ``device``."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or
            t.device != device or not t.is_contiguous()):
        raise MoeError(MOE_ERR_INVALID_ARG, "%s: %s must be a contiguous %s tensor of shape %s on %s"
                       % (what, name, dtype, tuple(shape), device))


class _on:
    """Makes ``device`` and ``stream`` (None: the device's current stream) current, so results
    allocated inside belong to the stream that writes them; gives the stream's handle.  Entering
    with the current device and no stream, the usual case, changes nothing."""

    __slots__ = ("device", "stream", "guards")

    def __init__(self, device, stream):
        self.device, self.stream, self.guards = device, stream, None

    def __enter__(self):
        index = self.device.index
        if self.device.type != "cuda":
            raise MoeError(MOE_ERR_INVALID_ARG, "tensors must be on a CUDA device, not on %s" % self.device)
        if self.stream is None and index == torch._C._cuda_getDevice():
            return torch._C._cuda_getCurrentRawStream(index)
        with contextlib.ExitStack() as guards:             # (undone if the stream cannot be used)
            guards.enter_context(torch.cuda.device(self.device))
            if self.stream is not None:
                guards.enter_context(torch.cuda.stream(self._stream()))
            self.guards = guards.pop_all()
        return torch._C._cuda_getCurrentRawStream(index)

    def _stream(self):
        st = self.stream
        if hasattr(st, "cuda_stream"):
            if st.device != self.device:
                raise MoeError(MOE_ERR_INVALID_ARG, "stream is on %s, the tensors on %s"
                               % (st.device, self.device))
            return st
        try:
            handle = operator.index(st)
        except TypeError:
            raise MoeError(MOE_ERR_INVALID_ARG, "stream must be a CUDA stream or its handle") from None
        return torch.cuda.ExternalStream(handle, device=self.device)

    def __exit__(self, *exc):
        if self.guards is not None:
            self.guards.__exit__(*exc)
        return False


class W4Weights:
    """4-bit weights [E, N, K] with group scales: ``q`` [E, N, 16 ceil(K/128)] int32 words,
    ``scale`` and the optional offsets ``zero`` [E, ceil(K/group), N] bfloat16 (the layout of
    moe_w4).  :func:`quantize_w4` makes them.  The tensors' values may change in place; other
    tensors take another object."""

    q = property(lambda self: self._tensors[0])
    scale = property(lambda self: self._tensors[1])
    zero = property(lambda self: self._tensors[2])
    E = property(lambda self: self._sizes[0])
    N = property(lambda self: self._sizes[1])
    K = property(lambda self: self._sizes[2])
    group = property(lambda self: self._sizes[3])

    def __init__(self, q, scale, zero=None, *, K, group):
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise MoeError(MOE_ERR_INVALID_ARG, "W4Weights: q must be int32 words [E, N, ...]")
        if group not in (32, 64, 128):
            raise MoeError(MOE_ERR_INVALID_ARG, "W4Weights: group must be 32, 64 or 128")
        E, N, dev = q.shape[0], q.shape[1], q.device
        shapes = ((E, N, 16 * (-(-K // 128))), (E, -(-K // group), N))
        _need("W4Weights", "q", q, torch.int32, shapes[0], dev)
        _need("W4Weights", "scale", scale, torch.bfloat16, shapes[1], dev)
        if zero is not None:
            _need("W4Weights", "zero", zero, torch.bfloat16, shapes[1], dev)
        self._tensors, self._shapes = (q, scale, zero), shapes
        self._sizes, self._device = (E, N, int(K), int(group)), dev

    @property
    def c(self):
        """The tensors' present addresses as a moe_w4.  (A tensor can be given other storage or
        another shape in place, so each call looks at them.)"""
        q, scale, zero = self._tensors
        words, side = self._shapes
        if (q.shape != words or scale.shape != side or not q.is_contiguous() or
                not scale.is_contiguous() or q.device != self._device or
                scale.device != self._device or (zero is not None and (
                    zero.shape != side or not zero.is_contiguous() or
                    zero.device != self._device))):
            raise MoeError(MOE_ERR_INVALID_ARG, "W4Weights: a tensor was changed to another shape, "
                           "layout or device")
        return W4(q.data_ptr(), scale.data_ptr(), None if zero is None else zero.data_ptr(),
                  self._sizes[3])

    def _need(self, what, name, shape, device):
        if self._sizes[:3] != tuple(shape) or self._device != device:
            raise MoeError(MOE_ERR_INVALID_ARG, "%s: %s must be 4-bit weights of shape %s on %s"
                           % (what, name, tuple(shape), device))


def quantize_w4(W, group, zeros=False, stream=None) -> W4Weights:
    """Quantises ``W`` [E, N, K] (bfloat16 or float32) to 4 bits with a scale, and with ``zeros`` an
    offset, per ``group`` columns.  A group with a NaN or an infinity reads back as not finite."""
    if not isinstance(W, torch.Tensor) or W.dim() != 3 or W.dtype not in (torch.bfloat16,
                                                                         torch.float32):
        raise MoeError(MOE_ERR_INVALID_ARG, "quantize_w4: W must be bfloat16 or float32 [E, N, K]")
    if group not in (32, 64, 128):
        raise MoeError(MOE_ERR_INVALID_ARG, "quantize_w4: group must be 32, 64 or 128")
    E, N, K = W.shape
    _need("quantize_w4", "W", W, W.dtype, (E, N, K), W.device)
    with _on(W.device, stream) as st:
        q = torch.empty((E, N, 16 * (-(-K // 128))), dtype=torch.int32, device=W.device)
        side = (E, -(-K // group), N)
        scale = torch.empty(side, dtype=torch.bfloat16, device=W.device)
        zero = torch.empty(side, dtype=torch.bfloat16, device=W.device) if zeros else None
        moe_quantize_packed(W, E, N, K, group, q, scale, zero, st)
    return W4Weights(q, scale, zero, K=K, group=group)


def dequantize_w4(w: W4Weights, stream=None):
    """The values of 4-bit weights, bfloat16 [E, N, K]."""
    if not isinstance(w, W4Weights):
        raise MoeError(MOE_ERR_INVALID_ARG, "dequantize_w4: w must be W4Weights")
    with _on(w.q.device, stream) as st:
        W = torch.empty((w.E, w.N, w.K), dtype=torch.bfloat16, device=w.q.device)
        moe_dequantize_packed(w.c, w.E, w.N, w.K, W, st)
    return W


# ----------------------------------------------------------------------------------------------
# Convenience: a layer that owns its workspace (allocated once through torch).
# ----------------------------------------------------------------------------------------------
class MoELayer:
    """Holds a problem description and a workspace; calls the C ABI on torch tensors.

    The workspace serves one call at a time: calls of one layer that may overlap on the GPU (on
    other streams) take a layer each.

    ``w4``: size the workspace for 4-bit expert weights too (``expert_ffn_w4``,
    ``forward_block`` with :class:`W4Weights`); above 64 rows an expert that adds a bfloat16 copy of
    the larger weight.  (Weights are arguments: one object serves all layers of a model that have
    this shape and run one after the other, and so one workspace does.)"""

    def __init__(self, T, d_model, d_ff, E, k, capacity_factor=math.inf, dtype="bf16",
                 device="cuda", flags=0, w4=False):
        self.p = problem(T, d_model, d_ff, E, k, capacity_factor, dtype, flags)
        self.K = moe_capacity(self.p)
        self.device = torch.device(device)
        nbytes = moe_workspace_size_packed(self.p) if w4 else moe_workspace_size(self.p)
        # int64 elements keep the base 256-byte aligned through the caching allocator.
        self.ws = torch.zeros((nbytes + 7) // 8, dtype=torch.int64, device=self.device)
        self._p = ctypes.byref(self.p)
        self.max_rows = min(T * k, E * self.K)

    @property
    def _ws(self):
        return self.ws.data_ptr(), self.ws.numel() * self.ws.element_size()

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.p.dtype == MOE_BF16 else torch.float32

    def forward(self, x, Wr, br, W1, b1, W2, b2, out=None, want_routing=False, stream=None):
        p = self.p
        out = torch.empty_like(x) if out is None else out
        extra = {}
        if want_routing:
            dev = x.device
            extra = dict(
                logits_out=torch.empty((p.T, p.E), dtype=torch.float32, device=dev),
                ids_out=torch.empty((p.T, p.k), dtype=torch.int32, device=dev),
                w_out=torch.empty((p.T, p.k), dtype=torch.float32, device=dev),
                slot_out=torch.empty((p.T, p.k), dtype=torch.int32, device=dev),
                drop_out=torch.empty((p.T, p.k), dtype=torch.uint8, device=dev),
                counts_out=torch.empty(2 * p.E, dtype=torch.int32, device=dev))
        moe_forward(p, x, Wr, br, W1, b1, W2, b2, out, self.ws, stream=stream, **extra)
        return (out, extra) if want_routing else out

    def route(self, logits, stream=None):
        p, dev = self.p, logits.device
        r = dict(ids=torch.empty((p.T, p.k), dtype=torch.int32, device=dev),
                 w=torch.empty((p.T, p.k), dtype=torch.float32, device=dev),
                 slot=torch.empty((p.T, p.k), dtype=torch.int32, device=dev),
                 drop=torch.empty((p.T, p.k), dtype=torch.uint8, device=dev),
                 counts=torch.empty(2 * p.E, dtype=torch.int32, device=dev))
        moe_route(p, logits, r["ids"], r["w"], r["slot"], r["drop"], r["counts"], self.ws,
                  stream)
        return r

    def prepare_router(self, Wr, stream=None):
        """Splits Wr once into the workspace; later forwards skip the split (the problem's
        MOE_FLAG_ROUTER_PREPARED is set).  Call again after Wr changes."""
        self.p.flags |= FLAG_ROUTER_PREPARED
        moe_prepare_router(self.p, Wr, self.ws, stream)

    def router_logits(self, x, Wr, br, stream=None):
        logits = torch.empty((self.p.T, self.p.E), dtype=torch.float32, device=x.device)
        moe_router_logits(self.p, x, Wr, br, logits, self.ws, stream)
        return logits

    def capacity_dispatch(self, ids, w, K, stream=None):
        """Capacity selection of a given routing (ids, w [T, k]) with capacity K; returns slot,
        drop, counts and the expert-sorted layout (offsets, rowtok)."""
        p, dev = self.p, ids.device
        rows = max(min(p.T * p.k, p.E * int(K)), 1)
        r = dict(slot=torch.empty((p.T, p.k), dtype=torch.int32, device=dev),
                 drop=torch.empty((p.T, p.k), dtype=torch.uint8, device=dev),
                 counts=torch.empty(2 * p.E, dtype=torch.int32, device=dev),
                 offsets=torch.empty(p.E + 1, dtype=torch.int32, device=dev),
                 rowtok=torch.empty(rows, dtype=torch.int32, device=dev))
        moe_capacity_dispatch(p, K, ids, w, r["slot"], r["drop"], r["counts"], self.ws,
                              r["offsets"], r["rowtok"], stream)
        return r

    def dispatch(self, ids, slot, x=None, permute=False, stream=None):
        p, dev = self.p, ids.device
        offsets = torch.empty(p.E + 1, dtype=torch.int32, device=dev)
        rowtok = torch.empty(max(self.max_rows, 1), dtype=torch.int32, device=dev)
        xp = None
        if permute:
            xp = torch.empty((max(self.max_rows, 1), p.d_model), dtype=x.dtype, device=dev)
        moe_dispatch(p, ids, slot, offsets, rowtok, self.ws, x=x, x_perm=xp, stream=stream)
        return offsets, rowtok, xp

    def expert_ffn(self, x, offsets, rowtok, W1, b1, W2, b2, stream=None):
        p = self.p
        Y = torch.empty((max(self.max_rows, 1), p.d_model), dtype=x.dtype, device=x.device)
        moe_expert_ffn(p, x, offsets, rowtok, W1, b1, W2, b2, Y, self.ws, stream)
        return Y

    def combine(self, x, Y, w, ids, slot, offsets, stream=None):
        out = torch.empty_like(x)
        moe_combine(self.p, x, Y, w, ids, slot, offsets, out, self.ws, stream)
        return out

    # -- router training ------------------------------------------------------------------------
    def balance_loss(self, logits, ids, mask=None, stream=None):
        """Router losses of a routing: ``losses`` [2] (load balance, z-loss), ``counts`` [E+1]
        int32 (pairs per expert, then tokens), ``probs`` [E] (mean router probability).
        ``mask`` [T] uint8 or bool: 0 leaves a token out."""
        p, dev, what = self.p, self.ws.device, "balance_loss"
        T, E = p.T, p.E
        _need(what, "logits", logits, torch.float32, (T, E), dev)
        _need(what, "ids", ids, torch.int32, (T, p.k), dev)
        mask = None if mask is None else self._mask(what, mask)
        with _on(dev, stream) as st:
            losses = torch.empty(2, dtype=torch.float32, device=dev)
            counts = torch.empty(E + 1, dtype=torch.int32, device=dev)
            probs = torch.empty(E, dtype=torch.float32, device=dev)
            _check(_lib.moe_balance_loss(self._p, logits.data_ptr(), ids.data_ptr(), _at(mask),
                                         losses.data_ptr(), counts.data_ptr(), probs.data_ptr(),
                                         *self._ws, st), what)
        return losses, counts, probs

    def route_backward(self, logits, ids, counts=None, grad_losses=None, grad_w=None, mask=None,
                       stream=None):
        """dlogits [T, E] from the gradient of the losses (``grad_losses`` [2] on the device, with
        ``counts`` from :meth:`balance_loss`) and of the routing weights (``grad_w`` [T, k])."""
        p, dev, what = self.p, self.ws.device, "route_backward"
        T, E = p.T, p.E
        _need(what, "logits", logits, torch.float32, (T, E), dev)
        _need(what, "ids", ids, torch.int32, (T, p.k), dev)
        if grad_losses is not None:
            _need(what, "grad_losses", grad_losses, torch.float32, (2,), dev)
            _need(what, "counts", counts, torch.int32, (E + 1,), dev)
        if grad_w is not None:
            _need(what, "grad_w", grad_w, torch.float32, (T, p.k), dev)
        mask = None if mask is None else self._mask(what, mask)
        with _on(dev, stream) as st:
            dlogits = torch.empty_like(logits)
            _check(_lib.moe_route_backward(self._p, logits.data_ptr(), ids.data_ptr(), _at(mask),
                                           _at(counts), _at(grad_losses), _at(grad_w),
                                           dlogits.data_ptr(), *self._ws, st), what)
        return dlogits

    def _mask(self, what, mask):
        if isinstance(mask, torch.Tensor) and mask.dtype == torch.bool:
            mask = mask.view(torch.uint8)
        _need(what, "mask", mask, torch.uint8, (self.p.T,), self.ws.device)
        return mask

    # -- layer norm -----------------------------------------------------------------------------
    def layer_norm(self, x, gamma, beta, eps=1e-5, stream=None):
        """(y, mean, rstd) of the layer norm of x [T, d_model]; gamma, beta [d_model] float32."""
        p, dev, what = self.p, self.ws.device, "layer_norm"
        T, d = p.T, p.d_model
        _need(what, "x", x, self.torch_dtype, (T, d), dev)
        _need(what, "gamma", gamma, torch.float32, (d,), dev)
        _need(what, "beta", beta, torch.float32, (d,), dev)
        with _on(dev, stream) as st:
            y = torch.empty_like(x)
            mean = torch.empty(T, dtype=torch.float32, device=dev)
            rstd = torch.empty_like(mean)
            _check(_lib.moe_layer_norm(self._p, x.data_ptr(), gamma.data_ptr(), beta.data_ptr(),
                                       eps, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), st),
                   what)
        return y, mean, rstd

    def layer_norm_backward(self, dy, x, gamma, mean, rstd, dres=None, stream=None):
        """(dx, dgamma, dbeta) from dy and the forward's x, mean and rstd; ``dres`` [T, d_model]
        (the residual's gradient) is added to dx."""
        p, dev, what = self.p, self.ws.device, "layer_norm_backward"
        T, d, dtype = p.T, p.d_model, self.torch_dtype
        _need(what, "dy", dy, dtype, (T, d), dev)
        _need(what, "x", x, dtype, (T, d), dev)
        if dres is not None:
            _need(what, "dres", dres, dtype, (T, d), dev)
        _need(what, "gamma", gamma, torch.float32, (d,), dev)
        _need(what, "mean", mean, torch.float32, (T,), dev)
        _need(what, "rstd", rstd, torch.float32, (T,), dev)
        with _on(dev, stream) as st:
            dx = torch.empty_like(x)
            dgamma = torch.empty_like(gamma)
            dbeta = torch.empty_like(gamma)
            _check(_lib.moe_layer_norm_backward(self._p, dy.data_ptr(), x.data_ptr(),
                                                gamma.data_ptr(), mean.data_ptr(),
                                                rstd.data_ptr(), _at(dres), dx.data_ptr(),
                                                dgamma.data_ptr(), dbeta.data_ptr(), *self._ws,
                                                st), what)
        return dx, dgamma, dbeta

    # -- 4-bit expert weights -------------------------------------------------------------------
    def _need_experts(self, what, W1, b1, W2, b2):
        p, dev = self.p, self.ws.device
        F1 = 2 * p.d_ff if p.flags & FLAG_GATED else p.d_ff
        for name, W, shape in (("W1", W1, (p.E, F1, p.d_model)),
                               ("W2", W2, (p.E, p.d_model, p.d_ff))):
            if isinstance(W, W4Weights):
                W._need(what, name, shape, dev)
            else:
                _need(what, name, W, self.torch_dtype, shape, dev)
        for name, b, n in (("b1", b1, F1), ("b2", b2, p.d_model)):
            if b is not None:
                _need(what, name, b, torch.float32, (p.E, n), dev)

    def expert_ffn_w4(self, x, offsets, rowtok, W1, b1, W2, b2, stream=None):
        """:meth:`expert_ffn` over :class:`W4Weights`; the layer is made with ``w4=True``."""
        p, dev, what = self.p, self.ws.device, "expert_ffn_w4"
        if not (isinstance(W1, W4Weights) and isinstance(W2, W4Weights)):
            raise MoeError(MOE_ERR_INVALID_ARG, what + ": W1 and W2 must be W4Weights")
        _need(what, "x", x, torch.bfloat16, (p.T, p.d_model), dev)
        _need(what, "offsets", offsets, torch.int32, (p.E + 1,), dev)
        rows = rowtok.numel() if isinstance(rowtok, torch.Tensor) else 0
        _need(what, "rowtok", rowtok, torch.int32, (max(self.max_rows, rows),), dev)
        self._need_experts(what, W1, b1, W2, b2)
        with _on(dev, stream) as st:
            Y = torch.empty((max(self.max_rows, 1), p.d_model), dtype=x.dtype, device=dev)
            _check(_lib.moe_expert_ffn_packed(self._p, x.data_ptr(), offsets.data_ptr(),
                                              rowtok.data_ptr(), ctypes.byref(W1.c), _at(b1),
                                              ctypes.byref(W2.c), _at(b2), Y.data_ptr(),
                                              *self._ws, st), what)
        return Y

    # -- the layer as a block of a model --------------------------------------------------------
    def forward_block(self, x, Wr, br, W1, b1, W2, b2, norm=None, stream=None):
        """The whole layer with an optional layer norm in front, ``norm`` = (gamma, beta, eps):
        out = x + experts(norm(x)); W1 and W2 are tensors or both :class:`W4Weights`.  Returns
        (out, routing and norm results: logits_out, ids_out, ..., and y, mean, rstd)."""
        p, dev, what = self.p, self.ws.device, "forward_block"
        w4 = isinstance(W1, W4Weights)
        if w4 != isinstance(W2, W4Weights):
            raise MoeError(MOE_ERR_INVALID_ARG, what + ": W1 and W2 must both be 4-bit or neither")
        _need(what, "x", x, self.torch_dtype, (p.T, p.d_model), dev)
        _need(what, "Wr", Wr, torch.float32, (p.d_model, p.E), dev)
        if br is not None:
            _need(what, "br", br, torch.float32, (p.E,), dev)
        self._need_experts(what, W1, b1, W2, b2)
        if norm is not None:
            if not isinstance(norm, (tuple, list)) or len(norm) != 3:
                raise MoeError(MOE_ERR_INVALID_ARG, what + ": norm must be (gamma, beta, eps)")
            for name, t in (("gamma", norm[0]), ("beta", norm[1])):
                _need(what, name, t, torch.float32, (p.d_model,), dev)
        with _on(dev, stream) as st:
            def new(*shape, dtype=torch.float32):
                return torch.empty(shape, dtype=dtype, device=dev)

            out = torch.empty_like(x)
            extra = dict(logits_out=new(p.T, p.E), ids_out=new(p.T, p.k, dtype=torch.int32),
                         w_out=new(p.T, p.k), slot_out=new(p.T, p.k, dtype=torch.int32),
                         drop_out=new(p.T, p.k, dtype=torch.uint8),
                         counts_out=new(2 * p.E, dtype=torch.int32))
            n, kept = None, {}
            if norm is not None:
                kept = dict(y=torch.empty_like(x), mean=new(p.T), rstd=new(p.T))
                n = Norm(norm[0].data_ptr(), norm[1].data_ptr(), float(norm[2]),
                         *(kept[key].data_ptr() for key in ("y", "mean", "rstd")))
            moe_forward_block(p, x, n, Wr, br, None if w4 else W1, None if w4 else W2,
                              W1.c if w4 else None, W2.c if w4 else None, b1, b2, out, self.ws,
                              stream=st, **extra)
        return out, {**extra, **kept}
