"""GB300-native AdaComp: per-layer adaptive residual gradient compression.

A thin ctypes binding over the C ABI of ``libadacomp.so`` (``include/adacomp.h``).
Every function keeps the C name and only marshals arguments: torch tensors become
device pointers, the stream defaults to torch's current stream, and a non-OK status
raises :class:`AdacompError`. All computation runs in the library's CUDA kernels;
there is no CPU fallback, and using the binding without the built library raises.

Method: "AdaComp (Adaptive Residual Gradient Compression)", Claims > Mechanism
#r629-local-bin-soft-threshold-and-mean-gmax-quantization.
"""
from __future__ import annotations

import ctypes
import os
from typing import Sequence

import torch

from .build import lib_path as _lib_path

# libadacomp.so, or libadacomp_debug.so when ADACOMP_DEBUG_CHECKS=1 (a debug build)
_LIB_PATH = _lib_path()

OK, ERR_INVALID_ARG, ERR_ALIGNMENT, ERR_WORKSPACE, ERR_CAPACITY, ERR_CUDA, ERR_TIMEOUT, \
    ERR_BAD_MESSAGE = range(8)
F32, BF16 = 0, 1
RULE_ADACOMP, RULE_LOCAL_SELECTION = 0, 1
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = range(5)
MAX_GROUP = 128
MAX_LEARNERS = 256
DECODE_WS_FIXED = 10240
RECURRENCE_CHUNK = 64   # steps between the states that the recurrence's forward pass keeps
ADAMW_BLOCK = 256       # elements that share a scale of 8-bit optimiser states
MAX_TEACHER = 256       # tokens of a teacher's list
STATIC_WS_BYTES = 1 << 20  # ADACOMP_STATIC_WS_BYTES: the largest workspace adacomp_compress_static_ws holds

_lib = None


class AdacompError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {adacomp_status_string(status)} ({status})")


def lib() -> ctypes.CDLL:
    """The loaded libadacomp.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"{_LIB_PATH} is missing: build it with "
                              "residual_gradient_compression_gb300.build.build()")
        L = ctypes.CDLL(_LIB_PATH)
        vp, sz, i32, i64, u64 = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32,
                                 ctypes.c_int64, ctypes.c_uint64)
        P = ctypes.POINTER
        L.adacomp_init_layer.argtypes = [P(vp), i64, i32, ctypes.c_int, P(sz), P(sz), P(sz)]
        L.adacomp_init_group.argtypes = [P(vp), i32, P(i64), P(i32), P(i32), P(sz), P(sz), P(sz)]
        L.adacomp_compress.argtypes = [vp, vp, vp, vp, sz, vp, sz, vp]
        L.adacomp_compress_group.argtypes = [vp, P(vp), P(vp), P(vp), P(sz), vp, sz, vp]
        L.adacomp_decode_accumulate.argtypes = [vp, P(vp), P(u64), i32, vp, vp, sz, vp]
        L.adacomp_decode_accumulate_group.argtypes = [vp, P(vp), P(u64), i32, P(vp), vp, sz, vp]
        L.adacomp_query.argtypes = [vp, vp, i32, vp, P(u64), P(ctypes.c_float), P(i32)]
        L.adacomp_decode_status.argtypes = [vp, vp, vp, P(i32)]
        L.adacomp_set_timeout_ns.argtypes = [vp, u64]
        L.adacomp_set_timing_events.argtypes = [vp, vp, vp, vp]
        L.adacomp_set_fault_injection.argtypes = [vp, ctypes.c_uint32]
        L.adacomp_set_lazy_fixup.argtypes = [vp, i32, P(sz)]
        L.adacomp_set_selection_rule.argtypes = [vp, i32]
        f32 = ctypes.c_float
        L.adacomp_decode_sgd.argtypes = [vp, P(vp), P(u64), i32, vp, vp, f32, f32, f32, vp, sz, vp]
        L.adacomp_decode_sgd_group.argtypes = [vp, P(vp), P(u64), i32, P(vp), P(vp), f32, f32, f32, vp, sz, vp]
        L.adacomp_decode_adam.argtypes = [vp, P(vp), P(u64), i32, vp, vp, vp] + [f32] * 7 + [vp, sz, vp]
        L.adacomp_decode_adam_group.argtypes = [vp, P(vp), P(u64), i32, P(vp), P(vp), P(vp)] + [f32] * 7 + [vp, sz, vp]
        L.adacomp_materialize.argtypes = [vp, vp, vp, sz, vp]
        L.adacomp_materialize_group.argtypes = [vp, P(vp), vp, sz, vp]
        L.adacomp_free.argtypes = [vp]
        L.adacomp_free.restype = None
        L.adacomp_layer_norm_init.argtypes = [P(vp), i64, ctypes.c_int, ctypes.c_int, f32]
        L.adacomp_layer_norm_forward.argtypes = [vp, i64, vp, i64, vp, vp, vp, i64, vp, vp, vp]
        L.adacomp_layer_norm_backward_ws_bytes.argtypes = [vp, i64]
        L.adacomp_layer_norm_backward_ws_bytes.restype = sz
        L.adacomp_layer_norm_backward.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, vp, vp, sz, vp]
        L.adacomp_recurrence_init.argtypes = [P(vp), i64, ctypes.c_int]
        L.adacomp_recurrence_carry_bytes.argtypes = [vp, i64, i64]
        L.adacomp_recurrence_carry_bytes.restype = sz
        seq = [vp, i64, i64]
        L.adacomp_recurrence_forward.argtypes = [vp, i64, i64] + seq * 2 + [vp, vp] + seq + [vp, vp, vp]
        L.adacomp_recurrence_backward.argtypes = [vp, i64, i64] + seq * 3 + [vp, vp, vp] + seq * 2 + [vp, vp]
        L.adacomp_recurrence_set_timeout_ns.argtypes = [vp, u64]
        L.adacomp_recurrence_set_fault_injection.argtypes = [vp, ctypes.c_uint32]
        L.adacomp_adamw_init.argtypes = [P(vp), i32, P(i64), P(i32), P(i32), P(f32), i32, P(sz)]
        L.adacomp_grad_norm.argtypes = [vp, vp, f32, f32, vp, vp, sz, vp]
        L.adacomp_adamw_step.argtypes = [vp] * 8 + [f32] * 7 + [vp, vp]
        L.adacomp_linear_init.argtypes = [P(vp), i64, i64, ctypes.c_int, ctypes.c_int]
        row = [vp, i64]
        L.adacomp_linear_forward.argtypes = [vp, i64] + row * 2 + [vp] + row * 3 + [vp, sz, vp]
        L.adacomp_linear_backward.argtypes = [vp, i64] + row * 6 + [vp, vp, sz, vp]
        L.adacomp_vocab_init.argtypes = [P(vp), i64, i64, ctypes.c_int]
        L.adacomp_vocab_loss_forward.argtypes = [vp, i64] + row * 2 + [vp, i32, vp, vp, vp, sz, vp]
        L.adacomp_vocab_loss_backward.argtypes = [vp, i64] + row * 2 + [vp, i32, vp] + row * 3 + [vp, sz, vp]
        lists = [i32] + row * 2 + [ctypes.c_int, f32]
        L.adacomp_distill_forward.argtypes = [vp, i64] + row * 2 + lists + [vp, vp, vp, sz, vp]
        L.adacomp_distill_backward.argtypes = [vp, i64] + row * 2 + lists + [vp] + row * 3 + [vp, sz, vp]
        for name, more in (("linear_forward", []), ("linear_backward", []), ("vocab_loss_forward", []),
                           ("vocab_loss_backward", []), ("distill_forward", [i32]), ("distill_backward", [i32])):
            getattr(L, f"adacomp_{name}").restype = ctypes.c_int
            size = getattr(L, f"adacomp_{name}_ws_bytes")
            size.argtypes, size.restype = [vp, i64] + more, sz
        for kind in ("linear", "vocab"):
            for name, value in (("set_timeout_ns", u64), ("set_fault_injection", ctypes.c_uint32)):
                call = getattr(L, f"adacomp_{kind}_{name}")
                call.argtypes, call.restype = [vp, value], ctypes.c_int
        for name in ("adacomp_layer_norm_free", "adacomp_recurrence_free", "adacomp_adamw_free", "adacomp_linear_free",
                     "adacomp_vocab_free"):
            getattr(L, name).argtypes = [vp]
            getattr(L, name).restype = None
        L.adacomp_status_string.argtypes = [ctypes.c_int]
        L.adacomp_status_string.restype = ctypes.c_char_p
        for name in ("adacomp_init_layer", "adacomp_init_group", "adacomp_compress",
                     "adacomp_compress_group", "adacomp_decode_accumulate",
                     "adacomp_decode_accumulate_group", "adacomp_query", "adacomp_decode_status",
                     "adacomp_set_timeout_ns", "adacomp_set_timing_events",
                     "adacomp_set_fault_injection", "adacomp_set_lazy_fixup", "adacomp_set_selection_rule",
                     "adacomp_materialize", "adacomp_decode_sgd", "adacomp_decode_sgd_group",
                     "adacomp_decode_adam", "adacomp_decode_adam_group", "adacomp_materialize_group",
                     "adacomp_layer_norm_init", "adacomp_layer_norm_forward", "adacomp_layer_norm_backward",
                     "adacomp_recurrence_init", "adacomp_recurrence_forward", "adacomp_recurrence_backward",
                     "adacomp_recurrence_set_timeout_ns", "adacomp_recurrence_set_fault_injection",
                     "adacomp_adamw_init", "adacomp_grad_norm", "adacomp_adamw_step",
                     "adacomp_linear_init", "adacomp_vocab_init"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != OK:
        raise AdacompError(status, where)


# torch's current stream without the Stream object that torch.cuda.current_stream() makes (3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _device is not None and torch.cuda.is_initialized():
            return _raw_stream(_device())
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t) -> int:
    if isinstance(t, torch.Tensor):
        if not t.is_contiguous():
            raise ValueError("tensors passed to the library must be contiguous")
        return t.data_ptr()
    return int(t)


class Handle:
    """Host-side handle for one layer or a group of layers (no device memory)."""

    def __init__(self, ptr, num_layers, ns, bin_lens, dtypes, max_msg_bytes, ws, dws):
        self.ptr = ptr
        self.num_layers = num_layers
        self.n = list(ns)
        self.bin_len = list(bin_lens)
        self.dtype = list(dtypes)
        self.max_msg_bytes = list(max_msg_bytes)
        self.compress_ws_bytes = ws
        self.decode_ws_bytes_per_learner = dws

    def decode_ws_bytes(self, K: int) -> int:
        return DECODE_WS_FIXED + K * self.decode_ws_bytes_per_learner

    def __del__(self):
        if getattr(self, "ptr", None) and _lib is not None:
            _lib.adacomp_free(self.ptr)
            self.ptr = None


def adacomp_init_layer(n: int, bin_len: int, dw_dtype: int = F32) -> Handle:
    h = ctypes.c_void_p()
    mm, ws, dws = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().adacomp_init_layer(ctypes.byref(h), n, bin_len, dw_dtype, ctypes.byref(mm),
                                    ctypes.byref(ws), ctypes.byref(dws)), "adacomp_init_layer")
    return Handle(h.value, 1, [n], [bin_len], [dw_dtype], [mm.value], ws.value, dws.value)


def adacomp_init_group(ns: Sequence[int], bin_lens: Sequence[int], dw_dtypes: Sequence[int]) -> Handle:
    L = len(ns)
    h = ctypes.c_void_p()
    mm = (ctypes.c_size_t * L)()
    ws, dws = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().adacomp_init_group(ctypes.byref(h), L, (ctypes.c_int64 * L)(*ns),
                                    (ctypes.c_int32 * L)(*bin_lens), (ctypes.c_int32 * L)(*dw_dtypes),
                                    mm, ctypes.byref(ws), ctypes.byref(dws)), "adacomp_init_group")
    return Handle(h.value, L, ns, bin_lens, dw_dtypes, list(mm), ws.value, dws.value)


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def adacomp_compress(h: Handle, residue, dW, msg, ws, stream=None):
    _check(lib().adacomp_compress(h.ptr, _ptr(residue), _ptr(dW), _ptr(msg), _nbytes(msg),
                                  _ptr(ws), _nbytes(ws), _stream(stream)), "adacomp_compress")


def adacomp_compress_group(h: Handle, residues, dWs, msgs, ws, stream=None):
    L = h.num_layers
    VP = ctypes.c_void_p * L
    _check(lib().adacomp_compress_group(
        h.ptr, VP(*[_ptr(r) for r in residues]), VP(*[_ptr(d) for d in dWs]),
        VP(*[_ptr(m) for m in msgs]), (ctypes.c_size_t * L)(*[_nbytes(m) for m in msgs]),
        _ptr(ws), _nbytes(ws), _stream(stream)), "adacomp_compress_group")


def _lengths(msg_bytes, count: int):
    lens = [int(b) for b in msg_bytes]
    if len(lens) != count:
        raise ValueError(f"expected {count} message lengths, got {len(lens)}")
    return (ctypes.c_uint64 * count)(*lens)


def adacomp_decode_accumulate(h: Handle, msgs, msg_bytes, dense, ws, stream=None):
    """msgs: K device buffers; msg_bytes: the K message lengths in bytes."""
    K = len(msgs)
    arr = (ctypes.c_void_p * K)(*[_ptr(m) for m in msgs])
    _check(lib().adacomp_decode_accumulate(h.ptr, arr, _lengths(msg_bytes, K), K, _ptr(dense), _ptr(ws),
                                           _nbytes(ws), _stream(stream)), "adacomp_decode_accumulate")


def adacomp_decode_accumulate_group(h: Handle, msgs, msg_bytes, denses, ws, stream=None):
    """msgs[l][k]: learner k's message for layer l, msg_bytes[l][k] its length;
    denses[l]: layer l's dense buffer."""
    L = h.num_layers
    K = len(msgs[0])
    flat = [_ptr(m) for per_layer in msgs for m in per_layer]
    lens = _lengths([b for per_layer in msg_bytes for b in per_layer], L * K)
    _check(lib().adacomp_decode_accumulate_group(
        h.ptr, (ctypes.c_void_p * (L * K))(*flat), lens, K, (ctypes.c_void_p * L)(*[_ptr(d) for d in denses]),
        _ptr(ws), _nbytes(ws), _stream(stream)), "adacomp_decode_accumulate_group")


def adacomp_query(h: Handle, ws, layer: int = 0, stream=None):
    """(message bytes, s, device status) of the last compress that used ws."""
    mb, s, st = ctypes.c_uint64(), ctypes.c_float(), ctypes.c_int32()
    _check(lib().adacomp_query(h.ptr, _ptr(ws), layer, _stream(stream), ctypes.byref(mb),
                               ctypes.byref(s), ctypes.byref(st)), "adacomp_query")
    return mb.value, s.value, st.value


def adacomp_decode_status(h: Handle, ws, stream=None) -> int:
    st = ctypes.c_int32()
    _check(lib().adacomp_decode_status(h.ptr, _ptr(ws), _stream(stream), ctypes.byref(st)),
           "adacomp_decode_status")
    return st.value


def adacomp_set_timeout_ns(h: Handle, ns: int):
    _check(lib().adacomp_set_timeout_ns(h.ptr, ns), "adacomp_set_timeout_ns")


def adacomp_set_timing_events(h: Handle, before=None, mid=None, after=None):
    """Record caller-owned torch.cuda.Event objects around the two compress kernels."""
    def raw(ev):
        return None if ev is None else ctypes.c_void_p(ev.cuda_event)
    _check(lib().adacomp_set_timing_events(h.ptr, raw(before), raw(mid), raw(after)),
           "adacomp_set_timing_events")


def adacomp_set_fault_injection(h: Handle, skip_tile: int = 0xFFFFFFFF):
    """Test hook: the given tile never publishes, so its successors time out."""
    _check(lib().adacomp_set_fault_injection(h.ptr, skip_tile), "adacomp_set_fault_injection")


def adacomp_decode_sgd(h: Handle, msgs, msg_bytes, weights, momentum, lr: float, mu: float, ws,
                       grad_scale: float = 1.0, stream=None):
    K = len(msgs)
    arr = (ctypes.c_void_p * K)(*[_ptr(m) for m in msgs])
    _check(lib().adacomp_decode_sgd(h.ptr, arr, _lengths(msg_bytes, K), K, _ptr(weights), _ptr(momentum), lr, mu,
                                    grad_scale, _ptr(ws), _nbytes(ws), _stream(stream)), "adacomp_decode_sgd")


def adacomp_decode_sgd_group(h: Handle, msgs, msg_bytes, weights, momentum, lr: float, mu: float, ws,
                             grad_scale: float = 1.0, stream=None):
    """msgs, msg_bytes: per layer a list of K messages and their lengths (layer-major, as
    adacomp_decode_accumulate_group)."""
    L = h.num_layers
    K = len(msgs[0])
    arr = (ctypes.c_void_p * (L * K))(*[_ptr(m) for layer in msgs for m in layer])
    lens = _lengths([b for layer in msg_bytes for b in layer], L * K)
    VP = ctypes.c_void_p * L
    _check(lib().adacomp_decode_sgd_group(h.ptr, arr, lens, K, VP(*[_ptr(w) for w in weights]),
                                          VP(*[_ptr(v) for v in momentum]), lr, mu, grad_scale, _ptr(ws),
                                          _nbytes(ws), _stream(stream)), "adacomp_decode_sgd_group")


def adacomp_decode_adam(h: Handle, msgs, msg_bytes, weights, m, v, lr: float, beta1: float, beta2: float,
                        eps: float, bias_correction1: float, bias_correction2: float, ws, grad_scale: float = 1.0,
                        stream=None):
    K = len(msgs)
    arr = (ctypes.c_void_p * K)(*[_ptr(x) for x in msgs])
    _check(lib().adacomp_decode_adam(h.ptr, arr, _lengths(msg_bytes, K), K, _ptr(weights), _ptr(m), _ptr(v), lr,
                                     beta1, beta2, eps, bias_correction1, bias_correction2, grad_scale, _ptr(ws),
                                     _nbytes(ws), _stream(stream)), "adacomp_decode_adam")


def adacomp_decode_adam_group(h: Handle, msgs, msg_bytes, weights, m, v, lr: float, beta1: float, beta2: float,
                              eps: float, bias_correction1: float, bias_correction2: float, ws,
                              grad_scale: float = 1.0, stream=None):
    """msgs, msg_bytes: per layer a list of K messages and their lengths (layer-major);
    weights, m, v: one buffer per layer."""
    L = h.num_layers
    K = len(msgs[0])
    arr = (ctypes.c_void_p * (L * K))(*[_ptr(x) for layer in msgs for x in layer])
    lens = _lengths([b for layer in msg_bytes for b in layer], L * K)
    VP = ctypes.c_void_p * L
    _check(lib().adacomp_decode_adam_group(h.ptr, arr, lens, K, VP(*[_ptr(x) for x in weights]),
                                           VP(*[_ptr(x) for x in m]), VP(*[_ptr(x) for x in v]), lr, beta1, beta2,
                                           eps, bias_correction1, bias_correction2, grad_scale, _ptr(ws),
                                           _nbytes(ws), _stream(stream)), "adacomp_decode_adam_group")


def adacomp_set_selection_rule(h: Handle, rule: int):
    """RULE_ADACOMP (default) or RULE_LOCAL_SELECTION (abs(G) >= g_max, no probe)."""
    _check(lib().adacomp_set_selection_rule(h.ptr, rule), "adacomp_set_selection_rule")


def adacomp_set_lazy_fixup(h: Handle, enable: bool = True) -> int:
    """Defers the residue fix-up to the next compress call; returns (and records on
    the handle) the compress workspace size the mode needs."""
    ws = ctypes.c_size_t()
    _check(lib().adacomp_set_lazy_fixup(h.ptr, int(bool(enable)), ctypes.byref(ws)), "adacomp_set_lazy_fixup")
    h.compress_ws_bytes = ws.value
    return ws.value


def adacomp_materialize(h: Handle, residue, ws, stream=None):
    _check(lib().adacomp_materialize(h.ptr, _ptr(residue), _ptr(ws), _nbytes(ws), _stream(stream)),
           "adacomp_materialize")


def adacomp_materialize_group(h: Handle, residues, ws, stream=None):
    VP = ctypes.c_void_p * h.num_layers
    _check(lib().adacomp_materialize_group(h.ptr, VP(*[_ptr(r) for r in residues]), _ptr(ws), _nbytes(ws),
                                           _stream(stream)), "adacomp_materialize_group")


def adacomp_free(h: Handle):
    if h.ptr:
        lib().adacomp_free(h.ptr)
        h.ptr = None


def adacomp_status_string(status: int) -> str:
    return lib().adacomp_status_string(status).decode()


# ---------------------------------------------------------------------------------------
# Training operators around the compressor: layer norm, a gated linear recurrence, the norm
# of many gradients and an AdamW step. Tensors may be strided as the header states.

_DTYPES = {F32: torch.float32, BF16: torch.bfloat16}


class _TrainHandle:
    """Host-side handle of a training operator (sizes and types only)."""

    def __init__(self, ptr, free):
        self.ptr = ptr
        self._free = free

    def __del__(self):
        if getattr(self, "ptr", None) and _lib is not None:
            getattr(_lib, self._free)(self.ptr)
            self.ptr = None


def _bad(what: str):
    raise ValueError(what)


def _array(t, count: int, dtype, what: str):
    """The address of a contiguous CUDA tensor of `count` elements; None stays None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != count or not t.is_cuda or not t.is_contiguous():
        _bad(f"{what} must be a contiguous CUDA tensor of {count} {dtype} elements")
    return t.data_ptr()


def _matrix(t, h, what: str):
    """(address, rows, row stride) of a tensor whose last axis is a row of h.dim elements."""
    shape, dim = t.shape, h.dim
    if t.dtype is not h.torch_dtype or not t.is_cuda or not shape or shape[-1] != dim:
        _bad(f"{what} must be a CUDA tensor of {h.torch_dtype} with rows of {dim}")
    if len(shape) == 2:
        stride, one = t.stride()
        if one != 1 and dim > 1:
            _bad(f"{what}: the elements of a row must be contiguous")
        return t.data_ptr(), shape[0], stride
    if not t.is_contiguous():
        _bad(f"{what}: a tensor that is not a matrix must be contiguous")
    return t.data_ptr(), t.numel() // dim, dim


def _sequence(t, h, shape, what: str):
    """(address, batch stride, step stride) of a [batch, steps, channels] tensor."""
    if t.dtype is not h.torch_dtype or not t.is_cuda or t.shape != shape:
        _bad(f"{what} must be a CUDA tensor of {h.torch_dtype} and shape {tuple(shape)}")
    batch, step, one = t.stride()
    if one != 1 and shape[2] > 1:
        _bad(f"{what}: the channels of a step must be contiguous")
    return t.data_ptr(), batch, step


def adacomp_layer_norm_init(dim: int, x_dtype: int = F32, w_dtype: int = F32, eps: float = 1e-5) -> _TrainHandle:
    p = ctypes.c_void_p()
    _check(lib().adacomp_layer_norm_init(ctypes.byref(p), dim, x_dtype, w_dtype, eps), "adacomp_layer_norm_init")
    h = _TrainHandle(p.value, "adacomp_layer_norm_free")
    h.dim, h.torch_dtype, h.w_torch_dtype = dim, _DTYPES[x_dtype], _DTYPES[w_dtype]
    return h


def adacomp_layer_norm_forward(h, x, w, b, y, mean=None, rstd=None, stream=None):
    """y = norm of the rows of x; mean and rstd (fp32, one value per row) are for the backward pass."""
    xp, rows, xs = _matrix(x, h, "x")
    yp, yrows, ys = _matrix(y, h, "y")
    if yrows != rows:
        _bad("x and y have unlike numbers of rows")
    _check(lib().adacomp_layer_norm_forward(
        h.ptr, rows, xp, xs, _array(w, h.dim, h.w_torch_dtype, "w"), _array(b, h.dim, h.w_torch_dtype, "b"), yp, ys,
        _array(mean, rows, torch.float32, "mean"), _array(rstd, rows, torch.float32, "rstd"), _stream(stream)),
        "adacomp_layer_norm_forward")


def adacomp_layer_norm_backward_ws_bytes(h, rows: int) -> int:
    return lib().adacomp_layer_norm_backward_ws_bytes(h.ptr, rows)


def adacomp_layer_norm_backward(h, dy, x, w, mean, rstd, dx, dw, db, ws, stream=None):
    """dx, dw and db (which may be None) from dy and the forward pass's x, mean and rstd."""
    xp, rows, xs = _matrix(x, h, "x")
    gp, grows, gs = _matrix(dy, h, "dy")
    op, orows, os_ = _matrix(dx, h, "dx")
    if grows != rows or orows != rows:
        _bad("dy, x and dx have unlike numbers of rows")
    wt = h.w_torch_dtype
    _check(lib().adacomp_layer_norm_backward(
        h.ptr, rows, gp, gs, xp, xs, _array(w, h.dim, wt, "w"), _array(mean, rows, torch.float32, "mean"),
        _array(rstd, rows, torch.float32, "rstd"), op, os_, _array(dw, h.dim, wt, "dw"), _array(db, h.dim, wt, "db"),
        _ptr(ws), _nbytes(ws), _stream(stream)), "adacomp_layer_norm_backward")


def adacomp_layer_norm_free(h):
    h.__del__()


def adacomp_recurrence_init(channels: int, dtype: int = F32) -> _TrainHandle:
    p = ctypes.c_void_p()
    _check(lib().adacomp_recurrence_init(ctypes.byref(p), channels, dtype), "adacomp_recurrence_init")
    h = _TrainHandle(p.value, "adacomp_recurrence_free")
    h.channels, h.torch_dtype = channels, _DTYPES[dtype]
    return h


def adacomp_recurrence_carry_bytes(h, batch: int, steps: int) -> int:
    return lib().adacomp_recurrence_carry_bytes(h.ptr, batch, steps)


def _carry(h, carry, batch, steps):
    return _array(carry, batch * -(-steps // RECURRENCE_CHUNK) * h.channels, torch.float32, "carry")


def adacomp_recurrence_forward(h, z, x, y, h0=None, lengths=None, h_last=None, carry=None, stream=None):
    """y_t = h_t = a_t h_{t-1} + (1 - a_t) x_t with a = sigmoid(z); [batch, steps, channels] tensors."""
    shape = z.shape
    if len(shape) != 3 or shape[2] != h.channels:
        _bad(f"z must have the shape [batch, steps, {h.channels}]")
    batch, steps, n = shape[0], shape[1], shape[0] * h.channels
    _check(lib().adacomp_recurrence_forward(
        h.ptr, batch, steps, *_sequence(z, h, shape, "z"), *_sequence(x, h, shape, "x"),
        _array(h0, n, torch.float32, "h0"), _array(lengths, batch, torch.int32, "lengths"),
        *_sequence(y, h, shape, "y"), _array(h_last, n, torch.float32, "h_last"), _carry(h, carry, batch, steps),
        _stream(stream)), "adacomp_recurrence_forward")


def adacomp_recurrence_backward(h, z, x, dy, carry, dz, dx, lengths=None, dh_last=None, dh0=None, stream=None):
    """dz, dx and dh0 from dy, dh_last, and the inputs and the carry of the forward pass."""
    shape = z.shape
    if len(shape) != 3 or shape[2] != h.channels:
        _bad(f"z must have the shape [batch, steps, {h.channels}]")
    batch, steps, n = shape[0], shape[1], shape[0] * h.channels
    _check(lib().adacomp_recurrence_backward(
        h.ptr, batch, steps, *_sequence(z, h, shape, "z"), *_sequence(x, h, shape, "x"),
        *_sequence(dy, h, shape, "dy"), _carry(h, carry, batch, steps), _array(lengths, batch, torch.int32, "lengths"),
        _array(dh_last, n, torch.float32, "dh_last"), *_sequence(dz, h, shape, "dz"), *_sequence(dx, h, shape, "dx"),
        _array(dh0, n, torch.float32, "dh0"), _stream(stream)), "adacomp_recurrence_backward")


def adacomp_recurrence_set_timeout_ns(h, ns: int):
    """Bound on a wait within a cluster; results behind one that runs out are NaN."""
    _check(lib().adacomp_recurrence_set_timeout_ns(h.ptr, ns), "adacomp_recurrence_set_timeout_ns")


def adacomp_recurrence_set_fault_injection(h, silent_cta: int = 0xFFFFFFFF):
    """Test hook: the given CTA of every cluster writes nothing to the others, whose waits run out."""
    _check(lib().adacomp_recurrence_set_fault_injection(h.ptr, silent_cta), "adacomp_recurrence_set_fault_injection")


def adacomp_recurrence_free(h):
    h.__del__()


class Pointers:
    """Tensors whose addresses are passed together; made once, used by many calls."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        for t in self.tensors:
            if t is not None and not (t.is_cuda and t.is_contiguous()):
                _bad("the tensors must be contiguous CUDA tensors")
        self.array = (ctypes.c_void_p * max(1, len(self.tensors)))(
            *[None if t is None else t.data_ptr() for t in self.tensors])
        self.kinds = [None if t is None else (t.numel(), t.dtype) for t in self.tensors]
        self.checked = None  # the sizes and types that these tensors have been compared with


def adacomp_pointers(tensors) -> Pointers:
    """Tensors to pass to adacomp_grad_norm or adacomp_adamw_step (which also take plain lists).
    Their addresses are taken here, and their memory is kept: a tensor that is given other memory
    afterwards (t.data = ..., resize_) is not followed, and wants new pointers."""
    return Pointers(None if t is None else t.detach() for t in tensors)


def _pointers(tensors, expect, what: str, may_miss: bool = False):
    if tensors is None:
        return None
    p = tensors if isinstance(tensors, Pointers) else Pointers(tensors)
    if p.checked is not expect:
        if len(p.kinds) != len(expect):
            _bad(f"{what}: {len(expect)} tensors are wanted, got {len(p.kinds)}")
        for i, (k, e) in enumerate(zip(p.kinds, expect)):
            if (k is None and not may_miss) or (k is not None and k != e):
                _bad(f"{what}[{i}] must be a tensor of {e[0]} elements of {e[1]}")
        p.checked = expect
    return p.array


def adacomp_adamw_init(ns: Sequence[int], w_dtypes: Sequence[int], g_dtypes: Sequence[int], weight_decay=None,
                       state_bits: int = 32) -> _TrainHandle:
    """Tensor i has ns[i] elements; weight_decay: one value per tensor (None: none decays).
    The handle's norm_ws_bytes is the workspace size of adacomp_grad_norm."""
    ns, count = [int(n) for n in ns], len(ns)
    if len(w_dtypes) != count or len(g_dtypes) != count or (weight_decay is not None and len(weight_decay) != count):
        _bad("one type and one weight decay are wanted for each tensor")
    p, ws = ctypes.c_void_p(), ctypes.c_size_t()
    I32 = ctypes.c_int32 * max(1, count)
    _check(lib().adacomp_adamw_init(
        ctypes.byref(p), count, (ctypes.c_int64 * max(1, count))(*ns), I32(*w_dtypes), I32(*g_dtypes),
        None if weight_decay is None else (ctypes.c_float * max(1, count))(*weight_decay), state_bits,
        ctypes.byref(ws)), "adacomp_adamw_init")
    h = _TrainHandle(p.value, "adacomp_adamw_free")
    h.norm_ws_bytes, h.state_bits = ws.value, state_bits
    h.weights = [(n, _DTYPES[d]) for n, d in zip(ns, w_dtypes)]
    h.grads = [(n, _DTYPES[d]) for n, d in zip(ns, g_dtypes)]
    h.states = [(n, torch.float8_e4m3fn if state_bits == 8 else torch.float32) for n in ns]
    h.scales = [(-(-n // ADAMW_BLOCK), torch.float32) for n in ns]
    h.copies = [(n, torch.bfloat16) for n in ns]
    return h


def adacomp_grad_norm(h, grads, result, ws, max_norm: float = 0.0, grad_scale: float = 1.0, stream=None):
    """result[0] = grad_scale times the norm of all gradients, result[1] the coefficient that
    scales and clips them to max_norm (0: no clipping; NaN when the norm is not finite)."""
    _check(lib().adacomp_grad_norm(h.ptr, _pointers(grads, h.grads, "grads"), grad_scale, max_norm,
                                   _array(result, 2, torch.float32, "result"), _ptr(ws), _nbytes(ws),
                                   _stream(stream)), "adacomp_grad_norm")


def adacomp_adamw_step(h, weights, grads, m, v, lr: float, beta1: float, beta2: float, eps: float,
                       bias_correction1: float, bias_correction2: float, m_scale=None, v_scale=None, copies=None,
                       grad_scale: float = 1.0, coefficient=None, stream=None):
    """weights, grads, m, v (and the scales of 8-bit states, and bf16 copies): lists of tensors or
    adacomp_pointers. coefficient: one fp32 on the device, e.g. result[1:] of adacomp_grad_norm."""
    _check(lib().adacomp_adamw_step(
        h.ptr, _pointers(weights, h.weights, "weights"), _pointers(grads, h.grads, "grads"),
        _pointers(m, h.states, "m"), _pointers(v, h.states, "v"), _pointers(m_scale, h.scales, "m_scale"),
        _pointers(v_scale, h.scales, "v_scale"), _pointers(copies, h.copies, "copies", may_miss=True), lr, beta1,
        beta2, eps, bias_correction1, bias_correction2, grad_scale,
        _array(coefficient, 1, torch.float32, "coefficient"), _stream(stream)), "adacomp_adamw_step")


def adacomp_adamw_free(h):
    h.__del__()


# ---------------------------------------------------------------------------------------
# Linear layers and losses over a vocabulary.

_CODES = {v: k for k, v in _DTYPES.items()}


def _rows(t, dtype, rows: int, cols: int, what: str):
    """(address, row stride) of a tensor of rows x cols elements: a matrix with contiguous rows, or
    anything contiguous whose last axis is a row. None stays None."""
    if t is None:
        return None, 0
    shape = t.shape
    if t.dtype is not dtype or not t.is_cuda or not shape or shape[-1] != cols or t.numel() != rows * cols:
        _bad(f"{what} must be a CUDA tensor of {dtype}, {rows} rows of {cols}")
    if len(shape) == 2:
        stride, one = t.stride()
        if one != 1 and cols > 1:
            _bad(f"{what}: the elements of a row must be contiguous")
        return t.data_ptr(), stride
    if not t.is_contiguous():
        _bad(f"{what}: a tensor that is not a matrix must be contiguous")
    return t.data_ptr(), cols


def _count(t, cols: int, what: str) -> int:
    if not t.dim() or t.shape[-1] != cols:
        _bad(f"{what} must have rows of {cols}")
    return t.numel() // cols


def adacomp_linear_init(in_dim: int, out_dim: int, dtype: int = F32, activation: int = ACT_NONE) -> _TrainHandle:
    p = ctypes.c_void_p()
    _check(lib().adacomp_linear_init(ctypes.byref(p), in_dim, out_dim, dtype, activation), "adacomp_linear_init")
    h = _TrainHandle(p.value, "adacomp_linear_free")
    h.in_dim, h.out_dim, h.torch_dtype, h.activation = in_dim, out_dim, _DTYPES[dtype], activation
    return h


def adacomp_linear_forward_ws_bytes(h, rows: int) -> int:
    return lib().adacomp_linear_forward_ws_bytes(h.ptr, rows)


def adacomp_linear_backward_ws_bytes(h, rows: int) -> int:
    return lib().adacomp_linear_backward_ws_bytes(h.ptr, rows)


def adacomp_linear_forward(h, x, w, y, ws, bias=None, residual=None, pre=None, stream=None):
    """y = act(x w^T + bias) + residual; pre receives the value before the activation, for the backward pass."""
    t, n = h.torch_dtype, h.out_dim
    rows = _count(x, h.in_dim, "x")
    _check(lib().adacomp_linear_forward(
        h.ptr, rows, *_rows(x, t, rows, h.in_dim, "x"), *_rows(w, t, n, h.in_dim, "w"), _array(bias, n, t, "bias"),
        *_rows(residual, t, rows, n, "residual"), *_rows(y, t, rows, n, "y"), *_rows(pre, t, rows, n, "pre"), _ptr(ws),
        _nbytes(ws), _stream(stream)), "adacomp_linear_forward")


def adacomp_linear_backward(h, dy, x, w, ws, pre=None, dx=None, dw=None, db=None, stream=None):
    """dx, dw and db (those that are given) from dy and the forward pass's x, w and pre. x may be None
    without dw, w without dx."""
    t, n, k = h.torch_dtype, h.out_dim, h.in_dim
    rows = _count(dy, n, "dy")
    _check(lib().adacomp_linear_backward(
        h.ptr, rows, *_rows(dy, t, rows, n, "dy"), *_rows(x, t, rows, k, "x"), *_rows(w, t, n, k, "w"),
        *_rows(pre, t, rows, n, "pre"), *_rows(dx, t, rows, k, "dx"), *_rows(dw, t, n, k, "dw"),
        _array(db, n, t, "db"), _ptr(ws), _nbytes(ws), _stream(stream)), "adacomp_linear_backward")


def adacomp_linear_set_timeout_ns(h, ns: int):
    """Bound on a wait within a product; results behind one that runs out are NaN."""
    _check(lib().adacomp_linear_set_timeout_ns(h.ptr, ns), "adacomp_linear_set_timeout_ns")


def adacomp_linear_set_fault_injection(h, silent_cta: int = 0xFFFFFFFF):
    """Test hook: the given CTA (0 or 1) of every pair copies nothing, so that the pair's waits run out."""
    _check(lib().adacomp_linear_set_fault_injection(h.ptr, silent_cta), "adacomp_linear_set_fault_injection")


def adacomp_linear_free(h):
    h.__del__()


def adacomp_vocab_init(dim: int, vocab: int, dtype: int = F32) -> _TrainHandle:
    p = ctypes.c_void_p()
    _check(lib().adacomp_vocab_init(ctypes.byref(p), dim, vocab, dtype), "adacomp_vocab_init")
    h = _TrainHandle(p.value, "adacomp_vocab_free")
    h.dim, h.vocab, h.torch_dtype = dim, vocab, _DTYPES[dtype]
    return h


def adacomp_vocab_loss_forward_ws_bytes(h, rows: int) -> int:
    return lib().adacomp_vocab_loss_forward_ws_bytes(h.ptr, rows)


def adacomp_vocab_loss_backward_ws_bytes(h, rows: int) -> int:
    return lib().adacomp_vocab_loss_backward_ws_bytes(h.ptr, rows)


def adacomp_distill_forward_ws_bytes(h, rows: int, k: int) -> int:
    return lib().adacomp_distill_forward_ws_bytes(h.ptr, rows, k)


def adacomp_distill_backward_ws_bytes(h, rows: int, k: int) -> int:
    return lib().adacomp_distill_backward_ws_bytes(h.ptr, rows, k)


def _target(target, rows: int):
    if target.dtype not in (torch.int32, torch.int64):
        _bad("target must be a tensor of int32 or int64")
    return _array(target, rows, target.dtype, "target"), target.dtype.itemsize


def _teacher(index, logit, rows: int):
    if index.dim() < 2 or logit.shape != index.shape or logit.dtype not in _CODES:
        _bad("index and logit must be [rows, k], logit of float32 or bfloat16")
    k = index.shape[-1]
    return (k, *_rows(index, torch.int32, rows, k, "index"), *_rows(logit, logit.dtype, rows, k, "logit"),
            _CODES[logit.dtype])


def _dloss(dloss, rows: int):
    """(address, stride): one value per row, or one for all."""
    if dloss.numel() == 1 and rows != 1:
        return _array(dloss, 1, torch.float32, "dloss"), 0
    return _array(dloss, rows, torch.float32, "dloss"), 1


def _hidden(h, x, w):
    rows = _count(x, h.dim, "x")
    return rows, (*_rows(x, h.torch_dtype, rows, h.dim, "x"), *_rows(w, h.torch_dtype, h.vocab, h.dim, "w"))


def _vocab_gradients(h, rows, dx, dw):
    return (*_rows(dx, h.torch_dtype, rows, h.dim, "dx"), *_rows(dw, h.torch_dtype, h.vocab, h.dim, "dw"))


def adacomp_vocab_loss_forward(h, x, w, target, loss, lse, ws, stream=None):
    """Each row's softmax cross entropy of the logits x w^T; a negative target is a row without a loss.
    loss and lse: fp32, one value per row."""
    rows, operands = _hidden(h, x, w)
    _check(lib().adacomp_vocab_loss_forward(
        h.ptr, rows, *operands, *_target(target, rows), _array(loss, rows, torch.float32, "loss"),
        _array(lse, rows, torch.float32, "lse"), _ptr(ws), _nbytes(ws), _stream(stream)), "adacomp_vocab_loss_forward")


def adacomp_vocab_loss_backward(h, x, w, target, lse, dloss, ws, dx=None, dw=None, stream=None):
    """dx and dw (those that are given) from dloss (fp32, one per row or one for all) and the forward pass's lse."""
    rows, operands = _hidden(h, x, w)
    _check(lib().adacomp_vocab_loss_backward(
        h.ptr, rows, *operands, *_target(target, rows), _array(lse, rows, torch.float32, "lse"), *_dloss(dloss, rows),
        *_vocab_gradients(h, rows, dx, dw), _ptr(ws), _nbytes(ws), _stream(stream)), "adacomp_vocab_loss_backward")


def adacomp_distill_forward(h, x, w, index, logit, temperature: float, loss, lse, ws, stream=None):
    """Each row's temperature^2 KL(teacher || student), the teacher given by the logits of the tokens index
    (int32 [rows, k]; a negative one is none). loss and lse: fp32, one value per row."""
    rows, operands = _hidden(h, x, w)
    _check(lib().adacomp_distill_forward(
        h.ptr, rows, *operands, *_teacher(index, logit, rows), temperature, _array(loss, rows, torch.float32, "loss"),
        _array(lse, rows, torch.float32, "lse"), _ptr(ws), _nbytes(ws), _stream(stream)), "adacomp_distill_forward")


def adacomp_distill_backward(h, x, w, index, logit, temperature: float, lse, dloss, ws, dx=None, dw=None, stream=None):
    """dx and dw (those that are given) from dloss (fp32, one per row or one for all) and the forward pass's lse."""
    rows, operands = _hidden(h, x, w)
    _check(lib().adacomp_distill_backward(
        h.ptr, rows, *operands, *_teacher(index, logit, rows), temperature, _array(lse, rows, torch.float32, "lse"),
        *_dloss(dloss, rows), *_vocab_gradients(h, rows, dx, dw), _ptr(ws), _nbytes(ws), _stream(stream)),
        "adacomp_distill_backward")


def adacomp_vocab_set_timeout_ns(h, ns: int):
    """As adacomp_linear_set_timeout_ns."""
    _check(lib().adacomp_vocab_set_timeout_ns(h.ptr, ns), "adacomp_vocab_set_timeout_ns")


def adacomp_vocab_set_fault_injection(h, silent_cta: int = 0xFFFFFFFF):
    """As adacomp_linear_set_fault_injection."""
    _check(lib().adacomp_vocab_set_fault_injection(h.ptr, silent_cta), "adacomp_vocab_set_fault_injection")


def adacomp_vocab_free(h):
    h.__del__()
