"""Python binding of the GB300 BitLinear W1.58A8 C-ABI library (libbitlinear.so).

Argument marshalling only: every function below forwards torch CUDA tensors
(as raw device pointers, sizes and the current CUDA stream) to the
``extern "C"`` entry point of the same name declared in ``include/bitlinear.h``.
All arithmetic runs in the library's CUDA kernels; there is no CPU fallback.
If the library has not been built, importing works but every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import sys

__all__ = [
    "BitLinearError", "load_library", "library_path",
    "bitlinear_abi_version", "bitlinear_status_string", "bitlinear_packed_bytes",
    "bitlinear_quantize_weights_workspace", "bitlinear_quantize_weights",
    "bitlinear_quant_act", "bitlinear_forward", "bitlinear_forward_ex",
    "bitlinear_forward_workspace", "bitlinear_forward_ws",
    "bitlinear_device_status", "bitlinear_quantize_weights_noalloc",
    "bitlinear_selftest_wait_timeout", "bitlinear_linear", "bitlinear_linear_ws", "bitlinear_argmax",
    "bitlinear_rope_frequencies", "bitlinear_rope", "bitlinear_kv_append", "bitlinear_kv_read",
    "bitlinear_attention_workspace", "bitlinear_attention",
    "bitlinear_attention_shared_workspace", "bitlinear_attention_shared", "bitlinear_kv_summarise",
    "bitlinear_attention_select", "bitlinear_attention_blocks", "bitlinear_softmax", "bitlinear_verify",
    "BitLinearWeight", "BitLinearKVPages", "BitLinearRopeSpec", "BitLinearKVSummary",
    "EXPORTED_SYMBOLS",
    "ALGO_AUTO", "ALGO_DECODE", "ALGO_PREFILL", "ALGO_BATCHED", "ALGO_WIDE", "FLAG_PDL",
    "KV_INT8", "KV_FP8", "KV_BF16", "ROPE_HALF", "ROPE_INTERLEAVED",
    "ROPE_SCALE_NONE", "ROPE_SCALE_LINEAR", "ROPE_SCALE_BASE", "ROPE_SCALE_PARTS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_build", "libbitlinear.so")

ALGO_AUTO, ALGO_DECODE, ALGO_PREFILL, ALGO_BATCHED, ALGO_WIDE = 0, 1, 2, 3, 4
FLAG_PDL = 1
FLAG_GATED = 2  # bitlinear_linear: gate, up pair; the first output receives (r * r) * up, r = max(gate, 0)

KV_INT8, KV_FP8, KV_BF16 = 0, 1, 2
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_SCALE_NONE, ROPE_SCALE_LINEAR, ROPE_SCALE_BASE, ROPE_SCALE_PARTS = 0, 1, 2, 3

STATUS = {0: "OK", -1: "ERR_NULL", -2: "ERR_SHAPE", -3: "ERR_ALIGN", -4: "ERR_UNSUPPORTED",
          -5: "ERR_CUDA", -6: "ERR_TIMEOUT", -7: "ERR_WORKSPACE"}

# Every entry point include/bitlinear.h declares.
EXPORTED_SYMBOLS = (
    "bitlinear_abi_version", "bitlinear_status_string", "bitlinear_packed_bytes",
    "bitlinear_quantize_weights_workspace", "bitlinear_quantize_weights",
    "bitlinear_quant_act", "bitlinear_forward", "bitlinear_forward_ex",
    "bitlinear_forward_workspace", "bitlinear_forward_ws",
    "bitlinear_device_status", "bitlinear_quantize_weights_noalloc",
    "bitlinear_selftest_wait_timeout", "bitlinear_linear", "bitlinear_linear_ws", "bitlinear_argmax",
    "bitlinear_rope_frequencies", "bitlinear_rope", "bitlinear_kv_append", "bitlinear_kv_read",
    "bitlinear_attention_workspace", "bitlinear_attention",
    "bitlinear_attention_shared_workspace", "bitlinear_attention_shared", "bitlinear_kv_summarise",
    "bitlinear_attention_select", "bitlinear_attention_blocks", "bitlinear_softmax", "bitlinear_verify",
)

# The calls of a serving step that the compiled marshal takes, in bind_serving's order.
_SERVING = ("attention_shared", "kv_summarise", "attention_select", "attention_blocks", "softmax", "verify")

_lib = None
torch = None     # imported by the first attention call: the C ABI alone needs no torch
_marshal = None  # the compiled common case of the attention calls (csrc/marshal.cpp), where it was built
_ready = False   # both of them sought


class BitLinearWeight(ctypes.Structure):
    """ctypes mirror of the C struct bitlinear_weight."""
    _fields_ = [("packed", ctypes.c_void_p), ("w_scale", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("acc", ctypes.c_void_p)]


class BitLinearKVPages(ctypes.Structure):
    """ctypes mirror of the C struct bitlinear_kv_pages."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_step", ctypes.c_void_p),
                ("v_step", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("num_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("format", ctypes.c_int32)]


class BitLinearRopeSpec(ctypes.Structure):
    """ctypes mirror of the C struct bitlinear_rope_spec."""
    _fields_ = [("freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("amplitude", ctypes.c_float)]


class BitLinearKVSummary(ctypes.Structure):
    """ctypes mirror of the C struct bitlinear_kv_summary."""
    _fields_ = [("bounds", ctypes.c_void_p), ("step", ctypes.c_void_p)]


class BitLinearError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {bitlinear_status_string(status)} ({status})")


def library_path() -> str:
    return _LIB_PATH


def load_library(path: str | None = None):
    """Load libbitlinear.so (raises if it was not built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libbitlinear.so not found at {p}: build it with "
                           "bitlinear_w1_a8_gb300.build.build() (needs nvcc)")
    lib = ctypes.CDLL(p)
    i64, vp, sz, st = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    lib.bitlinear_abi_version.argtypes = []
    lib.bitlinear_abi_version.restype = ctypes.c_int
    lib.bitlinear_status_string.argtypes = [st]
    lib.bitlinear_status_string.restype = ctypes.c_char_p
    lib.bitlinear_packed_bytes.argtypes = [i64, i64]
    lib.bitlinear_packed_bytes.restype = sz
    lib.bitlinear_quantize_weights_workspace.argtypes = [i64, i64]
    lib.bitlinear_quantize_weights_workspace.restype = sz
    lib.bitlinear_quantize_weights.argtypes = [vp, i64, i64, vp, vp, vp, sz, vp]
    lib.bitlinear_quantize_weights.restype = st
    lib.bitlinear_quant_act.argtypes = [vp, vp, i64, i64, vp, ctypes.c_double, vp, vp, vp]
    lib.bitlinear_quant_act.restype = st
    lib.bitlinear_forward.argtypes = [vp, vp, i64, vp, vp, i64, i64, vp, vp, vp]
    lib.bitlinear_forward.restype = st
    lib.bitlinear_forward_ex.argtypes = [vp, vp, i64, vp, vp, i64, i64, vp, vp, ctypes.c_int,
                                         ctypes.c_int, vp]
    lib.bitlinear_forward_ex.restype = st
    lib.bitlinear_forward_workspace.argtypes = [i64, i64]
    lib.bitlinear_forward_workspace.restype = sz
    lib.bitlinear_forward_ws.argtypes = [vp, vp, i64, vp, vp, i64, i64, vp, vp, ctypes.c_int,
                                         ctypes.c_int, vp, sz, vp]
    lib.bitlinear_forward_ws.restype = st
    lib.bitlinear_quantize_weights_noalloc.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.bitlinear_quantize_weights_noalloc.restype = st
    lib.bitlinear_selftest_wait_timeout.argtypes = [i64, vp]
    lib.bitlinear_selftest_wait_timeout.restype = st
    lib.bitlinear_linear.argtypes = [vp, vp, i64, i64, vp, ctypes.c_double, ctypes.POINTER(BitLinearWeight),
                                     ctypes.c_int, vp, vp, ctypes.c_int, vp]
    lib.bitlinear_linear.restype = st
    lib.bitlinear_linear_ws.argtypes = [vp, vp, i64, i64, vp, ctypes.c_double, ctypes.POINTER(BitLinearWeight),
                                        ctypes.c_int, vp, vp, ctypes.c_int, vp, sz, vp]
    lib.bitlinear_linear_ws.restype = st
    lib.bitlinear_argmax.argtypes = [vp, i64, i64, vp, vp]
    lib.bitlinear_argmax.restype = st
    ci, dbl, pages, spec = ctypes.c_int, ctypes.c_double, ctypes.POINTER(BitLinearKVPages), ctypes.POINTER(BitLinearRopeSpec)
    lib.bitlinear_rope_frequencies.argtypes = [ci, dbl, ci, dbl, dbl, dbl, dbl, vp]
    lib.bitlinear_rope_frequencies.restype = st
    lib.bitlinear_rope.argtypes = [vp, i64, i64, ci, ci, vp, spec, vp, i64, ci, vp]
    lib.bitlinear_rope.restype = st
    lib.bitlinear_kv_append.argtypes = [vp, i64, ci, vp, i64, vp, i64, vp, i64, i64, vp, vp, vp, i64, i64, i64, spec,
                                        pages, ci, vp]
    lib.bitlinear_kv_append.restype = st
    lib.bitlinear_kv_read.argtypes = [pages, i64, vp, vp, vp, i64, i64, i64, vp, i64, vp, i64, ci, vp]
    lib.bitlinear_kv_read.restype = st
    lib.bitlinear_attention_workspace.argtypes = [i64, ci, ci, ci]
    lib.bitlinear_attention_workspace.restype = sz
    lib.bitlinear_attention.argtypes = [vp, i64, i64, ci, pages, vp, i64, i64, vp, i64, ctypes.c_float, vp, i64, vp,
                                        sz, ci, vp]
    lib.bitlinear_attention.restype = st
    summary, f32 = ctypes.POINTER(BitLinearKVSummary), ctypes.c_float
    lib.bitlinear_attention_shared_workspace.argtypes = [i64, ci, ci, ci, i64]
    lib.bitlinear_attention_shared_workspace.restype = sz
    lib.bitlinear_attention_shared.argtypes = [vp, i64, i64, ci, pages, vp, i64, i64, vp, vp, i64, f32, vp, i64, vp, sz, ci, vp]
    lib.bitlinear_attention_shared.restype = st
    lib.bitlinear_kv_summarise.argtypes = [pages, summary, vp, i64, i64, i64, vp, vp, ci, vp]
    lib.bitlinear_kv_summarise.restype = st
    lib.bitlinear_attention_select.argtypes = [vp, i64, i64, ci, pages, summary, vp, i64, i64, vp, ci, ci, vp, ci, ci, vp]
    lib.bitlinear_attention_select.restype = st
    lib.bitlinear_attention_blocks.argtypes = [vp, i64, i64, ci, pages, vp, i64, i64, vp, vp, ci, f32, vp, i64, ci, vp]
    lib.bitlinear_attention_blocks.restype = st
    lib.bitlinear_softmax.argtypes = [vp, i64, i64, vp, vp, ci, vp]
    lib.bitlinear_softmax.restype = st
    lib.bitlinear_verify.argtypes = [vp, vp, i64, ci, i64, vp, vp, vp, vp, ci, vp]
    lib.bitlinear_verify.restype = st
    lib.bitlinear_device_status.argtypes = [vp, ctypes.c_int]
    lib.bitlinear_device_status.restype = st
    if path is None:
        _lib = lib
        if "torch" in sys.modules:
            _get_ready()
    return lib


def _get_ready():
    """Imports torch and, once the library is there, the marshal."""
    global torch, _ready
    import torch
    if _lib is not None and not _ready:
        _ready = True
        _load_marshal(_lib)


def _load_marshal(lib):
    """The module built from these sources for this Python and torch, if it is there."""
    global _marshal
    import importlib.machinery
    import importlib.util
    from .build import marshal_path
    try:
        at = marshal_path()
    except (OSError, AttributeError):  # without its sources, or with half a torch, none is known to belong
        return
    if at is None or not os.path.exists(at):
        return
    loader = importlib.machinery.ExtensionFileLoader("bitlinear_marshal", at)
    try:
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("bitlinear_marshal", loader))
        loader.exec_module(module)
    except ImportError:
        return
    module.bind(*(ctypes.cast(getattr(lib, "bitlinear_" + name), ctypes.c_void_p).value
                  for name in ("rope", "kv_append", "kv_read", "attention")))
    module.bind_serving(*(ctypes.cast(getattr(lib, "bitlinear_" + name), ctypes.c_void_p).value for name in _SERVING))
    _marshal = module


def _check(status: int, what: str):
    if status != 0:
        raise BitLinearError(status, what)


# Addresses go to ctypes as plain ints (the argtypes are c_void_p; None is NULL).
def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        try:  # the handle alone: a third of the time of building a Stream object
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        except AttributeError:
            return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _need(t, dtype, name, shape=None):
    try:  # the common case in one expression; the detailed checks only on failure
        if t.is_cuda and t.dtype == dtype and t.is_contiguous() and (shape is None or t.shape == shape):
            return
    except AttributeError:
        pass
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def bitlinear_abi_version() -> int:
    return load_library().bitlinear_abi_version()


def bitlinear_status_string(status: int) -> str:
    try:
        return load_library().bitlinear_status_string(status).decode()
    except RuntimeError:
        return STATUS.get(status, "unknown status")


@functools.lru_cache(maxsize=256)
def bitlinear_packed_bytes(N: int, K: int) -> int:
    """Bytes of the packed layout of an [N, K] matrix (asked of the library)."""
    return int(load_library().bitlinear_packed_bytes(int(N), int(K)))


def bitlinear_quantize_weights_workspace(N: int, K: int) -> int:
    return int(load_library().bitlinear_quantize_weights_workspace(N, K))


def bitlinear_quantize_weights(W, packed, w_scale, workspace, stream=None):
    """weight_quant + pack of W [N, K] fp32 into `packed` (uint8) and `w_scale` (fp32 [1])."""
    import torch
    _need(W, torch.float32, "W")
    N, K = W.shape
    _need(packed, torch.uint8, "packed", (bitlinear_packed_bytes(N, K),))
    _need(w_scale, torch.float32, "w_scale")
    _need(workspace, torch.uint8, "workspace")
    _check(load_library().bitlinear_quantize_weights(
        _ptr(W), N, K, _ptr(packed), _ptr(w_scale), _ptr(workspace), workspace.numel(),
        _stream(stream)), "bitlinear_quantize_weights")


def bitlinear_quantize_weights_noalloc(W, packed, w_scale, stream=None):
    """weight_quant + pack like bitlinear_quantize_weights, for callers that cannot
    allocate device memory: the scratch is a fixed array inside the library
    (calls on one device must not overlap on the GPU; see include/bitlinear.h)."""
    import torch
    _need(W, torch.float32, "W")
    N, K = W.shape
    _need(packed, torch.uint8, "packed", (bitlinear_packed_bytes(N, K),))
    _need(w_scale, torch.float32, "w_scale")
    _check(load_library().bitlinear_quantize_weights_noalloc(
        _ptr(W), N, K, _ptr(packed), _ptr(w_scale), _stream(stream)),
        "bitlinear_quantize_weights_noalloc")


def bitlinear_quant_act(x, xq, x_scale, mul=None, rms_weight=None, rms_eps: float = 1e-6,
                        stream=None):
    """activation_quant of x [M, K] fp32 (optional ReLU^2*mul gating, optional RMSNorm)."""
    import torch
    _need(x, torch.float32, "x")
    M, K = x.shape
    _need(xq, torch.int8, "xq", (M, K))
    _need(x_scale, torch.float32, "x_scale", (M,))
    if mul is not None:
        _need(mul, torch.float32, "mul", (M, K))
    if rms_weight is not None:
        _need(rms_weight, torch.float32, "rms_weight", (K,))
    _check(load_library().bitlinear_quant_act(
        _ptr(x), _ptr(mul), M, K, _ptr(rms_weight), float(rms_eps), _ptr(xq), _ptr(x_scale),
        _stream(stream)), "bitlinear_quant_act")


def bitlinear_forward_ex(xq, x_scale, packed, w_scale, N: int, y, acc=None,
                         algo: int = ALGO_AUTO, flags: int = 0, stream=None):
    """y [M, N] = (xq . Wq^T) / (sx * sw) with an explicit algorithm and flags."""
    import torch
    _need(xq, torch.int8, "xq")
    M, K = xq.shape
    _need(x_scale, torch.float32, "x_scale", (M,))
    _need(packed, torch.uint8, "packed", (bitlinear_packed_bytes(N, K),))
    _need(w_scale, torch.float32, "w_scale")
    _need(y, torch.float32, "y", (M, N))
    if acc is not None:
        _need(acc, torch.int32, "acc", (M, N))
    _check(load_library().bitlinear_forward_ex(
        _ptr(xq), _ptr(x_scale), M, _ptr(packed), _ptr(w_scale), N, K, _ptr(y), _ptr(acc),
        int(algo), int(flags), _stream(stream)), "bitlinear_forward_ex")


@functools.lru_cache(maxsize=256)
def bitlinear_forward_workspace(M: int, K: int) -> int:
    """Bytes of device workspace bitlinear_forward_ws needs for M tokens of K."""
    return int(load_library().bitlinear_forward_workspace(int(M), int(K)))


def bitlinear_forward_ws(xq, x_scale, packed, w_scale, N: int, y, acc=None, workspace=None,
                         algo: int = ALGO_AUTO, flags: int = 0, stream=None):
    """bitlinear_forward_ex with a device workspace (a uint8 CUDA tensor of at
    least bitlinear_forward_workspace(M, K) bytes, or None: then no algorithm
    that needs one is chosen, and asking for ALGO_WIDE raises)."""
    import torch
    _need(xq, torch.int8, "xq")
    M, K = xq.shape
    _need(x_scale, torch.float32, "x_scale", (M,))
    _need(packed, torch.uint8, "packed", (bitlinear_packed_bytes(N, K),))
    _need(w_scale, torch.float32, "w_scale")
    _need(y, torch.float32, "y", (M, N))
    if acc is not None:
        _need(acc, torch.int32, "acc", (M, N))
    if workspace is not None:
        _need(workspace, torch.uint8, "workspace")
    _check(load_library().bitlinear_forward_ws(
        _ptr(xq), _ptr(x_scale), M, _ptr(packed), _ptr(w_scale), N, K, _ptr(y), _ptr(acc),
        int(algo), int(flags), _ptr(workspace), 0 if workspace is None else workspace.numel(),
        _stream(stream)), "bitlinear_forward_ws")


def bitlinear_forward(xq, x_scale, packed, w_scale, N: int, y, acc=None, stream=None):
    """y [M, N] = (xq . Wq^T) / (sx * sw); the kernel is chosen from M."""
    import torch
    _need(xq, torch.int8, "xq")
    M, K = xq.shape
    _need(x_scale, torch.float32, "x_scale", (M,))
    _need(packed, torch.uint8, "packed", (bitlinear_packed_bytes(N, K),))
    _need(w_scale, torch.float32, "w_scale")
    _need(y, torch.float32, "y", (M, N))
    if acc is not None:
        _need(acc, torch.int32, "acc", (M, N))
    _check(load_library().bitlinear_forward(
        _ptr(xq), _ptr(x_scale), M, _ptr(packed), _ptr(w_scale), N, K, _ptr(y), _ptr(acc),
        _stream(stream)), "bitlinear_forward")


def bitlinear_device_status(stream=None, clear: bool = True) -> int:
    """Synchronise the stream and return the library's device status (0 = OK)."""
    return int(load_library().bitlinear_device_status(_stream(stream), 1 if clear else 0))


def bitlinear_argmax(y, index, stream=None):
    """index[m] = first n of the largest y[m, n] (y [M, N] fp32, index [M] int32)."""
    import torch
    _need(y, torch.float32, "y")
    if y.dim() != 2:
        raise ValueError("y must be [M, N]")
    M, N = y.shape
    _need(index, torch.int32, "index", (M,))
    _check(load_library().bitlinear_argmax(_ptr(y), M, N, _ptr(index), _stream(stream)), "bitlinear_argmax")


def bitlinear_selftest_wait_timeout(limit_ns: int, stream=None):
    """Launch the bounded-wait self-test kernel (a wait nothing satisfies)."""
    _check(load_library().bitlinear_selftest_wait_timeout(int(limit_ns), _stream(stream)),
           "bitlinear_selftest_wait_timeout")


def _packed_size(N: int, K: int) -> int:
    """bitlinear_packed_bytes(N, K) without a call into the library (N * ceil(K/64) * 16,
    the layout the header documents); a CPU test holds the two equal."""
    return N * ((K + 63) // 64) * 16


def _weight_array(weights, M, K):
    import torch
    arr = (BitLinearWeight * len(weights))()
    for i, w in enumerate(weights):
        packed, w_scale, y = w[0], w[1], w[2]
        acc = w[3] if len(w) > 3 else None
        N = y.shape[1]
        _need(packed, torch.uint8, "packed", (_packed_size(N, K),))
        _need(w_scale, torch.float32, "w_scale")
        _need(y, torch.float32, "y", (M, N))
        if acc is not None:
            _need(acc, torch.int32, "acc", (M, N))
        arr[i] = BitLinearWeight(packed.data_ptr(), w_scale.data_ptr(), N, y.data_ptr(),
                                 acc.data_ptr() if acc is not None else None)
    return arr


def _linear_inputs(x, xq, x_scale, mul, rms_weight):
    import torch
    _need(x, torch.float32, "x")
    M, K = x.shape
    _need(xq, torch.int8, "xq", (M, K))
    _need(x_scale, torch.float32, "x_scale", (M,))
    if mul is not None:
        _need(mul, torch.float32, "mul", (M, K))
    if rms_weight is not None:
        _need(rms_weight, torch.float32, "rms_weight", (K,))
    return M, K


def bitlinear_linear(x, weights, xq, x_scale, mul=None, rms_weight=None, rms_eps: float = 1e-6,
                     flags: int = 0, stream=None):
    """act_quant + forward for 1..4 matrices sharing the input x [M, K].

    weights: sequence of (packed, w_scale, y) or (packed, w_scale, y, acc) tuples of
    CUDA tensors (y [M, N] fp32, acc [M, N] int32 or None).
    """
    M, K = _linear_inputs(x, xq, x_scale, mul, rms_weight)
    arr = _weight_array(weights, M, K)
    _check(load_library().bitlinear_linear(
        _ptr(x), _ptr(mul), M, K, _ptr(rms_weight), float(rms_eps), arr, len(weights), _ptr(xq),
        _ptr(x_scale), int(flags), _stream(stream)), "bitlinear_linear")


def bitlinear_linear_ws(x, weights, xq, x_scale, workspace, mul=None, rms_weight=None, rms_eps: float = 1e-6,
                        flags: int = 0, stream=None):
    """bitlinear_linear with a device workspace (uint8 CUDA tensor of at least
    bitlinear_forward_workspace(M, K) bytes, or None)."""
    import torch
    M, K = _linear_inputs(x, xq, x_scale, mul, rms_weight)
    arr = _weight_array(weights, M, K)
    if workspace is not None:
        _need(workspace, torch.uint8, "workspace")
    _check(load_library().bitlinear_linear_ws(
        _ptr(x), _ptr(mul), M, K, _ptr(rms_weight), float(rms_eps), arr, len(weights), _ptr(xq),
        _ptr(x_scale), int(flags), _ptr(workspace), 0 if workspace is None else workspace.numel(),
        _stream(stream)), "bitlinear_linear_ws")


# --- rotary positions, the paged key-value cache and attention over it ---
#
# These calls take many tensors and are made once or twice a layer and token, so the
# compiled marshal takes the common case (contiguous tensors that fit).  It answers None
# for every other; then, or where it was not built, each call checks its tensors here, in
# one expression, and one by one when that fails: for an unusual layout, or to say what
# is wrong.


def _current_device():
    try:  # without torch.cuda's lazy initialisation: a CUDA tensor is there already
        return torch._C._cuda_getDevice()
    except AttributeError:
        return torch.cuda.current_device()


def _device(t, name):
    """The index of the tensor's device, which must be the current one: the library launches there."""
    try:
        at = t.get_device()
    except AttributeError:
        at = -1
    if at < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if at != _current_device():
        raise ValueError(f"{name} must be on the current device cuda:{_current_device()}, got {t.device}")
    return at


def _need_on(t, at, dtype, name, shape=None):
    _need(t, dtype, name, shape)
    if t.get_device() != at:
        raise ValueError(f"{name} must be on cuda:{at}, got {t.device}")


def _rows(t, at, name, shape):
    """The row stride (elements) of fp32 [T, H, D] rows: heads side by side, rows any stride apart."""
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be torch.float32, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != at:
        raise ValueError(f"{name} must be on cuda:{at}, got {t.device}")
    T, H, D = shape
    if t.is_contiguous():  # strides of dims of size 1 say nothing
        return H * D
    strides = t.stride()
    if strides[2] != 1 or (H > 1 and strides[1] != D):
        raise ValueError(f"{name}'s heads must lie side by side in each row, got strides {tuple(strides)}")
    return strides[0] if T > 1 else H * D


def _page_table(t, at, rows=None):
    """(rows, columns, row stride) of the int32 page table: contiguous rows, any stride apart."""
    if not getattr(t, "is_cuda", False) or t.dtype != torch.int32:
        raise TypeError("page_table must be an int32 CUDA tensor")
    shape = t.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows):
        raise ValueError(f"page_table must be [{'sequences' if rows is None else rows}, pages], got {tuple(shape)}")
    if t.get_device() != at:
        raise ValueError(f"page_table must be on cuda:{at}, got {t.device}")
    n, cols = shape
    if t.is_contiguous():
        return n, cols, cols
    if cols > 1 and t.stride(1) != 1:
        raise ValueError("page_table's rows must be contiguous")
    return n, cols, t.stride(0) if n > 1 else cols


def _kv_pages(cache, at):
    """BitLinearKVPages of (k, v, k_step, v_step), the steps None or left out for bf16."""
    k, v = cache[0], cache[1]
    k_step, v_step = (cache[2], cache[3]) if len(cache) > 2 else (None, None)
    if not getattr(k, "is_cuda", False):
        raise TypeError("the cache must be CUDA tensors")
    dtype, shape = k.dtype, k.shape
    if len(shape) != 4:
        raise ValueError(f"the cache's k must be [pages, heads, page_size, head_dim], got {tuple(shape)}")
    if dtype is torch.bfloat16:
        if k_step is not None or v_step is not None:
            raise ValueError("a bfloat16 cache has no steps")
        _need_on(k, at, dtype, "the cache's k")
        _need_on(v, at, dtype, "the cache's v", shape)
        return BitLinearKVPages(k.data_ptr(), v.data_ptr(), None, None, *shape, KV_BF16)
    if dtype is not torch.int8 and dtype is not torch.float8_e4m3fn:
        raise TypeError(f"the cache must be int8, float8_e4m3fn or bfloat16, got {dtype}")
    rows = shape[:3]
    f32 = torch.float32
    if not (v_step is not None and k_step is not None and k.get_device() == v.get_device() == k_step.get_device()
            == v_step.get_device() == at and v.dtype is dtype and k_step.dtype is f32 and v_step.dtype is f32
            and v.shape == shape and k_step.shape == rows and v_step.shape == rows and k.is_contiguous()
            and v.is_contiguous() and k_step.is_contiguous() and v_step.is_contiguous()):
        _need_on(k, at, dtype, "the cache's k")
        _need_on(v, at, dtype, "the cache's v", shape)
        _need_on(k_step, at, f32, "the cache's k_step", rows)
        _need_on(v_step, at, f32, "the cache's v_step", rows)
    return BitLinearKVPages(k.data_ptr(), v.data_ptr(), k_step.data_ptr(), v_step.data_ptr(), *shape,
                            KV_INT8 if dtype is torch.int8 else KV_FP8)


def _rope_spec(rope, at):
    """BitLinearRopeSpec of (freq, layout) or (freq, layout, amplitude)."""
    freq = rope[0]
    if not (freq.get_device() == at and freq.dtype is torch.float64 and freq.is_contiguous()):
        _need_on(freq, at, torch.float64, "rope's freq")
    return BitLinearRopeSpec(freq.data_ptr(), 2 * freq.numel(), int(rope[1]), float(rope[2]) if len(rope) > 2 else 1.0)


def bitlinear_rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: int = ROPE_SCALE_NONE,
                               factor: float = 1.0, original_length: float = 0.0, low: float = 1.0,
                               high: float = 32.0):
    """The rot_dim / 2 rotary frequencies (radians a position) as a fp64 CPU tensor; move it
    to the device once."""
    n = max(0, int(rot_dim)) // 2
    out = (ctypes.c_double * max(1, n))()
    _check(load_library().bitlinear_rope_frequencies(
        int(rot_dim), float(base), int(scaling), float(factor), float(original_length), float(low), float(high),
        ctypes.addressof(out)), "bitlinear_rope_frequencies")
    import torch
    return torch.tensor(list(out), dtype=torch.float64)


def bitlinear_rope(x, positions, rope, y, flags: int = 0, stream=None):
    """y [T, H, D] = x [T, H, D] rotated to positions [T] (int32).

    rope: (freq, layout) or (freq, layout, amplitude) with freq a fp64 CUDA tensor
    (bitlinear_rope_frequencies) and layout ROPE_HALF or ROPE_INTERLEAVED.  y may be x.
    Rows may lie any multiple of 4 floats apart.
    """
    if not _ready:
        _get_ready()
    if _marshal is not None:
        status = _marshal.rope(x, positions, rope, y, flags, stream)
        if status is not None:
            return _check(status, "bitlinear_rope")
    at = _device(x, "x")
    shape = x.shape
    if len(shape) != 3:
        raise ValueError(f"x must be [rows, heads, head_dim], got {tuple(shape)}")
    T, H, D = shape
    x_stride = y_stride = H * D
    f32 = torch.float32
    if not (y.get_device() == positions.get_device() == at and x.dtype is f32 and y.dtype is f32
            and positions.dtype is torch.int32 and y.shape == shape and positions.shape == (T,)
            and x.is_contiguous() and y.is_contiguous() and positions.is_contiguous()):
        x_stride, y_stride = _rows(x, at, "x", shape), _rows(y, at, "y", shape)
        _need_on(positions, at, torch.int32, "positions", (T,))
    _check(load_library().bitlinear_rope(x.data_ptr(), x_stride, T, H, D, positions.data_ptr(), _rope_spec(rope, at),
                                         y.data_ptr(), y_stride, flags, _stream(stream)), "bitlinear_rope")


def _row_places(positions, page_table, seq, T, at):
    """(positions, seq, table addresses, table stride, sequences, pages) of T rows."""
    i32 = torch.int32
    if (positions.dtype is i32 and page_table.dtype is i32 and positions.get_device() == page_table.get_device() == at
            and positions.shape == (T,) and positions.is_contiguous() and page_table.is_contiguous()
            and len(page_table.shape) == 2):
        n, cols = page_table.shape
        stride = cols
    else:
        _need_on(positions, at, i32, "positions", (T,))
        n, cols, stride = _page_table(page_table, at)
    if seq is None:
        return positions.data_ptr(), None, page_table.data_ptr(), stride, n, cols
    if not (seq.dtype is i32 and seq.get_device() == at and seq.shape == (T,) and seq.is_contiguous()):
        _need_on(seq, at, i32, "seq", (T,))
    return positions.data_ptr(), seq.data_ptr(), page_table.data_ptr(), stride, n, cols


def bitlinear_kv_append(k, v, cache, positions, page_table, seq=None, q=None, q_out=None, rope=None,
                        flags: int = 0, stream=None):
    """Writes T new tokens into the paged cache: k and v [T, heads, head_dim] quantised as they
    are written, k and the optional q [T, q_heads, head_dim] rotated first (q into q_out).

    cache: (k, v, k_step, v_step), codes [pages, heads, page_size, head_dim] of int8 or
    float8_e4m3fn with fp32 steps [pages, heads, page_size], or (k, v) of bfloat16.
    positions, seq: int32 [T]; page_table: int32 [sequences, pages]; seq None: row i is of
    sequence i.  Rows with a negative position are padding.  rope: as for bitlinear_rope.
    """
    if not _ready:
        _get_ready()
    if _marshal is not None:
        status = _marshal.kv_append(k, v, cache, positions, page_table, seq, q, q_out, rope, flags, stream)
        if status is not None:
            return _check(status, "bitlinear_kv_append")
    at = _device(k, "k")
    pages = _kv_pages(cache, at)
    f32, T, Hk, D = torch.float32, k.shape[0], pages.num_heads, pages.head_dim
    shape = (T, Hk, D)
    k_stride = v_stride = Hk * D
    if not (v.get_device() == at and k.dtype is f32 and v.dtype is f32 and k.shape == shape and v.shape == shape
            and k.is_contiguous() and v.is_contiguous()):
        k_stride, v_stride = _rows(k, at, "k", shape), _rows(v, at, "v", shape)
    positions_at, seq_at, table_at, table_stride, num_seqs, max_pages = _row_places(positions, page_table, seq, T, at)
    Hq = q_stride = q_out_stride = 0
    q_at = q_out_at = None
    if q is not None:
        if q.dim() != 3:
            raise ValueError(f"q must be [rows, heads, head_dim], got {tuple(q.shape)}")
        Hq = q.shape[1]
        q_shape = (T, Hq, D)
        q_stride = q_out_stride = Hq * D
        if not (q_out is not None and q.get_device() == q_out.get_device() == at and q.dtype is f32
                and q_out.dtype is f32 and q.shape == q_shape and q_out.shape == q_shape and q.is_contiguous()
                and q_out.is_contiguous()):
            q_stride, q_out_stride = _rows(q, at, "q", q_shape), _rows(q_out, at, "q_out", q_shape)
        q_at, q_out_at = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    _check(load_library().bitlinear_kv_append(
        q_at, q_stride, Hq, q_out_at, q_out_stride, k.data_ptr(), k_stride, v.data_ptr(), v_stride, T, positions_at,
        seq_at, table_at, table_stride, num_seqs, max_pages, None if rope is None else _rope_spec(rope, at), pages,
        flags, _stream(stream)), "bitlinear_kv_append")


def bitlinear_kv_read(cache, positions, page_table, k_out, v_out, seq=None, flags: int = 0, stream=None):
    """k_out, v_out [T, heads, head_dim] fp32 = the cached rows at (seq[i], positions[i])."""
    if not _ready:
        _get_ready()
    if _marshal is not None:
        status = _marshal.kv_read(cache, positions, page_table, k_out, v_out, seq, flags, stream)
        if status is not None:
            return _check(status, "bitlinear_kv_read")
    at = _device(k_out, "k_out")
    pages = _kv_pages(cache, at)
    f32, T, Hk, D = torch.float32, k_out.shape[0], pages.num_heads, pages.head_dim
    shape = (T, Hk, D)
    k_stride = v_stride = Hk * D
    if not (v_out.get_device() == at and k_out.dtype is f32 and v_out.dtype is f32 and k_out.shape == shape
            and v_out.shape == shape and k_out.is_contiguous() and v_out.is_contiguous()):
        k_stride, v_stride = _rows(k_out, at, "k_out", shape), _rows(v_out, at, "v_out", shape)
    positions_at, seq_at, table_at, table_stride, num_seqs, max_pages = _row_places(positions, page_table, seq, T, at)
    _check(load_library().bitlinear_kv_read(
        pages, T, positions_at, seq_at, table_at, table_stride, num_seqs, max_pages, k_out.data_ptr(), k_stride,
        v_out.data_ptr(), v_stride, flags, _stream(stream)), "bitlinear_kv_read")


def bitlinear_attention_workspace(B: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    """Bytes of device workspace with which bitlinear_attention may split its sequences further."""
    return int(load_library().bitlinear_attention_workspace(int(B), int(num_q_heads), int(num_kv_heads), int(head_dim)))


def bitlinear_attention(q, cache, page_table, lengths, out, workspace=None, scale: float | None = None,
                        window: int = 0, flags: int = 0, stream=None):
    """out [B, q_heads, head_dim] = attention of q over the lengths[b] cached tokens of each
    sequence (the last `window` of them when it is not 0); scale None: 1 / sqrt(head_dim).
    cache and page_table: as for bitlinear_kv_append; lengths: int32 [B]."""
    if not _ready:
        _get_ready()
    if _marshal is not None:
        status = _marshal.attention(q, cache, page_table, lengths, out, workspace, scale, window, flags, stream)
        if status is not None:
            return _check(status, "bitlinear_attention")
    at = _device(q, "q")
    pages = _kv_pages(cache, at)
    shape = q.shape
    if len(shape) != 3 or shape[2] != pages.head_dim:
        raise ValueError(f"q must be [sequences, heads, {pages.head_dim}], got {tuple(shape)}")
    B, Hq, D = shape
    q_stride = out_stride = Hq * D
    f32, i32 = torch.float32, torch.int32
    if (out.get_device() == page_table.get_device() == lengths.get_device() == at and q.dtype is f32
            and out.dtype is f32 and page_table.dtype is i32 and lengths.dtype is i32 and out.shape == shape
            and lengths.shape == (B,) and page_table.shape[0] == B and len(page_table.shape) == 2
            and q.is_contiguous() and out.is_contiguous() and page_table.is_contiguous()
            and lengths.is_contiguous()):
        table_stride = max_pages = page_table.shape[1]
    else:
        q_stride, out_stride = _rows(q, at, "q", shape), _rows(out, at, "out", shape)
        _need_on(lengths, at, i32, "lengths", (B,))
        _, max_pages, table_stride = _page_table(page_table, at, B)
    space = None
    if workspace is not None:
        if not (workspace.get_device() == at and workspace.dtype is torch.uint8 and workspace.is_contiguous()):
            _need_on(workspace, at, torch.uint8, "workspace")
        space = workspace.data_ptr()
    _check(load_library().bitlinear_attention(
        q.data_ptr(), q_stride, B, Hq, pages, page_table.data_ptr(), table_stride, max_pages, lengths.data_ptr(),
        window, D ** -0.5 if scale is None else scale, out.data_ptr(), out_stride, space,
        0 if workspace is None else workspace.numel(), flags, _stream(stream)), "bitlinear_attention")


# --- a serving step: shared prefixes, chosen blocks, probabilities and drafted tokens ---
#
# As above: the compiled marshal takes the common case, and each call does every other here.


def bitlinear_attention_shared_workspace(B: int, num_q_heads: int, num_kv_heads: int, head_dim: int, num_groups: int) -> int:
    """Bytes of device workspace that bitlinear_attention_shared needs."""
    return int(load_library().bitlinear_attention_shared_workspace(int(B), int(num_q_heads), int(num_kv_heads), int(head_dim),
                                                                   int(num_groups)))


def _attention_tensors(q, cache, page_table, lengths, out):
    """(device, pages, the arguments q .. lengths and out, out_stride) of an attention call."""
    at = _device(q, "q")
    pages = _kv_pages(cache, at)
    shape = q.shape
    if len(shape) != 3 or shape[2] != pages.head_dim:
        raise ValueError(f"q must be [sequences, heads, {pages.head_dim}], got {tuple(shape)}")
    B, Hq, D = shape
    q_stride, out_stride = _rows(q, at, "q", shape), _rows(out, at, "out", shape)
    _need_on(lengths, at, torch.int32, "lengths", (B,))
    _, max_pages, table_stride = _page_table(page_table, at, B)
    return at, pages, (q.data_ptr(), q_stride, B, Hq, pages, page_table.data_ptr(), table_stride, max_pages,
                       lengths.data_ptr()), (out.data_ptr(), out_stride)


def bitlinear_attention_shared(q, cache, page_table, lengths, shared, out, workspace=None, scale: float | None = None,
                               flags: int = 0, stream=None):
    """bitlinear_attention of rows that share their first shared[g] (int32 [groups]) tokens in groups of
    B / groups consecutive rows: those tokens are read once for all of a group's rows.  page_table and
    lengths are each row's own, shared tokens included; workspace: uint8, at least
    bitlinear_attention_shared_workspace() bytes."""
    if not _ready:
        _get_ready()
    if _marshal is not None:
        status = _marshal.attention_shared(q, cache, page_table, lengths, shared, out, workspace, scale, flags, stream)
        if status is not None:
            return _check(status, "bitlinear_attention_shared")
    at, pages, tensors, written = _attention_tensors(q, cache, page_table, lengths, out)
    _need_on(shared, at, torch.int32, "shared")
    if shared.dim() != 1:
        raise ValueError(f"shared must be [groups], got {tuple(shared.shape)}")
    if workspace is not None:
        _need_on(workspace, at, torch.uint8, "workspace")
    _check(load_library().bitlinear_attention_shared(
        *tensors, shared.data_ptr(), shared.shape[0], pages.head_dim ** -0.5 if scale is None else scale, *written,
        _ptr(workspace), 0 if workspace is None else workspace.numel(), flags, _stream(stream)), "bitlinear_attention_shared")


def _kv_summary(summary, pages, at):
    """BitLinearKVSummary of (bounds, step)."""
    bounds, step = summary
    _need_on(bounds, at, torch.int8, "the summary's bounds", (pages.num_pages, pages.num_heads, 2, pages.head_dim))
    _need_on(step, at, torch.float32, "the summary's step", (pages.num_pages, pages.num_heads))
    return BitLinearKVSummary(bounds.data_ptr(), step.data_ptr())


def bitlinear_kv_summarise(cache, summary, page_table, first, lengths, flags: int = 0, stream=None):
    """Writes the bounds of the keys of the pages that hold tokens first[b] .. lengths[b] - 1 (int32 [B]).

    summary: (bounds, step), int8 [pages, heads, 2, head_dim] and fp32 [pages, heads]; cache and
    page_table as for bitlinear_attention."""
    if not _ready:
        _get_ready()
    if _marshal is not None:
        status = _marshal.kv_summarise(cache, summary, page_table, first, lengths, flags, stream)
        if status is not None:
            return _check(status, "bitlinear_kv_summarise")
    at = _device(page_table, "page_table")
    pages = _kv_pages(cache, at)
    B, max_pages, table_stride = _page_table(page_table, at)
    _need_on(first, at, torch.int32, "first", (B,))
    _need_on(lengths, at, torch.int32, "lengths", (B,))
    _check(load_library().bitlinear_kv_summarise(
        pages, _kv_summary(summary, pages, at), page_table.data_ptr(), table_stride, B, max_pages, first.data_ptr(),
        lengths.data_ptr(), flags, _stream(stream)), "bitlinear_kv_summarise")


def _blocks(blocks, B, pages, at):
    """How many pages a list of int32 [B, heads, count] names."""
    _need_on(blocks, at, torch.int32, "blocks")
    if blocks.dim() != 3 or blocks.shape[:2] != (B, pages.num_heads):
        raise ValueError(f"blocks must be [{B}, {pages.num_heads}, count], got {tuple(blocks.shape)}")
    return blocks.shape[2]


def _as_int(n) -> int:
    """n as a C int takes it: what is beyond 32 bits is the nearest inside, not its last 32 bits."""
    return max(-2 ** 31, min(2 ** 31 - 1, int(n)))


def bitlinear_attention_select(q, cache, summary, page_table, lengths, blocks, keep_first: int = 1, keep_last: int = 1,
                               flags: int = 0, stream=None):
    """blocks [B, heads, count] (int32) = the pages (columns of the page table) of the largest scores for
    each key head, the first keep_first and last keep_last of a sequence among them, in order, then -1.
    summary: as bitlinear_kv_summarise wrote it; other arguments as for bitlinear_attention."""
    if not _ready:
        _get_ready()
    if _marshal is not None:
        status = _marshal.attention_select(q, cache, summary, page_table, lengths, blocks, keep_first, keep_last, flags, stream)
        if status is not None:
            return _check(status, "bitlinear_attention_select")
    at = _device(q, "q")
    pages = _kv_pages(cache, at)
    shape = q.shape
    if len(shape) != 3 or shape[2] != pages.head_dim:
        raise ValueError(f"q must be [sequences, heads, {pages.head_dim}], got {tuple(shape)}")
    q_stride = _rows(q, at, "q", shape)
    _need_on(lengths, at, torch.int32, "lengths", (shape[0],))
    _, max_pages, table_stride = _page_table(page_table, at, shape[0])
    count = _blocks(blocks, shape[0], pages, at)
    _check(load_library().bitlinear_attention_select(
        q.data_ptr(), q_stride, shape[0], shape[1], pages, _kv_summary(summary, pages, at), page_table.data_ptr(), table_stride,
        max_pages, lengths.data_ptr(), _as_int(keep_first), _as_int(keep_last), blocks.data_ptr(), _as_int(count), flags,
        _stream(stream)), "bitlinear_attention_select")


def bitlinear_attention_blocks(q, cache, page_table, lengths, blocks, out, scale: float | None = None, flags: int = 0, stream=None):
    """bitlinear_attention over the tokens of the pages that blocks [B, heads, count] (int32) lists for each key
    head, in place of all tokens."""
    if not _ready:
        _get_ready()
    if _marshal is not None:
        status = _marshal.attention_blocks(q, cache, page_table, lengths, blocks, out, scale, flags, stream)
        if status is not None:
            return _check(status, "bitlinear_attention_blocks")
    at, pages, tensors, written = _attention_tensors(q, cache, page_table, lengths, out)
    count = _blocks(blocks, q.shape[0], pages, at)
    _check(load_library().bitlinear_attention_blocks(
        *tensors, blocks.data_ptr(), _as_int(count), pages.head_dim ** -0.5 if scale is None else scale, *written, flags,
        _stream(stream)), "bitlinear_attention_blocks")


def bitlinear_softmax(y, p, temperature=None, flags: int = 0, stream=None):
    """p [M, N] = softmax(y / temperature) of logits y [M, N] (fp32; p may be y); temperature: fp32 [M], 0 for the
    first maximum alone, or None for 1."""
    if not _ready:
        _get_ready()
    if _marshal is not None:
        status = _marshal.softmax(y, p, temperature, flags, stream)
        if status is not None:
            return _check(status, "bitlinear_softmax")
    at = _device(y, "y")
    _need_on(y, at, torch.float32, "y")
    if y.dim() != 2:
        raise ValueError(f"y must be [M, N], got {tuple(y.shape)}")
    _need_on(p, at, torch.float32, "p", y.shape)
    if temperature is not None:
        _need_on(temperature, at, torch.float32, "temperature", y.shape[:1])
    _check(load_library().bitlinear_softmax(y.data_ptr(), y.shape[0], y.shape[1], _ptr(temperature), p.data_ptr(), flags,
                                            _stream(stream)), "bitlinear_softmax")


def bitlinear_verify(p, q, draft, uniform, tokens, accepted, flags: int = 0, stream=None):
    """Verifies drafts [B, K] (int32) against the target's probabilities p [B, K + 1, N], given the draft's
    q [B, K, N] and random numbers uniform [B, K + 1] in [0, 1): tokens [B, K + 1] (int32) = the drafts taken, one token
    drawn, then -1; accepted [B] (int32) = how many were taken.  q and draft None: K = 0, a token is drawn."""
    if not _ready:
        _get_ready()
    if _marshal is not None:
        status = _marshal.verify(p, q, draft, uniform, tokens, accepted, flags, stream)
        if status is not None:
            return _check(status, "bitlinear_verify")
    at = _device(p, "p")
    f32, i32 = torch.float32, torch.int32
    _need_on(p, at, f32, "p")
    if p.dim() != 3 or p.shape[1] < 1:
        raise ValueError(f"p must be [sequences, drafts + 1, N], got {tuple(p.shape)}")
    B, K, N = p.shape[0], p.shape[1] - 1, p.shape[2]
    if K > 0 or q is not None:
        _need_on(q, at, f32, "q", (B, K, N))
    if K > 0 or draft is not None:
        _need_on(draft, at, i32, "draft", (B, K))
    _need_on(uniform, at, f32, "uniform", (B, K + 1))
    _need_on(tokens, at, i32, "tokens", (B, K + 1))
    _need_on(accepted, at, i32, "accepted", (B,))
    _check(load_library().bitlinear_verify(p.data_ptr(), _ptr(q) if K else None, B, _as_int(K), N, _ptr(draft) if K else None,
                                           uniform.data_ptr(), tokens.data_ptr(), accepted.data_ptr(), flags,
                                           _stream(stream)), "bitlinear_verify")
