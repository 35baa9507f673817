"""Python binding of libmoeq.so (include/moeq.h): argument marshalling only.

Every function here forwards to the C entry point of the same name; device
buffers are passed as torch CUDA tensors (their data pointers) and streams
as torch streams.  There is no fallback: if the library is missing this
module fails to import, and a non-OK status raises MoeqError.
"""
from __future__ import annotations

import ctypes as C
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libmoeq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built: run `python -m quantized_mixture_experts_affine_b200._build`"
                      " (nvcc, sm_100a) before using the layer library")

_lib = C.CDLL(LIB_PATH)

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_ALIGNMENT, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, \
    ERR_RANGE = range(8)
MODE_AUTO, MODE_DECODE, MODE_PREFILL = 0, 1, 2

EXPORTS = ("moeq_dequant", "moeq_qmv", "moeq_route_topk", "moeq_expert_ffn", "moeq_layer_forward",
           "moeq_workspace_bytes", "moeq_device_status", "moeq_status_str", "moeq_version",
           "moeq_set_profile_events", "moeq_launch_count", "moeq_layer_forward_static",
           "moeq_static_workspace_capacity", "moeq_selftest_wait_timeout",
           "moeq_layer_forward_norm", "moeq_cache_create", "moeq_cache_workspace_bytes",
           "moeq_cache_forward", "moeq_cache_stats", "moeq_cache_destroy",
           "moeq_route_groups", "moeq_add_rmsnorm", "moeq_linear", "moeq_linear_workspace_bytes",
           "moeq_layer_forward_routed", "moeq_routed_workspace_bytes")


class MoeqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_str(status)} (status {status})")


class QTensor(C.Structure):
    """moeq_qtensor."""
    _fields_ = [("w", C.c_void_p), ("scales", C.c_void_p), ("biases", C.c_void_p),
                ("out_dim", C.c_int32), ("in_dim", C.c_int32), ("bits", C.c_int32),
                ("group_size", C.c_int32), ("expert_stride_w", C.c_int64),
                ("expert_stride_sb", C.c_int64), ("format", C.c_int32)]


class Layer(C.Structure):
    """moeq_layer."""
    _fields_ = [("router", QTensor), ("gate", QTensor), ("up", QTensor), ("down", QTensor),
                ("has_shared", C.c_int32), ("sh_gate", QTensor), ("sh_up", QTensor),
                ("sh_down", QTensor), ("sh_expert_gate", QTensor), ("hidden", C.c_int32),
                ("inter", C.c_int32), ("n_experts", C.c_int32), ("top_k", C.c_int32),
                ("renorm", C.c_int32), ("router_scale", C.c_float)]


class Routing(C.Structure):
    """moeq_routing."""
    _fields_ = [("n_experts", C.c_int32), ("top_k", C.c_int32), ("score", C.c_int32),
                ("n_groups", C.c_int32), ("topk_groups", C.c_int32), ("group_top", C.c_int32),
                ("renorm", C.c_int32), ("router_scale", C.c_float), ("routed_scale", C.c_float)]


class NormArgs(C.Structure):
    """moeq_norm_args."""
    _fields_ = [("x", C.c_void_p), ("x_type", C.c_int32), ("x_stride", C.c_int64),
                ("residual", C.c_void_p), ("r_type", C.c_int32), ("r_stride", C.c_int64),
                ("r_out", C.c_void_p), ("r_out_stride", C.c_int64), ("gamma", C.c_void_p),
                ("eps", C.c_float), ("y", C.c_void_p), ("y_stride", C.c_int64),
                ("q", C.c_void_p), ("q_type", C.c_int32), ("q_stride", C.c_int64),
                ("q_scales", C.c_void_p), ("q_group", C.c_int32)]


class LinearArgs(C.Structure):
    """moeq_linear_args."""
    _fields_ = [("x", C.c_void_p), ("x_type", C.c_int32), ("x_stride", C.c_int64),
                ("x_scales", C.c_void_p), ("x_group", C.c_int32), ("bias", C.c_void_p),
                ("act", C.c_int32), ("mul", C.c_void_p), ("mul_stride", C.c_int64),
                ("residual", C.c_void_p), ("residual_stride", C.c_int64), ("y", C.c_void_p),
                ("out_type", C.c_int32), ("y_stride", C.c_int64)]


_P = C.c_void_p
_lib.moeq_dequant.argtypes = [C.POINTER(QTensor), C.c_int32, _P, _P, _P]
_lib.moeq_qmv.argtypes = [C.POINTER(QTensor), C.c_int32, _P, C.c_int32, _P, _P]
_lib.moeq_route_topk.argtypes = [_P, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_float, _P,
                                 _P, _P]
_lib.moeq_expert_ffn.argtypes = [C.POINTER(Layer), _P, C.c_int32, _P, _P, _P, _P, _P, C.c_size_t,
                                 C.c_int32, _P]
_lib.moeq_layer_forward.argtypes = [C.POINTER(Layer), _P, C.c_int32, _P, _P, _P, _P, _P,
                                    C.c_size_t, C.c_int32, _P]
_lib.moeq_layer_forward_static.argtypes = [C.POINTER(Layer), _P, C.c_int32, _P, _P, _P, _P, _P]
_lib.moeq_cache_create.argtypes = [C.POINTER(Layer), C.c_int32, C.c_int32, C.POINTER(C.c_void_p)]
_lib.moeq_cache_create.restype = C.c_int
_lib.moeq_cache_workspace_bytes.argtypes = [C.c_void_p, C.c_int32]
_lib.moeq_cache_workspace_bytes.restype = C.c_size_t
_lib.moeq_cache_forward.argtypes = [C.c_void_p, _P, C.c_int32, _P, _P, _P, _P, _P, C.c_size_t, _P]
_lib.moeq_cache_forward.restype = C.c_int
_lib.moeq_cache_stats.argtypes = [C.c_void_p, C.POINTER(C.c_uint64), C.POINTER(C.c_uint64),
                                  C.POINTER(C.c_uint64)]
_lib.moeq_cache_stats.restype = C.c_int
_lib.moeq_cache_destroy.argtypes = [C.c_void_p]
_lib.moeq_cache_destroy.restype = None
_lib.moeq_layer_forward_norm.argtypes = [C.POINTER(Layer), _P, C.c_int32, _P, _P, _P, C.c_float,
                                         _P, _P, _P, _P, C.c_size_t, C.c_int32, _P]
_lib.moeq_static_workspace_capacity.restype = C.c_size_t
_lib.moeq_workspace_bytes.argtypes = [C.POINTER(Layer), C.c_int32, C.c_int32]
_lib.moeq_workspace_bytes.restype = C.c_size_t
_lib.moeq_device_status.argtypes = [_P, C.POINTER(C.c_int32)]
_lib.moeq_selftest_wait_timeout.argtypes = [_P]
_lib.moeq_status_str.argtypes = [C.c_int32]
_lib.moeq_status_str.restype = C.c_char_p
_lib.moeq_version.restype = C.c_char_p
_lib.moeq_set_profile_events.argtypes = [_P, _P]
_lib.moeq_set_profile_events.restype = C.c_int
_lib.moeq_launch_count.restype = C.c_uint64
_lib.moeq_route_groups.argtypes = [C.POINTER(Routing), _P, C.c_int32, C.c_int64, _P, C.c_int32, _P,
                                   _P, _P]
_lib.moeq_add_rmsnorm.argtypes = [C.POINTER(NormArgs), C.c_int32, C.c_int32, _P]
_lib.moeq_linear.argtypes = [C.POINTER(QTensor), C.c_int32, C.POINTER(LinearArgs), C.c_int32, _P,
                             C.c_size_t, _P]
_lib.moeq_linear_workspace_bytes.argtypes = [C.POINTER(QTensor), C.c_int32, C.c_int32, C.c_int32]
_lib.moeq_linear_workspace_bytes.restype = C.c_size_t
_lib.moeq_layer_forward_routed.argtypes = [C.POINTER(Layer), C.POINTER(Routing), _P, _P, C.c_int32,
                                           _P, _P, _P, _P, _P, C.c_size_t, C.c_int32, _P]
_lib.moeq_routed_workspace_bytes.argtypes = [C.POINTER(Layer), C.c_int32, C.c_int32]
_lib.moeq_routed_workspace_bytes.restype = C.c_size_t
for _f in ("moeq_dequant", "moeq_qmv", "moeq_route_topk", "moeq_expert_ffn", "moeq_layer_forward",
           "moeq_layer_forward_static", "moeq_device_status", "moeq_selftest_wait_timeout",
           "moeq_layer_forward_norm", "moeq_route_groups", "moeq_add_rmsnorm", "moeq_linear",
           "moeq_layer_forward_routed"):
    getattr(_lib, _f).restype = C.c_int


def lib() -> C.CDLL:
    return _lib


def status_str(status: int) -> str:
    return _lib.moeq_status_str(int(status)).decode()


def version() -> str:
    return _lib.moeq_version().decode()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(s):
    if s is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(fn, rc):
    if rc != OK:
        raise MoeqError(fn, rc)


FMT_AFFINE, FMT_MXFP4 = 0, 1
F32, BF16, I8, E4M3 = range(4)
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
ACT_NONE, ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_RELU, ACT_SIGMOID = range(6)
_DTYPES = {}


def dtype_code(dtype) -> int:
    """moeq_dtype of a torch dtype."""
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: F32, torch.bfloat16: BF16, torch.int8: I8,
                        torch.float8_e4m3fn: E4M3})
    try:
        return _DTYPES[dtype]
    except KeyError:
        raise MoeqError(f"dtype {dtype}", ERR_UNSUPPORTED) from None


def _device(name, t) -> int:
    """Launches go to the current device: its tensors have to be there too."""
    import torch
    d = t.get_device()
    if d < 0 or d != torch.cuda.current_device():
        raise ValueError(f"{name}: on {t.device}, not on the current CUDA device")
    return d


def _rows(name, t, M, n, dtype=None, device=None):
    """Row stride of a [M][n] tensor whose rows are contiguous, of the given
    type and on the given device; raises ValueError otherwise."""
    if t.shape != (M, n) or (n > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected [{M}][{n}] with contiguous rows, got "
                         f"{tuple(t.shape)} with strides {t.stride()}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, not on CUDA device {device}")
    return t.stride(0) if M > 1 else n


def _dense(name, t, shape, dtype, device):
    """Address of a contiguous tensor of the given shape, type and device."""
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous() \
            or t.get_device() != device:
        raise ValueError(f"{name}: expected contiguous {dtype} {shape} on device {device}, got "
                         f"{t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _x_scales_shape(M, n, group):
    return (M, -(-n // group)) if group else (M, 1)


def qtensor(w, scales, biases, out_dim, in_dim, bits, group_size=64, n_mats=1,
            fmt: int = FMT_AFFINE) -> QTensor:
    """Descriptor of a bank of n_mats packed matrices stored back to back
    (MX FP4: scales are the uint8 exponents, biases unused)."""
    sw = out_dim * in_dim * bits // 32 if n_mats > 1 else 0
    ssb = out_dim * (in_dim // group_size) if n_mats > 1 else 0
    return QTensor(_ptr(w), _ptr(scales), _ptr(biases) if fmt == FMT_AFFINE else None, out_dim,
                   in_dim, bits, group_size, sw, ssb, fmt)


def moeq_dequant(t: QTensor, expert: int, q_out=None, w_out=None, stream=None) -> None:
    _check("moeq_dequant", _lib.moeq_dequant(C.byref(t), expert, _ptr(q_out), _ptr(w_out),
                                             _stream(stream)))


def moeq_qmv(t: QTensor, expert: int, x, M: int, y, stream=None) -> None:
    _check("moeq_qmv", _lib.moeq_qmv(C.byref(t), expert, _ptr(x), M, _ptr(y), _stream(stream)))


def moeq_route_topk(logits, M: int, E: int, K: int, renorm: bool, router_scale: float, idx, w,
                    stream=None) -> None:
    _check("moeq_route_topk", _lib.moeq_route_topk(_ptr(logits), M, E, K, int(renorm),
                                                   float(router_scale), _ptr(idx), _ptr(w),
                                                   _stream(stream)))


def routing(n_experts: int, top_k: int, score: int = SCORE_SOFTMAX, n_groups: int = 1,
            topk_groups: int = 1, group_top: int = 1, renorm: bool = True,
            router_scale: float = 1.0, routed_scale: float = 1.0) -> Routing:
    return Routing(n_experts, top_k, score, n_groups, topk_groups, group_top, int(renorm),
                   router_scale, routed_scale)


def moeq_route_groups(r: Routing, logits, idx, w, bias=None, stream=None) -> None:
    """Routing `r` of logits [M][E] (fp32 or bf16, rows may be strided) into
    idx int32 [M][K] and w fp32 [M][K]; bias: fp32 [E] or None."""
    import torch
    dev = _device("logits", logits)
    M, E, K = logits.shape[0], r.n_experts, r.top_k
    _check("moeq_route_groups",
           _lib.moeq_route_groups(
               C.byref(r), logits.data_ptr(), dtype_code(logits.dtype),
               _rows("logits", logits, M, E),
               None if bias is None else _dense("bias", bias, (E,), torch.float32, dev), M,
               _dense("idx", idx, (M, K), torch.int32, dev),
               _dense("w", w, (M, K), torch.float32, dev), _stream(stream)))


def moeq_add_rmsnorm(x, gamma, eps: float, residual=None, r_out=None, y=None, q=None,
                     q_scales=None, q_group: int = 0, stream=None) -> None:
    """r = x + residual (into r_out), y = bf16 RMS norm of r with weights
    gamma, q = its int8 or float8_e4m3fn codes with q_scales fp32 [M][1]
    (q_group 0) or [M][ceil(H / 128)] (q_group 128)."""
    import torch
    dev = _device("x", x)
    M, H = x.shape
    a = NormArgs(x.data_ptr(), dtype_code(x.dtype), _rows("x", x, M, H))
    a.gamma, a.eps = _dense("gamma", gamma, (H,), torch.bfloat16, dev), eps
    if residual is not None:
        a.residual, a.r_type = residual.data_ptr(), dtype_code(residual.dtype)
        a.r_stride = _rows("residual", residual, M, H, None, dev)
    if r_out is not None:
        a.r_out = r_out.data_ptr()
        a.r_out_stride = _rows("r_out", r_out, M, H,
                               None if residual is None else residual.dtype, dev)
    if y is not None:
        a.y, a.y_stride = y.data_ptr(), _rows("y", y, M, H, torch.bfloat16, dev)
    if q is not None:
        a.q, a.q_type, a.q_group = q.data_ptr(), dtype_code(q.dtype), q_group
        a.q_stride = _rows("q", q, M, H, None, dev)
        if q_scales is not None:
            a.q_scales = _dense("q_scales", q_scales, _x_scales_shape(M, H, q_group),
                                torch.float32, dev)
    _check("moeq_add_rmsnorm", _lib.moeq_add_rmsnorm(C.byref(a), M, H, _stream(stream)))


def moeq_linear_workspace_bytes(t: QTensor, M: int, x_dtype, out_dtype) -> int:
    return int(_lib.moeq_linear_workspace_bytes(C.byref(t), M, dtype_code(x_dtype),
                                                dtype_code(out_dtype)))


def moeq_linear(t: QTensor, expert: int, x, y, x_scales=None, x_group: int = 0, bias=None,
                act: int = ACT_NONE, mul=None, residual=None, ws=None, stream=None) -> None:
    """y = act(x W^T + bias) * mul + residual with matrix `expert` of t.
    x: bf16, int8 or float8_e4m3fn (with x_scales as moeq_add_rmsnorm writes
    them) [M][in_dim]; y, mul, residual: fp32 or bf16 [M][out_dim]; ws: uint8
    buffer of moeq_linear_workspace_bytes."""
    import torch
    dev = _device("x", x)
    M, n, o = x.shape[0], t.in_dim, t.out_dim
    a = LinearArgs(x.data_ptr(), dtype_code(x.dtype), _rows("x", x, M, n))
    if x_scales is not None:
        a.x_scales = _dense("x_scales", x_scales, _x_scales_shape(M, n, x_group), torch.float32,
                            dev)
        a.x_group = x_group
    a.act, a.y, a.out_type = act, y.data_ptr(), dtype_code(y.dtype)
    a.y_stride = _rows("y", y, M, o, None, dev)
    if bias is not None:
        a.bias = _dense("bias", bias, (o,), torch.bfloat16, dev)
    if mul is not None:
        a.mul, a.mul_stride = mul.data_ptr(), _rows("mul", mul, M, o, y.dtype, dev)
    if residual is not None:
        a.residual = residual.data_ptr()
        a.residual_stride = _rows("residual", residual, M, o, y.dtype, dev)
    n_ws = 0
    if ws is not None:
        n_ws = ws.numel() * ws.element_size()
        if ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError(f"ws: expected contiguous on device {dev}, got {ws.device}")
    _check("moeq_linear", _lib.moeq_linear(C.byref(t), expert, C.byref(a), M, _ptr(ws), n_ws,
                                           _stream(stream)))


def moeq_routed_workspace_bytes(L: Layer, M: int, mode: int = MODE_AUTO) -> int:
    return int(_lib.moeq_routed_workspace_bytes(C.byref(L), M, mode))


def moeq_layer_forward_routed(L: Layer, r: Routing, x, M: int, y, bias=None, residual=None,
                              idx_out=None, w_out=None, ws=None, ws_bytes: int = 0,
                              mode: int = MODE_AUTO, stream=None) -> None:
    """moeq_layer_forward with routing `r` (and its balance bias)."""
    _check("moeq_layer_forward_routed",
           _lib.moeq_layer_forward_routed(C.byref(L), C.byref(r), _ptr(bias), _ptr(x), M, _ptr(y),
                                          _ptr(residual), _ptr(idx_out), _ptr(w_out), _ptr(ws),
                                          ws_bytes, mode, _stream(stream)))


def moeq_workspace_bytes(L: Layer, M: int, mode: int = MODE_AUTO) -> int:
    return int(_lib.moeq_workspace_bytes(C.byref(L), M, mode))


def moeq_expert_ffn(L: Layer, x, M: int, idx, w, residual, y, ws, ws_bytes: int,
                    mode: int = MODE_AUTO, stream=None) -> None:
    _check("moeq_expert_ffn", _lib.moeq_expert_ffn(C.byref(L), _ptr(x), M, _ptr(idx), _ptr(w),
                                                   _ptr(residual), _ptr(y), _ptr(ws), ws_bytes,
                                                   mode, _stream(stream)))


def moeq_layer_forward(L: Layer, x, M: int, y, residual=None, idx_out=None, w_out=None, ws=None,
                       ws_bytes: int = 0, mode: int = MODE_AUTO, stream=None) -> None:
    _check("moeq_layer_forward",
           _lib.moeq_layer_forward(C.byref(L), _ptr(x), M, _ptr(y), _ptr(residual),
                                   _ptr(idx_out), _ptr(w_out), _ptr(ws), ws_bytes, mode,
                                   _stream(stream)))


def moeq_layer_forward_norm(L: Layer, x, M: int, y, gamma, eps: float, y_norm, residual=None,
                            idx_out=None, w_out=None, ws=None, ws_bytes: int = 0,
                            mode: int = MODE_AUTO, stream=None) -> None:
    """moeq_layer_forward plus y_norm = bf16 RMS norm of y with weights gamma."""
    _check("moeq_layer_forward_norm",
           _lib.moeq_layer_forward_norm(C.byref(L), _ptr(x), M, _ptr(y), _ptr(residual),
                                        _ptr(gamma), float(eps), _ptr(y_norm), _ptr(idx_out),
                                        _ptr(w_out), _ptr(ws), ws_bytes, mode, _stream(stream)))


def moeq_layer_forward_static(L: Layer, x, M: int, y, residual=None, idx_out=None, w_out=None,
                              stream=None) -> None:
    """Decode layer forward on the library's fixed per-device workspace."""
    _check("moeq_layer_forward_static",
           _lib.moeq_layer_forward_static(C.byref(L), _ptr(x), M, _ptr(y), _ptr(residual),
                                          _ptr(idx_out), _ptr(w_out), _stream(stream)))


def moeq_static_workspace_capacity() -> int:
    return int(_lib.moeq_static_workspace_capacity())


def moeq_set_profile_events(start=None, stop=None) -> None:
    """start/stop: torch.cuda.Event (or None to turn profiling off)."""
    _check("moeq_set_profile_events",
           _lib.moeq_set_profile_events(None if start is None else start.cuda_event,
                                        None if stop is None else stop.cuda_event))


def moeq_launch_count() -> int:
    return int(_lib.moeq_launch_count())


def moeq_selftest_wait_timeout(stream=None) -> None:
    _check("moeq_selftest_wait_timeout", _lib.moeq_selftest_wait_timeout(_stream(stream)))


def moeq_device_status(stream=None) -> int:
    v = C.c_int32(0)
    _check("moeq_device_status", _lib.moeq_device_status(_stream(stream), C.byref(v)))
    return int(v.value)


class ExpertCache:
    """moeq_expert_cache: routed expert banks in host memory, `slots` of
    them cached in HBM (see include/moeq.h).  Keeps the layer descriptor
    alive; frees the cache on close()."""

    def __init__(self, L: Layer, slots: int, max_tokens: int):
        self._L = L
        self._h = C.c_void_p()
        _check("moeq_cache_create", _lib.moeq_cache_create(C.byref(L), slots, max_tokens,
                                                           C.byref(self._h)))

    def workspace_bytes(self, M: int) -> int:
        return int(_lib.moeq_cache_workspace_bytes(self._h, M))

    def forward(self, x, M: int, y, ws, ws_bytes: int, residual=None, idx_out=None, w_out=None,
                stream=None) -> None:
        _check("moeq_cache_forward",
               _lib.moeq_cache_forward(self._h, _ptr(x), M, _ptr(y), _ptr(residual),
                                       _ptr(idx_out), _ptr(w_out), _ptr(ws), ws_bytes,
                                       _stream(stream)))

    def stats(self):
        h, m, b = C.c_uint64(), C.c_uint64(), C.c_uint64()
        _check("moeq_cache_stats", _lib.moeq_cache_stats(self._h, C.byref(h), C.byref(m),
                                                         C.byref(b)))
        return int(h.value), int(m.value), int(b.value)

    def close(self) -> None:
        if self._h:
            _lib.moeq_cache_destroy(self._h)
            self._h = C.c_void_p()
