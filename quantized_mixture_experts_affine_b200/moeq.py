"""Python binding of libmoeq.so (include/moeq.h): argument marshalling only.

Every function here forwards to the C entry point of the same name; device
buffers are passed as torch CUDA tensors (their data pointers) and streams
as torch streams.  There is no fallback: if the library is missing this
module fails to import, and a non-OK status raises MoeqError.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

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
_lib.moeq_add_rmsnorm.argtypes = [_P, C.c_int32, C.c_int32, _P]  # NormArgs
_lib.moeq_linear.argtypes = [C.POINTER(QTensor), C.c_int32, _P, C.c_int32, _P, C.c_size_t,
                             _P]  # the third: LinearArgs
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
        return torch.cuda.current_stream().cuda_stream
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
        _load_torch()
    try:
        return _DTYPES[dtype]
    except KeyError:
        raise MoeqError(f"dtype {dtype}", ERR_UNSUPPORTED) from None


def _load_torch() -> None:
    """torch's types and its current device and stream, looked up once: these
    calls are made thousands of times a second, a microsecond counts."""
    global _int32, _float32, _bfloat16, _current_device, _raw_stream
    import torch
    _int32, _float32, _bfloat16 = torch.int32, torch.float32, torch.bfloat16
    _current_device = torch._C._cuda_getDevice if torch.cuda.is_available() else lambda: -2
    _raw_stream = torch._C._cuda_getCurrentRawStream if torch.cuda.is_available() else None
    _DTYPES.update({torch.float32: F32, torch.bfloat16: BF16, torch.int8: I8,
                    torch.float8_e4m3fn: E4M3})


def _device(name, t) -> int:
    """Launches go to the current device: its tensors have to be there too."""
    if not _DTYPES:
        _load_torch()
    d = t.get_device()
    if d < 0 or d != _current_device():
        raise ValueError(f"{name}: on {t.device}, not on the current CUDA device")
    return d


def _rows(name, t, M, n, dtype=None, device=None):
    """Row stride of a [M][n] tensor whose rows are contiguous, of the given
    type and on the given device; raises ValueError otherwise."""
    stride = n
    if t.shape != (M, n) or not t.is_contiguous():
        if t.shape != (M, n) or (n > 1 and t.stride(1) != 1):
            raise ValueError(f"{name}: expected [{M}][{n}] with contiguous rows, got "
                             f"{tuple(t.shape)} with strides {t.stride()}")
        stride = t.stride(0) if M > 1 else n
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, not on CUDA device {device}")
    return stride


def _dense(name, t, shape, dtype, device):
    """Address of a contiguous tensor of the given shape, type and device."""
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous() \
            or t.get_device() != device:
        raise ValueError(f"{name}: expected contiguous {dtype} {shape} on device {device}, got "
                         f"{t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _first_rows(name, t, M, n, dtype, device):
    """Address of a contiguous tensor of at least M rows of n elements (None and
    raw addresses as they are)."""
    if t is None or isinstance(t, int):
        return t
    if t.dim() != 2 or t.shape[0] < M or t.shape[1] != n or t.dtype != dtype \
            or not t.is_contiguous() or (device is not None and t.get_device() != device):
        raise ValueError(f"{name}: expected contiguous {dtype} [{M}][{n}] on device {device}, got "
                         f"{t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return t.data_ptr()


# The argument structs packed in one step (native alignment; a null pointer
# is 0): several times faster than filling a ctypes Structure.
_NORM_ARGS = struct.Struct("@PiqPiqPqPfPqPiqPi0q")
_LINEAR_ARGS = struct.Struct("@PiqPiPiPqPqPiq0q")
assert _NORM_ARGS.size == C.sizeof(NormArgs) and _LINEAR_ARGS.size == C.sizeof(LinearArgs)


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
    dev = _device("logits", logits)
    M, E, K = logits.shape[0], r.n_experts, r.top_k
    rc = _lib.moeq_route_groups(
        C.byref(r), logits.data_ptr(), dtype_code(logits.dtype), _rows("logits", logits, M, E),
        None if bias is None else _dense("bias", bias, (E,), _float32, dev), M,
        _dense("idx", idx, (M, K), _int32, dev), _dense("w", w, (M, K), _float32, dev),
        _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check("moeq_route_groups", rc)


def moeq_add_rmsnorm(x, gamma, eps: float, residual=None, r_out=None, y=None, q=None,
                     q_scales=None, q_group: int = 0, stream=None) -> None:
    """r = x + residual (into r_out), y = bf16 RMS norm of r with weights
    gamma, q = its int8 or float8_e4m3fn codes with q_scales fp32 [M][1]
    (q_group 0) or [M][ceil(H / 128)] (q_group 128)."""
    dev = _device("x", x)
    M, H = x.shape
    pr = tr = sr = po = so = py = sy = pq = tq = sq = ps = 0
    if residual is not None:
        pr, tr = residual.data_ptr(), dtype_code(residual.dtype)
        sr = _rows("residual", residual, M, H, None, dev)
    if r_out is not None:
        po = r_out.data_ptr()
        so = _rows("r_out", r_out, M, H, None if residual is None else residual.dtype, dev)
    if y is not None:
        py, sy = y.data_ptr(), _rows("y", y, M, H, _bfloat16, dev)
    if q is not None:
        pq, tq, sq = q.data_ptr(), dtype_code(q.dtype), _rows("q", q, M, H, None, dev)
        if q_scales is not None:
            ps = _dense("q_scales", q_scales, _x_scales_shape(M, H, q_group), _float32, dev)
    a = _NORM_ARGS.pack(x.data_ptr(), dtype_code(x.dtype), _rows("x", x, M, H), pr, tr, sr, po, so,
                        _dense("gamma", gamma, (H,), _bfloat16, dev), eps, py, sy, pq, tq, sq, ps,
                        q_group)
    rc = _lib.moeq_add_rmsnorm(a, M, H, _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check("moeq_add_rmsnorm", rc)


def moeq_linear_workspace_bytes(t: QTensor, M: int, x_dtype, out_dtype) -> int:
    return int(_lib.moeq_linear_workspace_bytes(C.byref(t), M, dtype_code(x_dtype),
                                                dtype_code(out_dtype)))


def moeq_linear(t: QTensor, expert: int, x, y, x_scales=None, x_group: int = 0, bias=None,
                act: int = ACT_NONE, mul=None, residual=None, ws=None, stream=None) -> None:
    """y = act(x W^T + bias) * mul + residual with matrix `expert` of t.
    x: bf16, int8 or float8_e4m3fn (with x_scales as moeq_add_rmsnorm writes
    them) [M][in_dim]; y, mul, residual: fp32 or bf16 [M][out_dim]; ws: uint8
    buffer of moeq_linear_workspace_bytes."""
    dev = _device("x", x)
    M, n, o, yt = x.shape[0], t.in_dim, t.out_dim, y.dtype
    ps = pb = pm = sm = pr = sr = pw = nw = 0
    if x_scales is not None:
        ps = _dense("x_scales", x_scales, _x_scales_shape(M, n, x_group), _float32, dev)
    if bias is not None:
        pb = _dense("bias", bias, (o,), _bfloat16, dev)
    if mul is not None:
        pm, sm = mul.data_ptr(), _rows("mul", mul, M, o, yt, dev)
    if residual is not None:
        pr, sr = residual.data_ptr(), _rows("residual", residual, M, o, yt, dev)
    if ws is not None:
        pw, nw = ws.data_ptr(), ws.nbytes
        if ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError(f"ws: expected contiguous on device {dev}, got {ws.device}")
    a = _LINEAR_ARGS.pack(x.data_ptr(), dtype_code(x.dtype), _rows("x", x, M, n), ps, x_group, pb,
                          act, pm, sm, pr, sr, y.data_ptr(), dtype_code(yt),
                          _rows("y", y, M, o, None, dev))
    rc = _lib.moeq_linear(C.byref(t), expert, a, M, pw, nw,
                          _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check("moeq_linear", rc)


def moeq_routed_workspace_bytes(L: Layer, M: int, mode: int = MODE_AUTO) -> int:
    return int(_lib.moeq_routed_workspace_bytes(C.byref(L), M, mode))


def moeq_layer_forward_routed(L: Layer, r: Routing, x, M: int, y, bias=None, residual=None,
                              idx_out=None, w_out=None, ws=None, ws_bytes: int = 0,
                              mode: int = MODE_AUTO, stream=None) -> None:
    """moeq_layer_forward with routing `r` and its balance bias (fp32 [E]).  x:
    bf16 [M][H]; y, residual: fp32 [M][H]; idx_out: int32 [M][K]; w_out: fp32
    [M][K], at least M rows of each; ws: uint8 buffer of at least ws_bytes.  Raw
    addresses are taken as they are."""
    if not _DTYPES:
        _load_torch()
    dev = None if x is None or isinstance(x, int) else _device("x", x)
    H, E, K = L.hidden, L.n_experts, L.top_k
    px = _first_rows("x", x, M, H, _bfloat16, dev)
    py = _first_rows("y", y, M, H, _float32, dev)
    pr = _first_rows("residual", residual, M, H, _float32, dev)
    pi = _first_rows("idx_out", idx_out, M, K, _int32, dev)
    pw = _first_rows("w_out", w_out, M, K, _float32, dev)
    pb = _ptr(bias)
    if bias is not None and not isinstance(bias, int):
        pb = _dense("bias", bias, (E,), _float32, bias.get_device() if dev is None else dev)
    if ws is not None and not isinstance(ws, int):
        if not ws.is_contiguous() or ws.nbytes < ws_bytes or \
                (dev is not None and ws.get_device() != dev):
            raise ValueError(f"ws: expected {ws_bytes} contiguous bytes on device {dev}, got "
                             f"{ws.nbytes} on {ws.device}")
    _check("moeq_layer_forward_routed",
           _lib.moeq_layer_forward_routed(C.byref(L), C.byref(r), pb, px, M, py, pr, pi, pw,
                                          _ptr(ws), ws_bytes, mode, _stream(stream)))


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
