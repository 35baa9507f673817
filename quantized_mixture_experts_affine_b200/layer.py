"""Layer descriptors over device-resident packed weights.

``DeviceLayer`` owns the torch tensors of one layer and the ``moeq_layer``
struct that points at them.  ``synthetic_layer`` fills one from the seeded
generator; real weights can be wrapped the same way with ``moeq.qtensor``.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass, field

from . import moeq
from . import synth
from .config import CONFIGS, LayerConfig  # noqa: F401  (re-exported)


@dataclass
class DeviceLayer:
    cfg: LayerConfig
    router: synth.DevQ
    gate: synth.DevQ
    up: synth.DevQ
    down: synth.DevQ
    sh_gate: synth.DevQ | None = None
    sh_up: synth.DevQ | None = None
    sh_down: synth.DevQ | None = None
    sh_expert_gate: synth.DevQ | None = None
    desc: moeq.Layer = field(default=None)

    def __post_init__(self):
        c = self.cfg

        def q(t: synth.DevQ):
            return moeq.qtensor(t.w, t.s, t.b, t.out_dim, t.in_dim, t.bits, t.group_size,
                                t.n_mats, getattr(t, "fmt", 0))
        z = moeq.QTensor()
        self.desc = moeq.Layer(q(self.router), q(self.gate), q(self.up), q(self.down),
                               int(c.shared), q(self.sh_gate) if c.shared else z,
                               q(self.sh_up) if c.shared else z,
                               q(self.sh_down) if c.shared else z,
                               q(self.sh_expert_gate) if c.shared else z,
                               c.H, c.I, c.E, c.K, int(c.renorm), float(c.router_scale))

    def nbytes(self) -> int:
        ts = [self.router, self.gate, self.up, self.down]
        if self.cfg.shared:
            ts += [self.sh_gate, self.sh_up, self.sh_down, self.sh_expert_gate]
        return sum(t.nbytes for t in ts)


def synthetic_layer(cfg: LayerConfig, seed: int = 0, copy: int = 0, device="cuda") -> DeviceLayer:
    """All tensors of one layer drawn on the device from the seeded streams
    (stream tag = (tensor kind, copy), matrix m of a bank = tag + m)."""
    T = lambda kind: synth.tag(kind, copy)
    mk = lambda kind, n, o, i, b, rq=False: synth.tensor_dev(seed, T(kind), n, o, i, b, cfg.G, rq,
                                                             device)
    kw = {}
    if cfg.shared:
        kw = dict(sh_gate=mk(synth.SH_GATE, 1, cfg.shared_I, cfg.H, cfg.shared_bits),
                  sh_up=mk(synth.SH_UP, 1, cfg.shared_I, cfg.H, cfg.shared_bits),
                  sh_down=mk(synth.SH_DOWN, 1, cfg.H, cfg.shared_I, cfg.shared_bits),
                  sh_expert_gate=mk(synth.SH_EXPERT_GATE, 1, 1, cfg.H, cfg.shared_gate_bits))
    return DeviceLayer(cfg,
                       router=mk(synth.ROUTER, 1, cfg.E, cfg.H, cfg.router_bits),
                       gate=mk(synth.GATE, cfg.E, cfg.I, cfg.H, cfg.expert_bits, cfg.requant_from4),
                       up=mk(synth.UP, cfg.E, cfg.I, cfg.H, cfg.expert_bits, cfg.requant_from4),
                       down=mk(synth.DOWN, cfg.E, cfg.H, cfg.I, cfg.expert_bits, cfg.requant_from4),
                       **kw)


class Workspace:
    """A device workspace sized for a layer, a token count and a mode."""

    def __init__(self, L: DeviceLayer, M: int, mode: int = moeq.MODE_AUTO, device="cuda"):
        import torch
        self.bytes = moeq.moeq_workspace_bytes(L.desc, M, mode)
        if self.bytes == 0:
            raise moeq.MoeqError("moeq_workspace_bytes", moeq.ERR_UNSUPPORTED)
        # 256-byte aligned (torch's caching allocator aligns to 512)
        self.buf = torch.empty(self.bytes, dtype=torch.uint8, device=device)


class _Buffers:
    """Where a call on `stream` (None: the current one; a stream object or a raw
    handle) gets its buffers: from that stream's own memory, so that neither a
    workspace nor a dropped result is handed out again before `stream` is past
    the call.  What the caller keeps is recorded on the current stream as well.
    Inputs are the caller's: they have to outlive the call."""

    def __init__(self, stream, device):
        self.device, self.side = device, None
        if stream is None:
            return
        import torch
        handle = int(stream if isinstance(stream, int) else stream.cuda_stream)
        self.current = torch.cuda.current_stream(device)
        if handle == self.current.cuda_stream:
            return
        if isinstance(stream, torch.cuda.Stream):
            self.side = stream
        elif handle in (0, 1):  # (the legacy default stream has two names)
            self.side = torch.cuda.default_stream(device)
        else:
            self.side = torch.cuda.ExternalStream(handle, device)

    def scope(self):
        """Allocations in it are the stream's."""
        import torch
        return contextlib.nullcontext() if self.side is None else torch.cuda.stream(self.side)

    def scratch(self, nbytes: int):
        import torch
        with self.scope():
            return torch.empty(nbytes, dtype=torch.uint8, device=self.device)

    def workspace(self, L: "DeviceLayer", M: int, mode: int) -> Workspace:
        with self.scope():
            return Workspace(L, M, mode, self.device)

    def result(self, shape, dtype):
        import torch
        if self.side is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with self.scope():
            t = torch.empty(shape, dtype=dtype, device=self.device)
        t.record_stream(self.current)
        return t


def layer_forward(L: DeviceLayer, x, y=None, residual=None, idx=None, w=None, ws=None,
                  mode: int = moeq.MODE_AUTO, stream=None):
    """y = layer(x) for bf16 x [M][H] on the device; returns (y, idx, w)."""
    import torch
    M, buf = x.shape[0], _Buffers(stream, x.device)
    if y is None:
        y = buf.result((M, L.cfg.H), torch.float32)
    if idx is None:
        idx = buf.result((M, L.cfg.K), torch.int32)
    if w is None:
        w = buf.result((M, L.cfg.K), torch.float32)
    if ws is None:
        ws = buf.workspace(L, M, mode)
    moeq.moeq_layer_forward(L.desc, x, M, y, residual, idx, w, ws.buf, ws.bytes, mode, stream)
    return y, idx, w


def layer_forward_norm(L: DeviceLayer, x, gamma, eps: float, y=None, y_norm=None, residual=None,
                       idx=None, w=None, ws=None, mode: int = moeq.MODE_AUTO, stream=None):
    """y = layer(x) and y_norm = bf16 RMS norm of y with weights gamma (bf16
    [H]); returns (y, y_norm, idx, w)."""
    import torch
    M, buf = x.shape[0], _Buffers(stream, x.device)
    if y is None:
        y = buf.result((M, L.cfg.H), torch.float32)
    if y_norm is None:
        y_norm = buf.result((M, L.cfg.H), torch.bfloat16)
    if idx is None:
        idx = buf.result((M, L.cfg.K), torch.int32)
    if w is None:
        w = buf.result((M, L.cfg.K), torch.float32)
    if ws is None:
        ws = buf.workspace(L, M, mode)
    moeq.moeq_layer_forward_norm(L.desc, x, M, y, gamma, eps, y_norm, residual, idx, w, ws.buf,
                                 ws.bytes, mode, stream)
    return y, y_norm, idx, w


def expert_ffn(L: DeviceLayer, x, idx, w, y=None, residual=None, ws=None,
               mode: int = moeq.MODE_AUTO, stream=None):
    import torch
    M, buf = x.shape[0], _Buffers(stream, x.device)
    if y is None:
        y = buf.result((M, L.cfg.H), torch.float32)
    if ws is None:
        ws = buf.workspace(L, M, mode)
    moeq.moeq_expert_ffn(L.desc, x, M, idx, w, residual, y, ws.buf, ws.bytes, mode, stream)
    return y


def route_groups(r: moeq.Routing, logits, bias=None, stream=None):
    """Routing `r` of logits [M][E]; returns (idx, w)."""
    import torch
    M, buf = logits.shape[0], _Buffers(stream, logits.device)
    idx = buf.result((M, r.top_k), torch.int32)
    w = buf.result((M, r.top_k), torch.float32)
    moeq.moeq_route_groups(r, logits, idx, w, bias, stream)
    return idx, w


def add_rmsnorm(x, gamma, eps: float, residual=None, want_y: bool = True, q_dtype=None,
                q_group: int = 0, stream=None):
    """RMS norm of x + residual; returns (r, y, q, q_scales): the new residual
    stream (None without a residual), the bf16 norm (with want_y) and its codes
    in q_dtype (torch.int8 or torch.float8_e4m3fn) with their scales."""
    import torch
    M, H = x.shape
    buf = _Buffers(stream, x.device)
    r = buf.result(residual.shape, residual.dtype) if residual is not None else None
    y = buf.result((M, H), torch.bfloat16) if want_y else None
    q = qs = None
    if q_dtype is not None:
        q = buf.result((M, H), q_dtype)
        qs = buf.result((M, -(-H // q_group) if q_group else 1), torch.float32)
    moeq.moeq_add_rmsnorm(x, gamma, eps, residual, r, y, q, qs, q_group, stream)
    return r, y, q, qs


def linear(t: moeq.QTensor, x, out_dtype=None, expert: int = 0, x_scales=None, x_group: int = 0,
           bias=None, act: int = moeq.ACT_NONE, mul=None, residual=None, y=None, ws=None,
           stream=None):
    """y = act(x W^T + bias) * mul + residual (out_dtype: fp32 or, by default,
    bf16); returns y.  The workspace is allocated where none is given."""
    import torch
    M, buf = x.shape[0], _Buffers(stream, x.device)
    if y is None:
        y = buf.result((M, t.out_dim), out_dtype or torch.bfloat16)
    if ws is None:
        need = moeq.moeq_linear_workspace_bytes(t, M, x.dtype, y.dtype)
        if need:
            ws = buf.scratch(need)
    moeq.moeq_linear(t, expert, x, y, x_scales, x_group, bias, act, mul, residual, ws, stream)
    return y


def layer_forward_routed(L: DeviceLayer, r: moeq.Routing, x, bias=None, residual=None,
                         mode: int = moeq.MODE_AUTO, ws=None, stream=None):
    """y = layer(x) under routing `r`; returns (y, idx, w).  ws: uint8 buffer of
    moeq_routed_workspace_bytes."""
    import torch
    M, buf = x.shape[0], _Buffers(stream, x.device)
    y = buf.result((M, L.cfg.H), torch.float32)
    idx = buf.result((M, L.cfg.K), torch.int32)
    w = buf.result((M, L.cfg.K), torch.float32)
    if ws is None:
        ws = buf.scratch(moeq.moeq_routed_workspace_bytes(L.desc, M, mode))
    moeq.moeq_layer_forward_routed(L.desc, r, x, M, y, bias, residual, idx, w, ws, ws.numel(),
                                   mode, stream)
    return y, idx, w
