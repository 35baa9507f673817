"""Which stream's memory the allocating forms of layer.py use: that of the
stream the call runs on, given as an object or as a raw handle.  The CUDA parts
of torch are stand-ins (no GPU needed)."""
import contextlib

import pytest

from quantized_mixture_experts_affine_b200 import layer, moeq
from quantized_mixture_experts_affine_b200.config import CONFIGS

torch = pytest.importorskip("torch")
CURRENT, SIDE = 7 << 8, 9 << 8
CALLS = ("moeq_layer_forward", "moeq_layer_forward_norm", "moeq_expert_ffn", "moeq_route_groups",
         "moeq_add_rmsnorm", "moeq_linear", "moeq_layer_forward_routed")


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


@pytest.fixture
def made(monkeypatch):
    """(allocations as (bytes, stream), streams that they were recorded on)"""
    active, allocated, recorded = [Stream(CURRENT)], [], {}
    empty = torch.empty

    @contextlib.contextmanager
    def use(s):
        active.append(s)
        yield
        active.pop()

    def counted(*a, **k):
        t = empty(*a, **dict(k, device="cpu"))
        allocated.append((t, active[-1].cuda_stream))
        return t

    def record(t, s):
        recorded.setdefault(t.data_ptr(), set()).add(s.cuda_stream)
    monkeypatch.setattr(torch, "empty", counted)
    monkeypatch.setattr(torch, "empty_like", lambda t, **k: counted(t.shape, dtype=t.dtype))
    monkeypatch.setattr(torch.Tensor, "record_stream", record)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: active[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: Stream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", use)
    for name in CALLS:
        monkeypatch.setattr(moeq, name, lambda *a, **k: None)
    monkeypatch.setattr(moeq, "moeq_workspace_bytes", lambda *a: 640)
    monkeypatch.setattr(moeq, "moeq_linear_workspace_bytes", lambda *a: 704)
    monkeypatch.setattr(moeq, "moeq_routed_workspace_bytes", lambda *a: 768)
    return allocated, recorded


class Layer:
    cfg, desc = CONFIGS["tiny"], None


def forms():
    x = torch.zeros(4, 64)
    r = moeq.routing(64, 2)
    t = moeq.QTensor()
    t.out_dim, t.in_dim = 32, 64
    gamma = torch.zeros(64, dtype=torch.bfloat16)
    return [
        lambda s: layer.linear(t, x, stream=s),
        lambda s: layer.route_groups(r, x, stream=s),
        lambda s: layer.add_rmsnorm(x, gamma, 1e-6, x, q_dtype=torch.int8, stream=s),
        lambda s: layer.layer_forward_routed(Layer, r, x, stream=s),
        lambda s: layer.layer_forward(Layer, x, stream=s),
        lambda s: layer.layer_forward_norm(Layer, x, gamma, 1e-6, stream=s),
        lambda s: layer.expert_ffn(Layer, x, x, x, stream=s),
    ]


@pytest.mark.parametrize("form", range(7))
@pytest.mark.parametrize("stream,want", [(None, CURRENT), (CURRENT, CURRENT), (SIDE, SIDE),
                                         (Stream(SIDE), SIDE), (0, 0), (1, 0)])
def test_buffers_belong_to_the_calls_stream(made, form, stream, want):
    allocated, recorded = made
    out = forms()[form](stream)
    assert allocated and all(s == want for _, s in allocated)
    kept = [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]
    for t in kept:
        assert recorded.get(t.data_ptr(), set()) == (set() if want == CURRENT else {CURRENT})
    given = {t.data_ptr() for t in kept}
    assert all(t.data_ptr() in given or t.data_ptr() not in recorded for t, _ in allocated)
