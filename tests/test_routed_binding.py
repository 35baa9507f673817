"""moeq_layer_forward_routed in moeq.py: types, shapes and devices of tensors
are checked before the library sees an address (no GPU needed: every call here
is refused, or has no rows)."""
import pytest

from quantized_mixture_experts_affine_b200 import moeq
from test_abi import A, layer

torch = pytest.importorskip("torch")
H, E, K, M = 256, 8, 2, 3


@pytest.fixture
def call(monkeypatch):
    if torch.cuda.is_available():
        pytest.skip("host tensors only")
    if hasattr(moeq, "_load_torch"):
        moeq._load_torch()
    monkeypatch.setattr(moeq, "_device", lambda name, t: t.get_device())  # host tensors: -1
    monkeypatch.setattr(moeq, "_stream", lambda s: None)
    L = layer()
    assert (L.hidden, L.n_experts, L.top_k) == (H, E, K)

    def run(m=M, **kw):
        a = dict(x=torch.zeros(M, H, dtype=torch.bfloat16), y=torch.zeros(M, H),
                 bias=torch.zeros(E), residual=torch.zeros(M, H),
                 idx_out=torch.zeros(M, K, dtype=torch.int32), w_out=torch.zeros(M, K),
                 ws=torch.zeros(512, dtype=torch.uint8), ws_bytes=512)
        a.update(kw)
        x, y = a.pop("x"), a.pop("y")
        moeq.moeq_layer_forward_routed(L, moeq.routing(E, K), x, m, y, **a)
    return run


def test_what_fits_reaches_the_library(call):
    with pytest.raises(moeq.MoeqError):  # the workspace is too small
        call()
    with pytest.raises(moeq.MoeqError):  # more rows than M, no optional buffers
        call(m=2, bias=None, residual=None, idx_out=None, w_out=None)
    with pytest.raises(moeq.MoeqError):  # raw addresses
        call(x=A, y=A, bias=A, residual=A, idx_out=A, w_out=A, ws=A)


@pytest.mark.parametrize("bad", [
    dict(bias=torch.zeros(E, dtype=torch.bfloat16)), dict(bias=torch.zeros(E - 1)),
    dict(bias=torch.zeros(2 * E)[::2]), dict(x=torch.zeros(M, H)),
    dict(x=torch.zeros(M - 1, H, dtype=torch.bfloat16)),
    dict(x=torch.zeros(M, 2 * H, dtype=torch.bfloat16)[:, :H]),
    dict(x=torch.zeros(M, H - 64, dtype=torch.bfloat16)),
    dict(y=torch.zeros(M, H, dtype=torch.bfloat16)), dict(y=torch.zeros(M, H + 1)),
    dict(y=torch.zeros(H, M).t()), dict(residual=torch.zeros(M, H, dtype=torch.bfloat16)),
    dict(residual=torch.zeros(M - 1, H)), dict(idx_out=torch.zeros(M, K, dtype=torch.int64)),
    dict(idx_out=torch.zeros(M, K + 1, dtype=torch.int32)), dict(w_out=torch.zeros(M)),
    dict(w_out=torch.zeros(M, K, dtype=torch.float64)),
    dict(ws=torch.zeros(511, dtype=torch.uint8)), dict(ws=torch.zeros(1024, dtype=torch.uint8)[::2]),
    dict(ws_bytes=513)])
def test_what_does_not_fit_is_refused(call, bad):
    with pytest.raises(ValueError):
        call(**bad)


@pytest.mark.parametrize("other", ["y", "bias", "residual", "idx_out", "w_out", "ws"])
def test_one_device_for_all(call, other, monkeypatch):
    """x on device 0, one of the others not."""
    monkeypatch.setattr(moeq, "_device", lambda name, t: 0)
    none = dict(bias=None, residual=None, idx_out=None, w_out=None, ws=A, y=A)
    none.pop(other)
    with pytest.raises(ValueError):
        call(**none)


def test_an_empty_batch_needs_no_buffers(call):
    """Empty tensors have no address: nothing is launched, nothing refused."""
    z = dict(x=torch.zeros(0, H, dtype=torch.bfloat16), y=torch.zeros(0, H),
             residual=torch.zeros(0, H), idx_out=torch.zeros(0, K, dtype=torch.int32),
             w_out=torch.zeros(0, K), ws=torch.zeros(0, dtype=torch.uint8), ws_bytes=0)
    assert z["x"].data_ptr() == 0
    call(m=0, **z)
    with pytest.raises(moeq.MoeqError):
        call(m=-1)
