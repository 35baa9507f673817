"""Refusals of the routing, norm and linear entry points: every call here
fails its argument checks before anything is launched (no GPU needed)."""
import ctypes as C

import pytest

from quantized_mixture_experts_affine_b200 import moeq
from test_abi import A, layer, qt


def rc_route(r, logits=A, lt=moeq.F32, ld=None, bias=None, M=4, idx=A, w=A):
    ld = r.n_experts if ld is None else ld
    return moeq.lib().moeq_route_groups(C.byref(r), logits, lt, ld, bias, M, idx, w, None)


def test_route_groups_refusals():
    ok = moeq.routing(64, 8, moeq.SCORE_SIGMOID, 8, 4, 2)
    assert rc_route(ok, M=0) == moeq.OK
    assert rc_route(ok, M=-1) == moeq.ERR_INVALID_ARG
    assert rc_route(ok, logits=None) == moeq.ERR_INVALID_ARG
    assert rc_route(ok, idx=None) == moeq.ERR_INVALID_ARG
    assert rc_route(ok, ld=63) == moeq.ERR_INVALID_ARG
    assert rc_route(ok, lt=moeq.I8) == moeq.ERR_UNSUPPORTED
    assert rc_route(ok, logits=A + 2) == moeq.ERR_ALIGNMENT
    assert rc_route(ok, bias=A + 1) == moeq.ERR_ALIGNMENT
    assert moeq.lib().moeq_route_groups(None, A, 0, 8, None, 1, A, A, None) == \
        moeq.ERR_INVALID_ARG
    for bad in (dict(n_groups=7), dict(topk_groups=9), dict(topk_groups=0), dict(group_top=3),
                dict(top_k=33), dict(top_k=0), dict(n_experts=0), dict(score=2),
                dict(router_scale=0.0), dict(router_scale=float("nan")),
                dict(router_scale=-1.0), dict(routed_scale=float("inf")), dict(renorm=2)):
        r = moeq.routing(64, 8, moeq.SCORE_SIGMOID, 8, 4, 2)
        for k, v in bad.items():
            setattr(r, k, v)
        want = moeq.ERR_UNSUPPORTED if bad == dict(top_k=33) else moeq.ERR_INVALID_ARG
        assert rc_route(r) == want, bad
    assert rc_route(moeq.routing(64, 9, 0, 8, 1, 1)) == moeq.ERR_INVALID_ARG  # 8 in one group
    assert rc_route(moeq.routing(5000, 8)) == moeq.ERR_UNSUPPORTED
    assert rc_route(moeq.routing(64, 1, 0, 64, 1, 1)) == moeq.ERR_UNSUPPORTED  # 64 groups


def rc_norm(M=2, H=64, **kw):
    a = moeq.NormArgs(A, moeq.BF16, 64)
    a.gamma, a.eps, a.y, a.y_stride = A, 1e-6, A, 64
    for k, v in kw.items():
        setattr(a, k, v)
    return moeq.lib().moeq_add_rmsnorm(C.byref(a), M, H, None)


def test_add_rmsnorm_refusals():
    assert rc_norm(M=0) == moeq.OK
    assert rc_norm(M=-1) == moeq.ERR_INVALID_ARG
    assert rc_norm(H=0) == moeq.ERR_INVALID_ARG
    assert rc_norm(H=32769, x_stride=40000) == moeq.ERR_UNSUPPORTED
    assert rc_norm(H=65) == moeq.ERR_INVALID_ARG            # strides shorter than the row
    assert rc_norm(y=None) == moeq.ERR_INVALID_ARG          # no output
    assert rc_norm(gamma=None) == moeq.ERR_INVALID_ARG
    assert rc_norm(x=None) == moeq.ERR_INVALID_ARG
    assert rc_norm(x=A + 1) == moeq.ERR_ALIGNMENT
    assert rc_norm(gamma=A + 1) == moeq.ERR_ALIGNMENT
    assert rc_norm(x_type=moeq.I8) == moeq.ERR_UNSUPPORTED
    assert rc_norm(x_type=moeq.F32, x=A + 2) == moeq.ERR_ALIGNMENT
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        assert rc_norm(eps=eps) == moeq.ERR_INVALID_ARG
    assert rc_norm(r_out=A, r_out_stride=64) == moeq.ERR_INVALID_ARG   # without a residual
    assert rc_norm(residual=A, r_type=moeq.E4M3, r_stride=64) == moeq.ERR_UNSUPPORTED
    assert rc_norm(residual=A, r_stride=63) == moeq.ERR_INVALID_ARG
    assert rc_norm(residual=A, r_stride=64, r_out=A, r_out_stride=1) == moeq.ERR_INVALID_ARG
    q = dict(q=A, q_type=moeq.I8, q_stride=64, q_scales=A)
    assert rc_norm(**{**q, "q_scales": None}) == moeq.ERR_INVALID_ARG
    assert rc_norm(**{**q, "q_type": moeq.BF16}) == moeq.ERR_UNSUPPORTED
    assert rc_norm(**{**q, "q_group": 64}) == moeq.ERR_UNSUPPORTED
    assert rc_norm(**{**q, "q_stride": 63}) == moeq.ERR_INVALID_ARG
    assert rc_norm(**{**q, "q_scales": A + 2}) == moeq.ERR_ALIGNMENT
    assert moeq.lib().moeq_add_rmsnorm(None, 1, 1, None) == moeq.ERR_INVALID_ARG


def rc_linear(t=None, M=2, expert=0, ws=None, ws_bytes=0, **kw):
    t = t or qt()
    a = moeq.LinearArgs(A, moeq.BF16, t.in_dim)
    a.y, a.out_type, a.y_stride = A, moeq.F32, t.out_dim
    for k, v in kw.items():
        setattr(a, k, v)
    return moeq.lib().moeq_linear(C.byref(t), expert, C.byref(a), M, ws, ws_bytes, None)


def test_linear_refusals():
    assert rc_linear(M=0) == moeq.OK
    assert rc_linear(M=-1) == moeq.ERR_INVALID_ARG
    assert rc_linear(qt(bits=7)) == moeq.ERR_UNSUPPORTED
    assert rc_linear(qt(G=48)) == moeq.ERR_UNSUPPORTED
    assert rc_linear(qt(w=A + 4)) == moeq.ERR_ALIGNMENT
    assert rc_linear(qt(inn=96, G=64)) == moeq.ERR_ALIGNMENT
    assert rc_linear(expert=-1) == moeq.ERR_INVALID_ARG
    assert rc_linear(expert=1) == moeq.ERR_INVALID_ARG       # a single matrix
    assert rc_linear(x=None) == moeq.ERR_INVALID_ARG
    assert rc_linear(y=None) == moeq.ERR_INVALID_ARG
    assert rc_linear(x=A + 8) == moeq.ERR_ALIGNMENT
    assert rc_linear(x_stride=255) == moeq.ERR_INVALID_ARG
    assert rc_linear(x_stride=257) == moeq.ERR_ALIGNMENT     # rows off 16 bytes
    assert rc_linear(x_type=moeq.F32) == moeq.ERR_UNSUPPORTED
    assert rc_linear(x_type=moeq.I8) == moeq.ERR_INVALID_ARG  # no scales
    assert rc_linear(x_type=moeq.I8, x_scales=A, x_group=64) == moeq.ERR_UNSUPPORTED
    assert rc_linear(x_type=moeq.I8, x_scales=A, x_stride=264) == moeq.ERR_ALIGNMENT
    assert rc_linear(x_type=moeq.E4M3, x_scales=A + 2) == moeq.ERR_ALIGNMENT
    assert rc_linear(out_type=moeq.I8) == moeq.ERR_UNSUPPORTED
    assert rc_linear(y_stride=127) == moeq.ERR_INVALID_ARG
    assert rc_linear(y_stride=2 ** 28 + 1) == moeq.ERR_UNSUPPORTED
    assert rc_linear(mul=A, mul_stride=2 ** 40) == moeq.ERR_UNSUPPORTED
    assert rc_linear(residual=A, residual_stride=2 ** 28 + 8) == moeq.ERR_UNSUPPORTED
    assert rc_linear(y=A + 2) == moeq.ERR_ALIGNMENT
    assert rc_linear(bias=A + 1) == moeq.ERR_ALIGNMENT
    assert rc_linear(mul=A, mul_stride=1) == moeq.ERR_INVALID_ARG
    assert rc_linear(residual=A, residual_stride=1) == moeq.ERR_INVALID_ARG
    assert rc_linear(residual=A + 2, residual_stride=128) == moeq.ERR_ALIGNMENT
    assert rc_linear(act=6) == moeq.ERR_INVALID_ARG
    assert rc_linear(act=-1) == moeq.ERR_INVALID_ARG
    assert moeq.lib().moeq_linear(None, 0, None, 1, None, 0, None) == moeq.ERR_INVALID_ARG


def test_routed_layer_refusals():
    L = layer()
    r = moeq.routing(8, 2)

    def call(r=r, M=1, x=A, ws=A, ws_bytes=None, bias=None, mode=moeq.MODE_DECODE, L=L):
        if ws_bytes is None:
            ws_bytes = moeq.moeq_routed_workspace_bytes(L, max(M, 1), mode) - 1
        return moeq.lib().moeq_layer_forward_routed(C.byref(L), C.byref(r), bias, x, M, A, None,
                                                    None, None, ws, ws_bytes, mode, None)
    assert moeq.moeq_routed_workspace_bytes(L, 1, moeq.MODE_DECODE) > \
        moeq.moeq_workspace_bytes(L, 1, moeq.MODE_DECODE)
    assert moeq.moeq_routed_workspace_bytes(L, 65, moeq.MODE_DECODE) == 0
    assert call() == moeq.ERR_WORKSPACE
    assert call(ws=None) == moeq.ERR_WORKSPACE
    assert call(ws=A + 16, ws_bytes=1 << 30) == moeq.ERR_ALIGNMENT
    assert call(x=None, ws_bytes=1 << 30) == moeq.ERR_INVALID_ARG
    assert call(bias=A + 2, ws_bytes=1 << 30) == moeq.ERR_ALIGNMENT
    assert call(moeq.routing(16, 2), ws_bytes=1 << 30) == moeq.ERR_INVALID_ARG
    assert call(moeq.routing(8, 3), ws_bytes=1 << 30) == moeq.ERR_INVALID_ARG
    assert call(M=0) == moeq.OK
    assert call(M=65, ws_bytes=1 << 30) == moeq.ERR_UNSUPPORTED
    # a layer whose rows the decode path refuses: before the router's launch
    big = layer(H=16384, bits=4)
    assert call(L=big, ws_bytes=1 << 40) == moeq.ERR_UNSUPPORTED


def test_binding_checks_shapes_and_devices():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("host tensors only")
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        moeq.moeq_linear(qt(), 0, x, torch.zeros(2, 128))
    with pytest.raises(moeq.MoeqError):
        moeq.dtype_code(torch.float64)
    with pytest.raises(ValueError):
        moeq._rows("x", x.t(), 256, 2)
    with pytest.raises(ValueError):
        moeq._rows("x", x, 2, 256, torch.float32, -1)
    with pytest.raises(ValueError):
        moeq._dense("w", x[:, ::2], (2, 128), torch.bfloat16, -1)
