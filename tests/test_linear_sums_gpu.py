"""moeq_linear with an fp32 y: what the tensor cores cut off their sums.

Relative 2-norm over the whole output.  A chain of n products of 16 columns comes
out n 2^-27 too small at most where all its products have the accumulator's size:
32 of them between two roundings to nearest (2.4e-7), as the rests of weights and
tokens are added first.  Operands of 22 bits: 2^-23 each (2.4e-7 together).  Sums
of parts, scaling and the epilogue: three roundings of 2^-24 (1.8e-7) and the
parts' own, at most eight, which differ from value to value (half a step each,
2^-25 sqrt(8) = 0.8e-7).  7.4e-7 in all; with the rests last it is 96 products,
7.2e-7 for the chain alone.
"""
import pytest

import ops_reference as ref
from quantized_mixture_experts_affine_b200 import moeq
from quantized_mixture_experts_affine_b200.layer import linear
from test_linear_gpu import T, gen, qt

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("xt,group", [("int8", 128), ("e4m3", 128), ("bf16", 0), ("int8", 0)])
@pytest.mark.parametrize("M,n,o", [(202, 1920, 640), (3000, 1920, 640), (300, 4096, 333),
                                   (1500, 512, 1024)])
@pytest.mark.parametrize("bits,mx", [(4, False), (8, False), (4, True)])
def test_sums_of_rests(M, n, o, bits, mx, xt, group):
    g = gen(M + n)
    G = 32 if mx else 64
    w = ref.matrix(o, n, bits, G, g, mx)
    x = torch.randn(M, n, device="cuda", generator=g)
    if xt == "bf16":
        x, xs = x.to(torch.bfloat16), None
    else:
        top = 127.0 if xt == "int8" else 448.0
        cols = x.view(M, -1, group or n)
        xs = (cols.abs().amax(-1) / top).contiguous()
        v = (cols / xs[..., None]).view(M, n).clamp(-top, top)
        x = (torch.round(v) if xt == "int8" else v).to(T[xt])
    y = linear(qt(w, o, n, bits, G, mx), x, torch.float32, x_scales=xs, x_group=group)
    torch.cuda.synchronize()
    assert moeq.moeq_device_status() == 0
    want = ref.dequant_x(x, xs, group) @ w["dense"].t()
    assert float((y.double() - want).norm() / want.norm()) <= 7.4e-7
