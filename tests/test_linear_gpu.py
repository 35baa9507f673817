"""moeq_linear against the 64-bit reference.

Bounds, per element, with S = sum_i |x_i| (|s q_i| + |b|), the size of what is
added up: fp32 sums in chains of at most `chain` additions are off by at most
chain * 2^-23 S (tensor-core additions may truncate, hence 2^-23); calls that
round the weights (bf16 y, many tokens) by 2^-11 S more; an x of 8 bits with
128-column scales there by another 2^-11 S (x * scale in fp16).  The activations'
slopes are at most 1.13; mul scales the error; y adds half a step of its type.
"""
import pytest

import ops_reference as ref
from quantized_mixture_experts_affine_b200 import moeq
from quantized_mixture_experts_affine_b200.layer import linear

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
T = {"f32": torch.float32, "bf16": torch.bfloat16, "int8": torch.int8,
     "e4m3": torch.float8_e4m3fn}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def qt(w, out_dim, in_dim, bits, G, mx=False):
    return moeq.qtensor(w["w"], w["s"], w["b"], out_dim, in_dim, bits, G,
                        fmt=moeq.FMT_MXFP4 if mx else moeq.FMT_AFFINE)


def tokens(M, n, xt, group, g):
    x = torch.randn(M, n, device="cuda", generator=g)
    x[:, ::max(1, n // 3)] *= 10
    if xt == "bf16":
        return x.to(torch.bfloat16), None
    s = 0.01 * (1 + torch.rand(M, -(-n // 128) if group else 1, device="cuda", generator=g))
    if xt == "int8":
        return torch.randint(-127, 128, (M, n), device="cuda", generator=g).to(torch.int8), s
    return (30 * x).clamp(-448, 448).to(torch.float8_e4m3fn), s


def bound(x, xs, group, w, pre, name, mul, out, y, rounded):
    d = ref.dequant_x(x, xs, group).abs()
    S = d @ w["spread"].t()
    chain = x.shape[1] / 16 + 64
    rel = chain * 2.0 ** -23 + (2.0 ** -11 if rounded else 0) + \
        (2.0 ** -11 if rounded and group else 0)
    e = 1.13 * S * rel + 1e-6 * pre.abs()
    if mul is not None:
        e = e * mul.double().abs()
    return e + (HALF[out] + 2.0 ** -22) * y.abs() + 1e-30


def check(M, n, o, bits, G, xt="bf16", group=0, mx=False, act="none", bias=False, mul=False,
          res=False, out="f32", seed=0):
    g = gen(seed + M * 7 + n * 3 + o + bits)
    w = ref.matrix(o, n, bits, G, g, mx)
    x, xs = tokens(M, n, xt, group, g)
    b = torch.randn(o, device="cuda", generator=g).to(torch.bfloat16) if bias else None
    mm = torch.randn(M, o, device="cuda", generator=g).to(T[out]) if mul else None
    rr = torch.randn(M, o, device="cuda", generator=g).to(T[out]) if res else None
    y = linear(qt(w, o, n, bits, G, mx), x, T[out], x_scales=xs, x_group=group, bias=b,
               act=getattr(moeq, "ACT_" + act.upper()), mul=mm, residual=rr)
    torch.cuda.synchronize()
    assert moeq.moeq_device_status() == 0
    pre = ref.dequant_x(x, xs, group) @ w["dense"].t()
    if bias:
        pre = pre + b.double()
    want = ref.act(pre, act)
    if mul:
        want = want * mm.double()
    if res:
        want = want + rr.double()
    rounded = out == "bf16"
    e = (y.double() - want).abs()
    lim = bound(x, xs, group, w, pre, act, mm, out, want, rounded)
    assert bool((e <= lim).all()), (float((e / lim).max()), int((e > lim).sum()))
    return y


# Sizes that take each of the three ways: products of the codes, weights
# unpacked inside the product, weights laid out before it.
WAYS = {"codes": (9, 130), "inside": (100, 700), "before": (2600, 1930)}
FORMATS = [(2, 64, False), (2, 32, False), (2, 128, False), (3, 64, False), (3, 32, False),
           (4, 32, False), (4, 64, False), (4, 128, False), (5, 32, False), (5, 128, False),
           (6, 32, False), (6, 64, False), (8, 32, False), (8, 64, False), (8, 128, False),
           (4, 32, True)]
ROWS = [1, 8, 9, 16, 17, 33, 64, 65, 130, 300]


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("bits,G,mx", FORMATS)
def test_formats(bits, G, mx, M):
    check(M, 384, 130, bits, G, mx=mx, out="f32")
    check(M, 1024, 67, bits, G, mx=mx, out="bf16", bias=True)


@pytest.mark.parametrize("way", list(WAYS))
@pytest.mark.parametrize("bits,G,mx", FORMATS)
def test_formats_every_way(bits, G, mx, way):
    M, o = WAYS[way]
    before = moeq.moeq_launch_count()
    check(M, 384, o, bits, G, mx=mx, out="f32")
    check(M, 640, o, bits, G, mx=mx, out="bf16", bias=True)
    # one kernel, two (tokens laid out first), three (weights too)
    assert moeq.moeq_launch_count() - before == 2 * (1 + list(WAYS).index(way))


@pytest.mark.parametrize("way", list(WAYS))
@pytest.mark.parametrize("n,bits,G", [(32, 4, 32), (32, 8, 32), (64, 2, 64), (64, 6, 32), (96, 4, 32),
                                      (160, 8, 32), (288, 4, 32), (320, 8, 64), (448, 2, 32),
                                      (1056, 4, 32), (2080, 8, 32), (128, 5, 32), (640, 3, 128)])
def test_odd_columns_every_way(n, bits, G, way):
    M, o = WAYS[way]
    check(M, n, o, bits, G, out="f32", res=True)
    check(M, n, o, bits, G, out="bf16")
    if G == 32 and bits == 4:
        check(M, n, o, 4, 32, mx=True, out="bf16")


@pytest.mark.parametrize("way", list(WAYS))
@pytest.mark.parametrize("xt,group", [("int8", 0), ("int8", 128), ("e4m3", 0), ("e4m3", 128)])
def test_eight_bit_tokens_every_way(xt, group, way):
    M, o = WAYS[way]
    for n, bits, G in ((640, 4, 64), (416, 8, 32)):
        check(M, n, o, bits, G, xt, group, out="f32", res=True)
        check(M, n, o, bits, G, xt, group, out="bf16", act="silu", mul=True)


@pytest.mark.parametrize("way", list(WAYS))
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
def test_epilogue_every_way(act, way):
    M, o = WAYS[way]
    for out in ("f32", "bf16"):
        check(M, 256, o, 4, 64, act=act, bias=True, mul=True, res=True, out=out)


@pytest.mark.parametrize("M,o,n", [(40, 2000, 8192), (20, 700, 12288), (20, 700, 12544), (300, 300, 16384),
                                   (2600, 1930, 4096), (17, 8200, 1024), (513, 260, 1024)])
def test_long_sums_in_fp32(M, o, n):
    """fp32 outputs over thousands of columns stay near the 64-bit sum: the
    tensor cores cut off at most 96 additions in a row at about 2^-27 each
    (7.2e-7), then parts are added with rounding (at most 32 of them, 2^-24
    each in the worst case, far less in norm): under 1.5e-6 in norm."""
    g = gen(n + M)
    w = ref.matrix(o, n, 4, 64, g)
    x, _ = tokens(M, n, "bf16", 0, g)
    y = linear(qt(w, o, n, 4, 64), x, T["f32"])
    want = x.double() @ w["dense"].t()
    assert float((y.double() - want).norm() / want.norm()) < 1.5e-6


def test_a_workspace_for_many_tokens_serves_fewer():
    g = gen(5)
    for n, o in ((1024, 1024), (4096, 2048), (288, 5000)):
        t = qt(ref.matrix(o, n, 4, 64 if n > 288 else 32, g), o, n, 4, 64 if n > 288 else 32)
        for xt in (torch.bfloat16, torch.int8):
            for out in (torch.bfloat16, torch.float32):
                need = [moeq.moeq_linear_workspace_bytes(t, M, xt, out) for M in range(1, 1200, 7)]
                assert need == sorted(need) and need[0] == 0


@pytest.mark.parametrize("M", [1, 5, 24, 100, 257])
@pytest.mark.parametrize("xt,group", [("int8", 0), ("int8", 128), ("e4m3", 0), ("e4m3", 128)])
@pytest.mark.parametrize("bits,G,mx", [(4, 64, False), (8, 128, False), (2, 32, False),
                                       (5, 64, False), (4, 32, True)])
def test_eight_bit_tokens(bits, G, mx, xt, group, M):
    check(M, 640, 96, bits, G, xt, group, mx, out="f32", res=True)
    check(M, 640, 200, bits, G, xt, group, mx, out="bf16", act="silu", mul=True)


@pytest.mark.parametrize("M", [1, 20, 300])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_epilogue(out, act, M):
    for bias in (False, True):
        for mul in (False, True):
            for res in (False, True):
                check(M, 256, 72, 4, 64, act=act, bias=bias, mul=mul, res=res, out=out)


@pytest.mark.parametrize("M", [1, 3, 40, 129, 260])
@pytest.mark.parametrize("n,o,bits,G", [(32, 1, 4, 32), (32, 5, 8, 32), (64, 3, 2, 64),
                                        (96, 17, 4, 32), (160, 31, 8, 32), (64, 2, 6, 32),
                                        (128, 1, 5, 128), (448, 513, 8, 64), (8192, 40, 4, 64),
                                        (8192, 9, 8, 128), (16384, 12, 2, 64)])
def test_odd_sizes(n, o, bits, G, M):
    check(M, n, o, bits, G, out="f32")
    check(M, n, o, bits, G, out="bf16", bias=True, res=True)


@pytest.mark.parametrize("M,n,o,bits,G,out", [
    (2048, 2048, 1024, 4, 64, "bf16"), (1111, 768, 4001, 8, 64, "bf16"),
    (700, 4096, 512, 8, 64, "f32"), (512, 4096, 4096, 4, 64, "bf16"), (1, 4096, 4096, 4, 64, "f32"),
    (64, 4096, 512, 8, 64, "f32"), (3000, 512, 256, 2, 64, "f32")])
def test_larger(M, n, o, bits, G, out):
    check(M, n, o, bits, G, out=out, act="silu", res=True)


@pytest.mark.parametrize("M,o", [(3, 45), (150, 45), (150, 701), (2600, 1931)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_strides_in_place_and_untouched_memory(out, M, o):
    """Rows inside wider ones, y in the residual's memory, rows behind the last
    left as they were; the same values as the plain call."""
    n = 256
    g = gen(M)
    w = ref.matrix(o, n, 4, 64, g)
    t = qt(w, o, n, 4, 64)
    x, _ = tokens(M, n, "bf16", 0, g)
    res = torch.randn(M, o, device="cuda", generator=g).to(T[out])
    mul = torch.randn(M, o, device="cuda", generator=g).to(T[out])
    want = linear(t, x, T[out], residual=res, mul=mul)
    xw = torch.full((M, n + 24), float("nan"), device="cuda", dtype=torch.bfloat16)
    xw[:, 8:8 + n] = x
    buf = torch.full((M + 2, o + 6), 5.0, device="cuda").to(T[out])
    buf[:M, 3:3 + o] = res
    mw = torch.full((M, o + 1), 5.0, device="cuda").to(T[out])
    mw[:, 1:] = mul
    view = buf[:M, 3:3 + o]
    linear(t, xw[:, 8:8 + n], y=view, residual=view, mul=mw[:, 1:])
    torch.cuda.synchronize()
    assert torch.equal(view, want)
    assert (buf[M:] == 5).all() and (buf[:, :3] == 5).all() and (buf[:, 3 + o:] == 5).all()
    linear(t, x[:0], T[out])


@pytest.mark.parametrize("M,o", [(2, 64), (9, 64), (200, 704), (2600, 1930)])
def test_expert_of_a_bank(M, o):
    n, E = 256, 3
    g = gen(3)
    ws = [ref.matrix(o, n, 4, 64, g) for _ in range(E)]
    bank = [torch.stack([w[k] for w in ws]).contiguous() for k in ("w", "s", "b")]
    t = moeq.qtensor(*bank, o, n, 4, 64, E)
    x, _ = tokens(M, n, "bf16", 0, g)
    for e in range(E):
        one = linear(qt(ws[e], o, n, 4, 64), x)
        assert torch.equal(linear(t, x, expert=e), one)


@pytest.mark.parametrize("M,o", [(4, 80), (40, 80), (300, 700), (2600, 1930)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_a_bad_token_stays_alone(out, M, o):
    """A row of NaN and infinities changes no other row; huge and tiny rows
    keep their own precision."""
    n = 512
    g = gen(9)
    w = ref.matrix(o, n, 4, 64, g)
    t = qt(w, o, n, 4, 64)
    x, _ = tokens(M, n, "bf16", 0, g)
    want = linear(t, x, T[out])
    y = x.clone()
    y[1] = float("inf")
    y[2, 7] = float("nan")
    got = linear(t, y, T[out])
    keep = torch.arange(M, device="cuda")
    keep = keep[(keep != 1) & (keep != 2)]
    assert torch.equal(got[keep], want[keep])
    assert not torch.isfinite(got[2]).any()
    z = x.clone()
    z[0] *= 2.0 ** 90
    z[3] *= 2.0 ** -90
    got = linear(t, z, T[out])
    assert torch.equal(got[0].float(), want[0].float() * 2.0 ** 90)
    assert torch.equal(got[3].float(), want[3].float() * 2.0 ** -90)


@pytest.mark.parametrize("way", list(WAYS))
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_huge_weights_and_tiny_tokens(out, way):
    """Powers of two that cancel change no bit."""
    M, o = WAYS[way]
    n = 512
    g = gen(31)
    w = ref.matrix(o, n, 4, 64, g)
    x, _ = tokens(M, n, "bf16", 0, g)
    x = torch.where(x.abs() < 2.0 ** -8, torch.full_like(x, 2.0 ** -8), x)
    y = linear(qt(w, o, n, 4, 64), x, T[out])
    h = dict(w, s=w["s"] * 2.0 ** 118, b=w["b"] * 2.0 ** 118)
    got = linear(qt(h, o, n, 4, 64), x * 2.0 ** -114, T[out])
    assert torch.equal(got.float(), y.float() * 16)


@pytest.mark.parametrize("M,o", [(1, 320), (31, 320), (400, 320), (60, 2000), (2600, 1930)])
def test_two_calls_at_once_and_in_a_graph(M, o):
    """Two streams with a workspace each, and a captured call replayed on new
    tokens, give the plain call's values."""
    n = 1024
    g = gen(12)
    w = ref.matrix(o, n, 4, 64, g)
    t = qt(w, o, n, 4, 64)
    a, _ = tokens(M, n, "bf16", 0, g)
    b, _ = tokens(M, n, "bf16", 0, g)
    ya, yb = linear(t, a), linear(t, b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(8):
        outs.append((linear(t, a, stream=s1), linear(t, b, stream=s2)))
    torch.cuda.synchronize()
    for p, q in outs:
        assert torch.equal(p, ya) and torch.equal(q, yb)
    x, y = a.clone(), torch.empty_like(ya)
    need = moeq.moeq_linear_workspace_bytes(t, M, x.dtype, y.dtype)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moeq.moeq_linear(t, 0, x, y, ws=ws)
    for src, want in ((a, ya), (b, yb), (a, ya)):
        x.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
