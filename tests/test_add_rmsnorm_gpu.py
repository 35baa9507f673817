"""moeq_add_rmsnorm against the 64-bit reference.

The residual stream and the codes are equal to the reference's.  Scales: the
sum of squares has at most 32 + 5 + 10 additions in a row in fp32 (47 * 2^-24,
halved by the root); 1 / H and the sum with eps (halved too), the reciprocal
root's 2 ulp and three more roundings are 8 * 2^-24: 1.9e-6 relative, under the
2.5e-6 asked for.  y: that, three roundings of the product and one half step of
bf16 (2^-8 relative at most).
"""
import pytest

import ops_reference as ref
from quantized_mixture_experts_affine_b200 import moeq
from quantized_mixture_experts_affine_b200.layer import add_rmsnorm

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
EPS = 1e-6
SCALE = 2.5e-6
Y = 2.0 ** -8 + 3e-6
T = {"f32": torch.float32, "bf16": torch.bfloat16, "int8": torch.int8,
     "e4m3": torch.float8_e4m3fn, None: None}


def check(x, gamma, residual=None, q=None, group=0, want_y=True, got=None):
    r, y, c, s = got or add_rmsnorm(x, gamma, EPS, residual, want_y, T[q], group)
    torch.cuda.synchronize()
    want = ref.add_rmsnorm(x, gamma, EPS, residual, q, group)
    if residual is not None:
        assert torch.equal(r, want["r"])
    if want_y:
        assert bool(((y.double() - want["y"]).abs() <= Y * want["y"].abs() + 1e-38).all())
    if q:
        assert torch.equal(c.float().double(), want["codes"])
        assert bool(((s.double() - want["scales"]).abs() <= SCALE * want["scales"]).all())
    return r, y, c, s


def draw(M, H, xt, rt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, H, device="cuda", generator=g)
    x[:, ::max(1, H // 5)] *= 9
    gamma = (1 + 0.25 * torch.randn(H, device="cuda", generator=g)).to(torch.bfloat16)
    res = None if rt is None else (2 * torch.randn(M, H, device="cuda", generator=g)).to(T[rt])
    return x.to(T[xt]), gamma, res


@pytest.mark.parametrize("q,group", [(None, 0), ("int8", 0), ("int8", 128), ("e4m3", 0),
                                     ("e4m3", 128)])
@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"),
                                   ("f32", "bf16"), ("bf16", None), ("f32", None)])
@pytest.mark.parametrize("M,H", [(1, 4096), (3, 1), (7, 127), (5, 1000), (2, 2049), (64, 768)])
def test_add_rmsnorm(M, H, xt, rt, q, group):
    x, gamma, res = draw(M, H, xt, rt, M * 10000 + H)
    check(x, gamma, res, q, group)


@pytest.mark.parametrize("H", [8192, 16384, 16392, 32768])
def test_long_rows(H):
    x, gamma, res = draw(3, H, "bf16", "f32", H)
    check(x, gamma, res, "int8", 0)
    check(x, gamma, res, "e4m3", 128, want_y=False)


def test_many_rows():
    x, gamma, res = draw(4099, 512, "f32", "f32", 1)
    check(x, gamma, res, "int8", 128)
    check(x, gamma, res, "e4m3", 0)


def test_exact_ties_of_the_rounding():
    """r gamma = (k + 1/2) a / 127 exactly, and e4m3 midpoints: to even."""
    x = torch.zeros(2, 256, device="cuda")
    x[0, :127] = torch.arange(127, device="cuda") + 0.5
    x[0, 127] = 127.0
    x[1, 0] = 448.0
    x[1, 1:129] = torch.arange(128, device="cuda") + 0.5   # midpoints of steps 1, and finer
    x[1, 129:200] = (torch.arange(71, device="cuda") + 0.5) * 2.0 ** -9  # subnormal midpoints
    x = torch.cat([x, -x])
    gamma = torch.ones(256, device="cuda", dtype=torch.bfloat16)
    check(x, gamma, None, "int8", 0)
    check(x, gamma, None, "e4m3", 0)


def test_values_next_to_a_border():
    """fp32 rows whose ratios lie one part in 10^8 beside a border."""
    g = torch.Generator(device="cuda").manual_seed(4)
    k = torch.randint(0, 127, (64, 1024), device="cuda", generator=g) + 0.5
    a = 1 + torch.rand(64, 1, device="cuda", generator=g, dtype=torch.float64)
    x = (k * a / 127).float()
    x = torch.where(torch.rand(64, 1024, device="cuda", generator=g) < 0.5, x,
                    torch.nextafter(x, torch.zeros_like(x)))
    x[:, 0] = a[:, 0].float()
    gamma = torch.ones(1024, device="cuda", dtype=torch.bfloat16)
    check(x, gamma, None, "int8", 0)
    check(x * 448 / 127, gamma, None, "e4m3", 0)


def test_zero_tiny_and_non_finite_rows():
    x, gamma, _ = draw(7, 384, "f32", None, 2)
    x[0] = 0
    x[1, 128:256] = 0
    x[2] *= 1e-30
    x[3] *= 1e-36
    check(x[:4], gamma, None, "int8", 128)
    check(x[:4], gamma, None, "e4m3", 0)
    x[4, 5] = float("inf")
    x[5, 5] = float("nan")
    x[6, 200] = float("-inf")
    for q in ("int8", "e4m3"):
        _, _, c, s = add_rmsnorm(x, gamma, EPS, None, True, T[q], 128)
        c = c.float()
        assert torch.isnan(s[4, 0]) and torch.isnan(s[6, 1]) and torch.isnan(s[5]).all()
        assert (c[4, :128] == 0).all() and (c[5, :128] == 0).all() and (c[6, 128:256] == 0).all()
        assert (s[4, 1:] == 0).all()      # n is 0 beside an infinity
    check(x[:4], gamma, None, "int8", 128)


def test_strides_in_place_and_untouched_memory():
    x, gamma, res = draw(9, 200, "bf16", "f32", 6)
    want = ref.add_rmsnorm(x, gamma, EPS, res, "e4m3", 128)
    wide = torch.zeros(9, 211, dtype=torch.bfloat16, device="cuda")
    wide[:, 5:205] = x
    rw = torch.zeros(9, 203, device="cuda")
    rw[:, 1:201] = res
    y = torch.full((11, 207), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.full((11, 209), 3, dtype=torch.int8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.full((11, 2), 9.0, device="cuda")
    moeq.moeq_add_rmsnorm(wide[:, 5:205], gamma, EPS, rw[:, 1:201], rw[:, 1:201], y[:9, 2:202],
                          q[:9, 1:201], s[:9], 128)
    torch.cuda.synchronize()
    check(x, gamma, res, "e4m3", 128,
          got=(rw[:, 1:201], y[:9, 2:202], q[:9, 1:201], s[:9]))
    assert torch.equal(rw[:, 1:201], want["r"])
    assert (rw[:, 0] == 0).all() and (rw[:, 201:] == 0).all()
    assert (y[9:] == 7).all() and (y[:, :2] == 7).all() and (y[:, 202:] == 7).all()
    b = q.view(torch.int8)
    assert (b[9:] == 3).all() and (b[:, 0] == 3).all() and (b[:, 201:] == 3).all()
    assert (s[9:] == 9).all()
    # no rows
    add_rmsnorm(x[:0], gamma, EPS, res[:0], True, torch.int8, 0)


def test_rows_do_not_depend_on_the_batch():
    x, gamma, res = draw(300, 2048, "bf16", "bf16", 7)
    r, y, c, s = check(x, gamma, res, "e4m3", 128)
    for m in (0, 150, 299):
        r1, y1, c1, s1 = add_rmsnorm(x[m:m + 1], gamma, EPS, res[m:m + 1], True, T["e4m3"], 128)
        assert torch.equal(r1[0], r[m]) and torch.equal(y1[0], y[m]) and torch.equal(s1[0], s[m])
        assert torch.equal(c1.view(torch.int8)[0], c.view(torch.int8)[m])
