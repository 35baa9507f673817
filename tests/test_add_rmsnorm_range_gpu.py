"""moeq_add_rmsnorm at the ends of fp32's range, and row by row against a batch.

Tolerances as in test_add_rmsnorm_gpu: scales 2.5e-6 relative (what is added here
are exact products by powers of two), y one half step of bf16 more; values below
fp32's normal range are off by its smallest step.
"""
import pytest

import ops_reference as ref
from quantized_mixture_experts_affine_b200 import moeq
from quantized_mixture_experts_affine_b200.layer import add_rmsnorm
from test_add_rmsnorm_gpu import SCALE, T, Y, draw

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
TINY = 2.0 ** -149


def check(x, gamma, q, group, eps=1e-6, residual=None):
    r, y, c, s = add_rmsnorm(x, gamma, eps, residual, True, T[q], group)
    torch.cuda.synchronize()
    want = ref.add_rmsnorm(x, gamma, float(torch.tensor(eps)), residual, q, group)
    if residual is not None:
        assert torch.equal(r, want["r"])
    assert torch.equal(c.float().double(), want["codes"])
    assert bool(((s.double() - want["scales"]).abs() <= SCALE * want["scales"] + TINY).all())
    assert bool(((y.double() - want["y"]).abs() <= Y * want["y"].abs() + 1e-38).all())


CASES = [(q, group, xt, H) for q in ("int8", "e4m3") for group in (0, 128)
         for xt in ("f32", "bf16") for H in (64, 1001, 4096)]


@pytest.mark.parametrize("q,group,xt,H", CASES)
def test_large_products(q, group, xt, H):
    """|r gamma| next to fp32's largest value, and beyond it."""
    x, gamma, _ = draw(4, H, "f32", None, H)
    x = (x.clamp(-8, 8) * 1e16).to(T[xt])
    check(x, (gamma.float().clamp(0.5, 1.5) * 2.0 ** 70).to(torch.bfloat16), q, group)
    check(x, (gamma.float() * 1e25).to(torch.bfloat16), q, group)


@pytest.mark.parametrize("q,group,xt,H", CASES + [("int8", 0, "f32", 32768),
                                                  ("e4m3", 128, "bf16", 8200)])
def test_small_products(q, group, xt, H):
    """|r gamma| below fp32's normal range: codes and scales all the same."""
    x, gamma, _ = draw(4, H, "f32", None, H + 1)
    for xs, gs in ((1e-20, 1e-19), (1e-24, 1e-20), (1e-30, 1e-18), (1e-36, 1.0)):
        check((x * xs).to(T[xt]), (gamma.float() * gs).to(torch.bfloat16), q, group, eps=1e-30)


def test_zero_rows_and_groups_beside_others():
    x, gamma, _ = draw(40, 2048, "f32", None, 9)
    x[::3] = 0
    x[1, 128:300] = 0
    x[4, :1024] = 0
    for q, group in (("int8", 0), ("e4m3", 128)):
        check(x, gamma, q, group)
        check(x[:, :1001].contiguous(), gamma[:1001].contiguous(), q, group)
        check(x.to(torch.bfloat16), gamma, q, group, residual=torch.zeros_like(x))


@pytest.mark.parametrize("H", [8, 1001, 4096, 8200, 32768])
@pytest.mark.parametrize("q,group", [("int8", 0), ("e4m3", 128)])
@pytest.mark.parametrize("xt,rt", [("f32", None), ("bf16", "f32"), ("bf16", "bf16")])
def test_large_rows(H, q, group, xt, rt):
    """The squares' sum passes fp32's range; the norm does not."""
    x, gamma, res = draw(3, H, "f32", rt, H + 2)
    x = x.clamp(-10, 10)
    for top in (1e17, 1e18, 1e24, 1e29):
        r = None if res is None else (res.float() * (top / 100)).to(T[rt])
        check((x * top).to(T[xt]), gamma, q, group, residual=r)


def test_large_rows_beside_ordinary_ones():
    x, gamma, _ = draw(6, 4096, "f32", None, 5)
    x[1] *= 1e25
    x[3] *= 1e18
    x[4, 100] = 1e22
    check(x, gamma, "int8", 0)
    check(x, gamma, "e4m3", 128)


@pytest.mark.parametrize("H", [8, 1000, 1001, 2048, 2056, 4096, 4091, 6000])
@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("f32", None)])
@pytest.mark.parametrize("q,group", [("int8", 0), ("e4m3", 128)])
def test_rows_are_those_of_a_large_batch(H, xt, rt, q, group):
    """One row and 1300 run other variants of the kernel: the same bits."""
    x, gamma, res = draw(1300, H, xt, rt, H)
    x[700] = x[700].float().clamp(-10, 10) * 1e24  # squares beyond fp32
    many = add_rmsnorm(x, gamma, 1e-6, res, True, T[q], group)
    for m in (0, 1, 700, 1299):
        one = add_rmsnorm(x[m:m + 1].clone(), gamma, 1e-6,
                          None if res is None else res[m:m + 1].clone(), True, T[q], group)
        for a, b in zip(one, many):
            if b is not None:
                assert torch.equal(a[0].view(torch.uint8), b[m].view(torch.uint8))


@pytest.mark.parametrize("H", [256, 1001])
@pytest.mark.parametrize("rt", ["f32", "bf16"])
def test_ends_of_the_range_in_place_strided_and_without_a_new_stream(H, rt):
    """Rows out of range beside ordinary ones: the stream in place, the stream not
    written at all, rows that are parts of wider ones, y alone."""
    x, gamma, res = draw(12, H, "f32", rt, H + 4)
    scale = torch.tensor([1.0, 1e-30, 1e24, 0.0, 1e-20, 1e29], device="cuda").repeat(2)[:, None]
    x, res = x.clamp(-10, 10) * scale, (res.float() * scale).to(T[rt])
    x[7] = float("nan")
    res[7] = 0
    x[8, 3] = float("inf")
    fine = [m for m in range(12) if m not in (7, 8)]
    for q, group in (("int8", 0), ("e4m3", 128)):
        want = ref.add_rmsnorm(x, gamma, 1e-6, res, q, group)
        n = -(-H // group) if group else 1
        wide = torch.zeros(12, H + 3, dtype=T[rt], device="cuda")
        for stream in ("in place", "none"):
            wide[:, 1:H + 1] = res
            r = wide[:, 1:H + 1]
            y = torch.zeros(12, H + 5, dtype=torch.bfloat16, device="cuda")
            c = torch.zeros(12, H + 7, dtype=torch.int8, device="cuda").view(T[q])
            s = torch.zeros(12, n, device="cuda")
            moeq.moeq_add_rmsnorm(x, gamma, 1e-6, r, r if stream == "in place" else None,
                                  y[:, 2:H + 2], c[:, 3:H + 3], s, group)
            torch.cuda.synchronize()
            after = want["r"] if stream == "in place" else res
            assert torch.equal(r[fine], after[fine])
            assert torch.equal(c[:, 3:H + 3].float().double()[fine], want["codes"][fine])
            for got, ref_, rel, least in ((s, want["scales"], SCALE, TINY),
                                          (y[:, 2:H + 2], want["y"], Y, 1e-38)):
                d = (got.double() - ref_).abs()[fine]
                assert bool((d <= rel * ref_.abs()[fine] + least).all())
            assert torch.isnan(s[7]).all() and bool((c[7].float() == 0).all())
            assert torch.isnan(s[8, 0]) and bool((c[8, 3:128].float() == 0).all())
        y1 = add_rmsnorm(x, gamma, 1e-6, res)[1]
        assert torch.equal(y1[fine], y[:, 2:H + 2][fine])
