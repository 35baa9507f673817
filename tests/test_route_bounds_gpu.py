"""moeq_route_groups where fp32 scores are least able to tell: sigmoid rows far
below zero, whose scores are off by their logits' size times fp32's rounding.

Weights: a score's relative error there is the rounding of the scaled logit,
|z| 2^-24 with |z| <= 91 (5.5e-6), and 8 * 2^-24 of the exponential and the
division; the sum it is divided by has the same and five additions: under
1.25e-5 in all.
"""
import pytest

import ops_reference as ref
from quantized_mixture_experts_affine_b200 import moeq
from quantized_mixture_experts_affine_b200.layer import route_groups

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
REL = 1.25e-5
STEP = 2.0 ** -17  # a whole number of units in the last place of every logit here


def check(logits, K, bias=None, groups=1, keep=1, group_top=1, scale=1.0, renorm=True):
    r = moeq.routing(logits.shape[1], K, moeq.SCORE_SIGMOID, groups, keep, group_top, renorm,
                     scale, 1.0)
    idx, w = route_groups(r, logits, bias)
    torch.cuda.synchronize()
    ri, rw = ref.route(logits, K, "sigmoid", bias, groups, keep, group_top, renorm,
                       float(torch.tensor(scale)), 1.0)
    assert torch.equal(idx.cpu(), ri)
    err = (w.cpu().double() - rw).abs()
    assert bool((err <= REL * rw.abs() + 1e-37).all()), float(err.max())


def paired(M, E, groups, z, scale, seed):
    """Rows whose groups hold z + i STEP and z - i STEP, another i in each, the
    rest lower: the sums of two differ by i^2 STEP^2 relative, 64-bit arithmetic
    alone can order them."""
    g = torch.Generator().manual_seed(seed)
    z0 = round(z / scale / STEP) * STEP
    l = torch.full((M, groups, E // groups), z0 - 3.0)
    for m in range(M):
        i = torch.randperm(5 * groups, generator=g)[:groups] * STEP
        l[m, :, 0] = z0 + i
        l[m, :, 1] = z0 - i
    return l.view(M, E).cuda()


@pytest.mark.parametrize("z", [-12.0, -30.0, -45.0, -60.0, -85.0, -88.0])
@pytest.mark.parametrize("scale", [1.0, 0.7])
@pytest.mark.parametrize("M,E,groups,keep,K", [
    (40, 8, 4, 2, 2), (30, 256, 8, 4, 8), (20, 512, 16, 5, 4), (2400, 128, 8, 3, 4),
    (2400, 256, 16, 6, 4), (20, 1024, 32, 11, 4), (20, 60, 12, 4, 4)])
def test_two_best_of_groups_far_below_zero(z, scale, M, E, groups, keep, K):
    check(paired(M, E, groups, z, scale, E - int(z)), K, None, groups, keep, 2, scale)


@pytest.mark.parametrize("z", [-30.0, -60.0, -85.0])
@pytest.mark.parametrize("M,E,K", [(24, 64, 8), (2400, 64, 8), (24, 512, 8), (8, 640, 6)])
def test_biased_picks_far_below_zero(z, M, E, K):
    """Biases that even the scores out but for one part in 10^7 or less."""
    l = z / 0.7 + torch.linspace(-0.5, 0.5, E).roll(7)
    s = torch.sigmoid(0.7 * l.double())
    b = (s.max() - s).float()
    rows = torch.stack([l] * M).cuda()
    check(rows, K, b.cuda(), scale=0.7)
    check(rows, K, b.cuda(), 4, 2, 2, scale=0.7)


@pytest.mark.parametrize("M", [3, 2400])
@pytest.mark.parametrize("E", [16, 64, 300])
def test_experts_under_a_bias_of_minus_infinity(M, E):
    """They come after every other, before those whose logits are out."""
    g = torch.Generator(device="cuda").manual_seed(E)
    l = torch.randn(M, E, device="cuda", generator=g)
    b = torch.zeros(E, device="cuda")
    l[:, : E - 6] = float("nan")
    l[1, 2] = float("-inf")
    b[E - 3:] = float("-inf")
    idx = list(range(E - 6, E - 3)) + list(range(E - 3, E)) + [0, 1]
    check(l, 8, b)
    r = moeq.routing(E, 8, moeq.SCORE_SIGMOID)
    got, w = route_groups(r, l, b)
    assert got[0].tolist()[3:] == idx[3:] and w[0, 6:].abs().sum() == 0 and (w[0, :6] > 0).all()
    # fewer experts than picks, and a bias that masks all but two
    b[:] = float("-inf")
    b[E - 2:] = 0.25
    check(l, 8, b)
    check(torch.randn(M, E, device="cuda", generator=g), 6, b)


@pytest.mark.parametrize("M,E,K,groups,keep", [(16, 512, 8, 1, 1), (16, 512, 8, 8, 4),
                                               (2400, 128, 8, 8, 3), (8, 2048, 8, 16, 8)])
def test_biased_softmax_of_many_like_logits(M, E, K, groups, keep):
    """Hundreds of terms of the normaliser with one exponent, and so one rounding;
    biases that even the scores out but for their own rounding."""
    for d in (2.7, 4.9, 6.3):
        l = torch.full((E,), -d)
        l[7] = 0.0
        l -= torch.linspace(0, 1e-3, E).roll(11)
        p = torch.softmax(l.double(), 0)
        b = (p.max() - p).float()
        rows = torch.stack([l] * M).cuda()
        r = moeq.routing(E, K, moeq.SCORE_SOFTMAX, groups, keep, 2, True)
        idx, _ = route_groups(r, rows, b.cuda())
        ri, _ = ref.route(rows, K, "softmax", b.cuda(), groups, keep, 2, True)
        assert torch.equal(idx.cpu(), ri)
