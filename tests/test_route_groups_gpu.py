"""moeq_route_groups against a token-by-token 64-bit reference: indices equal,
weights within fp32's own error.

Weights: a score's numerator is exp(d) in fp32, |d| <= 20 here: relative
20 * 2^-23 + 4 * 2^-24 < 2.7e-6; the sum it is divided by has the same error
and at most 45 additions in a row (2.7e-6): 8.1e-6 in all.
"""
import pytest

import ops_reference as ref
from quantized_mixture_experts_affine_b200 import moeq
from quantized_mixture_experts_affine_b200.layer import route_groups

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
REL = 8.1e-6
SCORE = {"softmax": moeq.SCORE_SOFTMAX, "sigmoid": moeq.SCORE_SIGMOID}


def check(logits, K, bias=None, score="softmax", groups=1, keep=1, group_top=1, renorm=True,
          scale=1.0, routed=1.0):
    r = moeq.routing(logits.shape[1], K, SCORE[score], groups, keep, group_top, renorm, scale,
                     routed)
    idx, w = route_groups(r, logits, bias)
    torch.cuda.synchronize()
    ri, rw = ref.route(logits, K, score, bias, groups, keep, group_top, renorm,
                       float(torch.tensor(scale)), float(torch.tensor(routed)))
    assert torch.equal(idx.cpu(), ri)
    err = (w.cpu().double() - rw).abs()
    assert bool((err <= REL * rw.abs() + 1e-37).all()), float(err.max())
    return idx, w


def draw(M, E, seed, dtype=torch.float32, spread=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = (spread * torch.randn(M, E, device="cuda", generator=g)).to(dtype)
    return l, 0.05 * torch.randn(E, device="cuda", generator=g)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("M,E,K,groups,keep,top", [
    (1, 512, 4, 1, 1, 1), (5, 1, 1, 1, 1, 1), (33, 7, 7, 1, 1, 1), (300, 256, 8, 8, 4, 2),
    (257, 160, 6, 8, 3, 1), (40, 96, 8, 32, 5, 2), (9, 130, 3, 13, 2, 2), (64, 64, 1, 1, 1, 2),
    (3, 4096, 32, 16, 16, 2), (2, 4095, 9, 1, 1, 1), (20, 32, 3, 32, 3, 2), (11, 600, 12, 3, 2, 2)])
def test_route_groups(M, E, K, groups, keep, top, with_bias, score):
    l, b = draw(M, E, E * 100 + M)
    check(l, K, b if with_bias else None, score, groups, keep, top, renorm=M % 2 == 0, scale=0.7,
          routed=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("E,K,groups,keep,top", [
    (128, 8, 8, 3, 1), (128, 8, 8, 4, 2), (100, 3, 1, 1, 1), (64, 8, 4, 2, 2), (16, 2, 2, 1, 1),
    (256, 8, 8, 4, 2), (200, 16, 1, 1, 1), (256, 9, 16, 5, 1), (128, 9, 8, 4, 2),
    (128, 8, 16, 4, 2), (512, 8, 8, 4, 2)])
def test_many_rows(E, K, groups, keep, top, with_bias, score):
    """More than 16 rows per SM: several rows share a warp."""
    M = 2371 if E < 512 else 2369
    l, b = draw(M, E, E + K)
    l[5, ::3] = float("-inf")
    l[7] = float("nan")
    l[8] = float("-inf")
    l[8, 1] = 0.5
    check(l, K, b if with_bias else None, score, groups, keep, top, renorm=K % 2 == 0)


def test_near_ties_in_many_rows():
    """Rows that need the second look, beside rows that do not, in one warp."""
    E, M = 64, 2500
    l, b = draw(M, E, 77)
    tie = torch.linspace(-1e-6, 1e-6, E, device="cuda")
    for m in range(0, M, 3):
        l[m] = tie.roll(m)
    flat = 0.5 - torch.sigmoid(l[0].double()).float()
    check(l, 8, flat, "sigmoid")
    check(l, 8, flat, "sigmoid", 8, 4, 2)
    check(l, 6, flat, "softmax", 4, 2, 1)
    check(l.to(torch.bfloat16), 6, (b * 20).round() / 20, "sigmoid", 8, 3, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_bf16_logits_tie_by_index(score):
    """bf16 logits tie often; so do equal biases."""
    l, b = draw(200, 256, 5, torch.bfloat16)
    check(l, 8, None, score)
    check(l, 8, torch.zeros_like(b), score, 8, 3, 2)
    check(l, 8, None, score, 8, 3, 2)
    check(l, 8, (b * 20).round() / 20, score, 8, 3, 1)


def test_near_ties_are_ordered_as_real_numbers():
    """Scores whose difference fp32 cannot hold: sigmoid values one part in
    10^9 apart, ordered by an opposing bias."""
    E, M = 64, 64
    l = torch.zeros(M, E, device="cuda")
    for m in range(M):
        l[m] = torch.linspace(-1e-6, 1e-6, E, device="cuda").roll(m)
    b = 0.5 - torch.sigmoid(l[0].double()).float()  # fp32: leaves differences near 1e-9
    check(l, 8, b, "sigmoid")
    check(l, 8, b, "sigmoid", 8, 4, 2)
    check(l, 8, torch.zeros_like(b), "sigmoid", 4, 2, 1)


def test_equal_rows_choose_the_lowest_indices():
    l = torch.full((3, 48), 0.25, device="cuda")
    idx, w = check(l, 6, None, "sigmoid", 4, 2, 2)
    assert idx[0].tolist() == [0, 1, 2, 3, 4, 5]
    check(l, 6, torch.full((48,), -0.125, device="cuda"), "softmax", 4, 2, 1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_experts(score, with_bias):
    """-inf and NaN take experts out; rows with fewer than K, or none, left."""
    l, b = draw(12, 40, 8)
    l[0, 3] = float("-inf")
    l[1] = float("-inf")
    l[2, :38] = float("nan")
    l[3, ::2] = float("-inf")
    l[4, :10] = float("-inf")   # a whole group
    l[5, 10:] = float("-inf")   # all but one group
    l[6] = float("nan")
    l[7, 0] = torch.finfo(torch.float32).min
    l[8] = torch.finfo(torch.float32).min
    b = b if with_bias else None
    idx, w = check(l, 4, b, score)
    assert w[1].abs().sum() == 0 and idx[1].tolist() == [0, 1, 2, 3]
    check(l, 4, b, score, 4, 2, 1)
    check(l, 4, b, score, 4, 2, 2, renorm=False)


def test_extreme_logits():
    l, b = draw(6, 64, 9)
    l[0, 5] = float("inf")
    l[1] *= 1e30
    l[2, 7] = 3e38
    l[3] = -60.0 - torch.arange(64, device="cuda") * 0.5   # sigmoid scores down to 1e-40
    l[4] = -300.0 - torch.arange(64, device="cuda")        # below fp32's smallest
    l[5] *= 1e-30
    for score in ("softmax", "sigmoid"):
        check(l, 5, None, score)
        check(l[3:], 5, b, score)


def test_strided_unaligned_rows_and_untouched_memory():
    g = torch.Generator(device="cuda").manual_seed(3)
    for dtype in (torch.float32, torch.bfloat16):
        wide = torch.randn(9, 77, device="cuda", generator=g).to(dtype)
        l = wide[:, 3:70]
        r = moeq.routing(67, 5)
        idx = torch.full((12, 5), -7, dtype=torch.int32, device="cuda")
        w = torch.full((12, 5), -7.0, device="cuda")
        moeq.moeq_route_groups(r, l, idx[:9], w[:9])
        ri, _ = ref.route(l, 5)
        assert torch.equal(idx[:9].cpu(), ri)
        assert (idx[9:] == -7).all() and (w[9:] == -7).all()
    check(torch.zeros(0, 8, device="cuda"), 2)


def test_deterministic_in_a_graph_on_another_stream():
    l, b = draw(2048, 256, 11)
    r = moeq.routing(256, 8, moeq.SCORE_SIGMOID, 8, 4, 2)
    i0, w0 = route_groups(r, l, b)
    idx, w = torch.empty_like(i0), torch.empty_like(w0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        moeq.moeq_route_groups(r, l, idx, w, b)
    for _ in range(2):
        idx.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, i0) and torch.equal(w, w0)


def test_as_many_rows_as_an_int_counts():
    M = 2 ** 31 - 1
    idx = torch.full((M, 1), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros(M, 1, device="cuda")
    l = torch.ones(M, 1, dtype=torch.bfloat16, device="cuda")
    moeq.moeq_route_groups(moeq.routing(1, 1), l, idx, w)
    assert int(idx.max()) == 0 and int(idx.min()) == 0
    assert float(w.max()) == 1 and float(w.min()) == 1


@pytest.mark.parametrize("M", [7, 2600])
@pytest.mark.parametrize("with_bias,score", [(True, "sigmoid"), (False, "softmax")])
@pytest.mark.parametrize("E,groups,keep,top,K", [
    (240, 4, 2, 2, 16), (60, 12, 3, 1, 8), (96, 32, 7, 2, 10), (33, 11, 5, 2, 6), (7, 7, 3, 1, 3),
    (368, 16, 12, 2, 6), (500, 5, 2, 2, 9), (26, 2, 1, 1, 8), (130, 2, 1, 2, 8), (300, 20, 6, 2, 8)])
def test_groups_of_any_size(E, groups, keep, top, K, with_bias, score, M):
    l, b = draw(M, E, E + groups + M, torch.bfloat16 if M == 7 else torch.float32)
    l[0] = float("-inf")
    l[1, : E // groups + 1] = float("nan")
    l[2] = l[2, 0].item()
    l[3, 1:] = float("-inf")
    check(l, K, b if with_bias else None, score, groups, keep, top)
