"""Calls on another stream than the current one, given as an object or a raw
handle, whose results are dropped or whose workspace is freed while they run."""
import pytest

import ops_reference as ref
from quantized_mixture_experts_affine_b200 import moeq
from quantized_mixture_experts_affine_b200.layer import (CONFIGS, add_rmsnorm, layer_forward_routed,
                                                         linear, route_groups, synthetic_layer)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def steps(M):
    H, O = 512, 640
    g = torch.Generator(device="cuda").manual_seed(M)
    w = ref.matrix(O, H, 4, 64, g)
    t = moeq.qtensor(w["w"], w["s"], w["b"], O, H, 4, 64)
    gamma = torch.ones(H, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(M, H, device="cuda", generator=g)
    L = synthetic_layer(CONFIGS["tiny"], 0, 0)
    c = L.cfg
    xl = torch.randn(M, c.H, device="cuda", generator=g).to(torch.bfloat16)
    R, RL = moeq.routing(O, 8, moeq.SCORE_SIGMOID, 8, 4, 2), moeq.routing(c.E, c.K)

    def run(stream, keep=(w,)):  # (the operands live as long as the calls)
        r, y, q, s = add_rmsnorm(x, gamma, 1e-6, x, q_dtype=torch.int8, stream=stream)
        l = linear(t, q, torch.float32, x_scales=s, stream=stream)
        return [r, y, q, s, l, linear(t, y, torch.bfloat16, stream=stream),
                *route_groups(R, l, stream=stream),
                *layer_forward_routed(L, RL, xl, stream=stream)]
    return run


@pytest.mark.parametrize("M", [3, 100, 2600])
@pytest.mark.parametrize("raw", [False, True])
def test_results_dropped_and_workspaces_freed_early(M, raw):
    run = steps(M)
    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2000000)
        kept = run(stream)
        dropped = [t.data_ptr() for t in run(stream)]  # (nothing of it is kept)
        # this stream takes as much memory again and writes it while the other runs
        mine = [torch.full_like(t, 3) for t in want for _ in range(2)]
        fill = [torch.full((1 << k,), 77, dtype=torch.uint8, device="cuda") for k in range(9, 25)]
        assert not {t.data_ptr() for t in mine} & set(dropped)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))
        assert all(bool((t.float() == 3).all()) for t in mine)
        assert all(bool((t == 77).all()) for t in fill)
        del kept, mine, fill
    assert moeq.moeq_device_status() == 0


def test_the_default_stream_by_its_handles():
    run = steps(40)
    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (0, 1):
        with torch.cuda.stream(side):
            got = run(handle)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
