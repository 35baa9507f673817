"""The routing, norm and linear operators together, as a model runs them:
norm with 8-bit output -> dense block (gate, up, down) -> norm -> layer under
a grouped sigmoid router."""
import os
import subprocess
import sys

import numpy as np
import pytest

import ops_reference as ref
from helpers import MAX_ABS, REL_L2, host_router, oracle_expert_outputs, rel_l2
import oracle
from quantized_mixture_experts_affine_b200 import moeq, synth
from quantized_mixture_experts_affine_b200.layer import (CONFIGS, add_rmsnorm, expert_ffn, linear,
                                                         layer_forward_routed, route_groups,
                                                         synthetic_layer)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
SEED = 0


def tokens(cfg, M, copy):
    xb = synth.normal_bf16_host(SEED, synth.tag(synth.X, copy), M * cfg.H).reshape(M, cfg.H)
    return xb, torch.from_numpy(xb.view(np.int16)).cuda().view(torch.bfloat16)


@pytest.mark.parametrize("name,M,mode,groups,keep", [
    ("tiny", 1, moeq.MODE_DECODE, 4, 2), ("decode_397b", 1, moeq.MODE_DECODE, 1, 1),
    ("decode_397b", 7, moeq.MODE_DECODE, 8, 4), ("decode_30b", 64, moeq.MODE_DECODE, 8, 3),
    ("prefill_8bit", 300, moeq.MODE_PREFILL, 8, 4), ("tiny", 200, moeq.MODE_AUTO, 2, 1)])
def test_layer_under_a_grouped_router(name, M, mode, groups, keep):
    cfg = CONFIGS[name]
    L = synthetic_layer(cfg, SEED, 0)
    xb, x = tokens(cfg, M, 500 + M)
    g = torch.Generator(device="cuda").manual_seed(M)
    bias = 0.05 * torch.randn(cfg.E, device="cuda", generator=g)
    r = moeq.routing(cfg.E, cfg.K, moeq.SCORE_SIGMOID, groups, keep, 2, True, 1.0, 2.5)
    res_np = np.linspace(-1, 1, M * cfg.H, dtype=np.float32).reshape(M, cfg.H)
    y, idx, w = layer_forward_routed(L, r, x, bias, torch.from_numpy(res_np).cuda(), mode)
    # the router's product and choice, each against its definition
    logits = linear(L.desc.router, x, torch.float32)
    torch.cuda.synchronize()
    assert moeq.moeq_device_status() == 0
    want = oracle.qmv(host_router(cfg, SEED, 0), xb)
    assert rel_l2(logits.cpu().numpy(), want) <= 1e-5
    ri, rw = ref.route(logits, cfg.K, "sigmoid", bias, groups, keep, 2, True, 1.0, 2.5)
    assert torch.equal(idx.cpu(), ri)
    assert float((w.cpu().double() - rw).abs().max()) < 1e-5
    rows = np.arange(M) if M <= 16 else np.unique(np.linspace(0, M - 1, 12).astype(int))
    out = oracle_expert_outputs(cfg, SEED, 0, xb[rows], ri.numpy()[rows], rw.numpy()[rows],
                                res_np[rows])
    got = y.cpu().numpy()[rows]
    # weights sum to 2.5 here: the layer's tolerances are for a sum of 1
    assert rel_l2(got, out) <= REL_L2 and np.abs(got - out).max() <= 2.5 * MAX_ABS


@pytest.mark.parametrize("M", [1, 6, 130])
@pytest.mark.parametrize("q,group", [(torch.int8, 0), (torch.float8_e4m3fn, 128)])
def test_block_between_two_layers(M, q, group):
    """norm(8 bit) -> dense SwiGLU -> residual -> norm -> route -> experts, each
    step against the 64-bit form of the same step on the library's own inputs."""
    cfg = CONFIGS["tiny"]
    H, I = cfg.H, 192
    g = torch.Generator(device="cuda").manual_seed(M)
    mats = {k: ref.matrix(o, n, 4, 64, g) for k, o, n in
            (("gate", I, H), ("up", I, H), ("down", H, I))}
    t = {k: moeq.qtensor(m["w"], m["s"], m["b"], *m["dense"].shape, 4, 64)
         for k, m in mats.items()}
    x = torch.randn(M, H, device="cuda", generator=g)
    stream = torch.randn(M, H, device="cuda", generator=g)
    gamma = (1 + 0.1 * torch.randn(H, device="cuda", generator=g)).to(torch.bfloat16)

    r, _, qx, qs = add_rmsnorm(x, gamma, 1e-6, stream, False, q, group)
    want = ref.add_rmsnorm(x, gamma, 1e-6, stream, "int8" if q == torch.int8 else "e4m3", group)
    assert torch.equal(r, want["r"]) and torch.equal(qx.float().double(), want["codes"])
    up = linear(t["up"], qx, x_scales=qs, x_group=group)
    h = linear(t["gate"], qx, x_scales=qs, x_group=group, act=moeq.ACT_SILU, mul=up)
    d = ref.dequant_x(qx, qs, group)
    ref_h = ref.act(d @ mats["gate"]["dense"].t(), "silu") * up.double()
    # two bf16 half steps at most (h's and, by the weights, an eighth of one)
    assert float((h.double() - ref_h).norm() / ref_h.norm()) < 2.0 ** -7
    r2 = linear(t["down"], h, torch.float32, residual=r)
    ref_r2 = h.double() @ mats["down"]["dense"].t() + r.double()
    assert float((r2.double() - ref_r2).abs().max()) < 1e-4
    L = synthetic_layer(cfg, SEED, 0)
    _, y2, _, _ = add_rmsnorm(r2, gamma, 1e-6)
    R = moeq.routing(cfg.E, cfg.K, moeq.SCORE_SOFTMAX, 4, 2, 1, False, 1.0, 1.5)
    logits = linear(L.desc.router, y2, torch.float32)
    idx, w = route_groups(R, logits)
    ri, rw = ref.route(logits, cfg.K, "softmax", None, 4, 2, 1, False, 1.0, 1.5)
    assert torch.equal(idx.cpu(), ri)
    out = expert_ffn(L, y2, idx, w, residual=r2)
    o, i2, w2 = layer_forward_routed(L, R, y2, residual=r2)
    torch.cuda.synchronize()
    assert torch.equal(i2, idx) and torch.equal(w2, w) and torch.equal(o, out)


def test_the_chain_in_a_graph():
    """The whole step captured once and replayed on other tokens."""
    cfg = CONFIGS["decode_30b"]
    L = synthetic_layer(cfg, SEED, 0)
    M = 4
    g = torch.Generator(device="cuda").manual_seed(1)
    gamma = (1 + 0.1 * torch.randn(cfg.H, device="cuda", generator=g)).to(torch.bfloat16)
    R = moeq.routing(cfg.E, cfg.K, moeq.SCORE_SIGMOID, 8, 4, 2, True)
    bias = 0.05 * torch.randn(cfg.E, device="cuda", generator=g)
    xs = [torch.randn(M, cfg.H, device="cuda", generator=g) for _ in range(2)]
    stream = torch.randn(M, cfg.H, device="cuda", generator=g)

    def step(x):
        r, y, _, _ = add_rmsnorm(x, gamma, 1e-6, stream)
        return layer_forward_routed(L, R, y, bias, r, moeq.MODE_DECODE)
    want = [step(x) for x in xs]
    torch.cuda.synchronize()
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x)
    for k in (1, 0, 1):
        x.copy_(xs[k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[k]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [1, 40, 700, 2600])
def test_calls_one_after_the_other(M):
    """Calls that feed one another, through one workspace and in place, give
    what they give with the device idle in between."""
    H, E, O = 1024, 64, 1920
    g = torch.Generator(device="cuda").manual_seed(M)
    packed = []

    def qt(o, n):
        packed.append(ref.matrix(o, n, 4, 64, g))
        w = packed[-1]
        return moeq.qtensor(w["w"], w["s"], w["b"], o, n, 4, 64)
    tu, td, tg = qt(O, H), qt(H, O), qt(E, H)
    gamma = torch.ones(H, device="cuda", dtype=torch.bfloat16)
    bias = 0.05 * torch.randn(E, device="cuda", generator=g)
    R = moeq.routing(E, 6, moeq.SCORE_SIGMOID, 8, 4, 2)
    x0 = torch.randn(M, H, device="cuda", generator=g)
    need = max(moeq.moeq_linear_workspace_bytes(t, M, torch.int8, torch.float32)
               for t in (tu, td, tg))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def steps(wait):
        kept = []
        stream, x = x0.clone(), 0.25 * x0
        y = torch.empty(M, H, device="cuda", dtype=torch.bfloat16)
        q = torch.empty(M, H, device="cuda", dtype=torch.int8)
        s = torch.empty(M, 1, device="cuda")
        h = torch.empty(M, O, device="cuda", dtype=torch.bfloat16)
        l = torch.empty(M, E, device="cuda")
        idx = torch.empty(M, 6, device="cuda", dtype=torch.int32)
        w = torch.empty(M, 6, device="cuda")
        for i in range(12):
            for call in (
                    lambda: moeq.moeq_add_rmsnorm(x, gamma, 1e-6, stream, stream, y, q, s),
                    lambda: moeq.moeq_linear(tu, 0, q, h, x_scales=s, act=moeq.ACT_SILU, ws=ws),
                    lambda: moeq.moeq_linear(td, 0, h, x, ws=ws),
                    lambda: moeq.moeq_linear(tg, 0, y, l, ws=ws),
                    lambda: moeq.moeq_route_groups(R, l, idx, w, bias)):
                call()
                if wait:
                    torch.cuda.synchronize()
            if i % 4 == 3:
                kept += [idx.clone(), w.clone()]
        return kept + [stream, x, h, l]
    want = steps(True)
    for _ in range(3):
        for a, b in zip(steps(False), want):
            assert torch.equal(a, b)


def ops_on(M):
    """x -> (norm, its codes through a projection, that through a router)."""
    H, O = 512, 640
    g = torch.Generator(device="cuda").manual_seed(M)
    w = ref.matrix(O, H, 4, 64, g)
    t = moeq.qtensor(w["w"], w["s"], w["b"], O, H, 4, 64)
    gamma = torch.ones(H, device="cuda", dtype=torch.bfloat16)
    R = moeq.routing(O, 8, moeq.SCORE_SIGMOID, 8, 4, 2)
    need = max(moeq.moeq_linear_workspace_bytes(t, M, torch.int8, torch.float32),
               moeq.moeq_linear_workspace_bytes(t, M, torch.bfloat16, torch.bfloat16))
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")

    def run(x, keep=w):  # (the operands live as long as the calls)
        _, y, q, s = add_rmsnorm(x, gamma, 1e-6, q_dtype=torch.int8)
        l = linear(t, q, torch.float32, x_scales=s, ws=ws)
        return [y, q, s, l, linear(t, y, torch.bfloat16, ws=ws), *route_groups(R, l)]
    xs = [torch.randn(M, H, device="cuda", generator=g) for _ in range(2)]
    return run, xs


@pytest.mark.parametrize("M", [3, 100, 2600])
def test_inputs_from_another_stream(M):
    """A call waits for an event of another stream, with kernels of its own
    stream right before it."""
    run, xs = ops_on(M)
    want = [run(x) for x in xs]
    torch.cuda.synchronize()
    side, x = torch.cuda.Stream(), torch.zeros_like(xs[0])
    for i in range(6):
        with torch.cuda.stream(side):
            torch.cuda._sleep(200000)
            x.copy_(xs[i % 2])
        y = [v * 2 for v in xs]  # kernels of this stream, before the wait
        torch.cuda.current_stream().wait_stream(side)
        got = run(x)
        side.wait_stream(torch.cuda.current_stream())
        for a, b in zip(got, want[i % 2]):
            assert torch.equal(a, b)
        del y


@pytest.mark.parametrize("M", [3, 100, 2600])
def test_a_fork_and_a_copy_in_a_graph(M):
    """Captured calls after a copy, and after branches that join before them."""
    run, xs = ops_on(M)
    want = [run(2 * x) for x in xs]
    src, x, side = xs[0].clone(), torch.empty_like(xs[0]), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.cuda._sleep(100000)
            x.copy_(src)
            x += src
        z = src * 3
        main.wait_stream(side)
        got = run(x)
        z += 1
    for k in (1, 0, 1):
        src.copy_(xs[k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[k]):
            assert torch.equal(a, b)


FIRST = """
import sys
sys.path[:0] = {path!r}
import torch
import ops_reference as ref
from quantized_mixture_experts_affine_b200 import moeq
from quantized_mixture_experts_affine_b200.layer import add_rmsnorm, linear, route_groups
g = torch.Generator(device="cuda").manual_seed(1)
w = ref.matrix(1930, 256, 4, 64, g)
t = moeq.qtensor(w["w"], w["s"], w["b"], 1930, 256, 4, 64)
gamma = torch.ones(256, device="cuda", dtype=torch.bfloat16)
xs = [torch.randn(M, 256, device="cuda", generator=g) for M in (3, 100, 2600)]
R = moeq.routing(1930, 8, moeq.SCORE_SIGMOID, 10, 4, 2)
def step():
    outs = []
    for x in xs:
        _, y, q, s = add_rmsnorm(x, gamma, 1e-6, q_dtype=torch.int8)
        l = linear(t, y, torch.float32)
        outs += [l, linear(t, q, torch.bfloat16, x_scales=s), *route_groups(R, l)]
    return outs
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    outs = step()
graph.replay()
torch.cuda.synchronize()
assert moeq.moeq_device_status() == 0
for a, b in zip(outs, step()):
    assert torch.equal(a, b)
"""


def test_first_calls_inside_a_capture():
    """A process that has made no call before captures its first ones."""
    here = os.path.dirname(os.path.abspath(__file__))
    code = FIRST.format(path=[os.path.dirname(here), here])
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)
