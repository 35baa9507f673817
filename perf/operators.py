"""Cases of the routing, norm and linear operators, with their plain forms.

Three operators of the serving path around the mixture-of-experts layer:
  route   grouped top-k routing (moeq_route_groups)
  norm    residual addition, RMS norm, 8-bit output with scales (moeq_add_rmsnorm)
  linear  packed-weight matrix product with bias, activation, multiplier and
          residual in its epilogue (moeq_linear)
``run`` computes them with elementary torch operations, or through the
library where ``own`` is true; ``exact`` computes them in 64 bits.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of the 512-expert layer under a sigmoid router with a balance bias
        dict(name="route_token", op="route", M=1, E=512, K=4, score="sigmoid", groups=1,
             keep=1, top=1, bias=True, renorm=True, scale=1.0, routed=1.0, dtype="f32"),
        # a prompt chunk under group-limited routing (two-best group scores)
        dict(name="route_groups", op="route", M=2048, E=256, K=8, score="sigmoid", groups=8,
             keep=4, top=2, bias=True, renorm=True, scale=1.0, routed=2.5, dtype="f32"),
        # the 16,068-token prompt of the 128-expert layer, softmax router, best-expert groups
        dict(name="route_prompt", op="route", M=16068, E=128, K=8, score="softmax", groups=8,
             keep=3, top=1, bias=False, renorm=False, scale=1.0, routed=16.0, dtype="bf16"),
        # one token: the layer's fp32 output joins the fp32 residual stream, int8 row out
        dict(name="norm_token", op="norm", M=1, H=4096, x="f32", res="f32", y=True, q="int8",
             group=0),
        # a ragged batch of odd-sized rows in bf16, e4m3 with a partial last group
        dict(name="norm_odd", op="norm", M=333, H=1000, x="bf16", res="bf16", y=True, q="e4m3",
             group=128),
        # the 16,068-token prompt of the hidden-4096 layers, bf16 stream, e4m3 rows by 128
        dict(name="norm_prompt", op="norm", M=16068, H=4096, x="bf16", res="bf16", y=False,
             q="e4m3", group=128),
        # one token through a 4-bit projection with its residual
        dict(name="linear_token", op="linear", M=1, IN=4096, OUT=4096, bits=4, G=64, mx=False,
             x="bf16", group=0, bias=True, act="none", mul=False, res=True, out="f32"),
        # eight tokens in int8 through the gate rows of a dense 4-bit block
        dict(name="linear_batch", op="linear", M=8, IN=4096, OUT=1024, bits=4, G=64, mx=False,
             x="int8", group=0, bias=False, act="silu", mul=True, res=False, out="bf16"),
        # router logits of a decode batch: 8-bit, fp32 out
        dict(name="linear_router", op="linear", M=64, IN=4096, OUT=512, bits=8, G=64, mx=False,
             x="bf16", group=0, bias=False, act="none", mul=False, res=False, out="f32"),
        # a ragged chunk: odd rows and columns, 2-bit codes, e4m3 input by 128
        dict(name="linear_odd", op="linear", M=301, IN=2048, OUT=4001, bits=2, G=32, mx=False,
             x="e4m3", group=128, bias=True, act="gelu", mul=False, res=True, out="bf16"),
        # a prompt chunk through an MX FP4 projection
        dict(name="linear_chunk", op="linear", M=2048, IN=2048, OUT=4096, bits=4, G=32, mx=True,
             x="bf16", group=0, bias=True, act="gelu_tanh", mul=False, res=True, out="bf16"),
        # the whole prompt through an 8-bit projection
        dict(name="linear_prompt", op="linear", M=16068, IN=4096, OUT=4096, bits=8, G=64,
             mx=False, x="bf16", group=0, bias=True, act="silu", mul=False, res=True, out="bf16"),
    ]


MOST_MACS = 16068 * 4096 * 4096  # of one linear pass


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "norm", "linear", "linear"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        E = groups * _log(rng, 4, 512 // groups)
        keep = rng.randint(1, groups)
        K = min(rng.randint(1, 16), keep * (E // groups))
        return dict(op="route", M=_log(rng, 1, 16384), E=E, K=K,
                    score=rng.choice(["softmax", "sigmoid"]), groups=groups, keep=keep,
                    top=rng.choice([1, 2]), bias=rng.random() < 0.6, renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 1.0, 0.7]), routed=rng.choice([1.0, 2.5]),
                    dtype=rng.choice(["f32", "bf16"]))
    if op == "norm":
        H = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            H = (H + 63) // 64 * 64
        return dict(op="norm", M=min(_log(rng, 1, 16384), 16068 * 4096 // H), H=H,
                    x=rng.choice(["f32", "bf16"]), res=rng.choice(["none", "f32", "bf16"]),
                    y=rng.random() < 0.5, q=rng.choice(["int8", "e4m3"]),
                    group=rng.choice([0, 128]))
    bits = rng.choice([2, 3, 4, 4, 4, 5, 6, 8, 8])
    mx = bits == 4 and rng.random() < 0.25
    x = rng.choice(["bf16", "bf16", "int8", "e4m3"])
    IN = 128 * _log(rng, 1, 64)
    OUT = _log(rng, 16, 8192)
    if rng.random() < 0.5:
        OUT = (OUT + 63) // 64 * 64
    return dict(op="linear", M=max(1, min(_log(rng, 1, 16384), MOST_MACS // (IN * OUT))), IN=IN,
                OUT=OUT, bits=bits, G=32 if mx else rng.choice([32, 64, 64, 128]), mx=mx, x=x,
                group=0 if x == "bf16" else rng.choice([0, 128]), bias=rng.random() < 0.5,
                act=rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu", "sigmoid"]),
                mul=rng.random() < 0.3, res=rng.random() < 0.5,
                out=rng.choice(["bf16", "bf16", "f32"]))


# ------------------------------------------------------------------ inputs
_T = {"f32": torch.float32, "bf16": torch.bfloat16, "int8": torch.int8,
      "e4m3": torch.float8_e4m3fn}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pack(q, bits):
    """Codes [out][in] as int32 words, each row one little-endian bit stream."""
    o, i = q.shape
    q = q.view(o, i // 32, 32).to(torch.int64)
    w = torch.zeros(o, i // 32, bits, dtype=torch.int64, device=q.device)
    for j in range(32):
        k, sh = divmod(j * bits, 32)
        w[..., k] |= (q[..., j] << sh) & 0xFFFFFFFF
        if sh + bits > 32:
            w[..., k + 1] |= q[..., j] >> (32 - sh)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32).view(o, -1).contiguous()


def _weights(case, gen):
    """Normal weights quantised as the packed formats hold them."""
    o, i, G = case["OUT"], case["IN"], case["G"]
    w = 0.02 * torch.randn(o, i, device="cuda", generator=gen)
    wg = w.view(o, i // G, G)
    if case["mx"]:
        e = torch.floor(torch.log2(wg.abs().amax(-1))) - 2
        mag = (wg / torch.exp2(e)[..., None]).abs()
        mid = torch.tensor([(a + b) / 2 for a, b in zip(_E2M1, _E2M1[1:])], device="cuda")
        q = torch.bucketize(mag, mid) + 8 * (wg < 0)
        return dict(w=_pack(q.view(o, i), 4), s=(e + 127).to(torch.uint8).contiguous(), b=None)
    lo, hi = wg.amin(-1), wg.amax(-1)
    top = 2 ** case["bits"] - 1
    s = ((hi - lo) / top).to(torch.bfloat16)
    b = lo.to(torch.bfloat16)
    q = torch.round((wg - b.float()[..., None]) / s.float()[..., None]).clamp_(0, top)
    return dict(w=_pack(q.view(o, i), case["bits"]), s=s.contiguous(), b=b.contiguous())


def _columns(per, n, group):
    """A value per row or per 128 columns, laid over the n columns."""
    return per if not group else per.repeat_interleave(group, 1)[:, :n]


def _tokens(case, M, n, gen):
    """Activations with a few channels larger than the rest, in the case's type."""
    x = torch.randn(M, n, device="cuda", generator=gen)
    x[:, :: max(1, n // 4)] *= 8.0
    if case["x"] in ("f32", "bf16"):
        return x.to(_T[case["x"]]), None
    group = case["group"]
    gs = group or n
    pad = torch.nn.functional.pad(x.abs(), (0, -n % gs)).view(M, -1, gs)
    sc = pad.amax(-1) / (127.0 if case["x"] == "int8" else 448.0)
    v = x / _columns(sc, n, group)
    q = torch.round(v).clamp_(-127, 127) if case["x"] == "int8" else v.clamp_(-448, 448)
    return q.to(_T[case["x"]]), sc.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    M = case["M"]
    if case["op"] == "route":
        E = case["E"]
        s["logits"] = (1.5 * torch.randn(M, E, device="cuda", generator=gen)).to(_T[case["dtype"]])
        s["bias"] = 0.05 * torch.randn(E, device="cuda", generator=gen) if case["bias"] else None
    elif case["op"] == "norm":
        H = case["H"]
        s["x"] = _tokens(case, M, H, gen)[0]
        s["gamma"] = (1 + 0.25 * torch.randn(H, device="cuda", generator=gen)).to(torch.bfloat16)
        s["res"] = None if case["res"] == "none" else \
            (2 * torch.randn(M, H, device="cuda", generator=gen)).to(_T[case["res"]])
    else:
        n, t = case["OUT"], _T[case["out"]]
        s.update(_weights(case, gen))
        s["x"], s["xs"] = _tokens(case, M, case["IN"], gen)
        s["bias"] = torch.randn(n, device="cuda", generator=gen).to(torch.bfloat16) \
            if case["bias"] else None
        s["mul"] = torch.randn(M, n, device="cuda", generator=gen).to(t) if case["mul"] else None
        s["res"] = torch.randn(M, n, device="cuda", generator=gen).to(t) if case["res"] else None
    if own:  # the descriptors, workspace and output buffers that a serving program keeps
        from quantized_mixture_experts_affine_b200 import moeq
        s["lib"] = moeq
        if case["op"] == "route":
            s["plan"] = moeq.routing(
                case["E"], case["K"], score=moeq.SCORE_SIGMOID if case["score"] == "sigmoid"
                else moeq.SCORE_SOFTMAX, n_groups=case["groups"], topk_groups=case["keep"],
                group_top=case["top"], renorm=case["renorm"], router_scale=case["scale"],
                routed_scale=case["routed"])
            s["idx"] = torch.empty(M, case["K"], dtype=torch.int32, device="cuda")
            s["wts"] = torch.empty(M, case["K"], device="cuda")
        elif case["op"] == "norm":
            H = case["H"]
            s["y"] = torch.empty(M, H, dtype=torch.bfloat16, device="cuda") if case["y"] else None
            s["q"] = torch.empty(M, H, dtype=_T[case["q"]], device="cuda")
            s["qs"] = torch.empty(M, -(-H // 128) if case["group"] else 1, device="cuda")
            s["r"] = None if s["res"] is None else torch.empty_like(s["res"])
        else:
            s["t"] = moeq.qtensor(s["w"], s["s"], s["b"], n, case["IN"], case["bits"], case["G"],
                                  fmt=moeq.FMT_MXFP4 if case["mx"] else moeq.FMT_AFFINE)
            s["y"] = torch.empty(M, n, dtype=t, device="cuda")
            need = moeq.moeq_linear_workspace_bytes(s["t"], M, s["x"].dtype, t)
            s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
            s["act"] = getattr(moeq, "ACT_" + case["act"].upper())
    return s


# ------------------------------------------------------------------ plain forms
def _plain_route(s):
    c = s["case"]
    M, E, K, G = c["M"], c["E"], c["K"], c["groups"]
    # 64 bits: which of two near scores is larger decides an index
    z = s["logits"].double() * c["scale"]
    if c["score"] == "softmax":
        p = torch.exp(z - z.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-z))
    v = p if s["bias"] is None else p + s["bias"].double()
    sel = z if s["bias"] is None else v  # without a bias the order is the logits' own
    if G > 1:
        if c["top"] == 1:
            score = sel.view(M, G, -1).amax(-1)
        else:
            score = torch.sort(v.view(M, G, -1), dim=-1, descending=True)[0][..., :2].sum(-1)
        kept = torch.sort(score, dim=1, descending=True, stable=True)[1][:, :c["keep"]]
        mask = torch.zeros(M, G, dtype=torch.bool, device=z.device).scatter_(1, kept, True)
        sel = torch.where(mask.repeat_interleave(E // G, 1), sel, -math.inf)
    idx = torch.sort(sel, dim=1, descending=True, stable=True)[1][:, :K]
    w = p.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"idx": idx.to(torch.int32), "w": (w * c["routed"]).float()}


def _to_e4m3(v):
    """Nearest e4m3 value (ties to even) of 64-bit values of magnitude <= 448."""
    e = torch.frexp(v)[1].clamp(min=-5) - 1
    step = torch.exp2((e - 3).double())
    return torch.round(v / step) * step


def _plain_norm(s):
    c = s["case"]
    M, H = c["M"], c["H"]
    r = s["x"].float()
    if s["res"] is not None:
        r = (r + s["res"].float()).to(s["res"].dtype)
    out = {} if s["res"] is None else {"r": r}
    r = r.float()
    inv = 1.0 / torch.sqrt((r * r).mean(1, keepdim=True) + EPS)
    g = s["gamma"].float()
    if c["y"]:
        out["y"] = (r * inv * g).to(torch.bfloat16)
    # 64 bits for the codes: a value next to a rounding border decides a code
    t = r.double() * g.double()
    gs = c["group"] or H
    a = torch.nn.functional.pad(t.abs(), (0, -H % gs)).view(M, -1, gs).amax(-1)
    top = 127.0 if c["q"] == "int8" else 448.0
    scale = (a * inv.double() / top).float()
    v = t * top / _columns(torch.where(a > 0, a, 1.0), H, c["group"])
    if c["q"] == "int8":
        out["values"] = torch.round(v).float() * _columns(scale, H, c["group"])
    else:
        out["codes"] = _to_e4m3(v).to(torch.float8_e4m3fn)
    out["scales"] = scale
    return out


EPS = 1e-6


def _act(v, name):
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "relu":
        return v.clamp(min=0)
    return 1.0 / (1.0 + torch.exp(-v)) if name == "sigmoid" else v


def _codes(w, bits, n):
    """The codes of packed rows, [out][n]."""
    o = w.shape[0]
    w = (w.to(torch.int64) & 0xFFFFFFFF).view(o, n // 32, bits)
    at = torch.arange(32, device=w.device) * bits
    lo = at // 32
    v = w[..., lo] | (w[..., (lo + 1).clamp(max=bits - 1)] << 32)
    return ((v >> (at % 32)) & (2 ** bits - 1)).view(o, n)


def _dense(s, t):
    """The weight matrix in floating type t."""
    c = s["case"]
    q = _codes(s["w"], c["bits"], c["IN"])
    if c["mx"]:
        v = torch.tensor(_E2M1 + tuple(-e for e in _E2M1), dtype=t, device="cuda")[q]
        sc, b = torch.exp2(s["s"].to(t) - 127), None
    else:
        v, sc, b = q.to(t), s["s"].to(t), s["b"].to(t)
    v = v.view(c["OUT"], -1, c["G"]) * sc[..., None]
    if b is not None:
        v = v + b[..., None]
    return v.view(c["OUT"], c["IN"])


def _plain_linear(s):
    c = s["case"]
    x = s["x"].float()
    if s["xs"] is not None:
        x = x * _columns(s["xs"], c["IN"], c["group"])
    v = x @ _dense(s, torch.float32).T
    if s["bias"] is not None:
        v = v + s["bias"].float()
    v = _act(v, c["act"])
    if s["mul"] is not None:
        v = v * s["mul"].float()
    if s["res"] is not None:
        v = v + s["res"].float()
    return v.to(_T[c["out"]])


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"route": _plain_route, "norm": _plain_norm, "linear": _plain_linear}[c["op"]](s)
    lib = s["lib"]
    if c["op"] == "route":
        lib.moeq_route_groups(s["plan"], s["logits"], s["idx"], s["wts"], bias=s["bias"])
        return {"idx": s["idx"], "w": s["wts"]}
    if c["op"] == "norm":
        lib.moeq_add_rmsnorm(s["x"], s["gamma"], EPS, residual=s["res"], r_out=s["r"], y=s["y"],
                             q=s["q"], q_scales=s["qs"], q_group=c["group"])
        out = {"scales": s["qs"]}
        if s["r"] is not None:
            out["r"] = s["r"]
        if c["y"]:
            out["y"] = s["y"]
        if c["q"] == "int8":
            out["values"] = s["q"] * _columns(s["qs"], c["H"], c["group"])
        else:
            out["codes"] = s["q"]
        return out
    lib.moeq_linear(s["t"], 0, s["x"], s["y"], x_scales=s["xs"], x_group=c["group"],
                    bias=s["bias"], act=s["act"], mul=s["mul"], residual=s["res"], ws=s["ws"])
    return s["y"]


# ------------------------------------------------------------------ work and 64-bit values
def work(case):
    c, M = case, case["M"]
    size = {"f32": 4, "bf16": 2, "int8": 1, "e4m3": 1, "none": 0}
    if c["op"] == "route":
        return {"bytes": M * c["E"] * size[c["dtype"]] + 8 * M * c["K"] + 4 * c["E"] * c["bias"],
                "flops": 4 * M * c["E"]}
    if c["op"] == "norm":
        H = c["H"]
        n = size[c["x"]] + 2 * size[c["res"]] + 2 * c["y"] + 1
        return {"bytes": M * H * n + 2 * H + 4 * M * (-(-H // 128) if c["group"] else 1),
                "flops": 6 * M * H}
    n, o, t = c["IN"], c["OUT"], size[c["out"]]
    packed = o * n * c["bits"] // 8 + o * (n // c["G"]) * (1 if c["mx"] else 4)
    xs = 0 if c["x"] == "bf16" else 4 * M * (-(-n // 128) if c["group"] else 1)
    return {"bytes": M * n * size[c["x"]] + xs + packed + 2 * o * c["bias"]
            + M * o * t * (1 + c["mul"] + c["res"]), "flops": 2 * M * n * o}


def _exact_route(c, s):
    l = s["logits"].double() * c["scale"]
    if c["score"] == "softmax":
        p = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    else:
        p = torch.sigmoid(l)
    v = p if s["bias"] is None else p + s["bias"].double()
    order = l if s["bias"] is None else v
    per = c["E"] // c["groups"]
    if c["top"] == 1:
        gs = order.unflatten(1, (c["groups"], per)).max(-1).values
    else:
        gs = torch.topk(v.unflatten(1, (c["groups"], per)), min(2, per), dim=-1).values.sum(-1)
    # rank of each group and expert: how many come before it (larger, or equal and earlier)
    earlier = torch.ones(c["groups"], c["groups"], dtype=torch.bool, device="cuda").triu(1)
    before = (gs[:, :, None] > gs[:, None, :]) | ((gs[:, :, None] == gs[:, None, :]) & earlier)
    in_group = (before.sum(1) < c["keep"])[:, torch.arange(c["E"], device="cuda") // per]
    idx = torch.empty(c["M"], c["K"], dtype=torch.int32, device="cuda")
    left = torch.where(in_group, order, -math.inf)
    for k in range(c["K"]):
        top = left.max(1, keepdim=True).values
        first = (left == top).to(torch.int8).argmax(1)
        idx[:, k] = first
        left = left.scatter(1, first[:, None], -math.inf)
    w = p.gather(1, idx.long())
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"idx": idx, "w": w * c["routed"]}


def _exact_norm(c, s):
    x = s["x"].double()
    out = {}
    if s["res"] is not None:
        x = x + s["res"].double()
        out["r"] = x
        x = x.to(s["res"].dtype).double()  # the norm is of the stored residual
    n = x * torch.rsqrt(x.square().sum(1, keepdim=True) / c["H"] + EPS) * s["gamma"].double()
    if c["y"]:
        out["y"] = n
    top = 127.0 if c["q"] == "int8" else 448.0
    parts = torch.split(n, c["group"] or c["H"], dim=1)
    scale = torch.stack([p.abs().max(1).values for p in parts], 1) / top
    v = n / _columns(scale, c["H"], c["group"])
    if c["q"] == "int8":
        out["values"] = torch.round(v) * _columns(scale, c["H"], c["group"])
    else:
        m = 2.0 ** (torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        out["codes"] = torch.round(v / m) * m
    out["scales"] = scale
    return out


def _exact_dense(c, s):
    """The weight matrix from the bits of each row's stream."""
    o, n, b = c["OUT"], c["IN"], c["bits"]
    bit = (s["w"][..., None] >> torch.arange(32, dtype=torch.int32, device="cuda")) & 1
    bit = bit.to(torch.uint8).reshape(o, n, b)
    q = sum(bit[..., k].double() * 2 ** k for k in range(b))
    sc = s["s"].double().repeat_interleave(c["G"], 1)
    if not c["mx"]:
        return q * sc + s["b"].double().repeat_interleave(c["G"], 1)
    m, e = bit[..., 0].double(), bit[..., 1].double() + 2 * bit[..., 2].double()
    mag = torch.where(e > 0, (1 + m / 2) * torch.pow(2.0, e - 1), m / 2)
    return (1 - 2 * bit[..., 3].double()) * mag * torch.pow(2.0, sc - 127)


def _exact_linear(c, s):
    x = s["x"].double()
    if s["xs"] is not None:
        x = x * _columns(s["xs"].double(), c["IN"], c["group"])
    v = torch.matmul(x, _exact_dense(c, s).t())
    if s["bias"] is not None:
        v += s["bias"].double()
    F = torch.nn.functional
    v = {"none": lambda a: a, "silu": F.silu, "gelu": F.gelu, "relu": F.relu,
         "gelu_tanh": lambda a: F.gelu(a, approximate="tanh"), "sigmoid": torch.sigmoid}[c["act"]](v)
    if s["mul"] is not None:
        v *= s["mul"].double()
    return v if s["res"] is None else v + s["res"].double()


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "norm": _exact_norm, "linear": _exact_linear}[case["op"]](case, s)
