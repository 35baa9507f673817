"""64-bit references of the routing, norm and linear operators, and packed
test matrices (torch tensors on any device, no code of the library)."""
import math

import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ routing
def route(logits, K, score="softmax", bias=None, groups=1, keep=1, group_top=1, renorm=True,
          scale=1.0, routed=1.0):
    """(idx int32 [M][K], w fp64 [M][K]), token by token."""
    l = logits.double().cpu()
    M, E = l.shape
    b = None if bias is None else bias.double().cpu()
    idx = torch.zeros(M, K, dtype=torch.int32)
    w = torch.zeros(M, K, dtype=torch.float64)
    for m in range(M):
        z = [scale * v for v in l[m].tolist()]
        out = [not v > -math.inf for v in z]
        top = max((v for v, o in zip(z, out) if not o), default=0.0)
        if score == "softmax":
            s = [0.0 if o else 1.0 if v == top else math.exp(v - top) for v, o in zip(z, out)]
            total = sum(s) or 1.0
            s = [v / total for v in s]
        else:
            s = [0.0 if o else 1 / (1 + math.exp(-v)) if v > -700 else 0.0
                 for v, o in zip(z, out)]
        v = s if b is None else [x + y for x, y in zip(s, b.tolist())]
        order = z if b is None else v
        gs = E // groups
        values = []
        for g in range(groups):
            live = [e for e in range(g * gs, (g + 1) * gs) if not out[e]]
            if not live:
                values.append(-math.inf)
            elif group_top == 1:
                values.append(max(order[e] for e in live))
            else:
                values.append(sum(sorted((v[e] for e in live), reverse=True)[:2]))
        kept = sorted(range(groups), key=lambda g: (-values[g], g))[:keep]
        cand = [e for g in kept for e in range(g * gs, (g + 1) * gs)]
        chosen = sorted(cand, key=lambda e: (out[e], -order[e] if not out[e] else 0.0, e))[:K]
        p = [s[e] for e in chosen]
        d = sum(p) if renorm else 1.0
        idx[m] = torch.tensor(chosen, dtype=torch.int32)
        if d > 0:
            w[m] = torch.tensor([x / d * routed for x in p])
    return idx, w


# ------------------------------------------------------------------ norm
def e4m3(v):
    """Nearest e4m3 value, ties to even, of |v| <= 448."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    # log2 may round up to the next integer just below a power of two
    e = torch.where(torch.exp2(e) > v.abs().clamp(min=2.0 ** -6), e - 1, e)
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def add_rmsnorm(x, gamma, eps, residual=None, q=None, group=0):
    """dict of r (in the residual's type), y, codes, scales (fp64)."""
    r = x
    if residual is not None:
        r = (x.float() + residual.float()).to(residual.dtype)
    d, g = r.double(), gamma.double()
    inv = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    out = {"r": r, "y": d * inv * g}
    if q:
        M, H = x.shape
        top = 127.0 if q == "int8" else 448.0
        t = d * g
        gs = group or H
        a = torch.nn.functional.pad(t.abs(), (0, -H % gs)).view(M, -1, gs).amax(-1)
        cols = a.repeat_interleave(gs, 1)[:, :H]
        v = t * top / torch.where(cols > 0, cols, 1.0)
        out["codes"] = torch.round(v) if q == "int8" else e4m3(v)
        out["scales"] = a * inv / top
    return out


# ------------------------------------------------------------------ linear
def pack(codes, bits):
    """Codes [out][in] as int32 words: each row one little-endian bit stream."""
    o, i = codes.shape
    bit = (codes.to(torch.int64)[..., None] >> torch.arange(bits, device=codes.device)) & 1
    bit = bit.view(o, i * bits // 32, 32) << torch.arange(32, device=codes.device)
    w = bit.sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32).contiguous()


def matrix(out_dim, in_dim, bits, G, gen, mx=False, scale=0.02):
    """A random packed matrix: dict of w, s, b (library operands) and dense (fp64)."""
    dev = gen.device
    q = torch.randint(0, 2 ** bits, (out_dim, in_dim), device=dev, generator=gen)
    if mx:
        s = torch.randint(119, 124, (out_dim, in_dim // G), device=dev, generator=gen)
        val = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=dev)[q]
        dense = val.view(out_dim, -1, G) * torch.exp2(s.double() - 127)[..., None]
        return dict(w=pack(q, 4), s=s.to(torch.uint8), b=None, q=q,
                    dense=dense.view(out_dim, in_dim), spread=dense.abs().view(out_dim, in_dim))
    u = torch.rand(out_dim, in_dim // G, device=dev, generator=gen)
    s = (scale * 5 / 2 ** bits * (0.5 + u)).to(torch.bfloat16)
    u = torch.rand(out_dim, in_dim // G, device=dev, generator=gen)
    b = (-scale * 2.5 * (0.5 + u)).to(torch.bfloat16)
    sq = q.double().view(out_dim, -1, G) * s.double()[..., None]
    bb = b.double()[..., None]
    return dict(w=pack(q, bits), s=s, b=b, q=q, dense=(sq + bb).view(out_dim, in_dim),
                spread=(sq.abs() + bb.abs()).view(out_dim, in_dim))


def act(v, name):
    F = torch.nn.functional
    return {"none": lambda a: a, "silu": F.silu, "gelu": F.gelu, "relu": F.relu,
            "gelu_tanh": lambda a: F.gelu(a, approximate="tanh"),
            "sigmoid": torch.sigmoid}[name](v)


def dequant_x(x, scales=None, group=0):
    d = x.double() if x.dtype != torch.float8_e4m3fn else x.float().double()
    if scales is None:
        return d
    s = scales.double()
    return d * (s.repeat_interleave(group, 1)[:, :x.shape[1]] if group else s)
