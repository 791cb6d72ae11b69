"""The mixture-of-experts layer's operators as a user's program calls them, with
their plain forms: routing tokens to experts, the experts' block-scaled matrix
products (forward, weight gradient, activation gradient) and the weighted
gather that ends the layer, with its gradient.

``listed()`` names the cases, ``prepare`` makes one case's inputs from a seed,
``run`` makes one pass (the library's calls where ``own`` is true, elementary
torch operations otherwise), ``exact`` evaluates the definition in binary64 and
``work`` counts the bytes and operations that a pass cannot do without.
"""
import math

import numpy as np
import torch

own = False

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one generated token through a 128-expert layer's router: the latency of a decode step
        dict(name="route_token", op="route", T=1, E=128, k=8, score="softmax", bias=False, groups=1, top_groups=1,
             renorm=True, scale=1.0, dtype="bf16", align=1),
        # prefill through a router with sigmoid scores, a balancing bias and 8 groups of experts
        dict(name="route_prefill", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, renorm=True, scale=2.5, dtype="fp32", align=128),
        # the router's backward pass in a training step
        dict(name="route_backward", op="route_grad", T=8192, E=128, k=8, score="softmax", renorm=True, scale=1.0,
             dtype="bf16"),
        # one generated token: the gate|up product of its 8 experts, quantized for the down product
        dict(name="product_token", op="product", fmt="mxfp8", T=1, E=128, k=8, N=768, K=2048, gather=True, gated=True,
             act="silu", bias=False, residual=False, q=True),
        # prefill of 4096 tokens: gate|up with SwiGLU, rows gathered from the quantized tokens
        dict(name="product_prefill", op="product", fmt="mxfp8", T=4096, E=128, k=8, N=768, K=2048, gather=True,
             gated=True, act="silu", bias=False, residual=False, q=True),
        # a long prefill on the rank that holds 16 experts: the largest product, bound by the tensor cores
        dict(name="product_long", op="product", fmt="nvfp4", T=8192, E=16, k=4, N=4096, K=2048, gather=True,
             gated=False, act="none", bias=False, residual=False, q=False),
        # a small layer of odd sizes with biases, a GELU and a residual; one expert gets nothing
        dict(name="product_odd", op="product", fmt="mxfp8", T=77, E=5, k=2, N=416, K=352, gather=False, gated=False,
             act="gelu", bias=True, residual=True, q=False),
        # weight gradients of a training step in MXFP8, over each expert's uneven rows
        dict(name="weight_grad", op="weight_grad", fmt="mxfp8", T=8192, E=32, k=2, N=1536, K=2048, out="fp32"),
        # the backward pass of SwiGLU with the bias gradients
        dict(name="activation_grad", op="act_grad", T=4096, E=128, k=8, N=768, gated=True, act="silu"),
        # the end of the layer: each token's weighted sum of its experts' rows plus the residual
        dict(name="combine_prefill", op="combine", T=4096, E=128, k=8, H=2048, residual=True),
        # the same for a few tokens of a decode step
        dict(name="combine_decode", op="combine", T=16, E=128, k=8, H=4096, residual=True),
        # its backward pass: the scattered rows' gradients and the routing weights' gradients
        dict(name="combine_backward", op="dispatch", T=4096, E=128, k=8, H=2048, weighted=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "product", "product", "product", "weight_grad", "act_grad",
                     "combine", "dispatch"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.choice([2, 5, 8, 16, 31, 32]) if groups > 1 else rng.choice([8, 17, 60, 64, 128, 256, 384])
        top = rng.randint(max(1, groups // 2), groups)
        k = min(rng.choice([1, 2, 4, 6, 8]), top * (E // groups))
        c = dict(op=op, T=_log(rng, 1, 16384), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                 renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["bf16", "fp32"]))
        if op == "route":
            c.update(bias=rng.random() < 0.5, groups=groups, top_groups=top, align=rng.choice([1, 16, 128]))
        return c
    E = rng.choice([1, 3, 8, 16, 60, 128])
    k = min(E, rng.choice([1, 2, 4, 8]))
    if op == "product":
        T = _log(rng, 1, 4096)
        gated = rng.random() < 0.5
        q = rng.random() < 0.4
        return dict(op=op, fmt=rng.choice(["mxfp8", "nvfp4"]), T=T, E=E, k=k,
                    N=rng.randint(1, 24) * 32 if q or gated else rng.randint(2, 192) * 8, K=rng.randint(1, 64) * 32,
                    gather=rng.random() < 0.6, gated=gated, act=rng.choice(["silu", "gelu"] if gated else
                                                                           ["none", "relu", "silu", "gelu"]),
                    bias=rng.random() < 0.4, residual=rng.random() < 0.4, q=q)
    if op == "weight_grad":
        return dict(op=op, fmt=rng.choice(["mxfp8", "nvfp4"]), T=_log(rng, 16, 8192), E=min(E, 32), k=min(k, 2),
                    N=rng.randint(2, 192) * 8, K=rng.randint(2, 256) * 8, out=rng.choice(["fp32", "bf16"]))
    if op == "act_grad":
        gated = rng.random() < 0.5
        return dict(op=op, T=_log(rng, 1, 4096), E=E, k=k, N=rng.randint(1, 96) * 8, gated=gated,
                    act=rng.choice(["silu", "gelu"] if gated else ["relu", "silu", "gelu"]))
    c = dict(op=op, T=_log(rng, 1, 4096), E=E, k=k, H=rng.randint(1, 256) * 8)
    c["residual" if op == "combine" else "weighted"] = rng.random() < 0.7
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _logits(g, T, E):
    """Token logits with a popularity of each expert, so that the experts' shares are uneven."""
    return _randn(g, T, E) * 1.2 + _randn(g, 1, E) * 0.4


def _slots_of(T, k, E, align):
    n = T * k
    return (n + min(E, n) * (align - 1) + align - 1) // align * align


def _order(ids, E, align):
    """The experts' order of the chosen pairs: offsets [E+1], counts [E], rows [slots], slots [T, k]."""
    T, k = ids.shape
    flat = ids.reshape(-1).to(torch.int64)
    live = flat >= 0
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    counts.scatter_add_(0, torch.where(live, flat, E), torch.ones_like(flat))
    counts = counts[:E]
    padded = (counts + align - 1) // align * align
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum(padded, 0)
    before = torch.cumsum(counts, 0) - counts
    key, by = torch.sort(torch.where(live, flat, E), stable=True)
    at = torch.arange(T * k, device=ids.device)
    e = torch.clamp(key, max=E - 1)
    place = torch.where(key < E, at - before[e] + offsets[e], -1)
    slots = torch.empty(T * k, dtype=torch.int64, device=ids.device)
    slots[by] = place
    n = _slots_of(T, k, E, align)
    rows = torch.full((n + 1,), -1, dtype=torch.int64, device=ids.device)
    rows[torch.where(place >= 0, place, n)] = torch.div(by, k, rounding_mode="floor")
    return (offsets.to(torch.int32), counts.to(torch.int32), rows[:n].to(torch.int32),
            slots.reshape(T, k).to(torch.int32))


def _mxfp8(x):
    """e4m3 codes and E8M0 bytes of fp32 [..., cols] in blocks of 32 (the smallest exponent that holds the block)."""
    b = x.unflatten(-1, (-1, 32))
    m, e = torch.frexp(b.abs().amax(-1))
    byte = torch.where(m > 0, e + 118 + (m > 0.875), 0).clamp(0, 254)
    q = torch.ldexp(b, (127 - byte).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.flatten(-2).view(torch.uint8), byte.to(torch.uint8)


def _nvfp4(x, amax):
    """Packed e2m1 codes and E4M3 bytes of fp32 [..., cols] in blocks of 16; amax broadcasts over [..., 1]."""
    g = amax / 2688.0
    b = x.unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) / 6.0 / g).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = s.to(torch.float32).unsqueeze(-1) * g.unsqueeze(-1)
    y = torch.where(step > 0, b / step, 0.0).flatten(-2)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(y.abs(), edges).to(torch.uint8) + 8 * (y < 0).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _swizzle(sf):
    """Scale bytes [..., rows, kv] as each matrix's swizzled 128x4 region (flat, zero padded)."""
    rows, kv = sf.shape[-2:]
    sf = torch.nn.functional.pad(sf, (0, -kv % 4, 0, -rows % 128))
    t = sf.unflatten(-1, (-1, 4)).unflatten(-3, (-1, 4, 32))  # [..., row tile, 4, 32, column tile, 4]
    return t.movedim(-2, -4).transpose(-3, -2).flatten(-5)


def _unswizzle(region, rows, kv):
    t = region.unflatten(-1, ((rows + 127) // 128, (kv + 3) // 4, 32, 4, 4))
    t = t.transpose(-3, -2).movedim(-4, -2)
    return t.flatten(-5, -3).flatten(-2)[..., :rows, :kv]


def _quantize(fmt, x, per_row):
    if fmt == "mxfp8":
        q, sf = _mxfp8(x)
        return q.contiguous(), sf.contiguous(), None
    amax = x.abs().amax(-1, keepdim=True) if per_row else x.abs().amax((-2, -1), keepdim=True)
    q, sf = _nvfp4(x, amax)
    return q.contiguous(), sf.contiguous(), amax.flatten().contiguous()


def _weights(g, fmt, E, N, K):
    q, sf, amax = _quantize(fmt, _randn(g, E, N, K) * 0.02, False)
    return q, _swizzle(sf).contiguous(), amax


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    if op in ("route", "route_grad"):
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s = dict(case=c, logits=_logits(g, c["T"], c["E"]).to(dt))
        if op == "route":
            s["bias"] = _randn(g, c["E"]) * 0.1 if c["bias"] else None
        else:
            s["ids"] = torch.topk(s["logits"].float(), c["k"], dim=-1).indices.to(torch.int32)
            s["dweights"] = _randn(g, c["T"], c["k"])
        return s
    T, E, k = c["T"], c["E"], c["k"]
    z = _logits(g, T, E)
    if E > 4 and E < 16:
        z[:, E // 2] = -100.0  # an expert that no token reaches
    ids = torch.topk(z, k, dim=-1).indices.to(torch.int32)
    align = 128 if op in ("weight_grad", "act_grad", "dispatch") else 1
    offsets, counts, rows, slots = _order(ids, E, align)
    S = rows.numel()
    s = dict(case=c, offsets=offsets, counts=counts, rows=rows, slots=slots)
    s["most"] = int(counts.max())
    bf = torch.bfloat16
    if op == "product":
        N, K = c["N"], c["K"]
        s["x"] = _quantize(c["fmt"], _randn(g, T if c["gather"] else S, K), True)
        s["w"] = _weights(g, c["fmt"], E, N, K)
        s["up"] = _weights(g, c["fmt"], E, N, K) if c["gated"] else None
        s["bias"] = (_randn(g, E, N) * 0.2).to(bf) if c["bias"] else None
        s["up_bias"] = (_randn(g, E, N) * 0.2).to(bf) if c["bias"] and c["gated"] else None
        s["residual"] = _randn(g, S, N).to(bf) if c["residual"] else None
        s["out"] = torch.zeros(S, N, dtype=bf, device="cuda")
        s["q"] = torch.zeros(S, N, dtype=torch.uint8, device="cuda") if c["q"] else None
        s["sf"] = torch.zeros(S, N // 32, dtype=torch.uint8, device="cuda") if c["q"] else None
    elif op == "weight_grad":
        live = (rows >= 0).float().unsqueeze(1)
        s["dz"] = s["xt"] = None
        for name, n in (("dz", c["N"]), ("xt", c["K"])):
            q, sf, amax = _quantize(c["fmt"], (_randn(g, S, n) * live).T.contiguous(), False)
            s[name] = (q, _swizzle(sf).contiguous(), amax)
        s["out"] = torch.zeros(E, c["N"], c["K"], dtype=torch.float32 if c["out"] == "fp32" else bf, device="cuda")
    elif op == "act_grad":
        w = 2 * c["N"] if c["gated"] else c["N"]
        s["pre"] = (_randn(g, S, w) * 1.5).to(bf)
        s["dout"] = _randn(g, S, c["N"]).to(bf)
        s["dpre"] = torch.zeros(S, w, dtype=bf, device="cuda")
        s["dbias"] = torch.zeros(E, w, dtype=torch.float32, device="cuda")
    else:
        w = torch.softmax(_randn(g, T, k), -1)
        if op == "combine":
            s["y"] = _randn(g, S, c["H"]).to(bf)
            s["weights"] = w
            s["residual"] = _randn(g, T, c["H"]).to(bf) if c["residual"] else None
            s["out"] = torch.zeros(T, c["H"], dtype=bf, device="cuda")
        else:
            s["x"] = _randn(g, T, c["H"]).to(bf)
            s["weights"] = w if c["weighted"] else None
            s["y"] = _randn(g, S, c["H"]).to(bf) if c["weighted"] else None
            s["out"] = torch.zeros(S, c["H"], dtype=bf, device="cuda")
            s["dots"] = torch.zeros(T, k, dtype=torch.float32, device="cuda") if c["weighted"] else None
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _decode(fmt, q, sf, amax=None):
    """fp32 values of quantized [..., rows, cols] with linear scales [..., rows, kv]; amax broadcasts."""
    if fmt == "mxfp8":
        v = q.view(torch.float8_e4m3fn).to(torch.float32).unflatten(-1, (-1, 32))
        return torch.ldexp(v, sf.to(torch.int32).unsqueeze(-1) - 127).flatten(-2)
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=q.device)
    v = torch.stack((table[(q & 15).long()], table[(q >> 4).long()]), -1).flatten(-2)
    s = sf.contiguous().view(torch.float8_e4m3fn).to(torch.float32) * (amax / 2688.0)
    return (v.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _column(amax):
    return None if amax is None else amax.unsqueeze(-1)


def _stacked(w, E, fmt, N, K):
    q, region, amax = w
    sf = _unswizzle(region, N, K // (32 if fmt == "mxfp8" else 16))
    return _decode(fmt, q, sf, None if amax is None else amax.reshape(E, 1, 1))


def _act(name, x):
    if name == "silu":
        return x / (1 + torch.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return torch.clamp(x, min=0.0) if name == "relu" else x


def _act_grad(name, x):
    if name == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    if name == "gelu":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (x + 0.044715 * x * x * x))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * a * (1 + 3 * 0.044715 * x * x)
    return (x > 0).to(x.dtype) if name == "relu" else torch.ones_like(x)


def _experts(s, E):
    """Per expert, the slots of its rows padded to the longest expert, and which of them are live: [E, most]."""
    at = torch.arange(s["most"], device="cuda")
    live = at < s["counts"].long().unsqueeze(1)
    return torch.where(live, s["offsets"][:E].long().unsqueeze(1) + at, 0), live


def _plain_route(s):
    c, x = s["case"], s["logits"].to(torch.float64)
    score = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.exp(x - x.amax(-1, keepdim=True))
    if c["score"] == "softmax":
        score = score / score.sum(-1, keepdim=True)
    by = score + s["bias"].to(torch.float64) if s["bias"] is not None else x
    if c["groups"] > 1:
        best = (by if s["bias"] is not None else score).unflatten(-1, (c["groups"], -1))
        best = torch.topk(best, min(2, best.shape[-1]), dim=-1).values.sum(-1)
        at = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, at, True)
        by = torch.where(keep.repeat_interleave(c["E"] // c["groups"], 1), by, -torch.inf)
    ids = torch.sort(by, dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    w = torch.gather(score, 1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    ids = ids.to(torch.int32)
    offsets, counts, rows, slots = _order(ids, c["E"], c["align"])
    return dict(ids=ids, weights=(w * c["scale"]).to(torch.float32), offsets=offsets, counts=counts, rows=rows,
                slots=slots)


def _plain_route_grad(s):
    c, x, ids, g = s["case"], s["logits"].to(torch.float32), s["ids"].long(), s["dweights"] * s["case"]["scale"]
    if c["score"] == "softmax":
        p = torch.exp(x - x.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        w = torch.gather(p, 1, ids)
        if c["renorm"]:
            w = w / w.sum(-1, keepdim=True)
            d = torch.zeros_like(x).scatter_(1, ids, w * (g - (g * w).sum(-1, keepdim=True)))
        else:
            d = torch.zeros_like(x).scatter_(1, ids, w * g) - p * (g * w).sum(-1, keepdim=True)
    else:
        v = torch.gather(x, 1, ids)
        w, rest = 1 / (1 + torch.exp(-v)), 1 / (1 + torch.exp(v))
        if c["renorm"]:
            total = w.sum(-1, keepdim=True)
            g = (g - (g * w).sum(-1, keepdim=True) / total) / total
        d = torch.zeros_like(x).scatter_(1, ids, g * w * rest)
    return dict(dlogits=d.to(s["logits"].dtype))


def _plain_product(s):
    c, fmt = s["case"], s["case"]["fmt"]
    E, N, K = c["E"], c["N"], c["K"]
    slot, live = _experts(s, E)
    x = _decode(fmt, s["x"][0], s["x"][1], _column(s["x"][2]))
    a = x[s["rows"].long()[slot]] if c["gather"] else x[slot]
    z = torch.bmm(a, _stacked(s["w"], E, fmt, N, K).transpose(1, 2))
    if s["bias"] is not None:
        z = z + s["bias"].to(torch.float32).unsqueeze(1)
    h = _act(c["act"], z)
    if c["gated"]:
        u = torch.bmm(a, _stacked(s["up"], E, fmt, N, K).transpose(1, 2))
        if s["up_bias"] is not None:
            u = u + s["up_bias"].to(torch.float32).unsqueeze(1)
        h = h * u
    flat = torch.zeros_like(s["out"], dtype=torch.float32)
    flat[slot[live]] = h[live]
    if s["residual"] is not None:
        flat = flat + s["residual"].to(torch.float32)
    out = flat.to(torch.bfloat16)
    if not c["q"]:
        return dict(out=out)
    q, sf = _mxfp8(out.to(torch.float32))
    return dict(out=out, q=q.view(torch.float8_e4m3fn), sf=sf.view(torch.float8_e8m0fnu))


def _plain_weight_grad(s):
    c, fmt = s["case"], s["case"]["fmt"]
    S = s["rows"].numel()
    kv = S // (32 if fmt == "mxfp8" else 16)
    slot, live = _experts(s, c["E"])
    dz, x = (_decode(fmt, s[n][0], _unswizzle(s[n][1], m, kv), s[n][2]).T for n, m in (("dz", c["N"]), ("xt", c["K"])))
    d = torch.bmm((dz[slot] * live.unsqueeze(-1)).transpose(1, 2), x[slot])
    return dict(dw=d.to(s["out"].dtype))


def _plain_act_grad(s):
    c, N = s["case"], s["case"]["N"]
    pre, d = s["pre"].to(torch.float32), s["dout"].to(torch.float32)
    z = pre[:, :N]
    dz = d * _act_grad(c["act"], z)
    if c["gated"]:
        dz = torch.cat((dz * pre[:, N:], d * _act(c["act"], z)), -1)
    dz = torch.where((s["rows"] >= 0).unsqueeze(1), dz, 0.0)
    slot, live = _experts(s, c["E"])
    return dict(dpre=dz.to(torch.bfloat16), dbias=(dz[slot] * live.unsqueeze(-1)).sum(1))


def _plain_combine(s):
    y = s["y"].to(torch.float32)[s["slots"].long()]
    y = (y * s["weights"].unsqueeze(-1)).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].to(torch.float32)
    return dict(out=y.to(torch.bfloat16))


def _plain_dispatch(s):
    c, at = s["case"], s["slots"].long().reshape(-1)
    x = s["x"].to(torch.float32)
    each = x.unsqueeze(1) * (s["weights"].unsqueeze(-1) if c["weighted"] else torch.ones(c["T"], c["k"], 1, device="cuda"))
    out = torch.zeros_like(s["out"])
    out[at] = each.reshape(-1, c["H"]).to(torch.bfloat16)
    if not c["weighted"]:
        return dict(out=out)
    return dict(out=out, dots=(s["y"].to(torch.float32)[s["slots"].long()] * x.unsqueeze(1)).sum(-1))


_PLAIN = dict(route=_plain_route, route_grad=_plain_route_grad, product=_plain_product,
              weight_grad=_plain_weight_grad, act_grad=_plain_act_grad, combine=_plain_combine,
              dispatch=_plain_dispatch)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own(s):
    import nvfp4_quantization_moe_b200 as qz
    c = s["case"]
    op = c["op"]
    acts = dict(none=qz.ACT_NONE, relu=qz.ACT_RELU, silu=qz.ACT_SILU, gelu=qz.ACT_GELU)
    if op in ("route", "route_grad"):
        score = qz.SCORE_SIGMOID if c["score"] == "sigmoid" else qz.SCORE_SOFTMAX
        if op == "route_grad":
            return dict(dlogits=qz.route_experts_grad(s["logits"], s["ids"], s["dweights"], score=score,
                                                      renormalize=c["renorm"], scale=c["scale"]))
        ids, weights = qz.route_experts(s["logits"], c["k"], score=score, bias=s["bias"], n_groups=c["groups"],
                                        top_groups=c["top_groups"], renormalize=c["renorm"], scale=c["scale"])
        plan = qz.plan_experts(ids, c["E"], align=c["align"])
        return dict(ids=ids, weights=weights, offsets=plan.offsets, counts=plan.counts, rows=plan.rows,
                    slots=plan.slots)
    fmt = qz.FMT_NVFP4 if c.get("fmt") == "nvfp4" else qz.FMT_MXFP8
    if op == "product":
        qz.expert_product(fmt, s["x"], s["w"], s["offsets"], s["counts"], s["out"],
                          rows=s["rows"] if c["gather"] else None, up=s["up"], bias=s["bias"], up_bias=s["up_bias"],
                          activation=acts[c["act"]], residual=s["residual"], q=s["q"], sf=s["sf"])
        if not c["q"]:
            return dict(out=s["out"])
        return dict(out=s["out"], q=s["q"].view(torch.float8_e4m3fn), sf=s["sf"].view(torch.float8_e8m0fnu))
    if op == "weight_grad":
        qz.expert_weight_grad(fmt, s["dz"], s["xt"], s["offsets"], s["counts"], s["out"])
        return dict(dw=s["out"])
    if op == "act_grad":
        qz.expert_activation_grad(s["dout"], s["pre"], s["offsets"], s["counts"], s["dpre"],
                                  activation=acts[c["act"]], gated=c["gated"], dbias=s["dbias"])
        return dict(dpre=s["dpre"], dbias=s["dbias"])
    if op == "combine":
        qz.combine_experts(s["y"], s["slots"], s["out"], weights=s["weights"], residual=s["residual"])
        return dict(out=s["out"])
    qz.dispatch_experts(s["x"], s["slots"], s["rows"], s["out"], weights=s["weights"], other=s["y"], dots=s["dots"])
    return dict(out=s["out"], dots=s["dots"]) if c["weighted"] else dict(out=s["out"])


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# work and the definition in binary64
# ---------------------------------------------------------------------------

def work(case):
    c = case
    op, T, E, k = c["op"], c["T"], c["E"], c["k"]
    if op in ("route", "route_grad"):
        each = 2 if c["dtype"] == "bf16" else 4
        if op == "route_grad":
            return dict(bytes=2 * T * E * each + T * k * 8, flops=8 * T * E)
        return dict(bytes=T * E * each + (4 * E if c["bias"] else 0) + T * k * 12 + 8 * E
                    + 4 * _slots_of(T, k, E, c["align"]), flops=T * E * (8 + k))
    S = T * k
    if op == "product":
        b, per = (1, 32) if c["fmt"] == "mxfp8" else (0.5, 16)
        N, K, ways = c["N"], c["K"], 2 if c["gated"] else 1
        rows = T if c["gather"] else S
        n = (rows + min(E, S) * N * ways) * K * (b + 1 / per) + S * N * 2 + 4 * S
        n += S * N * 2 if c["residual"] else 0
        n += min(E, S) * N * 2 * ways if c["bias"] else 0
        n += S * N * (1 + 1 / 32) if c["q"] else 0
        return dict(bytes=int(n), flops=2 * S * N * K * ways)
    if op == "weight_grad":
        b, per = (1, 32) if c["fmt"] == "mxfp8" else (0.5, 16)
        return dict(bytes=int(S * (c["N"] + c["K"]) * (b + 1 / per)
                              + E * c["N"] * c["K"] * (4 if c["out"] == "fp32" else 2)),
                    flops=2 * S * c["N"] * c["K"])
    if op == "act_grad":
        w = 2 if c["gated"] else 1
        return dict(bytes=S * c["N"] * 2 * (1 + 2 * w) + E * c["N"] * w * 4, flops=10 * S * c["N"] * w)
    if op == "combine":
        return dict(bytes=(S + T * (2 if c["residual"] else 1)) * c["H"] * 2 + S * 8, flops=2 * S * c["H"])
    pad = _slots_of(T, k, E, 128)
    return dict(bytes=(T + pad + (S if c["weighted"] else 0)) * c["H"] * 2 + S * (12 if c["weighted"] else 4) + 4 * pad,
                flops=(3 if c["weighted"] else 0) * S * c["H"])


def _sigma64(v):
    return torch.where(v >= 0, 1 / (1 + torch.exp(-v.abs())), torch.exp(-v.abs()) / (1 + torch.exp(-v.abs())))


def _f64(fmt, q, sf, g):
    """binary64 values of [rows, cols] codes with linear scales [rows, kv]; g: the second-level scales or None."""
    bits = np.arange(256)
    if fmt == "mxfp8":
        exp, man = (bits >> 3) & 15, bits & 7
        mag = np.where(exp == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (exp - 10.0))
        value = torch.from_numpy(np.where(bits > 127, -mag, mag)).cuda()[q.long()]
        scale = torch.from_numpy(2.0 ** (bits - 127.0)).cuda()[sf.long()]
        return value * scale.repeat_interleave(32, -1)
    mag = np.where(bits & 6, (2.0 + (bits & 1)) * 2.0 ** (((bits >> 1) & 3) - 2.0), (bits & 1) * 0.5)
    value = torch.from_numpy(np.where(bits & 8, -mag, mag)).cuda()
    both = torch.stack((value[(q & 15).long()], value[(q >> 4).long()]), -1).reshape(q.shape[0], -1)
    exp, man = (bits >> 3) & 15, bits & 7
    scale = torch.from_numpy(np.where(exp == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (exp - 10.0))).cuda()[sf.long()]
    return both * scale.repeat_interleave(16, -1) * g


def _linear64(region, rows, kv):
    """Linear scale bytes of one matrix, by the address of each byte in its swizzled region."""
    r = torch.arange(rows, device="cuda").unsqueeze(1)
    j = torch.arange(kv, device="cuda")
    at = ((r // 128) * ((kv + 3) // 4) + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4
    return region.reshape(-1)[at]


def _act64(name, v, derivative=False):
    if name == "silu":
        s = _sigma64(v)
        return s + v * s * _sigma64(-v) if derivative else v * s
    if name == "gelu":
        b = 2 * math.sqrt(2 / math.pi)
        s = _sigma64(b * (v + 0.044715 * v ** 3))
        return s + v * s * (1 - s) * b * (1 + 0.134145 * v ** 2) if derivative else v * s
    if name == "relu":
        return (v > 0).double() if derivative else v * (v > 0)
    return torch.ones_like(v) if derivative else v


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "route":
        x = s["logits"].double()
        p = _sigma64(x) if c["score"] == "sigmoid" else torch.exp(x - torch.logsumexp(x, -1, keepdim=True))
        pick = _plain_route(s)["ids"].long()  # whole numbers: compared with the plain form's
        w = torch.gather(p, 1, pick)
        w = (w / w.sum(-1, keepdim=True) if c["renorm"] else w) * c["scale"]
        return dict(ids=None, weights=w, offsets=None, counts=None, rows=None, slots=None)
    if op == "route_grad":
        x = s["logits"].double().requires_grad_()
        p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, -1)
        w = torch.gather(p, 1, s["ids"].long())
        w = (w / w.sum(-1, keepdim=True) if c["renorm"] else w) * c["scale"]
        return dict(dlogits=torch.autograd.grad(w, x, s["dweights"].double())[0])
    first, count, rows = s["offsets"].tolist(), s["counts"].tolist(), s["rows"].long()
    if op == "product":
        fmt, N, K = c["fmt"], c["N"], c["K"]
        kv = K // (32 if fmt == "mxfp8" else 16)

        def scale(a):
            return None if a is None else (a / 2688.0).double()

        q, sf, amax = s["x"]
        x = _f64(fmt, q, sf, None if amax is None else scale(amax).unsqueeze(1))
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            at = slice(first[e], first[e] + count[e])
            a = x[rows[at]] if c["gather"] else x[at]
            parts = []
            for w, b in ((s["w"], s["bias"]), (s["up"], s["up_bias"])):
                if w is None or not count[e]:
                    continue
                z = a @ _f64(fmt, w[0][e], _linear64(w[1][e], N, kv), scale(w[2][e]) if w[2] is not None else None).T
                parts.append(z if b is None else z + b[e].double())
            if parts:
                out[at] = _act64(c["act"], parts[0]) * (parts[1] if c["gated"] else 1.0)
        if s["residual"] is not None:
            out = out + s["residual"].double()
        return dict(out=out, q=None, sf=None) if c["q"] else dict(out=out)
    if op == "weight_grad":
        fmt, S = c["fmt"], rows.numel()
        kv = S // (32 if fmt == "mxfp8" else 16)
        dz, x = (_f64(fmt, s[n][0], _linear64(s[n][1], m, kv), None if s[n][2] is None else (s[n][2] / 2688.0).double())
                 for n, m in (("dz", c["N"]), ("xt", c["K"])))
        return dict(dw=torch.stack([dz[:, first[e]:first[e] + count[e]] @ x[:, first[e]:first[e] + count[e]].T
                                    for e in range(c["E"])]))
    if op == "act_grad":
        N, pre, d = c["N"], s["pre"].double(), s["dout"].double()
        dz = d * _act64(c["act"], pre[:, :N], True)
        if c["gated"]:
            dz = torch.cat((dz * pre[:, N:], d * _act64(c["act"], pre[:, :N])), -1)
        dz[rows < 0] = 0
        return dict(dpre=dz, dbias=torch.stack([dz[first[e]:first[e] + count[e]].sum(0) for e in range(c["E"])]))
    at = s["slots"].long()
    if op == "combine":
        out = torch.einsum("tk,tkh->th", s["weights"].double(), s["y"].double()[at])
        return dict(out=out if s["residual"] is None else out + s["residual"].double())
    x = s["x"].double()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        out[at[:, j]] = x if not c["weighted"] else x * s["weights"][:, j:j + 1].double()
    return dict(out=out) if not c["weighted"] else dict(out=out, dots=torch.einsum("th,tkh->tk", x, s["y"].double()[at]))
