"""binary64 reference of the mixture-of-experts entry points (numpy / torch on
the CPU, written from the definitions in include/qz.h) and input makers."""
from __future__ import annotations

import math

import numpy as np
import torch

HALF_BF16 = 2.0 ** -8  # half a bf16 step, relative to the value
HALF_F32 = 2.0 ** -24
HALF_E4M3 = 2.0 ** -4


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


def e4m3_table():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where(b > 127, -v, v)


def e2m1_table():
    v = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    return np.concatenate([v, -v])


def decode_scale(amax):
    """g = RN32(amax / 2688)"""
    return (amax.float() / torch.tensor(2688.0)).double()


def linear_sf(sf, rows, kv, swizzled):
    """[rows, kv] scale bytes of one region."""
    b = sf.cpu().numpy().reshape(-1)
    if not swizzled:
        return b[: rows * kv].reshape(rows, kv)
    r, k = np.arange(rows)[:, None], np.arange(kv)[None, :]
    at = ((r // 128) * ((kv + 3) // 4) + k // 4) * 512 + ((r % 32) * 4 + (r % 128) // 32) * 4 + k % 4
    return b[at]


def decode(q, sf, cols, nvfp4, swizzled, g=None):
    """binary64 [rows, cols] of one quantized matrix; g: its second-level scale(s)."""
    rows = q.shape[0]
    q = q.cpu().numpy().view(np.uint8)
    if nvfp4:
        s = e4m3_table()[linear_sf(sf, rows, cols // 16, swizzled)].repeat(16, 1)
        t = e2m1_table()
        v = np.stack([t[q & 15], t[q >> 4]], -1).reshape(rows, cols)
    else:
        s = (2.0 ** (linear_sf(sf, rows, cols // 32, swizzled) - 127.0)).repeat(32, 1)
        v = e4m3_table()[q]
    out = torch.from_numpy(v * s)
    return out if g is None else out * g


def act(kind, z):
    if kind == 1:
        return z.clamp(min=0)
    if kind == 2:
        return z * torch.sigmoid(z)
    if kind == 3:
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def act_grad(kind, z):
    z = z.clone().requires_grad_()
    return torch.autograd.grad(act(kind, z).sum(), z)[0] if kind != 0 else torch.ones_like(z)


def clean(x):
    x = torch.where(torch.isnan(x), -torch.inf, x.double())
    return x.clamp(max=float(np.finfo(np.float32).max))


def scores(x, sigmoid):
    if sigmoid:
        return torch.where(x > -torch.inf, torch.sigmoid(x), 0.0)
    m = x.amax(-1, keepdim=True)
    p = torch.where(x > -torch.inf, torch.exp(x - torch.where(m > -torch.inf, m, 0.0)), 0.0)
    return p / p.sum(-1, keepdim=True).clamp(min=1e-300)


def route(logits, k, sigmoid, bias, groups, top, renorm, scale):
    """ids and binary64 weights of the router's definition, one token at a time."""
    x = clean(logits.cpu())
    s = scores(x, sigmoid)
    T, E = x.shape
    ids = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    v = x if bias is None else s + bias.cpu().double()
    gv = s if bias is None else v
    size = E // groups
    for t in range(T):
        value = v[t].numpy().copy()
        masked = ~(x[t].numpy() > -np.inf) | np.isnan(value) | (value == -np.inf)
        if groups > 1 and top < groups:
            of = np.where(masked, -np.inf, gv[t].numpy())
            best = []
            for g in range(groups):
                u = np.sort(of[g * size:(g + 1) * size])[::-1][:2]
                u = u[u > -np.inf]
                best.append(u.sum() if len(u) else -np.inf)
            keep = sorted(range(groups), key=lambda g: (-best[g], g))[:top]
            for g in range(groups):
                if g not in keep:
                    masked[g * size:(g + 1) * size] = True
        order = sorted((i for i in range(E) if not masked[i]), key=lambda i: (-value[i], i))[:k]
        ids[t, :len(order)] = order
        c = s[t].numpy()[order]
        if renorm:
            if sigmoid:
                c = c / c.sum() if c.sum() > 0 else c * 0
            else:
                z = x[t].numpy()[order]
                c = np.exp(z - z.max()) if len(z) else z
                c = c / c.sum() if len(z) else c
        w[t, :len(order)] = c * scale
    return ids, w


def plan(ids, E, align):
    """offsets, counts, rows, slots by a stable sort."""
    T, k = ids.shape
    n = T * k
    total = (n + min(E, n) * (align - 1) + align - 1) // align * align
    offsets, counts = np.zeros(E + 1, np.int64), np.zeros(E, np.int64)
    rows, slots = np.full(total, -1, np.int64), np.full((T, k), -1, np.int64)
    at = 0
    for e in range(E):
        offsets[e] = at
        pairs = np.argwhere(ids == e)
        counts[e] = len(pairs)
        for i, (t, j) in enumerate(pairs):
            rows[at + i], slots[t, j] = t, at + i
        at += -(-len(pairs) // align) * align
    offsets[E] = at
    return offsets, counts, rows, slots


def split(g, E, total, empty=()):
    """Uneven counts of `total` rows over E experts, those in `empty` without any."""
    share = torch.rand(E, generator=g) ** 2 + 0.01
    for e in empty:
        share[e] = 0
    counts = (share / share.sum() * total).long()
    left = [e for e in range(E) if e not in empty]
    counts[left[0]] += total - int(counts.sum())
    return counts


def close(got, want, tol, what):
    got, want = got.detach().double().cpu(), want.double().cpu()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0].item()} against {want[bad][0].item()}, worst excess "
                           f"{((got - want).abs() / tol)[bad].max().item():.3g} times the tolerance")
