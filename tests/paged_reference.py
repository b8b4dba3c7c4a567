"""Plain 64-bit definitions of the paged-cache operators and the row sampler,
and the error bounds their tests use."""
from __future__ import annotations

import math

import torch


def unit(dtype) -> float:
    """Half a step of a rounding to `dtype`, relative to the value."""
    return torch.finfo(dtype).eps / 2


U32 = 2.0 ** -24


def plan(ctx, new, page, tables, free, count, width, room, cap):
    """One step's plan from Python lists; returns a dict (tables and free are changed copies)."""
    tables = [list(r) for r in tables]
    free = list(free)
    pages = lambda n: -(-n // page)
    stack = free[:count]
    for b, n in enumerate(new):
        if n < 0:
            stack += tables[b][:pages(ctx[b])]
    grown = [0 if n < 0 else pages(ctx[b] + n) - pages(ctx[b]) for b, n in enumerate(new)]
    total = sum(max(n, 0) for n in new)
    fails = (any(c < 0 for c in ctx) or count < 0 or len(stack) > cap or sum(grown) > len(stack) or total > room
             or any(n >= 0 and pages(ctx[b] + n) > width for b, n in enumerate(new)))
    if fails:
        return {"tables": tables, "free": free, "left": count, "seq": list(ctx), "cu": [0] * (len(ctx) + 1),
                "slots": [-1] * room, "pos": [-1] * room, "failed": True}
    free[:len(stack)] = stack
    seq, cu, slots, pos = [], [0], [], []
    for b, n in enumerate(new):
        if n < 0:
            seq.append(0)
            cu.append(cu[-1])
            continue
        for i in range(grown[b]):
            tables[b][pages(ctx[b]) + i] = stack.pop()
        seq.append(ctx[b] + n)
        cu.append(cu[-1] + n)
        for p in range(ctx[b], ctx[b] + n):
            pos.append(p)
            slots.append(tables[b][p // page] * page + p % page)
    pad = room - len(slots)
    return {"tables": tables, "free": free, "left": len(stack), "seq": seq, "cu": cu, "slots": slots + [-1] * pad,
            "pos": pos + [-1] * pad, "failed": False}


def rope_table(n, hd, theta=10000.0):
    j = torch.arange(hd // 2, dtype=torch.float64)
    ang = torch.arange(n, dtype=torch.float64)[:, None] * theta ** (-2.0 * j / hd)
    return torch.stack([ang.cos(), ang.sin()], -1)


def norm_rotate(x, w, eps, cs, out_dtype):
    """(value, bound) of x [T, heads, hd] (any float type) normed, rotated by cs [T, hd/2, 2] and rounded once.

    Bound: the sum of squares of up to 128 values in fp32 is off by at most 16
    roundings (chains of 8 in a lane, then at most 5 shuffle sums), halved by
    the square root; square root, reciprocal, two products: 12 in all before
    the rotation, whose two products and sum add 3: 16 fp32 roundings of
    |a| + |b|, and the final rounding of the value."""
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    a, b = x[..., 0::2], x[..., 1::2]
    c, s = cs[:, None, :, 0].double(), cs[:, None, :, 1].double()
    y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    size = (a.abs() + b.abs()).repeat_interleave(2, -1)
    return y, unit(out_dtype) * y.abs() + 16 * U32 * size + torch.finfo(out_dtype).smallest_normal


def attention(q, k, v, n, seq, scale):
    """(value, bound) for one request: q [n, nh, hd], k and v [seq, nkv, hd].

    Bound, with A = sum_j p_j |v_j| (p normalised): a score is off by at most
    d = (hd + 8) fp32 roundings of scale * sum |q k|, plus 2^-21 for the
    exponent's product, subtraction and exponential; p_j and the sum move by a
    factor within exp(+-d) each; sums over the keys add a rounding each (a
    chain is at most as long as the keys, and merges of partial sums count
    among them); in 16 bits p is rounded once more; the output is rounded once."""
    nh, nkv, hd = q.shape[1], k.shape[1], q.shape[2]
    rep = nh // nkv
    dt = q.dtype
    q, k, v = q.double(), k.double(), v.double()
    out = torch.zeros(n, nh, hd, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for i in range(n):
        keys = min(seq, seq - n + i + 1)
        if keys <= 0:
            continue
        kk = k[:keys].repeat_interleave(rep, 1)
        vv = v[:keys].repeat_interleave(rep, 1)
        s = torch.einsum("hd,jhd->hj", q[i], kk) * scale
        size = torch.einsum("hd,jhd->hj", q[i].abs(), kk.abs()) * abs(scale)
        p = torch.softmax(s, -1)
        out[i] = torch.einsum("hj,jhd->hd", p, vv)
        A = torch.einsum("hj,jhd->hd", p, vv.abs())
        d = (hd + 8) * U32 * size.amax(-1) + 2.0 ** -21
        rel = 2 * d.expm1() + (2 * keys + 16) * U32 + (unit(dt) if dt != torch.float32 else 0.0)
        tol[i] = A * rel[:, None] + unit(dt) * out[i].abs() * 1.01 + torch.finfo(dt).smallest_normal
    return out, tol


def sample(logits, temperature, top_k, top_p, min_p, u):
    """Token of one row (1-d tensor), from the definition."""
    V = logits.numel()
    l = logits.double().clone()
    l[l.isnan()] = -math.inf
    if not 0 <= temperature <= 1e30 or not top_p >= 0 or not 0 <= min_p <= 1:
        return -1
    order = torch.sort(l, descending=True, stable=True).indices
    top = l[order[0]]
    if top == -math.inf:
        return 0
    if temperature == 0:
        return int(order[0])
    x = l[order]
    e = torch.where(x == top, torch.ones_like(x), torch.exp((x - top) / temperature) if top < math.inf
                    else torch.zeros_like(x))
    k = top_k if 0 < top_k < V else V
    zk = e[:k].sum()
    cum = e.cumsum(0)
    keep = torch.arange(V) < k
    if top_p < 1:
        keep &= cum - e <= top_p * zk
    keep &= e >= min_p
    keep[0] = True
    n = int(keep.sum())
    z = cum[n - 1]
    hit = (cum > u * z).nonzero()
    return int(order[min(int(hit[0]), n - 1)])
