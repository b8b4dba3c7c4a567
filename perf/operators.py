"""What the paged-cache operators and the row sampler are measured on.

Four operators of a serving step over a paged KV cache, in the order in which
one step runs them:

  plan       paged_plan: block tables, slot maps, positions and offsets of a
             batch of requests, from their lengths
  append     paged_append: per-head RMSNorm of queries and keys (optional),
             rotation by position, K and V written to their cache slots
  attention  paged_attention: causal attention of each request's new tokens
             over its pages
  sample     sample_rows: temperature, top-k, top-p and min-p per row, drawn
             from given uniforms

With `own` false, `run` computes them from elementary torch operations; with
`own` true it makes the calls a user's program makes of this package.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a batch of running requests: each grows by one token
        {"name": "plan_decode_32", "op": "plan", "batch": 32, "ctx": 4000, "chunks": 0, "chunk": 1, "ended": 0,
         "page": 16},
        # a scheduler step of a busy server: long prompts admitted beside many decodes, finished requests released
        {"name": "plan_mixed_256", "op": "plan", "batch": 256, "ctx": 4000, "chunks": 15, "chunk": 1024, "ended": 9,
         "page": 32},
        # decode rows of the 64/8-head model: projections hand over 16-bit rows
        {"name": "append_decode_64", "op": "append", "tokens": 64, "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64, "in": "bf16", "cache": "bf16", "norm": True},
        # a prompt of the 32-head model through the fp32 output of op_linear, rotation only, odd length
        {"name": "append_prompt_2047", "op": "append", "tokens": 2047, "heads": 32, "kv_heads": 32, "dim": 128,
         "page": 16, "in": "f32", "cache": "f16", "norm": False},
        # many prompts packed into one step, with the norms
        {"name": "append_packed_16384", "op": "append", "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 32, "in": "bf16", "cache": "bf16", "norm": True},
        # decode of one short conversation: latency
        {"name": "attn_decode_1x190", "op": "attention", "chunks": 0, "chunk": 1, "decodes": 1, "ctx": 190,
         "heads": 32, "kv_heads": 32, "dim": 128, "page": 16, "cache": "bf16"},
        # decode of a batch of running requests, every context another length
        {"name": "attn_decode_32x2000", "op": "attention", "chunks": 0, "chunk": 1, "decodes": 32, "ctx": 2000,
         "heads": 32, "kv_heads": 32, "dim": 128, "page": 16, "cache": "bf16"},
        # decode of one long document with grouped queries: the work is split along its keys
        {"name": "attn_decode_1x60000", "op": "attention", "chunks": 0, "chunk": 1, "decodes": 1, "ctx": 60000,
         "heads": 64, "kv_heads": 8, "dim": 128, "page": 64, "cache": "f16"},
        # two prompts continued in large chunks over what they have in the cache
        {"name": "attn_chunk_2x2000", "op": "attention", "chunks": 2, "chunk": 2000, "decodes": 0, "ctx": 6000,
         "heads": 64, "kv_heads": 8, "dim": 128, "page": 64, "cache": "bf16"},
        # a mixed step: one prompt's chunk beside decodes, fp32 parity model with short heads
        {"name": "attn_mixed_f32", "op": "attention", "chunks": 1, "chunk": 300, "decodes": 11, "ctx": 500,
         "heads": 8, "kv_heads": 2, "dim": 32, "page": 16, "cache": "f32"},
        # next token of one conversation over the 32000-entry vocabulary
        {"name": "sample_1x32000", "op": "sample", "rows": 1, "vocab": 32000, "kinds": "all"},
        # a decode step's rows, each with parameters of its own, over a vocabulary four times as large
        {"name": "sample_64x128000", "op": "sample", "rows": 64, "vocab": 128000, "kinds": "mixed"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attention", "attention", "attention", "sample"])
    if op == "plan":
        batch = _log(rng, 1, 256)
        ended = rng.randint(0, batch // 4)
        chunks = rng.randint(0, min(16, batch - ended))
        return {"op": op, "batch": batch, "ctx": _log(rng, 1, 6000), "chunks": chunks,
                "chunk": _log(rng, 2, 1024), "ended": ended, "page": rng.choice([16, 32, 64, 128])}
    if op == "append":
        kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([32, 64, 128])
        cache = rng.choice(["bf16", "f16", "f32"])
        src = rng.choice(["f32", cache])
        return {"op": op, "tokens": _log(rng, 1, 6000), "heads": kv * rng.choice([1, 2, 4]), "kv_heads": kv,
                "dim": dim, "page": rng.choice([16, 32, 64, 128]), "in": src, "cache": cache,
                "norm": rng.random() < 0.5}
    if op == "attention":
        kv = rng.choice([1, 2, 4, 8])
        cache = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
        dim = rng.choice([64, 128, 128]) if cache != "f32" else rng.choice([32, 64])
        # fp32 models are the small parity ones: short chunks
        chunks = rng.randint(0, 2)
        return {"op": op, "chunks": chunks, "chunk": _log(rng, 2, 1500 if cache != "f32" else 200),
                "decodes": rng.randint(0 if chunks else 1, 24), "ctx": _log(rng, 1, 6000 if cache != "f32" else 500),
                "heads": kv * rng.choice([1, 2, 4, 8]), "kv_heads": kv, "dim": dim,
                "page": rng.choice([16, 32, 64, 128]), "cache": cache}
    return {"op": op, "rows": _log(rng, 1, 64), "vocab": _log(rng, 500, 128000),
            "kinds": rng.choice(["all", "mixed", "top_k", "top_p", "min_p", "plain"])}


# ---------------------------------------------------------------- inputs

def _ragged(n, top, salt):
    """n unequal lengths between about top/2 and top: part of the case, whatever the seed."""
    if n == 0:
        return []
    gen = torch.Generator().manual_seed(1000 * top + 10 * n + salt)
    return torch.randint(max(1, top - top // 2), top + 1, (n,), generator=gen).tolist()


def _plan_lengths(c):
    """(cached tokens, new tokens or -1) of each request of a plan case."""
    B = c["batch"]
    ctx = _ragged(B, c["ctx"], 1)
    new = [-1] * c["ended"] + _ragged(c["chunks"], c["chunk"], 2) + [1] * (B - c["ended"] - c["chunks"])
    for i in range(c["ended"], c["ended"] + c["chunks"], 2):
        ctx[i] = 0                    # every other chunk opens its request
    mix = torch.randperm(B, generator=torch.Generator().manual_seed(B)).tolist()
    return [ctx[i] for i in mix], [new[i] for i in mix]


def _lengths(c):
    """(new tokens, tokens with them) of each request of an attention case: chunks first, then decodes."""
    new = _ragged(c["chunks"], c["chunk"], 3) + [1] * c["decodes"]
    before = _ragged(len(new), c["ctx"], 4)
    return new, [n + b for n, b in zip(new, before)]


def _pages(total, gen):
    return torch.randperm(total, generator=gen).to(torch.int32)


def _prepare_plan(c, gen):
    B, ps = c["batch"], c["page"]
    ctx, new = (torch.tensor(v, dtype=torch.int32) for v in _plan_lengths(c))
    total = int(new.clamp(min=0).sum())
    have = (ctx + ps - 1) // ps
    width = (c["ctx"] + c["chunk"] + ps - 1) // ps
    need = (ctx + new.clamp(min=0) + ps - 1) // ps
    pool = int(need.sum()) + B
    perm = _pages(pool, gen)
    tables = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        n = int(have[b])
        tables[b, :n] = perm[at:at + n]
        at += n
    free = torch.full((pool,), -1, dtype=torch.int32)
    free[:pool - at] = perm[at:]
    room = total + 7            # the token arrays are a little wider than the step
    st = {"ctx": ctx, "new": new, "tables": tables, "free": free,
          "count": torch.tensor([pool - at], dtype=torch.int32), "seq": torch.zeros(B, dtype=torch.int32),
          "cu": torch.zeros(B + 1, dtype=torch.int32), "slots": torch.zeros(room, dtype=torch.int64),
          "pos": torch.zeros(room, dtype=torch.int32), "left": torch.zeros(1, dtype=torch.int32),
          "status": torch.zeros(1, dtype=torch.int32)}
    return {k: v.cuda() for k, v in st.items()}


def _rope(n, dim):
    j = torch.arange(dim // 2, dtype=torch.float64, device="cuda")
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2.0 * j / dim)
    return torch.stack([ang.cos(), ang.sin()], -1).float()


def _prepare_append(c, gen):
    T, nh, nkv, hd, ps = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    g = torch.Generator("cuda").manual_seed(int(torch.randint(1 << 30, (1,), generator=gen)))
    src, dst = _DT[c["in"]], _DT[c["cache"]]
    # one row per token: queries, keys and values of the fused projection side by side
    qkv = torch.randn(T, (nh + 2 * nkv) * hd, generator=g, device="cuda").to(src)
    pages = (T + ps - 1) // ps + 3
    perm = _pages(pages, gen).long()
    start = int(torch.randint(0, 3000, (1,), generator=gen))
    t = torch.arange(T)
    slots = perm[t // ps] * ps + t % ps
    pos = (start + t).to(torch.int32)
    st = {"T": T, "nh": nh, "nkv": nkv, "hd": hd, "ps": ps, "dst": dst,
          "q": qkv[:, :nh * hd].unflatten(1, (nh, hd)),
          "k": qkv[:, nh * hd:(nh + nkv) * hd].unflatten(1, (nkv, hd)),
          "v": qkv[:, (nh + nkv) * hd:].unflatten(1, (nkv, hd)),
          "slots": slots.cuda(), "pos": pos.cuda(), "rope": _rope(start + T, hd),
          "q_out": torch.zeros(T, nh, hd, dtype=dst, device="cuda"),
          "k_pages": torch.zeros(pages, nkv, ps, hd, dtype=dst, device="cuda"),
          "v_pages": torch.zeros(pages, nkv, ps, hd, dtype=dst, device="cuda"),
          "qw": None, "kw": None, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if c["norm"]:
        st["qw"] = 1.0 + 0.1 * torch.randn(hd, generator=g, device="cuda")
        st["kw"] = 1.0 + 0.1 * torch.randn(hd, generator=g, device="cuda")
    return st


def _prepare_attention(c, gen):
    nh, nkv, hd, ps, dt = c["heads"], c["kv_heads"], c["dim"], c["page"], _DT[c["cache"]]
    new, seq = _lengths(c)
    g = torch.Generator("cuda").manual_seed(int(torch.randint(1 << 30, (1,), generator=gen)))
    B, T = len(new), sum(new)
    used = [(s + ps - 1) // ps for s in seq]
    pages = sum(used) + 2
    perm = _pages(pages, gen)
    tables = torch.full((B, max(used) + 1), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        tables[b, :used[b]] = perm[at:at + used[b]]
        at += used[b]
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    # scores of standard deviation 1.5 after the scale
    st = {"new": new, "seq": seq, "nh": nh, "nkv": nkv, "hd": hd, "ps": ps, "T": T,
          "q": (1.5 * torch.randn(T, nh, hd, generator=g, device="cuda")).to(dt),
          "k_pages": torch.empty(pages, nkv, ps, hd, dtype=dt, device="cuda"),
          "v_pages": torch.empty(pages, nkv, ps, hd, dtype=dt, device="cuda"),
          "tables": tables.cuda(), "cu": cu.cuda(), "seq_lens": torch.tensor(seq, dtype=torch.int32).cuda(),
          "max_new": max(new), "out": torch.empty(T, nh, hd, dtype=dt, device="cuda"),
          "status": torch.zeros(1, dtype=torch.int32, device="cuda"), "ws": None}
    for name in ("k_pages", "v_pages"):
        for p in range(0, pages, 4096):      # drawn in pieces: no fp32 copy of the whole pool
            part = st[name][p:p + 4096]
            part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    if own:
        import decoder_only_transformer_llama_b200 as llb
        st["ws"] = llb.paged_attention_workspace(st["q"], nkv, st["max_new"])
    return st


def _prepare_sample(c, gen):
    B, V = c["rows"], c["vocab"]
    g = torch.Generator("cuda").manual_seed(int(torch.randint(1 << 30, (1,), generator=gen)))
    # logits with a few strong candidates and a long tail, as a trained model's
    logits = 2.0 * torch.randn(B, V, generator=g, device="cuda")
    peaks = torch.randint(0, V, (B, 40), generator=g, device="cuda")
    logits.scatter_add_(1, peaks, 8.0 * torch.rand(B, 40, generator=g, device="cuda"))
    kinds = c["kinds"]
    temperature = torch.full((B,), 0.8)
    top_k = torch.zeros(B, dtype=torch.int32)
    top_p = torch.ones(B)
    min_p = torch.zeros(B)
    for b in range(B):
        k = kinds if kinds != "mixed" else ("all", "top_k", "top_p", "min_p", "plain", "greedy")[b % 6]
        if k in ("all", "top_k"):
            top_k[b] = int(torch.randint(5, 200, (1,), generator=gen))
        if k in ("all", "top_p"):
            top_p[b] = 0.8 + 0.19 * float(torch.rand(1, generator=gen))
        if k in ("all", "min_p"):
            min_p[b] = 0.01 + 0.09 * float(torch.rand(1, generator=gen))
        temperature[b] = 0.0 if k == "greedy" else 0.5 + float(torch.rand(1, generator=gen))
    u = torch.rand(B, generator=gen)
    st = {"temperature": temperature, "top_k": top_k, "top_p": top_p, "min_p": min_p, "u": u}
    st = {k: v.cuda() for k, v in st.items()}
    st["logits"] = logits
    st["out"] = torch.empty(B, dtype=torch.int32, device="cuda")
    return st


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    st = {"plan": _prepare_plan, "append": _prepare_append, "attention": _prepare_attention,
          "sample": _prepare_sample}[case["op"]](case, gen)
    st["op"] = case["op"]
    if case["op"] == "plan":
        st["ps"] = case["page"]
    return st


# ---------------------------------------------------------------- plain forms

def _plain_plan(s):
    ps, ctx, new = s["ps"], s["ctx"].long(), s["new"].long()
    B, room = ctx.numel(), s["slots"].numel()
    dev = ctx.device
    ended = new < 0
    n = new.clamp(min=0)
    have = (ctx + ps - 1) // ps
    count = s["count"].long()
    cols = torch.arange(s["tables"].shape[1], device=dev)
    # pages of ended requests go back on the stack, in request order
    back = torch.where(ended, have, torch.zeros_like(have))
    back_at = back.cumsum(0) - back
    give = ended[:, None] & (cols[None] < have[:, None])
    at = (count + back_at[:, None] + cols[None]).clamp(max=s["free"].numel() - 1)
    free = s["free"].clone()
    free[at[give]] = s["tables"][give]
    count = count + back.sum()
    # pages of growing requests come off its top, in request order
    seq = torch.where(ended, torch.zeros_like(ctx), ctx + n)
    held = torch.where(ended, torch.zeros_like(have), have)
    want = (seq + ps - 1) // ps - held
    take_at = want.cumsum(0) - want
    i = cols[None] - held[:, None]
    take = (i >= 0) & (i < want[:, None])
    src = (count - 1 - (take_at[:, None] + i)).clamp(min=0)
    tables = torch.where(take, free[src], s["tables"])
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), n.cumsum(0)])
    t = torch.arange(room, device=dev)
    row = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=B - 1)
    live = t < cu[-1]
    pos = ctx[row] + t - cu[row]
    page = tables[row, (pos // ps).clamp(0, tables.shape[1] - 1)].long()
    none = torch.full_like(t, -1)
    return {"tables": tables, "free": free, "left": (count - want.sum()).int(), "seq": seq.int(), "cu": cu.int(),
            "slots": torch.where(live, page * ps + pos % ps, none), "pos": torch.where(live, pos, none).int()}


def _plain_norm(x, w, eps):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w


def _plain_rotate(x, cs):
    a, b = x[..., 0::2], x[..., 1::2]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def _plain_append(s):
    cs = s["rope"][s["pos"].long()]
    q = _plain_rotate(_plain_norm(s["q"].float(), s["qw"], 1e-5), cs)
    k = _plain_rotate(_plain_norm(s["k"].float(), s["kw"], 1e-5), cs)
    s["q_out"].copy_(q)
    page, off = s["slots"] // s["ps"], s["slots"] % s["ps"]
    s["k_pages"][page, :, off] = k.to(s["dst"])
    s["v_pages"][page, :, off] = s["v"].float().to(s["dst"])
    return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attention(s):
    nh, nkv, hd, ps = s["nh"], s["nkv"], s["hd"], s["ps"]
    rep = nh // nkv
    at = 0
    for b, (n, kv) in enumerate(zip(s["new"], s["seq"])):
        ids = s["tables"][b, :(kv + ps - 1) // ps].long()
        k = s["k_pages"][ids].float().transpose(0, 1).reshape(nkv, -1, hd)[:, :kv]
        v = s["v_pages"][ids].float().transpose(0, 1).reshape(nkv, -1, hd)[:, :kv]
        q = s["q"][at:at + n].float().reshape(n, nkv, rep, hd).permute(1, 2, 0, 3).reshape(nkv, rep * n, hd)
        sc = (q @ k.transpose(1, 2)).mul_(1.0 / math.sqrt(hd)).view(nkv, rep, n, kv)
        hidden = torch.arange(kv, device=q.device)[None] > (kv - n + torch.arange(n, device=q.device))[:, None]
        sc.masked_fill_(hidden, float("-inf"))
        p = sc.sub_(sc.amax(-1, keepdim=True)).exp_()
        p = p / p.sum(-1, keepdim=True)
        o = (p.view(nkv, rep * n, kv) @ v).view(nkv, rep, n, hd).permute(2, 0, 1, 3).reshape(n, nh, hd)
        s["out"][at:at + n] = o.to(s["out"].dtype)
        at += n
    return s["out"]


def _plain_sample(s):
    lg = s["logits"]
    B, V = lg.shape
    t = s["temperature"].double()
    order, ids = torch.sort(lg, dim=-1, descending=True, stable=True)
    x = (order.double() - order[:, :1].double()) / torch.where(t > 0, t, torch.ones_like(t))[:, None]
    e = x.exp()
    rank = torch.arange(V, device=lg.device)[None]
    k = s["top_k"].long()[:, None]
    in_k = (k <= 0) | (rank < k)
    cum = e.cumsum(-1)
    zk = torch.where(in_k, e, torch.zeros_like(e)).sum(-1, keepdim=True)
    keep = in_k & (cum - e <= s["top_p"].double()[:, None] * zk) & (e >= s["min_p"].double()[:, None])
    kept = keep.sum(-1, keepdim=True)
    z = cum.gather(1, kept - 1)
    hit = (cum > s["u"].double()[:, None] * z).int().argmax(-1, keepdim=True)
    pick = torch.minimum(hit, kept - 1)
    pick = torch.where(t[:, None] > 0, pick, torch.zeros_like(pick))
    return ids.gather(1, pick).squeeze(1).int()


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "attention": _plain_attention,
                "sample": _plain_sample}[op](s)
    import decoder_only_transformer_llama_b200 as llb
    if op == "plan":
        llb.paged_plan(s["ctx"], s["new"], s["tables"], s["free"], s["count"], s["ps"], s["seq"], s["cu"],
                       s["slots"], s["pos"], s["left"], status=s["status"])
        return {"tables": s["tables"], "free": s["free"], "left": s["left"], "seq": s["seq"], "cu": s["cu"],
                "slots": s["slots"], "pos": s["pos"]}
    if op == "append":
        llb.paged_append(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["rope"], s["q_out"], s["k_pages"],
                         s["v_pages"], q_norm=s["qw"], k_norm=s["kw"], eps=1e-5, status=s["status"])
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "attention":
        return llb.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["tables"], s["cu"], s["seq_lens"],
                                   s["out"], max_new=s["max_new"], workspace=s["ws"], status=s["status"])
    return llb.sample_rows(s["logits"], s["temperature"], s["u"], s["out"], top_k=s["top_k"], top_p=s["top_p"],
                           min_p=s["min_p"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "plan":
        ps, B = c["page"], c["batch"]
        ctx, new = _plan_lengths(c)
        pages = [-(-x // ps) for x in ctx]
        tokens = sum(n for n in new if n > 0)
        grown = sum(-(-(x + n) // ps) - h for x, n, h in zip(ctx, new, pages) if n > 0)
        freed = sum(h for n, h in zip(new, pages) if n < 0)
        # lengths in, lengths and offsets out, a page read and written per page moved, slot and position per token
        return {"bytes": 16 * B + 8 * (grown + freed) + 12 * tokens, "flops": 2 * tokens}
    if c["op"] == "append":
        T, nh, nkv, hd = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
        values = T * (nh + 2 * nkv) * hd
        rows = T * (12 + 4 * hd)         # slot, position and the position's cosines and sines
        per = 3 + (5 if c["norm"] else 0)
        return {"bytes": values * (_SIZE[c["in"]] + _SIZE[c["cache"]]) + rows, "flops": T * (nh + nkv) * hd * per}
    if c["op"] == "attention":
        nh, nkv, hd, e = c["heads"], c["kv_heads"], c["dim"], _SIZE[c["cache"]]
        new, seq = _lengths(c)
        seen = sum(n * (kv - n) + n * (n + 1) // 2 for n, kv in zip(new, seq))
        return {"bytes": 2 * sum(seq) * nkv * hd * e + 2 * sum(new) * nh * hd * e, "flops": 4 * nh * hd * seen}
    return {"bytes": c["rows"] * (4 * c["vocab"] + 24), "flops": 4 * c["rows"] * c["vocab"]}


# ---------------------------------------------------------------- 64 bits

def _exact_append(c, st):
    T, nh, nkv, hd, ps = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    pos = st["pos"].long()
    # the table the call is given holds the angles: its 32-bit entries are an input
    z = torch.view_as_complex(st["rope"].double().contiguous())[pos][:, None]

    def turn(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / hd + 1e-5).sqrt() * w.double()
        y = torch.view_as_complex(x.reshape(T, -1, hd // 2, 2).contiguous()) * z
        return torch.view_as_real(y).reshape(T, -1, hd)

    flat = {}
    for name, val in (("k_pages", turn(st["k"], st["kw"])), ("v_pages", st["v"].double())):
        pool = torch.zeros(st[name].shape[0] * ps, nkv, hd, dtype=torch.float64, device="cuda")
        pool.index_copy_(0, st["slots"], val)
        flat[name] = pool.view(-1, ps, nkv, hd).transpose(1, 2).contiguous()
    return {"q": turn(st["q"], st["qw"]), **flat}


def _exact_attention(c, st, new, seq):
    nh, nkv, hd, ps = c["heads"], c["kv_heads"], c["dim"], c["page"]
    out = torch.empty(sum(new), nh, hd, dtype=torch.float64, device="cuda")
    first = 0
    for b in range(len(new)):
        n, kv = new[b], seq[b]
        where = torch.arange(kv, device="cuda")
        page = st["tables"][b].long()[where // ps]
        for h in range(nh):
            g = h * nkv // nh
            keys = st["k_pages"][page, g, where % ps].double()
            vals = st["v_pages"][page, g, where % ps].double()
            for lo in range(0, n, 1024):
                hi = min(n, lo + 1024)
                a = torch.einsum("td,kd->tk", st["q"][first + lo:first + hi, h].double(), keys) / hd ** 0.5
                last = kv - n + torch.arange(lo, hi, device="cuda")
                a = torch.where(where[None, :] <= last[:, None], a, torch.full_like(a, -math.inf))
                out[first + lo:first + hi, h] = torch.einsum("tk,kd->td", torch.softmax(a, 1), vals)
        first += n
    return out


def exact(case, seed):
    if case["op"] in ("plan", "sample"):
        return None         # whole numbers only
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, st)
    return _exact_attention(case, st, *_lengths(case))
