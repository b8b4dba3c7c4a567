"""The operators of a serving step over a paged KV cache against their plain
64-bit definitions: plans are equal, values lie within derived bounds."""
import math

import pytest
import torch

import paged_reference as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def llb(cuda_device):
    import decoder_only_transformer_llama_b200 as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- plan

def plan_state(ctx, page, width, extra, seed, cap=None):
    g = torch.Generator().manual_seed(seed)
    used = [-(-max(c, 0) // page) for c in ctx]
    pool = sum(used) + extra
    perm = torch.randperm(pool, generator=g).tolist()
    tables, at = [], 0
    for n in used:
        tables.append(perm[at:at + n] + [-7] * (width - n))
        at += n
    cap = cap or pool
    free = perm[at:] + [-9] * (cap - extra)
    return tables, free, extra, cap


def run_plan(llb, ctx, new, page, tables, free, count, room, alias=False):
    B = len(ctx)
    c, n, t, f, fc = i32(ctx), i32(new), i32(tables), i32(free), i32([count])
    seq, left = (c, fc) if alias else (i32([99] * B), i32([99]))
    cu, st = i32([99] * (B + 1)), i32([0])
    slots = torch.full((room,), 99, dtype=torch.int64, device="cuda")
    pos = torch.full((room,), 99, dtype=torch.int32, device="cuda")
    llb.paged_plan(c, n, t, f, fc, page, seq, cu, slots, pos, left, status=st)
    torch.cuda.synchronize()
    return {"tables": t.tolist(), "free": f.tolist(), "left": int(left), "seq": seq.tolist(), "cu": cu.tolist(),
            "slots": slots.tolist(), "pos": pos.tolist()}, int(st)


PLANS = [
    ([0], [1], 16, 1),
    ([5], [0], 16, 0),
    ([16], [1], 16, 1),
    ([15, 16, 17, 31], [1, 1, 1, 1], 16, 9),
    ([0, 40, 0, 129, 7], [33, -1, 0, 128, -5], 32, 40),
    ([100, 0, 3], [300, 257, 1], 64, 20),
    ([1000, 255, 256, 257], [1, 1, 1, 700], 256, 6),
    ([300, 77], [-1, -1], 16, 3),
    (list(range(0, 1300, 5)), [(-1 if i % 9 == 4 else (i * 37) % 90) for i in range(260)], 16, 1500),
    ([i % 50 for i in range(1024)], [1 + i % 3 for i in range(1024)], 128, 1100),
]


@pytest.mark.parametrize("case", range(len(PLANS)))
@pytest.mark.parametrize("alias", [False, True])
def test_plan(llb, case, alias):
    ctx, new, page, extra = PLANS[case]
    width = max(-(-(c + max(n, 0)) // page) for c, n in zip(ctx, new)) + (case % 2)
    width = max(width, 1)
    tables, free, count, cap = plan_state(ctx, page, width, extra, case)
    total = sum(max(n, 0) for n in new)
    room = total + case % 4
    want = R.plan(ctx, new, page, tables, free, count, width, room, cap)
    assert not want.pop("failed")
    got, status = run_plan(llb, ctx, new, page, tables, free, count, room, alias)
    assert status == 0
    # a released page may be taken in the same step: compare the live part of the stack
    got["free"], want["free"] = got["free"][:want["left"]], want["free"][:want["left"]]
    assert got == want


@pytest.mark.parametrize("ctx,new,page,extra,width,room,cap,code", [
    ([10, 20], [7, 13], 16, 1, 4, 64, None, 2),          # two pages needed, one free
    ([10, 20], [7, 1], 16, 5, 2, 7, None, 2),            # eight tokens, seven rows
    ([10, 20], [7, 30], 16, 5, 3, 64, None, 2),          # four pages in a table of three
    ([10, -1], [7, 1], 16, 5, 3, 64, None, 1),
    ([64, 64], [-1, -1], 16, 2, 4, 4, 9, 1),             # ten free pages in a list of nine
    ([2147483000], [1000], 16, 5, 3, 64, None, 2),       # past the positions of an int
    ([3, -5, 70], [80, 1, 9], 16, 1, 6, 4, None, 1),     # several faults: a bad argument goes first
])
def test_plan_all_or_nothing(llb, ctx, new, page, extra, width, room, cap, code):
    real = [c if c < 1 << 20 else 0 for c in ctx]
    tables, free, count, cap_ = plan_state(real, page, width, extra, 3)
    if cap is not None:
        free, cap_ = free[:cap] + [-9] * max(0, cap - len(free)), cap
    want = R.plan(ctx, new, page, tables, free, count, width, room, cap_)
    assert want.pop("failed")
    got, status = run_plan(llb, ctx, new, page, tables, free, count, room)
    assert status == code
    assert got == want


def test_plan_steps_in_a_graph(llb):
    """Lengths and the free list updated in place by replays of one captured step."""
    page, width, B, steps = 16, 8, 5, 40
    ctx = [0, 3, 15, 16, 60]
    tables, free, count, cap = plan_state(ctx, page, width, 20, 11)
    new = [1] * B
    c, n, t, f, fc = i32(ctx), i32(new), i32(tables), i32(free), i32([count])
    cu, st = i32([0] * (B + 1)), i32([0])
    slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    step = lambda: llb.paged_plan(c, n, t, f, fc, page, c, cu, slots, pos, fc, status=st)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(steps):
        want = R.plan(ctx, new, page, tables, free, count, width, B, cap)
        assert not want["failed"]
        graph.replay()
        torch.cuda.synchronize()
        assert slots.tolist() == want["slots"] and pos.tolist() == want["pos"] and c.tolist() == want["seq"]
        assert t.tolist() == want["tables"] and int(fc) == want["left"]
        ctx, tables, free, count = want["seq"], want["tables"], want["free"], want["left"]
    assert int(st) == 0


# ---------------------------------------------------------------- append

def append_case(llb, T, nh, nkv, hd, page, src, dst, norm, seed, packed=True, eps=1e-5):
    g = torch.Generator().manual_seed(seed)
    src, dst = DT[src], DT[dst]
    flat = torch.randn(T, (nh + 2 * nkv) * hd, generator=g).to(src)
    if packed:
        dev = flat.cuda()
        parts = dev.split([nh * hd, nkv * hd, nkv * hd], 1)
    else:
        parts = [p.contiguous().cuda() for p in flat.split([nh * hd, nkv * hd, nkv * hd], 1)]
    q, k, v = (p.unflatten(1, (-1, hd)) for p in parts)
    n_pages = -(-T // page) + 2
    perm = torch.randperm(n_pages * page, generator=g)[:T]
    slots = perm.clone()
    pos = torch.randint(0, 500, (T,), generator=g).to(torch.int32)
    if T > 2:
        slots[T // 2] = -1                       # a padding row
    rope = torch.empty(500, hd // 2, 2, device="cuda")
    llb.rope_table(rope)
    qw = (1 + 0.1 * torch.randn(hd, generator=g)) if norm in ("both", "q") else None
    kw = (1 + 0.1 * torch.randn(hd, generator=g)) if norm in ("both", "k") else None
    q_out = torch.full((T, nh, hd), 7.0, dtype=dst, device="cuda")
    pools = [torch.full((n_pages, nkv, page, hd), 7.0, dtype=dst, device="cuda") for _ in range(2)]
    st = i32([0])
    cu = lambda w: None if w is None else w.cuda()
    llb.paged_append(q, k, v, pos.cuda(), slots.cuda(), rope, q_out, *pools, q_norm=cu(qw), k_norm=cu(kw), eps=eps,
                     status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    table = rope.cpu()
    want_table = R.rope_table(500, hd)
    # an fp32 rounding of fp64 cosines of angles below 500 (their fp64 error is far below it)
    assert ((table.double() - want_table).abs() <= R.U32 * want_table.abs() + 1e-12).all()
    cs = table[pos.long()]
    live = slots >= 0
    wq, tq = R.norm_rotate(q.cpu(), qw, eps, cs, dst)
    wk, tk = R.norm_rotate(k.cpu(), kw, eps, cs, dst)
    wv = v.cpu().to(dst)
    got_q = q_out.cpu().double()
    assert ((got_q - wq).abs() <= tq)[live].all()
    assert (got_q[~live] == 7.0).all()
    got_k, got_v = (p.cpu().transpose(1, 2).reshape(-1, nkv, hd) for p in pools)
    assert ((got_k[slots[live]].double() - wk[live]).abs() <= tk[live]).all()
    assert torch.equal(got_v[slots[live]], wv[live])
    rest = torch.ones(n_pages * page, dtype=torch.bool)
    rest[slots[live]] = False
    assert (got_k[rest] == 7.0).all() and (got_v[rest] == 7.0).all()


@pytest.mark.parametrize("T,nh,nkv,hd,page,src,dst,norm", [
    (1, 32, 32, 128, 16, "bf16", "bf16", None),
    (1, 64, 8, 128, 64, "f32", "bf16", "both"),
    (3, 8, 2, 32, 16, "f32", "f32", "both"),
    (7, 5, 5, 64, 32, "f16", "f16", "q"),
    (33, 40, 40, 128, 256, "f32", "f16", "k"),
    (129, 1, 1, 128, 16, "bf16", "bf16", "both"),
    (130, 3, 3, 32, 128, "bf16", "bf16", "both"),
    (257, 8, 1, 64, 16, "f32", "bf16", None),
    (1000, 16, 4, 128, 16, "f16", "f16", "both"),
    (2049, 4, 4, 32, 16, "f32", "f32", None),
])
@pytest.mark.parametrize("packed", [True, False])
def test_append(llb, T, nh, nkv, hd, page, src, dst, norm, packed):
    append_case(llb, T, nh, nkv, hd, page, src, dst, norm, T + nh, packed)


def test_append_in_place_and_out_of_range(llb):
    T, nh, nkv, hd, page = 6, 4, 2, 64, 16
    g = torch.Generator().manual_seed(5)
    q = torch.randn(T, nh, hd, generator=g).bfloat16()
    k = torch.randn(T, nkv, hd, generator=g).bfloat16()
    rope = R.rope_table(32, hd).float()
    pos = torch.tensor([0, 31, 32, -1, 4, 5], dtype=torch.int32)
    slots = torch.tensor([0, 1, 2, 3, 32, 5])
    qd, kd = q.cuda(), k.cuda()
    pools = [torch.full((2, nkv, page, hd), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    st = i32([0])
    llb.paged_append(qd, kd, kd, pos.cuda(), slots.cuda(), rope.cuda(), qd, *pools, status=st)
    assert int(st) == llb.LLAMA_ERR_CAPACITY
    good = [0, 1, 5]
    want, tol = R.norm_rotate(q, None, 0.0, rope[pos.long().clamp(0, 31)], torch.bfloat16)
    assert ((qd.cpu().double() - want).abs() <= tol)[good].all()
    assert torch.equal(qd.cpu()[[2, 3, 4]], q[[2, 3, 4]])
    flat = pools[1].cpu().transpose(1, 2).reshape(-1, nkv, hd)
    assert torch.equal(flat[[0, 1, 5]], k[good])
    assert (flat[[2, 3, 4]] == 7.0).all() and (flat[6:] == 7.0).all()


# ---------------------------------------------------------------- attention

def paged_cache(seqs, page, nkv, hd, dt, g, width_extra=1, fill=float("nan")):
    """Pools whose unused slots hold `fill`; dense k, v per request."""
    used = [-(-s // page) for s in seqs]
    n_pages = sum(used) + 2
    perm = torch.randperm(n_pages, generator=g).tolist()
    pools = [torch.full((n_pages, nkv, page, hd), fill, dtype=dt) for _ in range(2)]
    tables = torch.full((len(seqs), max(used + [1]) + width_extra), -1, dtype=torch.int32)
    dense, at = [], 0
    for b, s in enumerate(seqs):
        ids = perm[at:at + used[b]]
        at += used[b]
        tables[b, :used[b]] = torch.tensor(ids, dtype=torch.int32)
        kv = [torch.randn(s, nkv, hd, generator=g).to(dt) for _ in range(2)]
        for pool, x in zip(pools, kv):
            for i, p in enumerate(ids):
                part = x[i * page:(i + 1) * page]
                pool[p, :, :len(part)] = part.transpose(0, 1)
        dense.append(kv)
    return pools, tables, dense


def attn_case(llb, new, seqs, nh, nkv, hd, page, dtype, seed=0, scale=None, tail=3, max_new=None, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    pools, tables, dense = paged_cache(seqs, page, nkv, hd, dt, g)
    total = sum(new)
    q = (spread * torch.randn(total + tail, nh, hd, generator=g)).to(dt)
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    out = torch.full((total + tail, nh, hd), 7.0, dtype=dt, device="cuda")
    st = i32([0])
    args = [q.cuda(), pools[0].cuda(), pools[1].cuda(), tables.cuda(), cu.cuda(), i32(seqs)]
    mx = max_new or max(new + [1])
    ws = llb.paged_attention_workspace(args[0], nkv, mx)
    llb.paged_attention(*args, out, max_new=mx, scale=scale, workspace=ws, status=st)
    first = out.cpu()
    out.fill_(7.0)
    llb.paged_attention(*args, out, max_new=mx, scale=scale, workspace=ws, status=st)
    got = out.cpu()
    assert int(st) == 0
    assert torch.equal(first, got)                   # the same bits from call to call, the workspace left usable
    assert (got[total:] == 7.0).all()
    for b, n in enumerate(new):
        lo = int(cu[b])
        want, tol = R.attention(q[lo:lo + n], dense[b][0], dense[b][1], n, seqs[b],
                                hd ** -0.5 if scale is None else scale)
        err = (got[lo:lo + n].double() - want).abs()
        assert (err <= tol).all(), (b, float((err - tol).max()), float(err.max()))


ATTN = [
    # new, seqs, nh, nkv, hd, page
    ([1], [1], 32, 32, 128, 16),
    ([1], [190], 32, 32, 128, 16),
    ([1, 1, 1], [64, 65, 63], 8, 8, 128, 16),
    ([1] * 9, [1, 2, 15, 16, 17, 128, 129, 500, 1000], 16, 2, 128, 32),
    ([1], [3001], 8, 1, 128, 64),
    ([0, 1, 0, 2, 0], [0, 5, 40, 33, 9], 4, 4, 64, 16),
    ([3, 1, 4], [300, 70, 4], 8, 2, 128, 16),
    ([16, 17], [16, 140], 4, 4, 128, 128),
    ([128], [128], 2, 2, 128, 16),
    ([129, 1, 300], [129, 77, 513], 8, 2, 128, 32),
    ([260], [1000], 8, 1, 128, 256),
    ([65, 1, 31], [65, 200, 95], 8, 4, 64, 64),
    ([40, 1], [99, 258], 4, 1, 32, 16),
    ([257], [700], 2, 2, 64, 16),
    ([700], [700], 1, 1, 128, 64),
]


@pytest.mark.parametrize("case", range(len(ATTN)))
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_attention(llb, case, dtype):
    attn_case(llb, *ATTN[case], dtype, seed=case)


@pytest.mark.parametrize("dtype,hd,max_new", [("bf16", 128, 1), ("f16", 128, 300), ("bf16", 64, 300), ("f32", 32, 1)])
def test_attention_a_thousand_requests(llb, dtype, hd, max_new):
    """As many requests as a call may hold, a third of them without new tokens, some with a few."""
    new = [(0, 1, 1, 0, 1, 3)[b % 6] for b in range(1024)]
    seqs = [new[b] + (b * 7) % 40 for b in range(1024)]
    attn_case(llb, new, seqs, 2, 1, hd, 16, dtype, seed=1, max_new=max_new)


@pytest.mark.parametrize("max_new", [1, 300])
@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("f16", 64), ("f32", 128)])
def test_attention_any_max_new(llb, max_new, dtype, hd):
    """max_new only chooses the kernel: a request with more new tokens, or far fewer, is still right."""
    attn_case(llb, [5, 1, 90], [64, 1, 300], 8, 2, hd, 16, dtype, seed=5, max_new=max_new)


@pytest.mark.parametrize("new,seqs", [([1, 1], [5, 600]), ([200, 3], [200, 333])])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_attention_sharp_scores(llb, new, seqs, dtype):
    """Scores in the hundreds: the running maximum moves often, most weights vanish."""
    attn_case(llb, new, seqs, 4, 2, 128, 32, dtype, seed=2, spread=16.0)


@pytest.mark.parametrize("hd,n", [(128, 1), (64, 40)])
def test_attention_many_small_weights(llb, hd, n):
    """fp16, one key far above 20000 others: most of the output comes from weights near 2^-17 of the largest, below
    fp16's normal range. They are rounded with a factor 2^7 at least, so by at most 2^-32 of the largest each."""
    g = torch.Generator().manual_seed(14)
    page, nkv, nh, seq, dt = 64, 1, 2, 20000, torch.float16
    pools, tables, dense = paged_cache([seq], page, nkv, hd, dt, g)
    k, v = dense[0]
    k.zero_()
    k[17] = 1.0                                       # 11.5 after the scale: weights of e^-11.5 = 2^-16.6 elsewhere
    v.copy_(1.0 + v * 0.25)
    for j in range(seq):
        p, o = int(tables[0, j // page]), j % page
        pools[0][p, 0, o] = k[j, 0]
        pools[1][p, 0, o] = v[j, 0]
    q = torch.full((n, nh, hd), 11.5 / hd ** 0.5).to(dt)
    out = torch.empty(n, nh, hd, dtype=dt, device="cuda")
    llb.paged_attention(q.cuda(), pools[0].cuda(), pools[1].cuda(), tables.cuda(), i32([0, n]), i32([seq]), out,
                        max_new=n)
    got = out.cpu().double()
    for i in sorted({0, n - 1}):
        s1 = seq - n + i + 1
        want, tol = R.attention(q[i:i + 1], k, v, 1, s1, hd ** -0.5)
        # against the largest weight 1, the sum is at least 1: s1 * 2^-32 more of the mean |v| < 2
        assert ((got[i] - want[0]).abs() <= tol[0] + s1 * 2.0 ** -31).all()


def test_attention_negative_scale(llb):
    attn_case(llb, [1, 70], [100, 200], 4, 2, 64, 16, "bf16", seed=9, scale=-0.3)


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("f16", 64), ("bf16", 32), ("f32", 64)])
@pytest.mark.parametrize("max_new", [3, 400])
def test_attention_rows_without_keys(llb, dtype, hd, max_new):
    """seq_lens below the new tokens: rows at negative positions see nothing and give zeros."""
    g = torch.Generator().manual_seed(1)
    dt, page, nkv, nh = DT[dtype], 16, 2, 4
    new, seqs = [3, 5, 2], [0, 2, 40]
    pools, tables, dense = paged_cache(seqs, page, nkv, hd, dt, g)
    q = torch.randn(10, nh, hd, generator=g).to(dt)
    out = torch.full((10, nh, hd), 7.0, dtype=dt, device="cuda")
    st = i32([0])
    llb.paged_attention(q.cuda(), pools[0].cuda(), pools[1].cuda(), tables.cuda(), i32([0, 3, 8, 10]), i32(seqs), out,
                        max_new=max_new, status=st)
    got = out.cpu().double()
    assert int(st) == 0
    assert (got[:6] == 0).all()
    for lo, n, b in ((3, 5, 1), (8, 2, 2)):
        want, tol = R.attention(q[lo:lo + n], dense[b][0], dense[b][1], n, seqs[b], hd ** -0.5)
        assert ((got[lo:lo + n] - want).abs() <= tol).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype,hd,max_new", [("bf16", 128, 1), ("bf16", 128, 400), ("f16", 64, 400), ("f16", 32, 40),
                                              ("f32", 64, 40)])
def test_attention_bad_values_stay_behind_the_mask(llb, bad, dtype, hd, max_new):
    """Keys and values a row may not see hold NaN or infinities: rows before them are untouched by them,
    rows that see them are not finite."""
    g = torch.Generator().manual_seed(4)
    dt, page, nkv, nh, n, seq = DT[dtype], 16, 2, 8, 40, 100
    pools, tables, dense = paged_cache([seq], page, nkv, hd, dt, g, fill=bad)
    first = seq - n + 21                              # the position from which on V is bad
    k, v = dense[0]
    where = [(int(tables[0, j // page]), j % page) for j in range(seq)]
    for j in range(first, seq):
        p, o = where[j]
        pools[1][p, 0, o, 3] = bad
        pools[1][p, 1, o, hd - 1] = bad
    q = torch.randn(n, nh, hd, generator=g).to(dt)
    out = torch.empty(n, nh, hd, dtype=dt, device="cuda")
    llb.paged_attention(q.cuda(), pools[0].cuda(), pools[1].cuda(), tables.cuda(), i32([0, n]), i32([seq]), out,
                        max_new=max_new)
    got = out.cpu().double()
    want, tol = R.attention(q, k, v, n, seq, hd ** -0.5)
    assert ((got - want).abs() <= tol)[:21].all()
    rest = got[21:].clone()
    for h in range(nh):
        d = 3 if h < nh // 2 else hd - 1
        assert not torch.isfinite(rest[:, h, d]).any()
        if not math.isnan(bad):
            assert (rest[:, h, d] == bad).all()
        rest[:, h, d] = want[21:, h, d]
    assert ((rest - want[21:]).abs() <= tol[21:]).all()


@pytest.mark.parametrize("dtype,hd,max_new", [("bf16", 128, 1), ("f16", 128, 400), ("f32", 32, 4)])
def test_attention_bad_tables_and_offsets(llb, dtype, hd, max_new):
    """Pages outside the pool, lengths past the table and rows outside q are reported; the other requests stand."""
    g = torch.Generator().manual_seed(8)
    dt, page, nkv, nh = DT[dtype], 16, 2, 4
    new, seqs = [2, 2, 2], [50, 60, 70]
    pools, tables, dense = paged_cache(seqs, page, nkv, hd, dt, g)
    q = torch.randn(6, nh, hd, generator=g).to(dt)
    args = [q.cuda(), pools[0].cuda(), pools[1].cuda()]

    def check(tab, cu, sl, code, good):
        out = torch.full((6, nh, hd), 7.0, dtype=dt, device="cuda")
        st = i32([0])
        llb.paged_attention(*args, tab.cuda(), i32(cu), i32(sl), out, max_new=max_new, status=st)
        got = out.cpu().double()
        assert int(st) == code
        for b in good:
            want, tol = R.attention(q[2 * b:2 * b + 2], dense[b][0], dense[b][1], 2, seqs[b], hd ** -0.5)
            assert ((got[2 * b:2 * b + 2] - want).abs() <= tol).all()
        return got

    for wrong in (-1, pools[0].shape[0], 1 << 30):
        tab = tables.clone()
        tab[1, 2] = wrong
        got = check(tab, [0, 2, 4, 6], seqs, llb.LLAMA_ERR_INVALID_ARG, [0, 2])
        assert torch.isfinite(got[2:4]).all()
    check(tables, [0, 2, 4, 6], [50, 16 * tables.shape[1] + 1, 70], llb.LLAMA_ERR_CAPACITY, [0, 2])
    check(tables, [0, 2, 4, 6], [50, -4, 70], llb.LLAMA_ERR_CAPACITY, [0, 2])
    got = check(tables, [0, 2, 4, 900], seqs, llb.LLAMA_ERR_INVALID_ARG, [0, 1])
    assert (got[4:] == 7.0).all()
    # request 1 ends before it starts and is skipped; request 2 starts inside request 0, whose row 1 both then hold
    got = check(tables, [0, 2, 1, 6], [50, 60, 70], llb.LLAMA_ERR_INVALID_ARG, [])
    want, tol = R.attention(q[:2], *dense[0], 2, seqs[0], hd ** -0.5)
    assert ((got[0] - want[0]).abs() <= tol[0]).all()


def test_attention_one_workspace_for_every_call(llb):
    """One workspace, sized for the longest chunk, serves calls of every kind in turn: long caches split over many
    CTAs, chunks on the tile kernel, short ones again."""
    g = torch.Generator().manual_seed(12)
    page, nkv, nh, hd, dt = 64, 1, 8, 128, torch.bfloat16
    jobs = [([1], [20000]), ([300], [2000]), ([1], [20001]), ([2, 200], [9000, 200]), ([1, 1], [5, 15000])]
    ws = None
    for new, seqs in jobs + jobs[::-1]:
        pools, tables, dense = paged_cache(seqs, page, nkv, hd, dt, g)
        q = torch.randn(sum(new), nh, hd, generator=g).to(dt)
        if ws is None:
            ws = llb.paged_attention_workspace(q.cuda(), nkv, 300)
        out = torch.empty(sum(new), nh, hd, dtype=dt, device="cuda")
        cu = [0] + torch.tensor(new).cumsum(0).tolist()
        llb.paged_attention(q.cuda(), pools[0].cuda(), pools[1].cuda(), tables.cuda(), i32(cu), i32(seqs), out,
                            max_new=max(new), workspace=ws)
        got = out.cpu().double()
        for b, n in enumerate(new):
            rows = sorted({0, n // 2, n - 1})            # the 64-bit attention of three rows of each request
            for i in rows:
                want, tol = R.attention(q[cu[b] + i:cu[b] + i + 1], *dense[b], 1, seqs[b] - n + i + 1, hd ** -0.5)
                assert ((got[cu[b] + i] - want[0]).abs() <= tol[0]).all(), (new, seqs, b, i)


def test_attention_on_two_streams_and_in_graphs(llb):
    """Two captured calls with a workspace each, replayed at once on two streams beside eager calls."""
    g = torch.Generator().manual_seed(6)
    dt, page, nkv, nh, hd = torch.bfloat16, 16, 2, 16, 128
    jobs, kept = [], []
    for new, seqs in (([1] * 20, [700 + 13 * i for i in range(20)]), ([300, 1], [900, 1200])):
        pools, tables, dense = paged_cache(seqs, page, nkv, hd, dt, g)
        q = torch.randn(sum(new), nh, hd, generator=g).to(dt)
        a = [q.cuda(), pools[0].cuda(), pools[1].cuda(), tables.cuda(),
             i32([0] + torch.tensor(new).cumsum(0).tolist()), i32(seqs)]
        out = torch.empty_like(a[0])
        ws = llb.paged_attention_workspace(a[0], nkv, max(new))
        llb.paged_attention(*a, out, max_new=max(new), workspace=ws)
        torch.cuda.synchronize()
        want = out.clone()
        stream = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            llb.paged_attention(*a, out, max_new=max(new), workspace=ws)
        jobs.append((a, out, want, stream, graph, max(new)))
        kept.append(ws)                               # a graph's workspace lives as long as the graph
    for _ in range(20):
        for a, out, want, stream, graph, mx in jobs:
            with torch.cuda.stream(stream):
                graph.replay()
        eager = [torch.empty_like(j[1]) for j in jobs]
        for e, (a, _, _, _, _, mx) in zip(eager, jobs):
            llb.paged_attention(*a, e, max_new=mx)            # a workspace of its own
        torch.cuda.synchronize()
        for e, (_, out, want, _, _, _) in zip(eager, jobs):
            assert torch.equal(out, want) and torch.equal(e, want)
            out.zero_()
        torch.cuda.synchronize()


@pytest.mark.parametrize("hd,nkv,max_new", [(128, 8, 1), (128, 8, 200), (64, 8, 200)])
def test_far_pages(llb, hd, nkv, max_new):
    """Pools of more than 2^31 values: append to and attention over their last pages."""
    g = torch.Generator().manual_seed(19)
    page, nh, dt = 64, 8, torch.bfloat16
    n_pages = (1 << 31) // (nkv * page * hd) + 40
    pools = [torch.zeros(n_pages, nkv, page, hd, dtype=dt, device="cuda") for _ in range(2)]
    n, seq = max_new, 300
    ids = [n_pages - 1 - 2 * i for i in range(-(-seq // page))]
    k, v = (torch.randn(seq, nkv, hd, generator=g).to(dt) for _ in range(2))
    pos = torch.arange(seq, dtype=torch.int32)
    slots = torch.tensor([ids[p // page] * page + p % page for p in range(seq)])
    rope = torch.zeros(seq, hd // 2, 2)
    rope[..., 0] = 1.0                                # no rotation
    st = i32([0])
    q_out = torch.empty(seq, nh, hd, dtype=dt, device="cuda")
    q = torch.randn(seq, nh, hd, generator=g).to(dt)
    llb.paged_append(q.cuda(), k.cuda(), v.cuda(), pos.cuda(), slots.cuda(), rope.cuda(), q_out, *pools, status=st)
    assert torch.equal(q_out.cpu(), q)
    out = torch.empty(n, nh, hd, dtype=dt, device="cuda")
    llb.paged_attention(q_out[seq - n:].contiguous(), *pools, i32([ids]), i32([0, n]), i32([seq]), out, max_new=n,
                        status=st)
    assert int(st) == 0
    want, tol = R.attention(q[seq - n:], k, v, n, seq, hd ** -0.5)
    assert ((out.cpu().double() - want).abs() <= tol).all()
    assert int(pools[0][:n_pages - 2 * len(ids)].count_nonzero()) == 0
    del pools
    torch.cuda.empty_cache()


def test_on_a_side_stream(llb):
    """Calls on a stream given by argument and on the current one order themselves with that stream's work."""
    g = torch.Generator().manual_seed(3)
    page, nkv, nh, hd, dt, seq = 16, 2, 8, 128, torch.bfloat16, 500
    pools, tables, dense = paged_cache([seq], page, nkv, hd, dt, g)
    q = torch.randn(1, nh, hd, generator=g).to(dt)
    want, tol = R.attention(q, *dense[0], 1, seq, hd ** -0.5)
    dev = [x.cuda() for x in (pools[0], pools[1], tables)]
    cu, sl = i32([0, 1]), i32([seq])
    torch.cuda.synchronize()
    for given in (True, False):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            late = torch.zeros(1, nh, hd, dtype=dt, device="cuda")
            torch.cuda._sleep(20_000_000)             # the queries arrive late on s
            late.copy_(q.cuda())
            out = torch.empty_like(late)
            if not given:
                llb.paged_attention(late, *dev, cu, sl, out, max_new=1)
        if given:
            llb.paged_attention(late, *dev, cu, sl, out, max_new=1, stream=s)
        s.synchronize()
        assert ((out.cpu().double() - want).abs() <= tol).all()


# ---------------------------------------------------------------- refusals that need tensors

def test_wrong_tensors_are_refused(llb):
    z = lambda *shape, dt=torch.bfloat16: torch.zeros(*shape, dtype=dt, device="cuda")
    n0 = llb.launch_count()
    q, kv, pools, rope = z(4, 8, 64), z(4, 2, 64), [z(3, 2, 16, 64) for _ in range(2)], z(9, 32, 2, dt=torch.float32)
    pos, slots = i32([0, 1, 2, 3]), torch.arange(4, device="cuda")
    good = [q, kv, kv, pos, slots, rope, q.clone(), *pools]
    for i, bad in ((0, q.half()), (0, q.cpu()), (0, z(4, 8, 128)), (0, z(4, 8, 64).transpose(0, 1)), (1, z(4, 3, 64)),
                   (2, kv.float()), (3, pos.long()), (3, pos[:3]), (4, slots.int()), (4, slots[:3]), (5, rope.half()),
                   (5, z(9, 16, 2, dt=torch.float32)), (6, z(4, 8, 64, dt=torch.int16)), (6, z(3, 8, 64)),
                   (7, pools[0].float()), (8, z(3, 2, 32, 64)), (7, pools[0].transpose(1, 2)), (6, z(8, 4, 64).transpose(0, 1))):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            llb.paged_append(*args)
    with pytest.raises(ValueError):
        llb.paged_append(*good, q_norm=z(32, dt=torch.float32))
    with pytest.raises(ValueError):
        llb.paged_append(*good, status=z(1, dt=torch.int64))
    with pytest.raises(llb.LlamaError):
        llb.paged_append(*good, eps=-1.0)
    tab, cu, sl = i32([[0, 1]]), i32([0, 4]), i32([20])
    ws = llb.paged_attention_workspace(q, 2, 4)
    base = [q, *pools, tab, cu, sl, q.clone()]
    for i, bad in ((0, q.float()), (0, z(4, 8, 32)), (1, pools[0].half()), (3, tab.long()), (3, tab[0]), (4, i32([0])),
                   (5, i32([20, 3])), (6, z(4, 4, 64)), (6, q.cpu()), (4, cu.cpu())):
        args = list(base)
        args[i] = bad
        with pytest.raises(ValueError):
            llb.paged_attention(*args, workspace=ws)
    with pytest.raises(llb.LlamaError):
        llb.paged_attention(*base, workspace=ws[:1024])
    with pytest.raises(ValueError):
        llb.paged_attention(*base, workspace=ws.view(torch.int32))
    with pytest.raises(llb.LlamaError):
        llb.paged_attention(*base, workspace=ws, scale=float("nan"))
    lg, f, out = z(3, 50, dt=torch.float32), z(3, dt=torch.float32), i32([0] * 3)
    for args, kw in (((lg.half(), f, f, out), {}), ((lg, f[:2], f, out), {}), ((lg, f, f.double(), out), {}),
                     ((lg, f, f, out.long()), {}), ((lg[:, ::2], f, f, out), {}), ((lg, f, f, out), dict(top_k=f)),
                     ((lg, f, f, out), dict(top_p=f[:1])), ((lg, f, f, out), dict(min_p=f.cpu()))):
        with pytest.raises(ValueError):
            llb.sample_rows(*args, **kw)
    c = i32([1, 2])
    plan = [c, c, i32([[0, 1], [2, 3]]), i32([4, 5]), i32([2]), 16, c.clone(), i32([0] * 3), torch.zeros(4, dtype=torch.int64, device="cuda"),
            i32([0] * 4), i32([0])]
    for i, bad in ((1, i32([1])), (2, i32([[0, 1]])), (2, i32([0, 1])), (3, torch.zeros(2, device="cuda")), (4, i32([1, 2])),
                   (6, c.long()), (7, i32([0] * 2)), (8, i32([0] * 4)), (9, i32([0] * 3)), (10, i32([1, 2]))):
        args = list(plan)
        args[i] = bad
        with pytest.raises(ValueError):
            llb.paged_plan(*args)
    with pytest.raises(llb.LlamaError):
        llb.paged_plan(*plan[:5], 17, *plan[6:])
    assert llb.launch_count() == n0


# ---------------------------------------------------------------- a serving run

@pytest.mark.parametrize("dtype,hd,nh,nkv,page", [("bf16", 128, 8, 2, 16), ("f16", 64, 4, 4, 32), ("f32", 32, 8, 2, 16)])
def test_serving_steps(llb, dtype, hd, nh, nkv, page):
    """Requests come, grow in chunks and single tokens, and end; each step plans, appends, attends and samples.
    Every attention row is checked against the 64-bit attention over the very values the cache was given."""
    g = torch.Generator().manual_seed(21)
    dt = DT[dtype]
    B, width, n_pages, room = 4, 12, 30, 200
    rope = torch.empty(width * page, hd // 2, 2, device="cuda")
    llb.rope_table(rope)
    qw, kw = (1 + 0.1 * torch.randn(hd, generator=g) for _ in range(2))
    tables = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(n_pages, generator=g).to(torch.int32).cuda()
    count, seq, cu = i32([n_pages]), i32([0] * B), i32([0] * (B + 1))
    slots = torch.empty(room, dtype=torch.int64, device="cuda")
    pos = torch.empty(room, dtype=torch.int32, device="cuda")
    pools = [torch.full((n_pages, nkv, page, hd), float("nan"), dtype=dt, device="cuda") for _ in range(2)]
    st = i32([0])
    V = 300
    proj = torch.randn(nh * hd, V, generator=g).cuda() * 0.1
    held = [[] for _ in range(B)]                     # (k, v) rows each request holds, 64-bit rounded
    steps = [[5, 0, 100, 1], [1, 33, 1, 1], [1, 1, -1, 60], [70, 1, 9, 1], [1, 1, 1, -1], [-1, 1, 1, 40], [2, 2, 2, 2]]
    for new in steps:
        llb.paged_plan(seq, i32(new), tables, free, count, page, seq, cu, slots, pos, count, status=st)
        total = sum(max(n, 0) for n in new)
        qkv = torch.randn(total, (nh + 2 * nkv) * hd, generator=g)
        d = qkv.cuda()
        q, k, v = (x.unflatten(1, (-1, hd)) for x in d.split([nh * hd, nkv * hd, nkv * hd], 1))
        q_out = torch.empty(total, nh, hd, dtype=dt, device="cuda")
        out = torch.empty_like(q_out)
        llb.paged_append(q, k, v, pos, slots, rope, q_out, *pools, q_norm=qw.cuda(), k_norm=kw.cuda(), status=st)
        llb.paged_attention(q_out, *pools, tables, cu, seq, out, max_new=max(new), status=st)
        logits = (out.float().reshape(total, -1) @ proj).contiguous()
        u = torch.rand(total, generator=g)
        tok = torch.empty(total, dtype=torch.int32, device="cuda")
        params = [torch.full((total,), x, device="cuda") for x in (0.8, 0.95, 0.02)]
        llb.sample_rows(logits, params[0], u.cuda(), tok, top_k=i32([50] * total), top_p=params[1], min_p=params[2])
        torch.cuda.synchronize()
        assert int(st) == 0
        rows = cu.tolist()
        tab, flat = tables.cpu(), [p.cpu().transpose(1, 2).reshape(-1, nkv, hd) for p in pools]
        for b, n in enumerate(new):
            if n < 0:
                held[b] = []
                continue
            sl = slots[rows[b]:rows[b + 1]].cpu()
            held[b] += [(flat[0][s].clone(), flat[1][s].clone()) for s in sl]
            want_k, tol_k = R.norm_rotate(k[rows[b]:rows[b + 1]].cpu(), kw, 1e-5,
                                          rope.cpu()[pos[rows[b]:rows[b + 1]].cpu().long()], dt)
            assert ((flat[0][sl].double() - want_k).abs() <= tol_k).all()
            assert len(held[b]) == int(seq[b])
            if n == 0:
                continue
            ks, vs = (torch.stack([h[i] for h in held[b]]) for i in range(2))
            want, tol = R.attention(q_out[rows[b]:rows[b + 1]].cpu(), ks, vs, n, len(held[b]), hd ** -0.5)
            assert ((out[rows[b]:rows[b + 1]].cpu().double() - want).abs() <= tol).all()
        lg = logits.cpu()
        want_tok = [R.sample(lg[i], float(params[0][0]), 50, float(params[1][0]), float(params[2][0]), float(u[i]))
                    for i in range(total)]
        assert tok.tolist() == want_tok
