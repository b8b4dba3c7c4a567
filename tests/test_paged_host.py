"""Refusals of the paged-cache operators and the row sampler: every bad
argument is turned into an error on the host, before anything is launched (no
GPU needed; the pointers are never read)."""
import ctypes

import pytest
import torch

llb = pytest.importorskip("decoder_only_transformer_llama_b200",
                          reason="library not built (run decoder_only_transformer_llama_b200/build.py)")
import paged_reference as R  # noqa: E402

P = 1 << 20       # stands for a device address, 256-byte aligned
L = llb.lib()


def call(name, defaults, **change):
    args = dict(defaults)
    for k in change:
        assert k in args
    args.update(change)
    n = llb.launch_count()
    rc = getattr(L, name)(*args.values())
    assert llb.launch_count() == n
    return rc, llb.last_error()


PLAN = dict(ctx=P, new=P, B=4, page=16, tables=P, width=8, free=P, n_pages=9, count=P, T=8, seq=P, cu=P, slots=P,
            pos=P, left=P, status=None, stream=None)
APPEND = dict(q=P, qs=512, k=P, ks=256, v=P, vs=256, in_dtype=1, T=3, nh=4, nkv=2, hd=128, qw=None, kw=None, eps=1e-5,
              rope=P, rope_len=64, pos=P, slots=P, q_out=P, kp=P, vp=P, n_pages=4, page=16, dtype=1, status=None,
              stream=None)
ATTN = dict(q=P, kp=P, vp=P, dtype=1, T=3, nh=4, nkv=2, hd=128, B=2, cu=P, seq=P, tables=P, width=4, n_pages=4, page=16,
            max_new=1, scale=0.1, out=P, ws=P, ws_bytes=1 << 40, status=None, stream=None)
ROWS = dict(logits=P, B=2, V=100, t=P, k=None, p=None, m=None, u=P, out=P, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(ctx=None), 1), (dict(new=None), 1), (dict(tables=None), 1), (dict(free=None), 1), (dict(count=None), 1),
    (dict(seq=None), 1), (dict(cu=None), 1), (dict(slots=None), 1), (dict(pos=None), 1), (dict(left=None), 1),
    (dict(B=0), 1), (dict(B=-1), 1), (dict(B=1025), 2), (dict(page=0), 1), (dict(page=8), 1), (dict(page=48), 1),
    (dict(page=512), 1), (dict(width=0), 1), (dict(n_pages=0), 1), (dict(T=-1), 1)])
def test_plan_refusals(change, code):
    rc, msg = call("llama_paged_plan", PLAN, **change)
    assert rc == code and msg


@pytest.mark.parametrize("change", [
    dict(q=None), dict(k=None), dict(v=None), dict(q_out=None), dict(kp=None), dict(vp=None), dict(rope=None),
    dict(pos=None), dict(slots=None), dict(T=-1), dict(nh=0), dict(nkv=0), dict(nh=3), dict(nh=32, qs=4096), dict(hd=96),
    dict(hd=256), dict(in_dtype=2), dict(in_dtype=7), dict(dtype=3), dict(dtype=0), dict(eps=-1.0),
    dict(eps=float("nan")), dict(rope_len=0), dict(n_pages=0), dict(page=24), dict(qs=511), dict(qs=508), dict(ks=255),
    dict(vs=0), dict(q=P + 8), dict(k=P + 2), dict(v=P + 4), dict(q_out=P + 8), dict(kp=P + 8), dict(vp=P + 8),
    dict(rope=P + 8), dict(qw=P + 4), dict(kw=P + 4), dict(qs=516), dict(ks=260), dict(vs=260)])
def test_append_refusals(change):
    rc, msg = call("llama_paged_append", APPEND, **change)
    assert rc == 1 and msg


@pytest.mark.parametrize("change,code", [
    (dict(q=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(cu=None), 1), (dict(seq=None), 1),
    (dict(tables=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(ws=P + 16), 1), (dict(ws_bytes=8), 1),
    (dict(T=-1), 1), (dict(nh=6), 1), (dict(nh=32), 1), (dict(hd=48), 1), (dict(dtype=5), 1), (dict(B=0), 1),
    (dict(B=1025), 2), (dict(width=0), 1), (dict(width=1 << 27), 1), (dict(n_pages=0), 1), (dict(page=20), 1),
    (dict(max_new=0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(q=P + 8), 1),
    (dict(out=P + 2), 1), (dict(kp=P + 8), 1), (dict(vp=P + 8), 1), (dict(nh=2048, nkv=256), 1)])
def test_attention_refusals(change, code):
    rc, msg = call("llama_paged_attention", ATTN, **change)
    assert rc == code and msg


@pytest.mark.parametrize("change", [
    dict(logits=None), dict(t=None), dict(u=None), dict(out=None), dict(B=-1), dict(V=0), dict(V=262145)])
def test_sample_rows_refusals(change):
    rc, msg = call("llama_sample_rows", ROWS, **change)
    assert rc == 1 and msg


def test_rope_table_refusals():
    for args in ((None, 4, 64, 1e4), (P, 0, 64, 1e4), (P, 4, 63, 1e4), (P, 4, 64, 0.0), (P + 4, 4, 64, 1e4),
                 (P, 1 << 30, 128, 1e4)):
        assert L.llama_rope_table(*args, None) == 1 and llb.last_error()


def test_empty_calls_launch_nothing():
    n = llb.launch_count()
    assert call("llama_paged_append", APPEND, T=0)[0] == 0
    assert call("llama_paged_attention", ATTN, T=0)[0] == 0
    assert call("llama_sample_rows", ROWS, B=0)[0] == 0
    assert llb.launch_count() == n


def test_sample_rows_of_no_rows_and_of_too_many():
    n = llb.launch_count()
    assert call("llama_sample_rows", ROWS, B=0, logits=None, t=None, u=None, out=None)[0] == 0    # empty tensors have no address
    rc, msg = call("llama_sample_rows", ROWS, B=1 << 29, V=1)             # past the grid's 31 bits
    assert rc == 1 and msg
    assert llb.launch_count() == n


def test_workspace_sizes():
    f = L.llama_paged_attention_workspace_bytes
    for dt in (0, 1, 2):
        for hd in (32, 64, 128):
            sizes = [f(8, 2, hd, dt, n) for n in (1, 2, 16, 100, 5000)]
            assert all(s > 0 for s in sizes)
            assert sizes == sorted(sizes)                # one for the longest chunk serves the shorter
    assert f(8, 3, 64, 1, 1) == 0 and f(8, 2, 60, 1, 1) == 0 and f(8, 2, 64, 9, 1) == 0 and f(8, 2, 64, 1, 0) == 0


def test_cpu_tensors_are_refused():
    t = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        llb.paged_plan(t, t, t, t, t, 16, t, t, t, t, t)
    with pytest.raises(ValueError, match="CUDA"):
        llb.sample_rows(torch.zeros(2, 5), t, t, t)
    with pytest.raises(ValueError, match="CUDA"):
        llb.rope_table(torch.zeros(4, 16, 2))
    x = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        llb.paged_append(x, x, x, t, t, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        llb.paged_attention(x, x, x, t, t, t, x)


# ---------------------------------------------------------------- the definitions themselves

def test_reference_plan_by_hand():
    got = R.plan([3, 32, 16], [14, -1, 1], 16, [[4, -7], [0, 1], [2, -7]], [5, 3, -9, -9, -9, -9], 2, 2, 16, 6)
    # pages 0 and 1 return on top of 5 and 3; request 0 takes 1, request 2 takes 0
    assert got["tables"] == [[4, 1], [0, 1], [2, 0]]
    assert got["left"] == 2 and got["seq"] == [17, 0, 17] and got["cu"] == [0, 14, 14, 15]
    assert got["slots"] == [4 * 16 + p for p in range(3, 16)] + [16] + [0] + [-1]
    assert got["pos"] == list(range(3, 17)) + [16, -1]


def test_reference_sample_by_hand():
    lg = torch.log(torch.tensor([0.1, 0.4, 0.2, 0.3]))
    pick = lambda u, k=0, p=1.0, m=0.0: R.sample(lg, 1.0, k, p, m, u)
    assert [pick(u) for u in (0.0, 0.39, 0.41, 0.69, 0.71, 0.89, 0.91)] == [1, 1, 3, 3, 2, 2, 0]
    assert [pick(u, k=2) for u in (0.5, 0.6)] == [1, 3]                  # 0.4 of 0.7
    assert [pick(u, p=0.5) for u in (0.5, 0.6, 0.99)] == [1, 3, 3]      # 0.4 lies before 3, 0.7 before 2
    assert [pick(u, k=2, p=0.5) for u in (0.5, 0.99)] == [1, 1]         # 0.4 lies before 3, above 0.5 * 0.7
    assert [pick(u, m=0.6) for u in (0.5, 0.99)] == [1, 3]


def test_argument_counts_match_the_header():
    for name, d in (("llama_paged_plan", PLAN), ("llama_paged_append", APPEND), ("llama_paged_attention", ATTN),
                    ("llama_sample_rows", ROWS)):
        assert len(getattr(L, name).argtypes) == len(d)
        assert getattr(L, name).restype is ctypes.c_int
