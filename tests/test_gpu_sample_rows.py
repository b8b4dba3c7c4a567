"""llama_sample_rows against its 64-bit definition: the same tokens, with each
row's own parameters, on ordinary, tied and degenerate rows."""
import math

import pytest
import torch

import paged_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def llb(cuda_device):
    import decoder_only_transformer_llama_b200 as m
    return m


def draw(llb, logits, t, k, p, m, u):
    B = logits.shape[0]
    out = torch.full((B,), -5, dtype=torch.int32, device="cuda")
    f = lambda x: torch.as_tensor(x, dtype=torch.float32).cuda()
    llb.sample_rows(logits.cuda(), f(t), f(u), out, top_k=None if k is None else torch.tensor(k, dtype=torch.int32).cuda(),
                    top_p=None if p is None else f(p), min_p=None if m is None else f(m))
    return out.tolist()


def f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


def check(llb, logits, t, k, p, m, u):
    got = draw(llb, logits, t, k, p, m, u)
    B = logits.shape[0]
    want = [R.sample(logits[b], f32(t[b]), 0 if k is None else k[b], 1.0 if p is None else f32(p[b]),
                     0.0 if m is None else f32(m[b]), f32(u[b])) for b in range(B)]
    assert got == want


def rows(B, V, seed):
    g = torch.Generator().manual_seed(seed)
    return 3.0 * torch.randn(B, V, generator=g), torch.rand(B, generator=g).tolist()


@pytest.mark.parametrize("V", [1, 2, 7, 32, 1000, 1025, 32000, 32001, 100003, 131072, 262144])
def test_every_filter(llb, V):
    B = 12 if V <= 40000 else 5
    lg, u = rows(B, V, V)
    t = [0.6, 1.0, 0.0, 1.7, 0.05, 30.0, 1.0, 1.0, 0.9, 0.7, 1.0, 2.0][:B]
    k = [0, 50, 3, 1, 0, 0, V, V + 9, -3, 2, 700, 40][:B]
    p = [0.9, 0.95, 0.5, 1.0, 0.9, 0.8, 0.0, 1.0, 0.3, 2.0, 0.99, 0.999][:B]
    m = [0.0, 0.05, 0.5, 0.0, 0.1, 0.0, 0.0, 1.0, 0.02, 0.3, 0.001, 0.0][:B]
    check(llb, lg, t, k, p, m, u)
    check(llb, lg, t, k, None, None, u)
    check(llb, lg, t, None, p, None, u)
    check(llb, lg, t, None, None, m, u)
    check(llb, lg, t, None, None, None, u)


@pytest.mark.parametrize("B,V", [(33, 9000), (33, 70001), (64, 40002), (65, 9000), (65, 70001), (100, 131073)])
def test_every_filter_in_batches(llb, B, V):
    """The narrower clusters, whose slices stay in shared memory or are read again."""
    lg, u = rows(B, V, B + V)
    lg[1::7] *= 0.05                                      # near ties: crowded bins
    t = [(0.7, 1.0, 0.0, 1.6)[b % 4] for b in range(B)]
    k = [(0, 50, 0, 3, 5000)[b % 5] for b in range(B)]
    p = [(0.9, 1.0, 0.99)[b % 3] for b in range(B)]
    m = [(0.0, 0.0, 0.02)[b // 3 % 3] for b in range(B)]
    check(llb, lg, t, k, p, m, u)
    check(llb, lg, t, None, p, None, u)
    check(llb, lg, t, None, None, m, u)


@pytest.mark.parametrize("u", [0.0, 1.0 - 2.0 ** -24])
def test_ends_of_the_draw(llb, u):
    lg, _ = rows(6, 5000, 3)
    check(llb, lg, [1.0] * 6, [0, 1, 2, 10, 100, 4999], [1.0, 1.0, 0.5, 0.9, 0.99, 1.0], [0.0, 0.0, 0.0, 0.01, 0.0, 0.0],
          [u] * 6)


@pytest.mark.parametrize("grid", [0.25, 2.0, 100.0])
def test_ties_go_to_the_lowest_id(llb, grid):
    """Logits on a coarse grid: whole runs of equal masses, cut in their middle by top-k and top-p."""
    lg, u = rows(10, 20000, 17)
    lg = (lg / grid).round() * grid + 0.0
    check(llb, lg, [1.0] * 10, [0, 7, 100, 3000, 0, 0, 19999, 1, 5, 12000], [1.0, 0.9, 0.5, 0.99, 0.7, 0.2, 1.0, 1.0, 0.6, 0.95],
          [0.0, 0.0, 0.01, 0.0, 0.2, 0.0, 0.0, 0.0, 0.0, 0.0], u)


@pytest.mark.parametrize("V", [500, 32000, 150000])
def test_equal_rows(llb, V):
    lg = torch.full((6, V), 1.5)
    u = [0.0, 0.1, 0.5, 0.73, 0.999, 0.25]
    # equal masses: the draw is the first id whose count exceeds u * kept
    check(llb, lg, [1.0] * 6, [0, 10, 0, 77, 0, 0], [1.0, 1.0, 0.5, 0.3, 1.0, 0.0], [0.0, 0.0, 0.0, 0.0, 1.0, 0.0], u)


def test_many_wide_rows_of_near_ties(llb):
    """More than 2^17 tokens of one mass in each of many rows: a CTA's share of a
    bin's sums must not pass 32 bits (0.5 below the maximum at T = 0.8, the 16-bit
    parts of the mass are 0xb92b and 0xed6d)."""
    B, V = 66, 262144
    _, u = rows(B, 1, 41)
    lg = torch.zeros(V)
    lg[77777] = 0.5
    check(llb, lg.repeat(B, 1), [0.8] * B, None, None, None, u)
    check(llb, lg.repeat(B, 1), [0.8] * B, [200000] * B, [0.95] * B, None, u)


@pytest.mark.parametrize("scale,offset,t", [
    (1e-38, 0.0, 1.0), (1e-38, 0.0, 1e-38), (1e-44, 0.0, 1e-43), (4.0, 1e8, 0.15), (64.0, -1e8, 20.0), (1e30, 0.0, 1e30), (1e30, 0.0, 9e29),
    (3e37, 0.0, 1e30), (3e37, 0.0, 9e29), (1e-3, 5.0, 1e30), (1e-3, 5.0, 9e29), (0.02, 0.0, 1e-4), (40.0, 0.0, 1.0), (1.0, 1e4, 1.0)])
def test_extreme_scales(llb, scale, offset, t):
    """Distances from denormal to overflowing, temperatures as small and as large."""
    for V in (300, 40000, 140000):
        lg, u = rows(5, V, 51)
        lg = (lg / 3.0 * scale + offset).contiguous()
        check(llb, lg, [t] * 5, None, None, None, u)
        check(llb, lg, [t] * 5, [0, 3, 60, 290, 20000], [0.9, 0.5, 0.9, 1.0, 0.99], [0.0, 0.0, 0.1, 0.0, 0.0], u)
        check(llb, lg, [t] * 5, None, None, [0.1, 0.5, 0.9, 0.01, 1e-30], u)


def test_masked_logits(llb):
    """-inf, NaN and +inf entries, rows with one token left, rows with none."""
    lg, u = rows(12, 3000, 8)
    inf, nan = math.inf, math.nan
    lg[0, ::2] = -inf
    lg[1, 1:] = -inf
    lg[2, :-1] = -inf
    lg[3, :] = -inf
    lg[4, :] = nan
    lg[5, 100:2900] = nan
    lg[6, 17] = inf
    lg[7, [5, 900, 2999]] = inf
    lg[8, 7] = inf
    lg[8, 0] = -inf
    lg[9, :] = -3.4e38
    lg[10, 0] = 3.4e38
    lg[10, 1] = -3.4e38
    lg[11] = 0.0
    lg[11, 1::2] = -0.0
    ones = [1.0] * 12
    u[2] = 1.0 - 2.0 ** -24
    check(llb, lg, ones, [0] * 12, ones, [0.0] * 12, u)
    check(llb, lg, ones, [50] * 12, [0.9] * 12, [0.02] * 12, u)
    check(llb, lg, [0.0] * 12, [50] * 12, [0.9] * 12, [0.02] * 12, u)


def test_parameters_out_of_range_give_minus_one(llb):
    nan, inf = math.nan, math.inf
    lg, u = rows(9, 100, 2)
    t = [-1.0, nan, inf, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0]
    p = [0.9, 0.9, 0.9, -0.1, nan, 0.9, 0.9, 0.9, 0.9]
    m = [0.0, 0.0, 0.0, 0.0, 0.0, -0.1, 1.1, nan, 0.1]
    got = draw(llb, lg, t, None, p, m, u)
    assert got[:8] == [-1] * 8
    assert 0 <= got[8] < 100


def test_uniforms_are_clamped(llb):
    lg, _ = rows(4, 1000, 5)
    lg[:, 500:] = -math.inf
    got = draw(llb, lg, [1.0] * 4, None, None, None, [1.0, 2.0, -1.0, math.nan])
    ends = draw(llb, lg, [1.0] * 4, None, None, None, [1.0 - 2.0 ** -24] * 2 + [0.0] * 2)
    assert got == ends


def test_agrees_with_sample(llb):
    """The picks of llama_sample for one temperature and top-p, and its argmax."""
    lg, u = rows(16, 32000, 23)
    d = lg.cuda()
    for t, p in ((0.6, 0.9), (1.3, 0.5), (0.0, 0.9)):
        want = torch.empty(16, dtype=torch.int32, device="cuda")
        llb.sample(d, t, p, torch.tensor(u).cuda(), want)
        assert draw(llb, lg, [t] * 16, None, [p] * 16, None, u) == want.tolist()


def test_many_rows_in_a_graph(llb):
    """More rows than SMs, captured once and replayed on new logits."""
    B, V = 300, 4000
    lg, u = rows(B, V, 31)
    d, ud = torch.empty(B, V, device="cuda"), torch.tensor(u).cuda()
    t = torch.full((B,), 0.9, device="cuda")
    k = torch.full((B,), 40, dtype=torch.int32, device="cuda")
    out = torch.empty(B, dtype=torch.int32, device="cuda")
    d.copy_(lg)
    llb.sample_rows(d, t, ud, out, top_k=k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        llb.sample_rows(d, t, ud, out, top_k=k)
    for seed in (32, 33):
        lg, _ = rows(B, V, seed)
        d.copy_(lg)
        graph.replay()
        torch.cuda.synchronize()
        assert out.tolist() == [R.sample(lg[b], f32(0.9), 40, 1.0, 0.0, f32(u[b])) for b in range(B)]
