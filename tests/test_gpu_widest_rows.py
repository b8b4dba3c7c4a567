"""The samplers on rows of the widest vocabulary whose tokens all have the full
mass: sums of 2^18 such masses must fit 64 bits."""
import math

import pytest
import torch

import paged_reference as R
from test_gpu_sample_rows import check, f32, rows

pytestmark = pytest.mark.gpu
WIDEST = 262144


@pytest.fixture(scope="module")
def llb(cuda_device):
    import decoder_only_transformer_llama_b200 as m
    return m


def uniforms(B):
    """Among them the borders of the draw and of whole numbers of tokens."""
    u = torch.rand(B, generator=torch.Generator().manual_seed(B)).tolist()
    u[:5] = [0.0, 1.0 - 2.0 ** -24, 0.5, 0.75, 0.3]
    return u


@pytest.mark.parametrize("V", [WIDEST - 1, WIDEST])
@pytest.mark.parametrize("B", [6, 40, 66])
def test_rows_of_equal_logits(llb, B, V):
    lg, u = torch.full((B, V), 1.5), uniforms(B)
    t = [(1.0, 0.05, 7.0)[b % 3] for b in range(B)]
    k = [(0, 10, 3000, 200000, V - 1, V)[b % 6] for b in range(B)]
    p = [(1.0, 0.5, 0.95, 0.0, 0.3)[b % 5] for b in range(B)]
    m = [(0.0, 1.0, 0.25, 0.0)[b % 4] for b in range(B)]
    check(llb, lg, t, None, None, None, u)
    check(llb, lg, t, k, None, None, u)
    check(llb, lg, t, None, p, None, u)
    check(llb, lg, t, None, None, m, u)
    check(llb, lg, t, k, p, m, u)


@pytest.mark.parametrize("B", [6, 40, 66])
def test_rows_of_infinite_logits(llb, B):
    lg, u = torch.full((B, WIDEST), math.inf), uniforms(B)
    k = [(0, 7, 100000)[b % 3] for b in range(B)]
    p = [(1.0, 0.9, 0.5, 0.99)[b % 4] for b in range(B)]
    check(llb, lg, [1.0] * B, None, None, None, u)
    check(llb, lg, [1.0] * B, k, p, None, u)


@pytest.mark.parametrize("B", [5, 40, 66])
def test_distinct_logits_of_equal_mass(llb, B):
    """Temperatures that leave every exponential at 1: the order still counts."""
    lg, _ = rows(B, WIDEST, 7)
    u = uniforms(B)
    k = [(0, 3, 60, 290, 20000)[b % 5] for b in range(B)]
    p = [(0.9, 0.5, 1.0, 0.99)[b % 4] for b in range(B)]
    m = [(0.1, 0.0, 1.0)[b % 3] for b in range(B)]
    check(llb, lg, [9e29] * B, None, None, None, u)
    check(llb, lg, [9e29] * B, k, p, None, u)
    check(llb, lg, [9e29] * B, None, p, m, u)


@pytest.mark.parametrize("B", [6, 40, 66])
def test_ordinary_widest_rows(llb, B):
    lg, u = rows(B, WIDEST, 19)
    t = [(0.7, 1.0, 3.0, 30.0)[b % 4] for b in range(B)]
    k = [(0, 50, 0, 3, 5000)[b % 5] for b in range(B)]
    p = [(0.9, 1.0, 0.99)[b % 3] for b in range(B)]
    m = [(0.0, 0.0, 0.02)[b // 3 % 3] for b in range(B)]
    check(llb, lg, t, k, p, m, u)
    check(llb, lg, t, None, p, None, u)
    check(llb, lg, t, None, None, m, u)


@pytest.mark.parametrize("V", [WIDEST - 1, WIDEST])
def test_llama_sample_of_full_masses(llb, V):
    """The scalar sampler on the same rows: equal logits, and distinct ones of equal mass."""
    distinct, _ = rows(6, V, 29)
    for lg, t in ((torch.full((6, V), -2.25), 0.8), (distinct, 9e29)):
        d, u = lg.cuda(), uniforms(6)
        for p in (0.3, 0.9, 1.0):
            out = torch.full((6,), -5, dtype=torch.int32, device="cuda")
            llb.sample(d, t, p, torch.tensor(u).cuda(), out)
            assert out.tolist() == [R.sample(lg[b], f32(t), 0, f32(p), 0.0, f32(u[b])) for b in range(6)]
