"""One request over a long cache, split over more contributors than one merge
takes: partial results are merged in place level by level, and every call
gives the same bits."""
import pytest
import torch

import paged_reference as R
from test_gpu_paged import DT, i32, paged_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def llb(cuda_device):
    import decoder_only_transformer_llama_b200 as m
    return m


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("new,nh,nkv,hd", [(1, 1, 1, 32), (3, 2, 1, 32), (5, 1, 1, 64), (2, 8, 1, 64), (1, 1, 1, 128),
                                           (7, 2, 2, 128)])
def test_deep_merges_repeat(llb, dtype, new, nh, nkv, hd):
    """1 to 16 rows a tile, so that the merging warps are full, partly filled or idle."""
    g = torch.Generator().manual_seed(61)
    dt, seq = DT[dtype], 30011
    pools, tables, dense = paged_cache([seq], 64, nkv, hd, dt, g)
    q = torch.randn(new, nh, hd, generator=g).to(dt)
    want, tol = R.attention(q, *dense[0], new, seq, hd ** -0.5)
    args = [q.cuda(), pools[0].cuda(), pools[1].cuda(), tables.cuda(), i32([0, new]), i32([seq])]
    ws = llb.paged_attention_workspace(args[0], nkv, 1)
    st = i32([0])
    outs = [torch.full((new, nh, hd), 7.0, dtype=dt, device="cuda") for _ in range(60)]
    for out in outs:
        llb.paged_attention(*args, out, max_new=1, workspace=ws, status=st)
    got = torch.stack(outs).cpu()
    assert int(st) == 0
    assert ((got[0].double() - want).abs() <= tol).all()
    assert (got == got[0]).all()
