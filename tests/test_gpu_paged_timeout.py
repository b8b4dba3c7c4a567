"""The bounded waits of the chunk kernel, exercised without a GPU fault: one
ring stage of CTA 0 never comes (llama_debug_stall without a model), every
wait of that launch gives up after 1 ms, the call returns with
LLAMA_ERR_DEVICE_TIMEOUT in its status word, and the next call with a zeroed
workspace is right."""
import time

import pytest
import torch

import paged_reference as R
from test_gpu_paged import DT, i32, paged_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def llb(cuda_device):
    import decoder_only_transformer_llama_b200 as m
    yield m
    m.paged_debug_stall(-1)


def call(llb, args, nkv, ws, n):
    out = torch.full_like(args[0], 7.0)
    st = i32([0])
    t0 = time.monotonic()
    llb.paged_attention(*args, out, max_new=n, workspace=ws, status=st)
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 5.0
    return out.cpu(), int(st)


# CTA 0 owns three or four units: stages 0 .. 5 at least (K and V of each)
@pytest.mark.parametrize("dtype,hd,stages", [("bf16", 128, [0, 1, 2, 3, 5]), ("f16", 64, [0, 3, 5])])
@pytest.mark.parametrize("new,seq", [(300, 2000), (40, 4000)])
def test_a_stage_that_never_comes(llb, dtype, hd, stages, new, seq):
    """Chunks of two sub-tiles and of one."""
    g = torch.Generator().manual_seed(71)
    nh, nkv, dt = 4, 2, DT[dtype]
    pools, tables, dense = paged_cache([seq], 32, nkv, hd, dt, g)
    q = torch.randn(new, nh, hd, generator=g).to(dt)
    want, tol = R.attention(q, *dense[0], new, seq, hd ** -0.5)
    args = [q.cuda(), pools[0].cuda(), pools[1].cuda(), tables.cuda(), i32([0, new]), i32([seq])]
    ws = llb.paged_attention_workspace(args[0], nkv, new)
    good, st = call(llb, args, nkv, ws, new)
    assert st == 0 and ((good.double() - want).abs() <= tol).all()
    for stage in stages:
        llb.paged_debug_stall(stage, wait_limit_ns=1_000_000)
        _, st = call(llb, args, nkv, ws, new)
        assert st == llb.LLAMA_ERR_DEVICE_TIMEOUT, stage
        ws.zero_()
        out, st = call(llb, args, nkv, ws, new)
        assert st == 0 and torch.equal(out, good), stage


def test_a_stall_is_taken_once_by_the_chunk_kernel(llb):
    g = torch.Generator().manual_seed(72)
    pools, tables, dense = paged_cache([500], 16, 1, 64, torch.bfloat16, g)
    q = torch.randn(100, 1, 64, generator=g).bfloat16().cuda()
    rest = [pools[0].cuda(), pools[1].cuda(), tables.cuda()]
    one = [q[:1].contiguous(), *rest, i32([0, 1]), i32([500])]
    many = [q, *rest, i32([0, 100]), i32([500])]
    ws = llb.paged_attention_workspace(q, 1, 100)
    good, st = call(llb, many, 1, ws, 100)
    assert st == 0
    llb.paged_debug_stall(1000)                           # past the end of CTA 0's run
    assert call(llb, one, 1, ws, 1)[1] == 0               # not the chunk kernel: still armed
    out, st = call(llb, many, 1, ws, 100)
    assert st == 0 and torch.equal(out, good)
    llb.paged_debug_stall(0)
    llb.paged_debug_stall(-1)                             # disarmed before any launch took it
    out, st = call(llb, many, 1, ws, 100)
    assert st == 0 and torch.equal(out, good)
