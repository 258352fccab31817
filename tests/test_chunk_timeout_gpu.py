"""The timeout path of the chunk attention kernel, in a form that faults and hangs
nothing (as tests/test_serving_timeout_gpu.py does for the others): an instance
whose waits have a 200 us budget never loads its first K stage, the waits for it
run out, every role of both CTAs leaves its loop, and the grid ends with
MLA_ERR_TIMEOUT in the status word.  A normal call right after gives the usual
result."""

import time

import pytest
import torch

import mla_paged_kv_gb300 as mla

pytestmark = pytest.mark.gpu

MLA_ERR_TIMEOUT, UNSUPPORTED = 4, 2


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("new,ctx", [([3, 1, 5], [100, 40, 700]), ([40], [900])])
@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_wait_runs_out_and_the_next_call_is_as_ever(new, ctx, fp8):
    g = torch.Generator().manual_seed(len(new))
    lens = [a + b for a, b in zip(new, ctx)]
    q = torch.randn(sum(new), 16, 576, generator=g).to(torch.bfloat16).cuda()
    cache = torch.randn(60, 64, 576, generator=g).to(torch.bfloat16).cuda()
    if fp8:
        rows, cache = cache.view(-1, 576), torch.zeros(60, 64, 656, dtype=torch.uint8, device="cuda")
        table = torch.arange(60, dtype=torch.int32, device="cuda")[None]
        mla.cache_append(rows[:, :512], rows[:, 512:], cache, table, i32([60 * 64]))
    table = torch.arange(60, dtype=torch.int32, device="cuda").view(len(new), -1).contiguous()
    cu = i32([sum(new[:i]) for i in range(len(new) + 1)])
    pl = mla.plan_chunks(cu, i32(lens), sum(new), 16)
    if fp8:
        pl.workspace = mla.chunk_workspace(pl)
    want = mla.chunk_attention(q, cache, table, i32(lens), cu, pl=pl)
    out, lse, status = torch.zeros_like(want[0]), torch.zeros_like(want[1]), i32([0])
    for _ in range(2):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        mla.mla_test_chunk_timeout(q, cache, table, pl, out, lse, status)
        torch.cuda.synchronize()
        assert int(status) == MLA_ERR_TIMEOUT
        assert time.perf_counter() - t0 < 1.5  # the 200 us budgets, not the 2 s ones
        status.zero_()
        out.fill_(float("nan"))
        mla.mla_chunk_attention_fwd(q, cache, table, pl, out, lse, status)
        assert int(status) == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    if not fp8:
        with pytest.raises(mla.MlaError) as e:
            mla.mla_test_chunk_timeout(q.half(), cache.half(), table, pl, out, lse, status)
        assert e.value.code == UNSUPPORTED
