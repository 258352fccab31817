"""A plan of offsets or lengths out of range is empty.  Its maker reports it, into the
status that it was given; a call that gives the same offsets or lengths reports it
again, for its outputs are memory that nobody has written."""

import pytest
import torch

import mla_paged_kv_gb300 as mla
from tests.test_chunk_gpu import Case

pytestmark = pytest.mark.gpu

BAD_INDEX, STALE_PLAN = 5, 7


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cu,lens", [([0, 4, 3], [43, 53]), ([-1, 3, 6], [43, 53]), ([0, 3, 7], [43, 53]),
                                     ([0, 3, 6], [43, (1 << 24) + 1])])
def test_a_call_with_an_empty_plan_reports_it(cu, lens, fp8):
    c = Case([3, 3], [40, 50], heads=16, seed=23, fp8=fp8)
    q, cache, table, good_lens, good_cu = c.device()
    cu, lens, ignored, status = i32(cu), i32(lens), i32([0]), i32([0])
    pl = mla.plan_chunks(cu, lens, 6, 16, status=ignored)
    assert int(ignored) == BAD_INDEX
    mla.chunk_attention(q, cache, table, lens, cu, pl=pl, status=status)
    assert int(status) == BAD_INDEX
    with pytest.raises(mla.MlaError) as e:
        mla.chunk_attention(q, cache, table, lens, cu, pl=pl)
    assert e.value.code == BAD_INDEX
    if fp8:
        pl.workspace = mla.chunk_workspace(pl, 2)
    for some in (dict(cu_seqlens_q=cu), dict(cache_seqlens=lens), dict(cu_seqlens_q=cu, cache_seqlens=lens)):
        out, lse = torch.full((6, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((6, 16), 7.0, device="cuda")
        status.zero_()
        mla.mla_chunk_attention_fwd(q, cache, table, pl, out, lse, status, **some)
        assert int(status) == BAD_INDEX and bool((out == 7.0).all()) and bool((lse == 7.0).all())
    # the same memory with a good plan, and that one told of other offsets
    mla.mla_chunk_get_plan(good_cu, good_lens, 6, 16, True, pl.num_parts, pl.plan, status.zero_())
    out, lse = mla.chunk_attention(q, cache, table, good_lens, good_cu, pl=pl, status=status)
    assert int(status) == 0
    c.check(out, lse, True, scale=1.0 / 24.0)
    mla.chunk_attention(q, cache, table, lens, cu, pl=pl, status=status)
    assert int(status) == STALE_PLAN
