"""The timeout paths of the serving attention kernels, in a form that faults and
hangs nothing (as tests/test_timeout_gpu.py does for the plain decode).

Test instances whose waits have a 200 us budget never load their first key
tile (FP8 records: never compute the first scores): the issuing warp's wait
runs out, its CTA unwinds every role, the other CTA of a pair runs out of its
own waits, and the grid ends with MLA_ERR_TIMEOUT in the status word.  A
normal call right after gives the usual result."""

import time

import pytest
import torch

import mla_paged_kv_gb300 as mla

pytestmark = pytest.mark.gpu

MLA_ERR_TIMEOUT, UNSUPPORTED = 4, 2


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def runs_out(call, status):
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    assert int(status) == MLA_ERR_TIMEOUT
    assert elapsed < 1.5  # the 200 us budgets, not the 2 s ones
    status.zero_()


@pytest.mark.parametrize("lens", [[100, 40], [700, 300], [1100, 5, 900]])  # single CTAs, pairs of CTAs
def test_prompt_wait_runs_out_and_the_next_call_is_as_ever(lens):
    g = torch.Generator().manual_seed(sum(lens))
    q, k, v = (torch.randn(sum(lens), 4, d, generator=g).to(torch.bfloat16).cuda() for d in (192, 192, 128))
    cu = i32([sum(lens[:i]) for i in range(len(lens) + 1)])
    pl = mla.plan_prompt(cu, None, sum(lens))
    want = mla.prompt_attention(q, k, v, cu, pl=pl)
    out, lse, status = torch.zeros_like(want[0]), torch.zeros_like(want[1]), i32([0])
    for _ in range(2):
        runs_out(lambda: mla.mla_test_prompt_timeout(q, k, v, pl, out, lse, status), status)
        out.fill_(float("nan"))
        mla.mla_prompt_attention_fwd(q, k, v, pl, out, lse, status)
        assert int(status) == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    with pytest.raises(mla.MlaError) as e:
        mla.mla_test_prompt_timeout(q.half(), k.half(), v.half(), pl, out.half(), lse, status)
    assert e.value.code == UNSUPPORTED


@pytest.mark.parametrize("h_q", [16, 128])  # rows packed, requests alone
@pytest.mark.parametrize("fp8", [False, True])
def test_shared_prefix_wait_runs_out_and_the_next_call_is_as_ever(h_q, fp8):
    g = torch.Generator().manual_seed(h_q)
    table = torch.tensor([[0, 1, 2, 3, 4], [0, 1, 5, 6, 7], [0, 1, 8, 9, 10]], dtype=torch.int32, device="cuda")
    lens = i32([300, 160, 290])
    if fp8:
        kv = torch.randint(0, 100, (11, 64, 656), dtype=torch.uint8, generator=g)
        kv[..., 512:528] = torch.full((11, 64, 4), 0.01).view(torch.uint8)
        kv[..., 528:] = torch.randn(11, 64, 64, generator=g).to(torch.bfloat16).view(torch.uint8)
    else:
        kv = torch.randn(11, 64, 576, generator=g).to(torch.bfloat16)
    kv, q = kv.cuda(), torch.randn(3, 1, h_q, 576, generator=g).to(torch.bfloat16).cuda()
    pl = mla.plan_shared_prefix(table, lens, 1, h_q)
    want = mla.shared_prefix_decode(q, kv, table, lens, pl=pl)
    out, lse, status = torch.zeros_like(want[0]), torch.zeros_like(want[1]), i32([0])
    for _ in range(2):
        runs_out(lambda: mla.mla_test_shared_prefix_timeout(q, kv, table, pl, out, lse, status), status)
        out.fill_(float("nan"))
        mla.mla_shared_prefix_decode_fwd(q, kv, table, pl, out, lse, status)
        assert int(status) == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    if not fp8:
        with pytest.raises(mla.MlaError) as e:
            mla.mla_test_shared_prefix_timeout(q.half(), kv.half(), table, pl, out, lse, status)
        assert e.value.code == UNSUPPORTED
