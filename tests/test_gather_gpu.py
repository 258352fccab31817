"""Rows of a paged cache as packed rows.

16-bit rows are copies.  A value of an FP8 record is code x scale in fp32 (off by
2^-24 of it) rounded to bf16: half a step, 2^-8 of the value; the bf16 RoPE part
is a copy.
"""

import numpy as np
import pytest
import torch

import mla_paged_kv_gb300 as mla
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

BAD_INDEX = 5


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def pool(kind, pages, seed):
    g = torch.Generator().manual_seed(seed)
    if kind != "fp8":
        return torch.randn(pages, 64, 576, generator=g).to({"bf16": torch.bfloat16, "fp16": torch.float16}[kind])
    rec = torch.randint(0, 256, (pages, 64, 656), dtype=torch.uint8, generator=g)
    codes = rec[..., :512]
    codes[(codes & 0x7F) == 0x7F] = 0x7E  # no NaN codes
    rec[..., 512:528] = torch.exp2(4 * torch.randn(pages, 64, 4, generator=g)).view(torch.uint8)
    rec[..., 528:] = torch.randn(pages, 64, 64, generator=g).to(torch.bfloat16).view(torch.uint8)
    return rec


def check(got, cache, table, cu, starts, fill=None):
    """Every row; rows of no request, and those whose slot is outside the pool, hold `fill`."""
    host, live = cache.numpy() if cache.dtype == torch.uint8 else cache, np.zeros(got.shape[0], dtype=bool)
    got = got.cpu()
    for b in range(len(cu) - 1):
        for t in range(cu[b], cu[b + 1]):
            pos = starts[b] + t - cu[b]
            page = int(table[b][pos // 64]) if 0 <= pos < 64 * len(table[b]) else -1
            if not 0 <= page < cache.shape[0]:
                continue
            live[t] = True
            if cache.dtype != torch.uint8:
                assert torch.equal(got[t], host[page, pos % 64])
                continue
            rec = host[page, pos % 64]
            want = so.record_rows(rec[None])[0]
            row = got[t].double().numpy()
            assert np.all(np.abs(row - want) <= (2.0 ** -8 + 2.0 ** -24) * np.abs(want))
            assert np.array_equal(row[512:], want[512:])
    if fill is not None:
        assert bool((got[torch.from_numpy(~live)] == fill).all()), "another row was written"


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("lens", [[1], [64], [65, 1, 0, 130], [0, 0, 7], [700, 3, 800, 900, 200]])
def test_rows(kind, lens):
    need = [-(-n // 64) for n in lens]
    cache = pool(kind, sum(need) + 2, len(lens))
    perm = torch.randperm(cache.shape[0], generator=torch.Generator().manual_seed(1)).tolist()
    table = np.full((len(lens), max(need) + 1), -1, dtype=np.int32)
    for b in range(len(lens)):
        table[b, :need[b]] = [perm.pop() for _ in range(need[b])]
    cu = [0] + [int(v) for v in np.cumsum(lens)]
    got = mla.cache_gather(cache.cuda(), torch.from_numpy(table).cuda(), i32(cu))
    assert got.shape == (cu[-1], 576)
    check(got, cache, table, cu, [0] * len(lens))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("rows", [30, 3000])  # a row a warp, and four
def test_ranges_strides_and_rows_of_no_request(kind, rows):
    cache = pool(kind, 60, 3)
    table = np.stack([np.arange(60), np.arange(60)[::-1]]).astype(np.int32)
    n = rows // 2
    cu, starts = [3, 3 + n, 3 + n + rows // 3], [61, 130]
    wide = torch.full((rows, 600), 7.0, dtype=torch.bfloat16, device="cuda")
    mla.cache_gather(cache.cuda(), torch.from_numpy(table).cuda(), i32(cu), starts=i32(starts), out=wide[:, :576])
    check(wide[:, :576], cache, table, cu, starts, fill=7.0)
    assert bool((wide[:, 576:] == 7.0).all())


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_bad_slots_are_left_and_reported(kind):
    cache = pool(kind, 6, 5)
    table = np.array([[0, -1, 2], [99, 3, 4]], dtype=np.int32)
    cu, starts = [0, 195, 390], [-2, 0]  # positions below 0, past the table, pages outside the pool
    out, status = torch.full((390, 576), 7.0, dtype=torch.bfloat16, device="cuda"), i32([0])
    mla.cache_gather(cache.cuda(), torch.from_numpy(table).cuda(), i32(cu), starts=i32(starts), out=out, status=status)
    assert int(status) == BAD_INDEX
    check(out, cache, table, cu, starts, fill=7.0)
    with pytest.raises(mla.MlaError):
        mla.cache_gather(cache.cuda(), torch.from_numpy(table).cuda(), i32(cu), starts=i32(starts))


def test_all_codes():
    """Every E4M3 code times a scale, the code that is no number among them."""
    rec = torch.zeros(1, 64, 656, dtype=torch.uint8)
    rec[0, 0, :256] = torch.arange(256, dtype=torch.uint8)
    rec[..., 512:528] = torch.tensor([0.37, 2.0 ** -100, 1.0, 2.0 ** 100]).view(torch.uint8)
    got = mla.cache_gather(rec.cuda(), i32([[0]]), i32([0, 1]), 1).double().cpu().numpy()[0]
    want = so.record_rows(rec[0, :1].numpy())[0]
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    assert np.all(np.abs(got - want)[~nan] <= (2.0 ** -8 + 2.0 ** -24) * np.abs(want[~nan]))


def test_gather_undoes_append():
    g = torch.Generator().manual_seed(9)
    a = torch.randn(150, 576, generator=g).to(torch.bfloat16).cuda()
    cache = torch.zeros(6, 64, 576, dtype=torch.bfloat16, device="cuda")
    table, lens, cu = i32([[4, 0, -1], [3, 5, -1]]), i32([80, 70]), i32([0, 80, 150])
    mla.cache_append(a[:, :512], a[:, 512:], cache, table, lens, cu_seqlens=cu)
    assert torch.equal(mla.cache_gather(cache, table, cu, 150), a)


def test_no_rows():
    assert mla.cache_gather(pool("bf16", 1, 0).cuda(), i32([[0]]), i32([0, 0])).shape == (0, 576)
