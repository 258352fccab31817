"""Gathered rows at every number of rows around a warp's four and a block's sixteen, with requests that begin and
end inside them, and rows of no request before and behind."""

import numpy as np
import pytest
import torch

import mla_paged_kv_gb300 as mla
from tests.test_gather_gpu import check, i32, pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp8"])
def test_every_number_of_rows(kind):
    cache = pool(kind, 12, 7)
    dev, table = cache.cuda(), np.arange(12, dtype=np.int32).reshape(4, 3)[:, ::-1].copy()
    want = torch.float16 if kind == "fp16" else torch.bfloat16
    for rows in list(range(1, 37)) + [63, 64, 65, 127, 129]:
        for before, behind in ((0, 0), (rows // 3, rows // 4)):
            n = rows - before - behind
            cu = [before, before + n // 5, before + n // 5, before + n // 2, before + n]
            starts = [0, 5, 61, 63]
            out = torch.full((rows, 576), 7.0, dtype=want, device="cuda")
            mla.cache_gather(dev, torch.from_numpy(table).cuda(), i32(cu), starts=i32(starts), out=out)
            check(out, cache, table, cu, starts, fill=7.0)
