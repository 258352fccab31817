"""Chunk attention through the entry point's mirror: outputs that are missing are refused (CPU only)."""

import pytest
import torch

import mla_paged_kv_gb300 as mla


@pytest.mark.parametrize("name", ["mla_chunk_attention_fwd", "mla_test_chunk_timeout"])
@pytest.mark.parametrize("cache", [torch.zeros(8, 64, 576, dtype=torch.bfloat16),
                                   torch.zeros(8, 64, 656, dtype=torch.uint8)])
def test_missing_outputs_are_refused(name, cache):
    """(Outputs made in their place would be lost with the call.)"""
    q, block = torch.zeros(4, 16, 576, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32)
    pl = mla.ChunkPlan(torch.zeros(1 << 16, dtype=torch.uint8), 2, 4, 16, 4, True, torch.zeros(1 << 22, dtype=torch.uint8))
    st, out, lse = torch.zeros(1, dtype=torch.int32), torch.zeros(4, 16, 512), torch.zeros(4, 16)
    for o, l in ((None, lse), (out, None), (None, None)):
        with pytest.raises(ValueError, match="needed"):
            getattr(mla, name)(q, cache, block, pl, o, l, st)
