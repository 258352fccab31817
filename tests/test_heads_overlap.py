"""Outputs of the head rotation that overlap what the call reads, or themselves, are
refused (CPU only): every arrangement of small strides against the elements
themselves, and the layouts that a model's projections have, which are taken."""

import itertools
import random

import pytest
import torch

import mla_paged_kv_gb300 as mla
from mla_paged_kv_gb300.chunks import _apart, _output
from tests.test_chunks_abi import HEADS, INVALID

DIM = 8


def elements(t, tokens, dim):
    ptr, ts, hs, heads, _ = t
    return {ptr // 2 + i * ts + h * hs + d for i in range(tokens) for h in range(heads) for d in range(dim)}


def tensor(at, ts, hs, heads, tokens, dim):
    return 2 * at, ts, hs, heads, 2 * (at + (tokens - 1) * ts + (heads - 1) * hs + dim)


def test_overlaps_are_found_and_no_others():
    """Strides and offsets in units of the dim and of half of it."""
    rng, apart = random.Random(1), 0
    for _ in range(60000):
        tokens, ha, hb = rng.choice([1, 2, 3, 4]), rng.choice([1, 2, 3]), rng.choice([1, 2, 3])
        ts, hs = (DIM // 2 * rng.randint(0, 16) for _ in range(2))
        other = ts, hs
        if rng.random() < 0.3:
            other = tuple(DIM // 2 * rng.randint(0, 16) for _ in range(2))
        a = tensor(1000, ts, hs, ha, tokens, DIM)
        b = tensor(1000 + DIM // 2 * rng.randint(-20, 20), *other, hb, tokens, DIM)
        share = bool(elements(a, tokens, DIM) & elements(b, tokens, DIM))
        if _apart(a, b, tokens, DIM):
            apart += 1
            assert not share, (a, b, tokens)
        else:  # nothing that lies apart is refused, where both have the same strides
            assert share or other != (ts, hs) or ts == 0 or hs == 0, (a, b, tokens)
        assert _apart(a, b, tokens, DIM) == _apart(b, a, tokens, DIM)
    assert apart > 10000


def test_no_output_that_overlaps_itself_is_taken():
    for tokens, heads, ts, hs in itertools.product([1, 2, 3], [1, 2, 3], range(0, 65, 4), range(0, 65, 4)):
        t = tensor(0, ts, hs, heads, tokens, DIM)
        try:
            _output(t, tokens, DIM, (), None)
        except ValueError:
            continue
        assert len(elements(t, tokens, DIM)) == tokens * heads * DIM, (tokens, heads, ts, hs)


def refused(x, out, **more):
    """Whether the binding refuses out for its overlap (it stops at the device otherwise: these tensors are the CPU's)."""
    table, st = torch.zeros(64, 64), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError) as e:
        mla.rope_heads(x, table, positions=torch.zeros(x.shape[0], dtype=torch.int32), out=out, status=st, **more)
    text = str(e.value)
    assert "overlap" in text or "share memory" in text or "CUDA device" in text, text
    return "CUDA device" not in text


def buf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_windows_that_share_rows_are_refused():
    heads_first = buf(4, 9, 64)  # [heads, tokens, dim]
    assert refused(heads_first[:, 1:].transpose(0, 1), heads_first[:, :8].transpose(0, 1))
    rows = buf(4000)  # token stride 320, head stride 128: the heads of a token end 64 behind where the next begins
    assert refused(rows[64:].as_strided((4, 3, 64), (320, 128, 1), 64), rows.as_strided((4, 3, 64), (320, 128, 1), 0))
    tokens_first = buf(9, 4, 64)
    assert refused(tokens_first[1:], tokens_first[:8])
    assert refused(tokens_first[:8, 1:], tokens_first[:8, :3])
    wide = buf(5, 3, 128)
    assert refused(wide[..., :64], wide[..., 32:96])


def test_layouts_of_projections_are_taken():
    packed = buf(5, 10 * 64)  # queries, keys and values of grouped heads
    q, k = packed[:, :384].view(5, 6, 64), packed[:, 384:512].view(5, 2, 64)
    assert not refused(q, q, k=k, k_out=k)
    assert not refused(q, buf(5, 6, 64), k=k, k_out=k)
    wide = buf(5, 3, 128)  # parts of the same heads, either order
    assert not refused(wide[..., :64], wide[..., 64:]) and not refused(wide[..., 64:], wide[..., :64])
    padded = buf(5, 3 * 128 + 64)[:, :384].view(5, 3, 128)  # .. in rows that hold something else too
    assert not refused(padded[..., :64], padded[..., 64:]) and not refused(padded[..., 64:], padded[..., :64])
    swapped = buf(3, 5, 128).transpose(0, 1)  # .. with the heads outermost
    assert not refused(swapped[..., :64], swapped[..., 64:]) and not refused(swapped[..., 64:], swapped[..., :64])
    assert not refused(wide[:, :1, :64], wide[:, 1:2, :64]) and not refused(wide[:, 2:, :64], wide[:, :1, :64])
    assert not refused(wide[:1, :, :64], wide[:1, :, 64:]) and not refused(wide[:2, :, :64], wide[3:, :, :64])
    one = buf(5, 1, 64).expand(5, 3, 64)  # a head that is read for all
    assert not refused(one, buf(5, 3, 64))


@pytest.mark.parametrize("change", [dict(ot=0), dict(oh=0), dict(oh=56), dict(kot=0), dict(koh=0), dict(koh=32),
                                    dict(ot=32, oh=4096)])
def test_the_entry_point_refuses_outputs_on_top_of_each_other(change):
    """(Inputs may be: a stride of 0 reads one head for all.)"""
    args = {**HEADS, **change}
    assert mla.load_library().mla_rope_heads(*args.values()) == INVALID
