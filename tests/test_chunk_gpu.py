"""Attention of ragged chunks over a paged latent cache against 64-bit
attention, element by element.

Tolerances, from the arithmetic.  Each weight is rounded once to the cache's
type: half a step, u = 2^-8 (bf16) or 2^-11 (fp16), moves the output by at most
u * mix with mix = sum_j w_j |v_j|; rounding the output adds u |out| (2^-24 for
fp32).  A score is a sum of 576 products in fp32: off by at most 576 * 2^-23 *
reach, reach = max_j scale |q|.|k_j| (each add may lose one last place,
truncation allowed for), and the exponential, the reference's rounding and the
merge of pieces add 2^-20; both move weights, hence twice that on the output
(numerator and sum).  lse moves by the score error plus 2^-19 (sum, log, merge)
and one last place of its own value.  fp16 values below the smallest normal
are off by at most 2^-25.  Over FP8 records weights are fp16 (2^-11; those below
2^-14 of the largest are off by 2^-25 of it: 2^-25 sum_j |v_j| on the output), and a
value is off by the rounding of its scale and of the product, 2^-11 each.  Both are
taken without a power of two, 2^E, that the key's largest scale has in common with
those within a factor of 256: what is below the smallest normal is so after that.
"""

import math

import numpy as np
import pytest
import torch

import mla_paged_kv_gb300 as mla
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16
U = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, torch.float32: 2.0 ** -24}
BAD_INDEX, STALE_PLAN = 5, 7
SCALE = 1.0 / 24.0


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    """Requests with `new` tokens behind `ctx` keys; slots behind their last keys, and pages of nobody, hold `rest`."""

    def __init__(self, new, ctx, heads=2, dtype=BF16, seed=0, before=0, after=0, amp=1.0, rest=float("nan"), spare=3,
                 fp8=False):
        g = torch.Generator().manual_seed(seed)
        self.new, self.lens = list(new), [a + b for a, b in zip(new, ctx)]
        self.cu = [before + int(x) for x in np.concatenate([[0], np.cumsum(new)])]
        need = [-(-max(n, 0) // 64) for n in self.lens]
        pages = sum(need) + spare
        perm = torch.randperm(pages, generator=g).tolist()
        self.table = np.full((len(new), max(need) + 1), -1, dtype=np.int32)
        self.cache = torch.full((pages, 64, 576), rest).to(dtype)
        for b, n in enumerate(self.lens):
            for j in range(need[b]):
                page = perm.pop()
                self.table[b, j] = page
                k = min(64, n - 64 * j)
                self.cache[page, :k] = torch.randn(k, 576, generator=g).to(dtype)
        self.q = (amp * torch.randn(self.cu[-1] + after, heads, 576, generator=g)).to(dtype)
        self.values = self.cache.double().numpy()
        if fp8:  # records of those rows; what is no number in a row becomes codes and scales that are none
            c, r = self.cache[..., :512].float().reshape(pages, 64, 4, 128), self.cache[..., 512:]
            scale = torch.nan_to_num(c).abs().amax(3).clamp(min=1e-3) / 448.0
            scale = torch.where(torch.isfinite(c).all(3), scale, c[..., 0])
            codes = torch.where(torch.isfinite(c), (c / scale[..., None]).clamp(-448, 448), c).to(torch.float8_e4m3fn)
            self.cache = torch.cat([codes.view(torch.uint8).reshape(pages, 64, 512), scale.view(torch.uint8),
                                    r.contiguous().view(torch.uint8)], 2).contiguous()
            key = (codes.double() * scale.double()[..., None]).reshape(pages, 64, 512)
            self.values = torch.cat([key, r.double()], 2).numpy()
            self.scale = scale

    def keys(self):
        """Keys, and whether they are on a page of the pool, of each request."""
        rows = [so.request_keys(self.values, self.table[b], max(n, 0)) for b, n in enumerate(self.lens)]
        return [r[0] for r in rows], [r[1] for r in rows]

    def device(self):
        return (self.q.cuda(), self.cache.cuda(), torch.from_numpy(self.table).cuda(), i32(self.lens), i32(self.cu))

    def check(self, out, lse, causal, scale=SCALE, fill=None, split=False):
        u, uo = U[self.q.dtype], U[out.dtype]
        keys, seen = self.keys()
        want, wlse, mix, reach = so.chunk_attention(self.q.double().numpy(), keys, seen, self.cu, self.lens, causal,
                                                    scale)
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        live = np.zeros(o.shape[0], dtype=bool)
        live[self.cu[0]:self.cu[-1]] = True
        if fill is not None:
            assert np.all(o[~live] == fill) and np.all(l[~live] == fill), "rows of no chunk were written"
        o, l, want, wlse, mix, reach = (x[live] for x in (o, l, want, wlse, mix, reach))
        none = np.isneginf(wlse)
        assert np.array_equal(np.isneginf(l), none) and not o[none].any()
        score = 576 * 2.0 ** -23 * reach
        if split:
            most = np.abs(self.q.double().numpy()[live][..., :512]).max(2)
            score = score + 2.0 ** -17 * scale * most * max(np.abs(k[:, :512]).sum(1).max() for k in keys)
        half = self.q.dtype == FP16 or out.dtype == FP16
        tiny = 2.0 ** -25 * 8 if half else 0
        if self.cache.dtype == torch.uint8:
            u = 3 * 2.0 ** -11
            most = torch.nan_to_num(self.scale.double().abs().amax(2), posinf=1.0).clamp(2.0 ** -61, 2.0 ** 61)
            power = 2.0 ** (8 * torch.floor((torch.floor(torch.log2(most)) + 11) / 8) - 10)[..., None].numpy()
            power = [so.request_keys(power, self.table[b], max(n, 0))[0] for b, n in enumerate(self.lens)]
            tiny += max([2.0 ** -25 * e.max() * (8 + (np.abs(np.nan_to_num(k[:, :512])) / e).sum(0).max())
                         for k, e in zip(keys, power) if len(k)], default=0)
        tol = (u + 2 * score + 2.0 ** -19)[..., None] * mix + uo * np.abs(want) + tiny
        assert np.isfinite(o).all() and np.all(np.abs(o - want) <= tol), np.max(np.abs(o - want) / tol)
        l, wlse, score = l[~none], wlse[~none], score[~none]
        assert np.all(np.abs(l - wlse) <= score + 2.0 ** -19 + 2.0 ** -23 * np.abs(wlse))

    def run(self, causal=True, scale=SCALE, parts=None, out_fp32=False, split=False):
        q, cache, table, lens, cu = self.device()
        pl = None if parts is None else mla.plan_chunks(cu, lens, q.shape[0], q.shape[1], causal, num_parts=parts)
        out, lse = mla.chunk_attention(q, cache, table, lens, cu, causal, scale, out_fp32, pl=pl)
        self.check(out, lse, causal, scale, split=split)
        if cache.dtype == torch.uint8:  # without room for converted pages, and with room for some: the same to the bit
            pl = pl or mla.plan_chunks(cu, lens, q.shape[0], q.shape[1], causal)
            for room in (0, 3, 9):
                pl.workspace = mla.chunk_workspace(pl, room)
                o, l, status = torch.full_like(out, 7.0), torch.full_like(lse, 7.0), i32([0])
                mla.mla_chunk_attention_fwd(q, cache, table, pl, o, l, status, scale)
                live = slice(self.cu[0], self.cu[-1])  # (rows of no chunk are as they were)
                assert int(status) == 0 and torch.equal(o[live], out[live]) and torch.equal(l[live], lse[live])
        return out, lse


caches = pytest.mark.parametrize("fp8", [False, True])


@caches
@pytest.mark.parametrize("keys", [1, 2, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 191, 192, 193, 256, 257, 700])
def test_one_token(keys, fp8):
    Case([1], [keys - 1], seed=keys, fp8=fp8).run()


@caches
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 100])
def test_one_chunk(n, fp8):
    Case([n], [0], heads=4, seed=n, fp8=fp8).run()
    Case([n], [n + 70], heads=3, seed=n + 1, fp8=fp8).run()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("out_fp32", [True, False])
def test_types_and_masks(dtype, causal, out_fp32):
    Case([5, 1, 33], [200, 64, 0], heads=8, dtype=dtype, seed=3).run(causal, out_fp32=out_fp32)
    if dtype == BF16:
        Case([5, 1, 33], [200, 64, 0], heads=8, seed=4, fp8=True).run(causal, out_fp32=out_fp32)


@caches
@pytest.mark.parametrize("heads", [1, 5, 12, 16, 64, 128])
def test_heads(heads, fp8):
    """Blocks of 128 rows that begin and end inside a token among them."""
    Case([7, 1, 4], [130, 5, 250], heads=heads, seed=heads, fp8=fp8).run()


@caches
@pytest.mark.parametrize("parts", [1, 2, 3, 7, 76, 200])
def test_cuts(parts, fp8):
    """Units cut into up to as many pieces as they have tiles, and runs of many units."""
    Case([3, 20, 1], [1500, 100, 900], heads=16, seed=parts, fp8=fp8).run(parts=parts)
    Case([1], [3000], heads=16, seed=parts + 1, fp8=fp8).run(parts=parts)


@caches
def test_many_requests(fp8):
    new = [(5 * i) % 7 for i in range(60)]  # empty ones among them
    Case(new, [(37 * i) % 300 for i in range(60)], heads=16, seed=5, fp8=fp8).run()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("parts", [None, 1])
@caches
def test_rows_that_see_no_key(causal, parts, fp8):
    """Chunks longer than their keys (the first tokens see none), and requests without keys."""
    Case([40, 3, 2, 9], [-30, -3, 60, -9], heads=16, seed=7, fp8=fp8).run(causal, parts=parts)
    Case([4, 2], [-4, -2], heads=16, seed=8, fp8=fp8).run(causal, parts=parts)


@caches
@pytest.mark.parametrize("amp", [4.0, 30.0])
def test_growing_maxima(amp, fp8):
    """Scores that spread over hundreds of powers of two: the reference is raised again and again."""
    for parts in (1, None):
        Case([6, 40], [900, 500], heads=16, seed=11, amp=amp, fp8=fp8).run(parts=parts)


@pytest.mark.parametrize("spread", [0, 6, 14])
def test_queries_of_any_size_over_records(spread):
    """Over FP8 records a query is two E4M3 numbers an element, scaled by its largest one: elements below 2^-9 of that
    are off by 2^-17 of it at most, and so a score by that times the key's absolute sum (`split`).  Rows from 2^-60 to
    2^5, elements of a row within `spread` powers of two and one that is far above the others."""
    c = Case([9, 3], [130, 300], heads=16, seed=spread, fp8=True)
    g = torch.Generator().manual_seed(spread)
    q = c.q.float()
    q[..., :512] *= 2.0 ** -torch.randint(0, spread + 1, q[..., :512].shape, generator=g).float()
    q[:, 3, 77] *= 64
    for h, e in enumerate([-60, -35, -34, -20, -3, 5]):
        q[:, h] *= 2.0 ** e
    q[:, 7] = 0
    q[:, 8, :512] = 0
    q[:, 9, 512:] = 0
    c.q = q.to(BF16)
    c.run(split=True)


@pytest.mark.parametrize("parts", [None, 1])
def test_scales_far_apart(parts):
    """Keys (and groups of a key) whose scales are far from each other, in tiles of their own and side by side."""
    c = Case([9, 40, 200], [130, 300, 500], heads=16, seed=77, fp8=True, amp=0.5)
    g = torch.Generator().manual_seed(78)
    far = 2.0 ** torch.tensor([-50.0, -30.0, -12.0, -6.0, 0.0, 3.0])
    size = far[torch.randint(0, 6, c.scale.shape[:2], generator=g)][..., None].expand(-1, -1, 4).clone()
    size[::3] = 2.0 ** -9  # pages of keys that are alike
    size[1::3] *= 2.0 ** -torch.randint(0, 5, size[1::3].shape, generator=g).float()
    c.scale = c.scale * size
    rows, code = c.cache.clone(), c.cache[..., :512].contiguous().view(torch.float8_e4m3fn)
    rows[..., 512:528] = c.scale.contiguous().view(torch.uint8)
    key = (code.double().reshape(-1, 64, 4, 128) * c.scale.double()[..., None]).reshape(-1, 64, 512)
    c.cache, c.values = rows, np.concatenate([key.numpy(), c.values[..., 512:]], 2)
    c.run(parts=parts)
    c.run(False, parts=parts, out_fp32=True)


@caches
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_no_number_stays_with_its_row(what, fp8):
    c = Case([5, 40], [100, 200], heads=16, seed=5, fp8=fp8)
    want = c.run()
    for head, dim in ((2, 100), (9, 511), (15, 570)):
        c.q[3, head, dim] = what
    q, cache, table, lens, cu = c.device()
    out, lse = mla.chunk_attention(q, cache, table, lens, cu, True, SCALE)
    for head in range(16):
        if head in (2, 9, 15):
            assert not bool(torch.isfinite(out[3, head]).all())
        else:
            assert torch.equal(out[3, head], want[0][3, head]) and torch.equal(lse[3, head], want[1][3, head])
    keep = [t for t in range(45) if t != 3]
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


def test_rows_of_no_chunk_are_left():
    c = Case([3, 5], [100, 40], heads=16, seed=13, before=4, after=6)
    q, cache, table, lens, cu = c.device()
    for parts in (1, 76):
        pl = mla.plan_chunks(cu, lens, q.shape[0], 16, num_parts=parts)
        out = torch.full((q.shape[0], 16, 512), 7.0, dtype=BF16, device="cuda")
        lse = torch.full((q.shape[0], 16), 7.0, device="cuda")
        status = i32([0])
        mla.mla_chunk_attention_fwd(q, cache, table, pl, out, lse, status)
        assert int(status) == 0
        c.check(out, lse, True, fill=7.0)


@caches
@pytest.mark.parametrize("rest", [float("nan"), float("inf")])
def test_what_lies_behind_the_last_key(rest, fp8):
    """Slots behind a request's last key, and pages of nobody, hold no numbers; chunks end at every place of a tile."""
    for n in (1, 60, 64, 70, 127, 190):
        Case([2], [n], heads=64, seed=n, rest=rest, fp8=fp8).run()


@caches
def test_bad_pages_are_masked_and_reported(fp8):
    for heads, parts in ((16, None), (16, 1), (128, 2)):
        c = Case([4, 3, 2], [300, 500, 100], heads=heads, seed=17, fp8=fp8)
        c.table[0, 1], c.table[1, 0], c.table[1, 7] = -1, c.cache.shape[0], -5
        c.table[2, :2] = 99999  # all keys of a request
        q, cache, table, lens, cu = c.device()
        status = i32([0])
        pl = mla.plan_chunks(cu, lens, q.shape[0], heads, num_parts=parts)
        out, lse = mla.chunk_attention(q, cache, table, lens, cu, pl=pl, status=status)
        assert int(status) == BAD_INDEX
        c.check(out, lse, True)


@caches
def test_a_table_too_short_for_its_lengths(fp8):
    c = Case([2, 2], [200, 30], heads=16, seed=19, fp8=fp8)
    c.table = np.ascontiguousarray(c.table[:, :2])
    q, cache, table, lens, cu = c.device()
    status = i32([0])
    out, lse = mla.chunk_attention(q, cache, table, lens, cu, status=status)
    assert int(status) == BAD_INDEX
    c.check(out, lse, True)


def test_offsets_out_of_range():
    c = Case([3, 3], [40, 50], heads=16, seed=23)
    q, cache, table, lens, cu = c.device()
    for bad, ln in (([0, 4, 3], c.lens), ([-1, 3, 6], c.lens), ([0, 3, 7], c.lens), (c.cu, [43, (1 << 24) + 1])):
        status = i32([0])
        pl = mla.plan_chunks(i32(bad), i32(ln), 6, 16, status=status)
        assert int(status) == BAD_INDEX
        out, lse = torch.full((6, 16, 512), 7.0, dtype=BF16, device="cuda"), torch.full((6, 16), 7.0, device="cuda")
        status.zero_()
        mla.mla_chunk_attention_fwd(q, cache, table, pl, out, lse, status)
        assert int(status) == 0 and bool((out == 7.0).all()) and bool((lse == 7.0).all())
        with pytest.raises(mla.MlaError):
            mla.plan_chunks(i32(bad), i32(ln), 6, 16)


def test_an_empty_plan_over_records_converts_nothing():
    """A plan of offsets out of range, made where other numbers lay: no page and no query is looked at by it."""
    c = Case([200, 300], [40, 50], heads=16, seed=24, fp8=True)
    q, cache, table, lens, _ = c.device()
    parts = mla.mla_chunk_num_parts()
    plan = torch.full((mla.mla_chunk_plan_bytes(2, 500, 16, parts),), 0x3F, dtype=torch.uint8, device="cuda")
    status = i32([0])
    mla.mla_chunk_get_plan(i32([0, 300, 200]), lens, 500, 16, True, parts, plan, status)
    assert int(status) == BAD_INDEX
    pl = mla.ChunkPlan(plan, 2, 500, 16, parts, True, None)
    pl.workspace = mla.chunk_workspace(pl, 9).zero_()
    out, lse = torch.full((500, 16, 512), 7.0, dtype=BF16, device="cuda"), torch.full((500, 16), 7.0, device="cuda")
    status.zero_()
    mla.mla_chunk_attention_fwd(q, cache, table, pl, out, lse, status)
    assert int(status) == 0 and bool((out == 7.0).all()) and bool((lse == 7.0).all())
    base = mla.mla_chunk_workspace_bytes(parts)
    assert not bool(pl.workspace[base:base + 9 * mla.CHUNK_PAGE_BYTES].any())


def test_a_plan_of_others_is_reported():
    c = Case([3, 5], [100, 40], heads=16, seed=29)
    q, cache, table, lens, cu = c.device()
    pl = mla.plan_chunks(cu, lens, 8, 16)
    want = mla.chunk_attention(q, cache, table, lens, cu, pl=pl)
    for cu2, lens2 in ((i32([0, 4, 8]), lens), (cu, lens + 1), (cu + 0, lens - i32([0, 1]))):
        status = i32([0])
        got = mla.chunk_attention(q, cache, table, lens2, cu2, pl=pl, status=status)
        assert int(status) == STALE_PLAN
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])  # the plan's results
        with pytest.raises(mla.MlaError):
            mla.chunk_attention(q, cache, table, lens2, cu2, pl=pl)


@caches
def test_calls_repeat_to_the_bit(fp8):
    c = Case([30, 2, 1], [700, 1500, 90], heads=16, seed=31, fp8=fp8)
    q, cache, table, lens, cu = c.device()
    first = mla.chunk_attention(q, cache, table, lens, cu)
    for _ in range(3):
        again = mla.chunk_attention(q, cache, table, lens, cu)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_agrees_with_decode():
    """One token each: the plain decode of the same batch, within both calls' roundings."""
    c = Case([1] * 9, [70 * i for i in range(9)], heads=128, seed=37)
    q, cache, table, lens, cu = c.device()
    out, lse = mla.chunk_attention(q, cache, table, lens, cu, out_fp32=True)
    c.check(out, lse, True)
    # (the decode wants numbers behind the last key too)
    ref, rlse = mla.decode(q[:, None], torch.nan_to_num(cache), table, lens, softmax_scale=SCALE)
    assert float((out - ref[:, 0].float()).abs().max()) < 2.0 ** -6 * float(ref.abs().max())
    assert float((lse - rlse[:, 0]).abs().max()) < 1e-3


def test_records_against_the_rows_that_the_gather_gives():
    """Over FP8 records scores are the products' own; over a 16-bit cache of the gathered rows (the same values) keys are
    rounded, and lse and outputs are further from them."""
    c = Case([5, 2, 30], [130, 600, 64], heads=16, seed=41, fp8=True)
    q, cache, table, lens, cu = c.device()
    pages = torch.arange(cache.shape[0], dtype=torch.int32, device="cuda")
    rows = mla.cache_gather(cache, pages[None], i32([0, 64 * cache.shape[0]]), 64 * cache.shape[0])
    out, lse = mla.chunk_attention(q, cache, table, lens, cu)
    coarse = mla.chunk_attention(q, rows.view(-1, 64, 576), table, lens, cu)
    exact = c.cache[..., :512].contiguous().view(torch.float8_e4m3fn).double().reshape(-1, 64, 4, 128) * \
        c.cache[..., 512:528].contiguous().view(torch.float32).double()[..., None]
    exact = np.concatenate([exact.reshape(-1, 64, 512).numpy(), c.cache[..., 528:].contiguous().view(BF16).double().numpy()], 2)
    keys = [so.request_keys(exact, c.table[b], n) for b, n in enumerate(c.lens)]
    want, wlse, _, _ = so.chunk_attention(c.q.double().numpy(), [k[0] for k in keys], [k[1] for k in keys], c.cu, c.lens,
                                          True, SCALE)

    def off(x, y):
        return float(np.linalg.norm(x.double().cpu().numpy() - y) / np.linalg.norm(y))

    assert off(lse, wlse) < 1e-6 < 4e-6 < off(coarse[1], wlse)
    assert off(out, want) < off(coarse[0], want) < 4e-3
