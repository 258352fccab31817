"""Rotary tables and the rotation (and norm) of heads against 64-bit restatements.

Tolerances.  Table: an angle is the frequency's 64-bit value times the position,
off by 2^-52 of itself at most (its division by a turn and its rounding to 2^-64
turns), which numpy's own 64-bit product is too: together below 2^-51 p f.  The
fp32 part: the angle within an eighth of a turn rounded to 24 bits (2^-24 of it,
times at most 1 for sine and cosine), sincospif to 2 ulp, the magnitude's rounding
and the product: below 2^-21 magnitude in all.

Heads.  A stored value is one rounding (half a step, 2^-8 of a bf16 and 2^-11 of
an fp16 value, at least 2^-25 for fp16) of an fp32 result.  Norm: a sum of up to
1024 squares in any order (at most 1024 * 2^-24 relative for terms of one sign,
halved by the root), a division, a root, a reciprocal and two products: below
2^-14.  Rotation: a difference of two products, each with the norm's error: below
(2^-22 + 2^-14 with norm) (|x| + |y|).
"""

import numpy as np
import pytest
import torch

import mla_paged_kv_gb300 as mla
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16
HALF_STEP = {BF16: 2.0 ** -8, FP16: 2.0 ** -11}
BAD_INDEX = 5
EPS = 1e-6
SCALINGS = ["none", "linear", "ntk", "yarn", "wavelength"]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check_table(got, freq, size, first):
    p = np.arange(first, first + got.shape[0], dtype=np.float64)
    angle = np.multiply.outer(p, freq)
    want = np.concatenate([np.cos(angle), np.sin(angle)], 1) * size
    tol = size * (2.0 ** -21 + np.concatenate([angle, angle], 1) * 2.0 ** -51)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), (err / tol).max()


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("dim", [8, 32, 64, 128, 256])
def test_table(scaling, dim):
    freq, size = so.rope_frequencies(dim, 10000.0, scaling, 8.0, 4096, 1.0, 4.0 if scaling == "wavelength" else 32.0)
    for n in (1, 7, 300):
        check_table(mla.rope_table(n, dim, scaling=scaling, factor=8.0), freq, size, 0)


@pytest.mark.parametrize("first", [1, 1000, (1 << 20) - 3, (1 << 24) + 1, (1 << 31) - 400])
def test_table_of_far_positions(first):
    """2^31 steps of a frequency of 1: the angle's whole turns are left out exactly."""
    freq, size = so.rope_frequencies(64, 500000.0, "none", 1.0, 4096, 1.0, 32.0)
    check_table(mla.rope_table(400, 64, base=500000.0, first=first), freq, size, first)


def test_table_of_own_frequencies_and_magnitude():
    freq = [0.0, 1.0, 3.0, 6.283185307179586, 1000.0, 1e-9, 0.5, 2.0 ** -30]
    out = torch.empty(500, 16, device="cuda")
    mla.mla_rope_table(freq, 0.75, 5, out)
    check_table(out, np.array(freq), 0.75, 5)
    assert mla.rope_table(0, 64).shape == (0, 64)


def test_table_serves_the_append():
    """cache_append turns by the same table that rope_heads reads."""
    table = mla.rope_table(200, scaling="yarn", factor=4.0)
    r = torch.randn(130, 64, device="cuda").to(BF16)
    c = torch.zeros(130, 512, device="cuda", dtype=BF16)
    lens, cu = i32([150, 30]), i32([0, 100, 130])
    cache = torch.zeros(8, 64, 576, device="cuda", dtype=BF16)
    block = i32([[0, 1, 2], [3, 4, 5]])
    for inter in (False, True):
        mla.cache_append(c, r, cache, block, lens, cu_seqlens=cu, cos_sin=table, rope_interleaved=inter)
        turned = mla.rope_heads(r[:, None], table, lens, cu, interleaved=inter)[:, 0]
        rows = mla.cache_gather(cache, block, cu, starts=i32([50, 0]))
        assert torch.equal(rows[:, 512:], turned)


class Heads:
    def __init__(self, tokens, heads, dim, rope, k_heads=0, dtype=BF16, norm=False, seed=0, positions=500):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.x = (r(tokens, heads, dim) * torch.exp2(r(tokens, heads, 1))).to(dtype)
        self.k = r(tokens, k_heads, dim).to(dtype) if k_heads else None
        self.w = (1 + 0.3 * r(dim)).to(dtype) if norm else None
        self.kw = (1 + 0.3 * r(dim)).to(dtype) if norm and k_heads else None
        angle = np.multiply.outer(np.arange(positions), 10000.0 ** (-2.0 * np.arange(rope // 2) / max(rope, 1)))
        self.table = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float() if rope else None
        self.rope = rope

    def check(self, got, x, w, pos, offset, interleaved, skip=None, fill=None):
        got = got.double().cpu().numpy()
        step, dt = HALF_STEP[self.x.dtype], self.x.dtype
        for t in range(x.shape[0]):
            if pos[t] is None:
                if fill is not None:
                    assert np.all(got[t] == fill), "a token of no request was written"
                continue
            for h in range(x.shape[1]):
                src = x[t, h].double().numpy()
                row = None if self.table is None else self.table[pos[t]].numpy()
                want = so.rope_head(src, row, offset, interleaved, None if w is None else w.double().numpy(), EPS)
                plain = so.rope_head(src, None, 0, False, None if w is None else w.double().numpy(), EPS)
                mag, n = np.abs(plain), self.rope // 2
                part = mag[offset:offset + self.rope].copy()
                if interleaved:
                    mag[offset:offset + self.rope] = np.repeat(part[0::2] + part[1::2], 2)
                else:
                    mag[offset:offset + self.rope] = np.tile(part[:n] + part[n:], 2)
                tol = step * np.abs(want) + (2.0 ** -22 + (0 if w is None else 2.0 ** -14)) * mag + \
                    (2.0 ** -25 if dt == FP16 else 0)
                err = np.abs(got[t, h] - want)
                assert np.all(err <= tol), (t, h, (err / tol).max())

    def run(self, offset=None, interleaved=False, lens=None, cu=None, pos=None):
        dev = lambda v: None if v is None else v.cuda()  # noqa: E731
        if offset is None:
            offset = self.x.shape[2] - self.rope
        got = mla.rope_heads(self.x.cuda(), dev(self.table), None if lens is None else i32(lens),
                             None if cu is None else i32(cu), None if pos is None else i32(pos), k=dev(self.k),
                             norm_weight=dev(self.w), k_norm_weight=dev(self.kw), norm_eps=EPS, offset=offset,
                             interleaved=interleaved)
        if pos is None and lens is not None:
            each = self.x.shape[0] // len(lens)
            cu = cu or [each * b for b in range(len(lens) + 1)]
            pos = [lens[b] - (cu[b + 1] - t) for b in range(len(lens)) for t in range(cu[b], cu[b + 1])]
        pos = pos if pos is not None else [0] * self.x.shape[0]
        q, k = got if self.k is not None else (got, None)
        self.check(q, self.x, self.w, pos, offset, interleaved)
        if k is not None:
            self.check(k, self.k, self.kw, pos, offset, interleaved)


@pytest.mark.parametrize("dim,rope,offset", [(16, 16, 0), (64, 64, 0), (64, 32, 0), (64, 32, 16), (64, 16, 48),
                                             (128, 128, 0), (192, 64, 128), (192, 32, 8), (24, 16, 8), (576, 64, 512),
                                             (256, 256, 0), (1024, 128, 896), (200, 96, 24)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_dims(dim, rope, offset, interleaved, norm):
    Heads(5, 3, dim, rope, norm=norm, seed=dim + rope).run(offset, interleaved, lens=[40], cu=[0, 5])


@pytest.mark.parametrize("heads,k_heads", [(1, 0), (1, 1), (5, 2), (16, 1), (33, 8), (128, 0), (7, 40)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_queries_and_keys(heads, k_heads, dtype):
    for norm in (False, True):
        Heads(6, heads, 64, 64, k_heads, dtype, norm, seed=heads).run(lens=[30, 9], cu=[0, 4, 6])


def test_norm_of_one_side_alone():
    h = Heads(9, 4, 128, 64, 2, norm=True, seed=4)
    h.kw = None
    h.run(lens=[20, 20, 20])
    h = Heads(9, 4, 128, 64, 2, norm=True, seed=5)
    h.w = None
    h.run(lens=[20, 20, 20])


@pytest.mark.parametrize("dim", [64, 128, 192, 1000])
def test_norm_without_rotation(dim):
    Heads(5, 3, dim, 0, 2, norm=True, seed=dim).run()


def test_positions_of_their_own():
    """In any order, the same twice, the first and the last of the table."""
    Heads(6, 4, 64, 64, seed=6).run(pos=[499, 0, 7, 7, 120, 3])


@pytest.mark.parametrize("tokens", [1, 2, 31, 400])
def test_token_counts(tokens):
    Heads(tokens, 2, 64, 64, seed=tokens).run(lens=[tokens + 5], cu=[0, tokens])


def test_many_requests():
    new = [(3 * i) % 5 for i in range(70)]
    cu = [0] + [int(v) for v in np.cumsum(new)]
    Heads(cu[-1], 2, 64, 64, seed=70).run(lens=[n + 2 * i for i, n in enumerate(new)], cu=cu)


def test_in_place_and_strided():
    """The rotary part of projected heads into the decode's rows, and in place in the projection; the rest stays."""
    g = torch.Generator().manual_seed(8)
    proj = torch.randn(10, 12, 192, generator=g).to(BF16)
    h = Heads(10, 12, 64, 64, seed=9)
    h.x = proj[..., 128:]
    lens, cu = i32([50, 60]), i32([0, 7, 10])
    pos = [43 + t for t in range(7)] + [57 + t for t in range(3)]
    src, rows = proj.cuda(), torch.full((10, 12, 576), 7.0, dtype=BF16, device="cuda")
    mla.rope_heads(src[..., 128:], h.table.cuda(), lens, cu, out=rows[..., 512:], interleaved=True)
    h.check(rows[..., 512:], h.x, None, pos, 0, True)
    assert bool((rows[..., :512] == 7.0).all()) and torch.equal(src.cpu(), proj)
    again = mla.rope_heads(src, h.table.cuda(), lens, cu, out=src, interleaved=True)
    assert again.data_ptr() == src.data_ptr() and torch.equal(src[..., 128:], rows[..., 512:])
    assert torch.equal(src[..., :128].cpu(), proj[..., :128])
    # tokens and heads swapped in memory; a single key for all heads, read by a stride of 0
    swapped = proj.transpose(0, 1).contiguous().transpose(0, 1).cuda()
    assert torch.equal(mla.rope_heads(swapped, h.table.cuda(), lens, cu, interleaved=True), src)
    one = proj[:, :1].cuda().expand(10, 12, 192)
    got = mla.rope_heads(one, h.table.cuda(), lens, cu, interleaved=True)
    assert torch.equal(got, src[:, :1].expand(10, 12, 192))


def test_packed_projection_in_place():
    """Queries and keys side by side in one projection's rows, both turned where they lie; the values stay."""
    h = Heads(9, 6, 64, 32, 2, norm=True, seed=21)
    rows = torch.full((9, 10 * 64), 7.0, dtype=BF16, device="cuda")
    q, k = rows[:, :384].view(9, 6, 64), rows[:, 384:512].view(9, 2, 64)
    q.copy_(h.x)
    k.copy_(h.k)
    got = mla.rope_heads(q, h.table.cuda(), i32([30]), out=q, k=k, k_out=k, norm_weight=h.w.cuda(),
                         k_norm_weight=h.kw.cuda(), norm_eps=EPS)
    pos = list(range(21, 30))
    h.check(got[0], h.x, h.w, pos, 32, False)
    h.check(got[1], h.k, h.kw, pos, 32, False)
    assert bool((rows[:, 512:] == 7.0).all())
    # another part of the same heads as the output
    both = torch.zeros(9, 6, 128, dtype=BF16, device="cuda")
    both[..., :64] = h.x.cuda()
    mla.rope_heads(both[..., :64], h.table.cuda(), i32([30]), out=both[..., 64:])
    h.check(both[..., 64:], h.x, None, pos, 32, False)
    assert torch.equal(both[..., :64].cpu(), h.x)


@pytest.mark.parametrize("in_place", [False, True])
def test_tokens_that_are_left(in_place):
    """Tokens of no request, and those whose position is not in the table (reported)."""
    h = Heads(14, 3, 64, 64, 2, seed=10, positions=50)
    cu, lens = [2, 6, 10], [3, 52]  # positions -1 0 1 2 and 48 49 50 51
    pos = [None] * 2 + [None, 0, 1, 2] + [48, 49, None, None] + [None] * 4
    x, k = h.x.cuda(), h.k.cuda()
    out, k_out = (x, k) if in_place else (torch.full_like(x, 7.0), torch.full_like(k, 7.0))
    status = i32([0])
    mla.rope_heads(x, h.table.cuda(), i32(lens), i32(cu), out=out, k=k, k_out=k_out, status=status)
    assert int(status) == BAD_INDEX
    if in_place:
        for got, src in ((out, h.x), (k_out, h.k)):
            for t in range(14):
                if pos[t] is None:
                    assert torch.equal(got[t].cpu(), src[t])
        h.check(out, h.x, None, pos, 0, False)
    else:
        h.check(out, h.x, None, pos, 0, False, fill=7.0)
        h.check(k_out, h.k, None, pos, 0, False, fill=7.0)
    status.zero_()
    mla.rope_heads(h.x.cuda(), h.table.cuda(), positions=i32([-1, 50] + [49] * 12), status=status)
    assert int(status) == BAD_INDEX
    with pytest.raises(mla.MlaError):
        mla.rope_heads(h.x.cuda(), h.table.cuda(), positions=i32([-1] * 14))


def test_values_that_are_no_numbers_stay_in_their_heads():
    h = Heads(4, 5, 64, 64, norm=True, seed=12)
    x = h.x.clone()
    x[1, 2, 5], x[3, 0, 60] = float("nan"), float("inf")
    got = mla.rope_heads(x.cuda(), h.table.cuda(), i32([20]), norm_weight=h.w.cuda()).cpu()
    clean = mla.rope_heads(h.x.cuda(), h.table.cuda(), i32([20]), norm_weight=h.w.cuda()).cpu()
    for t in range(4):
        for n in range(5):
            if (t, n) in ((1, 2), (3, 0)):
                assert bool(torch.isnan(got[t, n]).any())
            else:
                assert torch.equal(got[t, n], clean[t, n])


def test_no_tokens():
    t = torch.empty(0, 3, 64, dtype=BF16, device="cuda")
    assert mla.rope_heads(t, mla.rope_table(8), i32([5])).shape == (0, 3, 64)
