"""mla_cache_append against a 64-bit restatement, token by token.

Tolerances.  A stored value is one rounding (half a step, 2^-8 of a bf16 and
2^-11 of an fp16 value) of an fp32 result.  The fp32 chain of the latent part
is a sum of 512 squares (any order: at most 512 * 2^-24 relative for terms of
one sign, halved by the square root), a square root, a reciprocal and two
products: below 2^-15.  The RoPE part is a difference of two products: below
2^-22 (|x| + |y|).
"""

import numpy as np
import pytest
import torch

import mla_paged_kv_gb300 as mla
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
CHAIN = 2.0 ** -15
EPS = 1e-6


class Case:
    def __init__(self, new, ctx, dtype=torch.bfloat16, fp8=False, seed=0, extra=0, before=0, norm=True, rope=True,
                 interleaved=False, layout="fused", uniform=False, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens = [a + b for a, b in zip(new, ctx)]
        self.cu = [before + int(x) for x in np.concatenate([[0], np.cumsum(new)])]
        t = self.cu[-1] + extra
        a = torch.randn(t, 576, generator=g) * torch.exp2(spread * torch.randn(t, 1, generator=g))
        a = a.to(dtype)
        width = max(-(-n // 64) for n in self.lens) + 1
        need = sum(-(-n // 64) for n in self.lens)
        self.pages = need + 3
        perm = torch.randperm(self.pages, generator=g).tolist()
        self.table = np.full((len(new), width), -1, dtype=np.int32)
        for b, n in enumerate(self.lens):
            for j in range(-(-n // 64)):
                self.table[b, j] = perm.pop()
        self.dtype, self.fp8, self.interleaved, self.uniform = dtype, fp8, interleaved, uniform
        self.w = (1 + 0.3 * torch.randn(512, generator=g)).to(dtype) if norm else None
        self.cos_sin = None
        if rope:
            ang = torch.arange(max(self.lens) + 1)[:, None] * 10000.0 ** (-torch.arange(32) / 32.0)[None]
            self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()
        if layout == "fused":  # slices of one projection
            self.c, self.r = a[:, :512], a[:, 512:]
        else:                  # two tensors, wide rows
            self.c = torch.nn.functional.pad(a[:, :512], (0, 24))[:, :512]
            self.r = a[:, 512:].contiguous()
        self.host = (a[:, :512].double().numpy(), a[:, 512:].double().numpy())
        self.refcount = None

    def run(self, status=None):
        dev = lambda x: None if x is None else x.cuda()  # noqa: E731

        def rows(x):  # onto the GPU with the same strides
            out = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
            return out.copy_(x)

        if self.fp8:
            cache = torch.full((self.pages, 64, 656), 0x5A, dtype=torch.uint8, device="cuda")
        else:
            cache = torch.full((self.pages, 64, 576), 777.0, dtype=self.dtype, device="cuda")
        mla.cache_append(rows(self.c), rows(self.r), cache, torch.from_numpy(self.table).cuda(),
                         torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
                         cu_seqlens=None if self.uniform else torch.tensor(self.cu, dtype=torch.int32, device="cuda"),
                         norm_weight=dev(self.w), norm_eps=EPS, cos_sin=dev(self.cos_sin),
                         rope_interleaved=self.interleaved, refcount=dev(self.refcount), status=status)
        return cache

    def check(self, cache, bad=False):
        ref = None if self.refcount is None else self.refcount.tolist()
        maxpos = None if self.cos_sin is None else self.cos_sin.shape[0]
        at, was_bad = so.append_targets(self.cu, self.lens, self.table, self.pages, maxpos, ref)
        assert was_bad == bad
        got = cache.cpu()
        written = torch.zeros(self.pages, 64, dtype=torch.bool)
        w = None if self.w is None else self.w.double().numpy()
        cs = None if self.cos_sin is None else self.cos_sin.numpy()
        for t, (page, row, pos) in at.items():
            written[page, row] = True
            c, r = so.latent_row(self.host[0][t], self.host[1][t], pos, w, EPS, cs, self.interleaved)
            # |x| + |y| of each rotated pair
            x = np.abs(self.host[1][t])
            mag = np.repeat(x[0::2] + x[1::2], 2) if self.interleaved else np.tile(x[:32] + x[32:], 2)
            rec = got[page, row]
            if self.fp8:
                rt = torch.bfloat16
                scale = rec[512:528].clone().view(torch.float32).double().numpy()
                top = np.abs(c.reshape(4, 128)).max(1)
                want = np.where(top > 0, top / 448.0, 1.0)
                assert np.all(np.abs(scale - want) <= 2 * CHAIN * want)
                val = so.e4m3_value(rec[:512].numpy()) * np.repeat(scale, 128)
                # half a step of E4M3: 2^-4 of a normal code's value, 2^-10 scale below that
                tol = np.maximum(2.0 ** -4 * np.abs(c), 2.0 ** -10 * np.repeat(scale, 128)) * (1 + 2 * CHAIN)
                assert np.all(np.abs(val - c) <= tol + 2 * CHAIN * np.abs(c))
                rope = rec[528:].clone().view(torch.bfloat16).double().numpy()
            else:
                rt = self.dtype
                val = rec[:512].double().numpy()
                tiny = 2.0 ** -25 if rt == torch.float16 else 0.0
                assert np.all(np.abs(val - c) <= (HALF_STEP[rt] + 2 * CHAIN) * np.abs(c) + tiny)
                rope = rec[512:].double().numpy()
            tiny = 2.0 ** -25 if rt == torch.float16 else 0.0
            assert np.all(np.abs(rope - r) <= HALF_STEP[rt] * np.abs(r) + 2.0 ** -21 * mag + tiny)
        rest = got[~written]
        assert torch.all(rest == (0x5A if self.fp8 else 777.0)), "a slot of no token was written"


@pytest.mark.parametrize("exponent", [-60, -64, -100, -120])
def test_tiny_rows_into_records(exponent):
    """Scales down to 2^-129, whose reciprocal is no fp32 number; groups of zeros beside them.  (The bars of
    check() hold: a scale of 2^-129 is rounded by 2^-21 of itself.)"""
    c = Case([5, 3], [2, 70], fp8=True, norm=False, seed=40)
    lat = c.c * 2.0 ** exponent  # exact, but for values below bf16's smallest
    lat[1, 128:256] = 0
    lat[3, 5:] = 0
    c.c = lat
    c.host = (lat.double().numpy(), c.host[1])
    c.check(c.run())


@pytest.mark.parametrize("fp8,dtype", [(False, torch.bfloat16), (False, torch.float16), (True, torch.bfloat16),
                                       (True, torch.float16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_ragged_batch(fp8, dtype, interleaved):
    c = Case([1, 70, 0, 64, 5, 129], [63, 0, 10, 64, 300, 1], dtype, fp8, seed=1, interleaved=interleaved)
    c.check(c.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("norm,rope", [(False, False), (True, False), (False, True)])
def test_without_norm_or_rope(fp8, norm, rope):
    c = Case([3, 65], [61, 2], fp8=fp8, seed=2, norm=norm, rope=rope, layout="wide")
    c.check(c.run())


@pytest.mark.parametrize("each", [1, 2, 7])
def test_decode_step_without_offsets(each):
    c = Case([each] * 9, list(range(60, 69)), fp8=True, seed=3, uniform=True)
    c.check(c.run())


@pytest.mark.parametrize("batch", [1, 31, 32, 33, 1100])
def test_many_requests_find_their_tokens(batch):
    c = Case([(i * 7) % 3 for i in range(batch - 1)] + [2], [i % 70 for i in range(batch)], seed=4, rope=False)
    c.check(c.run())


def test_tokens_outside_the_sequences_are_ignored():
    c = Case([4, 3], [0, 64], seed=5, before=6, extra=11)
    c.check(c.run())


def test_zero_and_large_groups():
    c = Case([6], [0], fp8=True, seed=6, norm=False, rope=False)
    c.c[0] = 0
    c.c[1, :128] = 0
    c.c[2, 5] = 3e38
    c.c[3] = 1e-30
    c.host = (c.c.double().numpy(), c.r.double().numpy())
    c.check(c.run())


def test_nan_stays_in_its_own_codes():
    c = Case([2], [0], fp8=True, seed=7, norm=False, rope=False)
    c.c[0, 3] = float("nan")
    cache = c.run()
    page = int(c.table[0, 0])
    codes = so.e4m3_value(cache[page, 0, :512].cpu().numpy())
    assert np.isnan(codes[3]) and np.isfinite(np.delete(codes, 3)).all()
    assert np.isfinite(so.e4m3_value(cache[page, 1, :512].cpu().numpy())).all()


@pytest.mark.parametrize("why", ["negative", "past_table", "past_rope", "page_low", "page_high", "shared", "free"])
def test_bad_targets_are_skipped_and_reported(why):
    c = Case([3, 66, 2], [62, 0, 9], seed=8)
    if why == "negative":
        c.lens[0] = 2
    elif why == "past_table":
        c.lens[0] = c.table.shape[1] * 64 + 1
        c.cos_sin = None
    elif why == "past_rope":
        c.cos_sin = c.cos_sin[:64].contiguous()
    elif why == "page_low":
        c.table[1, 1] = -1
    elif why == "page_high":
        c.table[1, 0] = c.pages
    else:
        c.refcount = torch.ones(c.pages, dtype=torch.int32)
        c.refcount[int(c.table[1, 0])] = 2 if why == "shared" else 0
    with pytest.raises(mla.MlaError) as e:
        c.run()
    assert e.value.code == 5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(c.run(status), bad=True)
    assert int(status) == 5


def test_no_tokens_is_no_work():
    c = Case([1], [3], seed=9)
    cache = torch.zeros(c.pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    mla.cache_append(torch.empty(0, 512, dtype=torch.bfloat16, device="cuda"),
                     torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), cache,
                     torch.from_numpy(c.table).cuda(), torch.tensor(c.lens, dtype=torch.int32, device="cuda"))
    assert not cache.any()


def test_slots_past_32_bits_of_bytes():
    """A pool of more than 2^32 bytes: the last page is written, the page that a
    32-bit byte offset would reach is not."""
    pages = (1 << 32) // (64 * 1152) + 70
    cache = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    a = torch.randn(2, 576, device="cuda").to(torch.bfloat16)
    table = torch.tensor([[pages - 1], [pages - 2]], dtype=torch.int32, device="cuda")
    mla.cache_append(a[:, :512], a[:, 512:], cache, table, torch.tensor([64, 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(cache[pages - 1, 63], a[0]) and torch.equal(cache[pages - 2, 0], a[1])
    cache[pages - 1, 63] = 0
    cache[pages - 2, 0] = 0
    assert not cache.any()


@pytest.mark.parametrize("cu", [[0, 40, 10, 50], [5, 5, 5, 5], [60, 0, 20, 30], [-9, 3, 2, 1000], [7, -3, 90, 20]])
def test_offsets_out_of_order_stay_inside_the_cache(cu):
    """Offsets that decrease or leave the batch: some tokens land somewhere or nowhere, all of it inside the pool."""
    pages = 8
    table = torch.arange(6, dtype=torch.int32, device="cuda").reshape(3, 2)
    whole = torch.zeros(pages + 4, 64, 576, dtype=torch.bfloat16, device="cuda")
    a = torch.ones(50, 576, device="cuda").to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.cache_append(a[:, :512], a[:, 512:], whole[2:2 + pages], table,
                     torch.tensor([100, 64, 20], dtype=torch.int32, device="cuda"),
                     cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), status=status)
    assert int(status) in (0, 5)
    assert not whole[:2].any() and not whole[2 + 6:].any()


def test_one_row_for_every_token():
    """A broadcast input (row stride 0) and a single token."""
    a = torch.randn(1, 576, device="cuda").to(torch.bfloat16)
    cache = torch.zeros(2, 64, 576, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    rows = a.expand(9, 576)
    mla.cache_append(rows[:, :512], rows[:, 512:], cache, table, torch.tensor([20], dtype=torch.int32, device="cuda"))
    assert torch.equal(cache[1, 11:20], rows) and not cache[0].any() and not cache[1, :11].any()
    mla.cache_append(a[:, :512], a[:, 512:], cache, table, torch.tensor([1], dtype=torch.int32, device="cuda"))
    assert torch.equal(cache[1, 0], a[0])


@pytest.mark.parametrize("exponent", [0, -40, -90, 30])
def test_codes_are_the_quotients_rounded(exponent):
    """codes = E4M3(c' / scale), the quotient in fp32, bit for bit; among the rows are quotients at ties, where a
    product with the reciprocal of the scale rounds to the other neighbour."""
    tops = [m / 128.0 for m in range(128, 256)]
    finite = torch.arange(0x7f80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    rows, g = [], torch.Generator().manual_seed(41)

    def code(v):
        return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    for top in tops:
        scale = torch.tensor(top) / 448
        x = finite[(finite <= top) & (finite > 0)]
        tie = x[code(x / scale) != code(x * (1 / scale))]
        fill = torch.randn(128, generator=g).clamp(-top, top).to(torch.bfloat16).float()
        fill[0] = top
        fill[1:1 + min(len(tie), 120)] = tie[:120]
        rows.append(fill)
    lat = (torch.stack(rows).reshape(32, 512) * 2.0 ** exponent).to(torch.bfloat16)
    c = Case([32], [40], fp8=True, norm=False, rope=False, seed=42)
    c.c, c.host = lat, (lat.double().numpy(), c.host[1])
    cache = c.run()
    c.check(cache)
    x = lat.float().reshape(32, 4, 128)
    scale = x.abs().amax(2) / 448
    want = code(x / scale[..., None])
    assert (want != code(x * (1 / scale)[..., None])).sum() > 50
    at, _ = so.append_targets(c.cu, c.lens, c.table, c.pages)
    got = torch.stack([cache[p, r].cpu() for p, r, _ in (at[t] for t in range(32))])
    assert torch.equal(got[:, :512].reshape(32, 4, 128), want)
    assert torch.equal(got[:, 512:528].contiguous().view(torch.float32), scale)


def test_infinity_takes_its_group():
    """A scale of infinity: finite values over it are zeros, infinities no number; other groups as ever."""
    c = Case([2], [0], fp8=True, seed=43, norm=False, rope=False)
    c.c[0, 130] = float("inf")
    c.c[0, 140] = -3e38
    cache = c.run()
    row = cache[int(c.table[0, 0]), 0].cpu()
    codes, scale = so.e4m3_value(row[:512].numpy()), row[512:528].clone().view(torch.float32).numpy()
    assert np.isinf(scale[1]) and np.isfinite(scale[[0, 2, 3]]).all()
    assert np.isnan(codes[130]) and not np.delete(codes[128:256], 2).any()
    assert np.isfinite(np.delete(codes, 130)).all() and codes[:128].any() and codes[256:].any()
