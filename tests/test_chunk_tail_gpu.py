"""A long tail behind one dominant key: weights held in fp16 (fp16 caches and FP8
records) must keep it, for the sum that they are divided by does.

The dominant key has values of zero, so that the output is the tail's alone:
out = sum_j w_j v_j.  Its score, and small differences between the tail's, come
from the RoPE dims alone, products of numbers with few bits.

Tolerance.  A row's largest weight lies in 2^7 .. 2^15 (over FP8 records: the
largest product of a weight and 2^E), so that rounding to fp16 moves a weight by
2^-11 of itself, or, below fp16's smallest normal number, by 2^-25, which is 2^-32
of the largest at most.  Each of n / 16 products adds to the output in fp32 and may
lose one last place, 2^-23 of it; each of n / 128 sums that go into l 2^-23 of l.
The exponent, of up to 30 powers of two, is off by 2^-23 of itself three times
(scale, product, difference), and so is its weight: 30 ln 2 3 2^-23 < 2^-17.
"""

import numpy as np
import pytest
import torch

import mla_paged_kv_gb300 as mla

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def exponent(scale):
    """E of a key over FP8 records, from its largest scale."""
    return 8.0 * np.floor((np.floor(np.log2(scale)) + 11) / 8) - 10


class Tail:
    """n keys of values about 1 and one of zeros, `bits` powers of two above them, at `at`; over FP8 records with scales
    tail_scale and top_scale."""

    def __init__(self, kind, bits, n, at, tail_scale=0.25, top_scale=0.25, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.scale = n + 1, float(np.float32(bits * np.log(2.0) / 64.0))
        value = torch.randint(8, 16, (n + 1, 512), generator=g).float() / 8.0  # 1 .. 1.875: numbers of E4M3
        value[at] = 0
        rope = torch.zeros(n + 1, 64)
        rope[:, 1] = torch.randint(-8, 9, (n + 1,), generator=g).float() / 4.0
        rope[at, 0], rope[at, 1] = 8.0, 0.0
        pages = -(-(n + 1) // 64)
        room = pages * 64
        scale = torch.full((room,), tail_scale)
        scale[at] = top_scale
        rows = torch.zeros(room, 576)
        rows[:n + 1] = torch.cat([value, rope], 1)
        self.dtype = FP16 if kind == "fp16" else BF16
        self.e = np.zeros(n + 1)
        if kind == "fp8":
            self.cache = torch.cat([rows[:, :512].to(torch.float8_e4m3fn).view(torch.uint8),
                                    scale[:, None].expand(-1, 4).contiguous().view(torch.uint8),
                                    rows[:, 512:].to(BF16).view(torch.uint8)], 1).view(pages, 64, 656).contiguous()
            value = value * scale[:n + 1, None]
            self.e = exponent(scale[:n + 1].double().numpy())
        else:
            self.cache = rows.to(self.dtype).view(pages, 64, 576)
        self.value, self.rope = value.double().numpy(), rope.double().numpy()
        self.table = torch.randperm(pages, generator=g).int()
        where = torch.empty(pages, dtype=torch.long)
        where[self.table.long()] = torch.arange(pages)
        self.cache = self.cache[where].contiguous()

    def check(self, heads=16, parts=1, tokens=1):
        q = torch.zeros(tokens, heads, 576, dtype=self.dtype, device="cuda")
        q[..., 512] = 8.0
        q[..., 513] = torch.arange(heads, device="cuda") / 16.0
        args = q, self.cache.cuda(), self.table[None].cuda(), i32([self.n]), i32([0, tokens])
        pl = mla.plan_chunks(args[4], args[3], tokens, heads, False, num_parts=parts)
        out, lse = mla.chunk_attention(*args, False, self.scale, True, pl=pl)
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        half = 2.0 ** -8 if self.cache.dtype == BF16 else 2.0 ** -11
        least = 0.0 if self.cache.dtype == BF16 else 2.0 ** -32
        for h in range(heads):
            s = self.scale * (8.0 * self.rope[:, 0] + h / 16.0 * self.rope[:, 1])
            top = s.max()
            w = np.exp(s - top)
            z = w.sum()
            w /= z
            want = w @ self.value
            lost = np.maximum(half * w, least * (w * 2.0 ** self.e).max() / 2.0 ** self.e)
            sums = self.n / 16 * 2.0 ** -23 + self.n / 128 * 2.0 ** -23
            tol = (lost + (2.0 ** -16 + sums) * w) @ self.value + 2.0 ** -24 * want
            for t in range(tokens):
                err = np.abs(out[t, h] - want)
                assert np.all(err <= tol), ((err / want).max(), (tol / want).min())
                assert abs(lse[t, h] - (top + np.log(z))) <= 2.0 ** -16 + self.n / 128 * 2.0 ** -23 + \
                    2.0 ** -22 * abs(top + np.log(z))


@pytest.mark.parametrize("kind", ["fp16", "fp8", "bf16"])
@pytest.mark.parametrize("bits", [12, 20, 23, 25, 28])
@pytest.mark.parametrize("at", [0, 700, 131072])
def test_a_tail_of_131072_keys(kind, bits, at):
    Tail(kind, bits, 131072, at, seed=bits).check()


@pytest.mark.parametrize("kind", ["fp16", "fp8"])
def test_rows_of_several_blocks_and_pieces(kind):
    """The dominant key among the first piece's keys, and chunks whose pages are converted once."""
    c = Tail(kind, 24, 100003, 37, seed=1)
    c.check(heads=128, tokens=3)
    c.check(heads=16, parts=3)


@pytest.mark.parametrize("tail,top,bits", [(0.25, 2.0 ** 8, 17), (0.25, 2.0 ** -9, 25), (2.0 ** -9, 0.25, 17)])
def test_scales_of_another_power(tail, top, bits):
    """Tiles of FP8 records whose keys differ in E, beside tiles of one E."""
    Tail("fp8", bits, 131072, 300, tail, top, seed=bits).check()
