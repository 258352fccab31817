"""Values of the rotary table next to the zeros of sine and cosine, and how far its
angles are from position times frequency.

Angles.  A frequency's turns, f / 2 pi in 64 bits (two roundings, 2^-52 of it), keep
64 bits behind the point (the rest is cut, up to 2^-64 turns); a position times that
modulo a turn has no rounding.  So an angle is off by 2^-52 of itself and 2^-64 turns
a position.

Values, in fp32, of that angle.  The nearest quarter turn comes off; what is left, x
half turns, |x| <= 1/4, is the sum of a high and a low word, each rounded to 24 bits,
the high one at most |x| + 2^-31, the low one 2^-31: off by 2^-23 |x| + 2^-54.  The
sine: the series is cut at 2^-28 of it, its last sum rounds by 2^-24, and what is
added there, a tenth of it, by a few 2^-24 of its own: 2^-23 in all.  The cosine, at
least 0.7 there, alike, with x's error times pi x tan(pi x) < 0.8.  The magnitude and
the product, 2^-24 each.  Together below 2^-21 of the value, and pi 2^-54 < 2^-52 of
the magnitude next to zero.
"""

from fractions import Fraction

import numpy as np
import pytest
import torch

import mla_paged_kv_gb300 as mla

pytestmark = pytest.mark.gpu

PI = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)


def cut_turns(freq):
    """Steps of 2^-64 turns a position, with the library's 64-bit division."""
    turns = np.float64(freq) / 6.283185307179586476925
    return int(np.ldexp(turns - np.floor(turns), 64)) % 2 ** 64


def values(turns):
    """Cosine and sine of a fraction of a turn, each to 2^-52 of itself."""
    quarter = round(4 * turns)
    x = float((turns - Fraction(quarter, 4)) * 2 * PI)
    c, s = np.cos(x), np.sin(x)
    return [(c, s), (-s, c), (-c, -s), (s, -c)][quarter % 4]


def table(freq, size, first, n):
    out = torch.empty(n, 2 * len(freq), device="cuda")
    mla.mla_rope_table(freq, size, first, out)
    return out.double().cpu().numpy()


def check(freq, size, first, n=40, rows=None):
    got = table(freq, size, first, n)
    for i, f in enumerate(freq):
        step = cut_turns(f)
        for r in rows or range(n):
            p = first + r
            mine = Fraction(p * step % 2 ** 64, 2 ** 64)
            true = Fraction(f) * p / (2 * PI)
            off = (mine - true) % 1
            off = float(min(off, 1 - off))
            assert off <= 2.0 ** -52 * float(true) + p * 2.0 ** -64, (f, p)
            for k, want in enumerate(values(mine)):
                err = abs(got[r, k * len(freq) + i] - size * want)
                assert err <= 2.0 ** -21 * abs(size * want) + 2.0 ** -52 * size, (f, p, k, err)


TURN = 6.283185307179586


@pytest.mark.parametrize("first", [0, 1, 12345, (1 << 24) - 20, (1 << 31) - 40])
def test_frequencies_of_a_model(first):
    for scaling in ("none", "yarn"):
        freq, size = mla.rope_frequencies(64, 500000.0, scaling, 40.0, 4096)
        check(freq, size, first)


@pytest.mark.parametrize("part", [0.0, 0.25, 0.5, 0.75, 1.0])
@pytest.mark.parametrize("away", [2.0 ** -20, 2.0 ** -33, 2.0 ** -45, 2.0 ** -52])
def test_angles_next_to_the_quarters_of_a_turn(part, away):
    """A position of 1, 5, 9, .. times a quarter and a little more or less: values down to 2^-50 of the others."""
    freq = [TURN * (part + away), TURN * abs(part - away), TURN * (part + 3 * away), TURN * part] * 4
    check(freq, 1.0, 0, 50)
    check(freq, 1.25, 4001, 12)


@pytest.mark.parametrize("size", [1.0, 0.1 * np.log(40.0) + 1.0, 2.0 ** -20])
def test_small_angles_keep_their_bits(size):
    """Sines of the slowest pairs at the first positions are their angles, to a few units in the last place."""
    freq = [10.0 ** -k for k in range(3, 11)]
    check(freq, size, 0, 70)
    got = table(freq, 1.0, 0, 70)
    assert np.all(np.abs(got[1:, 8:] / np.multiply.outer(np.arange(1, 70), freq) - 1) <= 2.0 ** -20 + 0.07 ** 2 / 6)
