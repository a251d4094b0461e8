"""Tables of rotary positions against their formulas, written out in Python numbers:
scaled frequencies, and frequencies as parts of a turn.  CPU only: no kernel runs."""
import math
from fractions import Fraction

import pytest

from segmented_gather_gemm_gb300 import binding as B


def yarn(rot, base, factor, original, fast=32.0, slow=1.0):
    """(frequencies, (first, last) index of the ramp).  The pair that makes t turns in the
    original context has the index rot ln(original / (2 pi t)) / (2 ln base), which may lie
    behind the last pair; the ramp goes from the one of `fast` turns, rounded down, to
    the one of `slow` turns, rounded up, within [0, rot - 1]."""
    def index(turns):
        return rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
    lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rot - 1)
    f = []
    for i in range(rot // 2):
        own = base ** (-2.0 * i / rot)
        ramp = (0.0 if i <= lo else 1.0) if hi <= lo else min(max((i - lo) / (hi - lo), 0.0), 1.0)
        f.append(own * (1.0 - ramp) + own / factor * ramp)
    return f, (lo, hi)


@pytest.mark.parametrize("rot", [2, 8, 16, 64, 96, 128, 256])
@pytest.mark.parametrize("base", [100.0, 10000.0, 500000.0, 1e6])
@pytest.mark.parametrize("original", [512, 8192, 32768, 65536, 131072, 1 << 20])
def test_yarn(rot, base, original):
    for more in ((), (32.0, 1.0), (64.0, 2.0), (4.0, 0.25), (7.0, 7.0)):
        got, scale = B.rope_frequencies(rot, base, ("yarn", 8.0, original, *more))
        want, _ = yarn(rot, base, 8.0, original, *more)
        # (a power, two products and a sum in 64 bits)
        assert all(abs(a - b) <= 1e-14 * b for a, b in zip(got.tolist(), want)) and len(got) == len(want)
        assert scale == 0.1 * math.log(8.0) + 1.0


@pytest.mark.parametrize("rot,base,original,lo,hi", [(128, 1e4, 8192, 25, 50), (128, 1e4, 65536, 40, 65), (128, 1e4, 131072, 45, 70),
                                                     (64, 1e4, 65536, 20, 33), (16, 1e4, 32768, 4, 8), (128, 5e5, 8192, 18, 35),
                                                     (128, 1e6, 32768, 23, 40)])
def test_the_ramp_of_yarn(rot, base, original, lo, hi):
    """Where it begins and ends, worked out by hand."""
    assert yarn(rot, base, 4.0, original)[1] == (lo, hi)
    f = B.rope_frequencies(rot, base)[0].tolist()
    g = B.rope_frequencies(rot, base, ("yarn", 4.0, original))[0].tolist()
    for i in range(rot // 2):
        part = min(max((i - lo) / (hi - lo), 0.0), 1.0)
        assert abs(g[i] / f[i] - (1.0 - 0.75 * part)) < 1e-14


def test_pairs_that_all_turn_fast_are_kept():
    """Where the ramp would begin behind all pairs, none is stretched."""
    for rot, base, original in ((4, 10.0, 1 << 20), (8, 2.0, 1 << 20), (2, 100.0, 1 << 20)):
        assert B.rope_frequencies(rot, base, ("yarn", 4.0, original))[0].tolist() == B.rope_frequencies(rot, base)[0].tolist()


def turns(*freq):
    return [t % 2 ** 64 for t in B.csgmv_rope_turns(list(freq)).tolist()]


TURN = Fraction(2 * math.pi)  # the double next to 2 pi, as a whole turn
# 2 pi to 60 decimal places
TWO_PI = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)
FREQ = [1.0, 0.3, 1e-6, 2.0 ** -40 / 3, 2.0 ** -63, 5e-324, 3.0, 6.283185307179586, 6.283185307179587, 12.566, 1e5 / 3, 2.0 ** 53 + 2,
        1e300 / 7] + [10000.0 ** (-2 * i / 128) for i in range(64)] + [500000.0 ** (-2 * i / 128) for i in range(64)]


def test_turns_are_rounded_once():
    for f in FREQ:
        whole = 2 ** 64 * Fraction(f) / TURN
        want = math.floor(whole + Fraction(1, 2)) % 2 ** 64  # (none of these lies between two)
        assert turns(f) == [want], f


def test_turns_of_negative_frequencies():
    """They are those of the positive ones, the other way round, to the last bit."""
    up, down = turns(*FREQ), turns(*[-f for f in FREQ])
    assert [(a + b) % 2 ** 64 for a, b in zip(up, down)] == [0] * len(FREQ)


def test_turns_keep_the_bits_of_a_frequency():
    """The double that stands for a turn is off by 2^-54 of it, less than a
    frequency's own rounding: so is every frequency below a turn."""
    for f in FREQ:
        if f < 6:
            exact = 2 ** 64 * Fraction(f) / TWO_PI
            for way in (1, -1):
                off = (turns(way * f)[0] - way * exact) % 2 ** 64  # (up to whole turns)
                assert min(off, 2 ** 64 - off) <= exact / 2 ** 54 + Fraction(1, 2), f


@pytest.mark.parametrize("base,scaling", [
    (10000.0, ("yarn", 4.0, 8192, 1.0, 32.0)), (0.5, ("yarn", 4.0, 8192)), (1.0, ("yarn", 4.0, 8192)), (10000.0, ("yarn", 4.0, math.inf)),
    (10000.0, ("yarn", math.nan, 8192)), (10000.0, ("linear", math.inf)), (math.inf, None), (math.nan, None), (0.0, None)])
def test_scalings_that_are_refused(base, scaling):
    """What makes no ramp, or one that runs backwards."""
    with pytest.raises(B.CsgmvError):
        B.rope_frequencies(64, base, scaling)
