"""The table of rotation angles against rational arithmetic, and what far positions make of it."""
import math
from fractions import Fraction

import numpy as np
import pytest

PI = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10**60)     # pi to 60 digits


@pytest.fixture(scope="module")
def k():
    import __graft_entry__
    __graft_entry__._builder().build()
    import kv_cache_pruning_gb300
    return kv_cache_pruning_gb300


def _off(got, want):
    """Distance of two angles in turns."""
    d = (got - want) % 1
    return min(d, 1 - d)


def test_entries_are_right_to_their_last_bit(k):
    """Half a unit of 2^-64 for the rounding, and the two-double quotient's 2^-74."""
    rng = np.random.default_rng(3)
    freqs = list(500000.0 ** (-np.arange(0, 128, 2) / 128)) + list(10000.0 ** (-np.arange(0, 64, 2) / 64))
    freqs += list(np.exp(rng.uniform(-60, 22, 400)) * rng.choice([-1, 1], 400))
    freqs += [0.0, -0.0, 1.0, -1.0, 2 * math.pi, math.pi, 5e-324, 1e-300, 2.0**32, -(2.0**32), 2.0**32 - 2.0**-20, 6.25]
    got = k.kvp_rope_turns(freqs, device="cpu").numpy().view(np.uint64)
    for f, g in zip(freqs, got):
        off = _off(Fraction(int(g), 2**64), Fraction(float(f)) / (2 * PI))
        assert off <= Fraction(1, 2**65) + Fraction(1, 2**74), (f, float(off) * 2.0**64)


def test_far_positions_keep_their_angles(k):
    """pos * turns modulo 2^64, as the kernel takes it, at the farthest positions: 2^31 units of 2^-64 and their sum's
    rounding, so 2^-33 of a turn, far below the 2^-26 of the angle's fp32 form."""
    freqs = list(10000.0 ** (-np.arange(0, 128, 2) / 128)) + [6.25, -3.0, 40.0]
    got = k.kvp_rope_turns(freqs, device="cpu").numpy().view(np.uint64)
    for pos in (2**31 - 1, -2**31, 2**30 + 7, 1999999999, 131071, 1, 0):
        for f, g in zip(freqs, got):
            assert _off(Fraction((pos * int(g)) % 2**64, 2**64), Fraction(float(f)) * pos / (2 * PI)) <= Fraction(1, 2**33)


def test_refusals(k):
    for f in (2.0**32 + 2.0**-19, -1e10, 1e300, math.inf, -math.inf, math.nan):
        with pytest.raises(k.KvpError):
            k.kvp_rope_turns([1.0, f], device="cpu")
