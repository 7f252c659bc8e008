"""Words of a rope's table against rational arithmetic (no GPU needed)."""
import ctypes
import math
from fractions import Fraction

import pytest

from tests.test_abi import K  # noqa: F401

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628621")


@pytest.mark.parametrize("freqs", [[1.0, 0.75, -1.0, 0.1, 1e-4, 1e-7, 1e-15, 0.0], [2 * math.pi, -2 * math.pi, 6.25, 3.0],
                                   [100.0, 12345.678, 1e9, 1.0e12, -1.0e12, 2.0 ** 40 - 1],
                                   [10000.0 ** (-2 * i / 128) for i in range(64)], [1e6 ** (-i / 32) for i in range(32)]])
def test_turns_are_within_a_unit(K, freqs):
    """Half a unit of 2^-62 for the rounding; what the two doubles of 1 / (2 pi) leave
    (2^-110 of it) and the remainder's own rounding (2^-53 of at most 2^-13) times
    2^40 stay below an eighth of one."""
    n = len(freqs)
    words = (ctypes.c_uint64 * n)()
    assert K.lib().kvq_rope_table((ctypes.c_double * n)(*freqs), None, n, words) == K.OK
    for f, w in zip(freqs, words):
        off = abs((Fraction(f) / TWO_PI) % 1 - Fraction(w >> 2, 1 << 62))
        assert w & 3 == 0 and min(off, 1 - off) <= Fraction(5, 8) / (1 << 62), (f, float(off * (1 << 62)))


def test_frequencies_of_any_size_make_a_word(K):
    freqs = [1e300, -1e300, 1.7e308, 5e-324, 2.0 ** 63]
    words = (ctypes.c_uint64 * 5)()
    assert K.lib().kvq_rope_table((ctypes.c_double * 5)(*freqs), None, 5, words) == K.OK
    assert (words[0] + words[1]) % (1 << 64) == 0 and words[3] == 0     # opposite turns; none at all
