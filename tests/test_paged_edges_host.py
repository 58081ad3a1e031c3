"""Edges of the paged-cache entry points without a GPU: exact phases, and refusals that come before the first CUDA call (fake addresses,
which no call may follow)."""
import os
from fractions import Fraction

import pytest

# 2 pi to 60 digits, far beyond what the products below need
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")


@pytest.fixture(scope="module")
def svx():
    from speculative_decoding_verification_chunked_gb300 import build
    if not all(os.path.exists(x) for x in (build.LIB, build.LIB_CHECKED)):
        build.build()
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


def test_turns_are_exact_for_every_frequency(svx):
    """turns is the fraction of a turn to one unit of 2^-64, so that no 32-bit position's phase is off by more than 2^-33 turns,
    for the fastest pairs that are taken too."""
    inv = [1.0, 0.1, 1e-3, 3e-7, 1e-17, 5e-324, 2.0 ** -60, 6.283185307179586, 10.0, 1e5, 524287.3, 2.0 ** 20 - 2.0 ** -32, 1048575.9999999999, 0.0,
           99999.99, 123456.789]
    for sign in (1.0, -1.0):
        r = svx.Rope(32, inv_freq=[sign * f for f in inv])
        for i, f in enumerate(inv):
            got, exact = Fraction(r.table.turns[i], 1 << 64), Fraction(sign * f) / TWO_PI
            off = (got - exact) % 1
            off = min(off, 1 - off)
            assert off <= Fraction(1, 1 << 64), (sign * f, float(off * 2 ** 64))
            for pos in (2 ** 31 - 1, -2 ** 31, 131071):
                phase = Fraction((pos * r.table.turns[i]) % (1 << 64), 1 << 64) - pos * exact
                assert min(phase % 1, 1 - phase % 1) <= Fraction(1, 1 << 33)
