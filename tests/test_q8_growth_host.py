"""The e4m3 scale's growth in the oracle, against exact rational arithmetic."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import quantized as oq

F32 = np.float32


def smallest(s, a):
    """s * 2^k with the smallest k >= 0 that makes room for a; room = fl(s * 448)."""
    room, k = Fraction(float(s * F32(448))), 0
    while room * 2 ** k < Fraction(float(a)):
        k += 1
    return Fraction(float(s)) * 2 ** k


@pytest.mark.parametrize("seed", range(4))
def test_smallest_power_of_two(seed):
    r = np.random.RandomState(seed)
    for _ in range(400):
        s = F32(np.ldexp(1 + r.rand(), r.randint(-109, 100)))
        a = F32(np.ldexp(1 + r.rand(), r.randint(-100, 127)))
        assert Fraction(float(oq.grown(s, a, "e4m3"))) == smallest(s, a)


@pytest.mark.parametrize("s,a", [(2.0 ** -109, 2.0 ** 100), (2.0 ** -100 / 448, 3.4e38), (2.0 ** -9, 3.5 * 2.0 ** 120),
                                 (1.0, 448.0), (1.0, 896.0), (1.0, np.nextafter(F32(896), F32(1e9))),
                                 (1.5, np.nextafter(F32(672), F32(0))), (1.5, np.nextafter(F32(672), F32(1e9)))])
def test_borders(s, a):
    s, a = F32(s), F32(a)
    assert Fraction(float(oq.grown(s, a, "e4m3"))) == smallest(s, a)
