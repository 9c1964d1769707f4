"""Angles of rotary positions without a GPU, against exact rational arithmetic: the reduction of a frequency to a 64-bit
fraction of a turn as the kernel does it, at positions beyond 32 bits and frequencies beyond one radian."""
from fractions import Fraction
import math

import pytest

from oracle import blocks as ob
from state_space_sequence_mamba_b200 import binding as bd

POSITIONS = (0, 1, -1, 12345, 131072, 2 ** 20, 2 ** 31 - 1, -2 ** 31, 2 ** 33, 2 ** 40 + 3, 2 ** 40 + 7, -2 ** 39 - 1, 2 ** 62 + 1)
HIGH, LOW = 0.15915494309189535, -9.839338337591243e-18      # 1 / 2 pi in two parts


def fma(a, b, c):
    return float(Fraction(a) * Fraction(b) + Fraction(c))


def fraction_of_a_turn(f):
    whole = f * HIGH
    t = (whole - round(whole)) + fma(f, LOW, fma(f, HIGH, -whole))
    t -= round(t)
    return max(-2 ** 63, min(2 ** 63 - 1, round(t * 2.0 ** 64))) % 2 ** 64


def distance(a, b):
    d = abs(a - b) % 1
    return min(d, 1 - d)


def test_two_pi():
    """The rational 2 pi and its inverse's two parts, against pi by the arctangents of 1/5 and 1/239 (Machin)."""
    def arctan_of_inverse(n):
        return sum(Fraction((-1) ** k, (2 * k + 1) * n ** (2 * k + 1)) for k in range(60))

    two_pi = 8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))
    assert abs(two_pi - ob.TWO_PI) < Fraction(1, 10 ** 59)
    assert abs(1 / two_pi - Fraction(HIGH) - Fraction(LOW)) < Fraction(1, 2 ** 108)


@pytest.mark.parametrize("pos", POSITIONS)
def test_angles_are_exact_to_a_share_of_a_turn(pos):
    """2^-54 turns for each position: the sum of two parts below one half is rounded at 2^-55, the fraction at 2^-64."""
    some = bd.rotary_frequencies(64)[0].tolist() + bd.rotary_frequencies(128, scaling="yarn", factor=16.0)[0].tolist()
    for f in some + [-0.3, 1.5, math.pi, -math.pi, 2 * math.pi, 10.0, 100.0, 1000.0, 12345.678, -1e6, 2.0 ** 40, 1e-30]:
        got = Fraction(pos * fraction_of_a_turn(f) % 2 ** 64, 2 ** 64)
        assert distance(got, ob.turns(f, pos)) <= abs(pos) * Fraction(1, 2 ** 54), f


def test_one_part_of_the_inverse_is_not_enough():
    """(what the two parts are for)"""
    turn = 1000.0 * HIGH
    got = Fraction((2 ** 31 - 1) * int((turn - math.floor(turn)) * 2.0 ** 64) % 2 ** 64, 2 ** 64)
    assert distance(got, ob.turns(1000.0, 2 ** 31 - 1)) > (2 ** 31 - 1) * Fraction(1, 2 ** 50)
