"""CPU: frequencies as fractions of a turn (csrc/sp_turns.h), against exact arithmetic.

A fraction is off by half a step of 2^-64 and by the double's own roundings of
w / 2 pi: the constant's (relative 2^-54.5) and the division's (2^-53), which are
1.35 * 2^-53 / (2 pi) < 2^-55 of |w| together."""
import math
import os
import random
import shutil
import subprocess
from fractions import Fraction

import pytest

from _angles import PI, turns

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "head_aware_paged_gb300", "csrc")


@pytest.fixture(scope="module")
def turn_of(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path_factory.mktemp("turns") / "turns_check")
    subprocess.run([cxx, "-std=c++17", "-O2", "-I", CSRC, os.path.join(HERE, "turns_check.cpp"), "-o", exe],
                   check=True, capture_output=True)

    def run(ws):
        out = subprocess.run([exe], input="".join(float(w).hex() + "\n" for w in ws), capture_output=True, text=True,
                             check=True).stdout.split()
        assert len(out) == len(ws)
        return [int(x) for x in out]
    return run


def _off(got, w):
    """Distance on the circle, in turns."""
    d = (Fraction(got, 1 << 64) - turns(w)) % 1
    return min(d, 1 - d)


def test_pi():
    assert abs(float(PI) - math.pi) == 0.0 and abs(PI - Fraction(math.pi)) < Fraction(1, 1 << 52)
    # its 40 decimals
    assert str(int(PI * 10 ** 40)) == "31415926535897932384626433832795028841971"


def _frequencies():
    r = random.Random(5)
    ws = [t ** (-2.0 * i / d) for t in (1e4, 5e5, 1e6) for d in (64, 128) for i in range(d // 2)]
    ws += [2.0 ** r.uniform(-60, 16) for _ in range(2000)]
    ws += [1e-6, 1e-9, 2.0 ** -70, 65536.0, 1.0, math.pi, 2 * math.pi, math.pi / 4, 5e-324, 0.0]
    # just below and above whole turns
    ws += [math.nextafter(2 * math.pi * k, s) for k in (1, 2, 7, 1000) for s in (0.0, 1e9)]
    return ws


def test_fractions_of_a_turn(turn_of):
    ws = _frequencies()
    for w, t in zip(ws, turn_of(ws)):
        assert _off(t, w) <= Fraction(1, 1 << 65) + Fraction(w) / (1 << 55), w


def test_negative_frequencies_turn_backwards(turn_of):
    ws = _frequencies()
    for w, t, b in zip(ws, turn_of(ws), turn_of([-w for w in ws])):
        assert (t + b) % (1 << 64) == 0, w
        assert _off(b, -w) <= Fraction(1, 1 << 65) + Fraction(w) / (1 << 55), w
