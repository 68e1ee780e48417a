"""pkv_rope_frequencies on the host: each scaling against its formula in
Python's 64-bit arithmetic, the fixed-point angle against exact rational
arithmetic, and the refusals."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

from paged_kv_cache_tables_gb300 import _binding as B

TURN = 2 ** 64


def frequencies(rot, base=10000.0, scaling=B.ROPE_PLAIN, factor=1.0, original=0.0, low=1.0, high=32.0):
    out, m = np.full(rot // 2 + 1, -77, np.int64), ctypes.c_float(0)
    rc = B.lib().pkv_rope_frequencies(out.ctypes.data, ctypes.byref(m), rot, base, scaling, factor, original, low, high)
    if rc == 0:
        assert out[-1] == -77
    return rc, out[:-1], m.value


def formula(rot, base, scaling, factor, original, low, high):
    f = []
    for i in range(rot // 2):
        w = base ** (-2 * i / rot)
        if scaling == B.ROPE_LINEAR:
            w /= factor
        elif scaling == B.ROPE_NTK:
            w = (base * factor ** (rot / (rot - 2))) ** (-2 * i / rot)
        elif scaling == B.ROPE_BANDS:
            turns = original * w / (2 * math.pi)
            if turns < low:
                w /= factor
            elif turns < high:
                s = (turns - low) / (high - low)
                w = s * w + (1 - s) * w / factor
        elif scaling == B.ROPE_YARN:
            pair = lambda t: rot * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base))   # noqa: E731
            a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
            r = min(max((i - a) / max(b - a, 1e-3), 0), 1)
            w = w * (1 - r) + w / factor * r
        f.append(w)
    return f


@pytest.mark.parametrize("rot", [16, 32, 48, 64, 112, 128])
@pytest.mark.parametrize("scaling,factor,original,low,high", [
    (B.ROPE_PLAIN, 1.0, 0.0, 0.0, 0.0), (B.ROPE_LINEAR, 4.0, 0.0, 0.0, 0.0), (B.ROPE_NTK, 8.0, 0.0, 0.0, 0.0),
    (B.ROPE_BANDS, 8.0, 8192.0, 1.0, 4.0), (B.ROPE_YARN, 16.0, 4096.0, 1.0, 32.0),
    (B.ROPE_YARN, 2.0, 10.0, 1.0, 32.0), (B.ROPE_BANDS, 1.0, 100.0, 0.5, 0.6)])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5])
def test_formula(rot, scaling, factor, original, low, high, base):
    rc, got, m = frequencies(rot, base, scaling, factor, original, low, high)
    assert rc == 0
    want = formula(rot, base, scaling, factor, original, low, high)
    for g, w in zip(got.tolist(), want):
        # a few double roundings of the formula and half a unit of the fixed point
        assert abs(g / TURN * 2 * math.pi - w) <= 1e-14 * w + 2 * math.pi / TURN
    assert m == pytest.approx(0.1 * math.log(factor) + 1 if scaling == B.ROPE_YARN else 1.0, rel=2 ** -23)


def test_angles_of_far_positions_modulo_a_turn():
    """position * frequency modulo 2^64 is the angle's fraction of a turn."""
    _, got, _ = frequencies(64)
    for f in got.tolist():
        exact = Fraction(f, TURN)
        for p in (0, 1, -1, 524287, 2 ** 31 - 1, -2 ** 31):
            assert Fraction((p * f) % TURN, TURN) == (p * exact) % 1


@pytest.mark.parametrize("kw,rc", [
    (dict(rot=8), -2), (dict(rot=24), -2), (dict(rot=144), -2), (dict(rot=64, scaling=5), -2),
    (dict(rot=64, scaling=-1), -2), (dict(rot=64, base=1.0), -1), (dict(rot=64, base=float("nan")), -1),
    (dict(rot=64, scaling=B.ROPE_LINEAR, factor=0.5), -1),
    (dict(rot=64, scaling=B.ROPE_NTK, factor=float("inf")), -1),
    (dict(rot=64, scaling=B.ROPE_YARN, factor=2.0), -1),
    (dict(rot=64, scaling=B.ROPE_BANDS, factor=2.0, original=4096.0, low=4.0, high=4.0), -1),
    (dict(rot=64, scaling=B.ROPE_BANDS, factor=2.0, original=4096.0, low=0.0, high=4.0), -1)])
def test_refusals(kw, rc):
    assert frequencies(**kw)[0] == rc


def test_null_pointers():
    L, m = B.lib(), ctypes.c_float(0)
    assert L.pkv_rope_frequencies(None, ctypes.byref(m), 64, 1e4, 0, 1.0, 0.0, 1.0, 32.0) == -1
    out = np.zeros(32, np.int64)
    assert L.pkv_rope_frequencies(out.ctypes.data, None, 64, 1e4, 0, 1.0, 0.0, 1.0, 32.0) == -1
