"""Angles of far positions: position * freqs modulo a turn against the scalings'
formulas in 60 digits.

Bound.  With u = 2^-53, a frequency f in double takes a rounding of the exponent
-2 i / r (f changes by |ln f| u relative), pow (2 u), and the division by 2 pi and
that constant's own rounding (2 u): f / 2 pi (|ln f| + 4) u turns, at most 0.64 u
since f (|ln f| + 4) grows up to f = 1.  LINEAR divides once more.  NTK's base
carries ((r / (r - 2)) ln factor + 3) u, which reaches f times the exponent: at most
(0.37 + 3) u / 2 pi more.  YARN's ramp and BANDS' share s add a few roundings of
f, s also t / (high - low) times the error of its t (high / (high - low) < 1.4
here).  All below 2 u = 2^-52 turns, and the fixed point half a unit of 2^-64."""
import ctypes
from decimal import ROUND_CEILING, ROUND_FLOOR, Decimal, localcontext

import numpy as np
import pytest

from paged_kv_cache_tables_gb300 import _binding as B

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def frequencies(rot, base, scaling, factor, original, low, high):
    out, m = np.zeros(rot // 2, np.int64), ctypes.c_float(0)
    assert B.lib().pkv_rope_frequencies(out.ctypes.data, ctypes.byref(m), rot, base, scaling, factor, original, low, high) == 0
    return out.tolist()


def formula(rot, base, scaling, factor, original, low, high):
    """Turns per position, in 60 digits."""
    base, factor, original, low, high = (Decimal(x) for x in (base, factor, original, low, high))
    one = Decimal(1)
    if scaling == B.ROPE_NTK:
        base *= (factor.ln() * rot / (rot - 2)).exp()
    if scaling == B.ROPE_YARN:
        pair = lambda turns: rot * (original / (turns * 2 * PI)).ln() / (2 * base.ln())   # noqa: E731
        first = max(pair(high).to_integral_value(ROUND_FLOOR), Decimal(0))
        last = min(pair(low).to_integral_value(ROUND_CEILING), Decimal(rot - 1))
    out = []
    for i in range(rot // 2):
        f = (base.ln() * -2 * i / rot).exp()
        if scaling == B.ROPE_LINEAR:
            f /= factor
        elif scaling == B.ROPE_BANDS:
            s = min(max((original * f / (2 * PI) - low) / (high - low), Decimal(0)), one)
            f = s * f + (one - s) * f / factor
        elif scaling == B.ROPE_YARN:
            ramp = min(max((i - first) / max(last - first, Decimal("0.001")), Decimal(0)), one)
            f = f / factor * ramp + f * (one - ramp)
        out.append(f / (2 * PI))
    return out


@pytest.mark.parametrize("rot", [16, 64, 96, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5])
@pytest.mark.parametrize("scaling,factor,original,low,high", [
    (B.ROPE_PLAIN, 1.0, 0.0, 0.0, 0.0), (B.ROPE_LINEAR, 3.0, 0.0, 0.0, 0.0), (B.ROPE_NTK, 8.0, 0.0, 0.0, 0.0),
    (B.ROPE_BANDS, 8.0, 8192.0, 1.0, 4.0), (B.ROPE_YARN, 16.0, 4096.0, 1.0, 32.0)])
def test_angles_of_far_positions(rot, base, scaling, factor, original, low, high):
    got = frequencies(rot, base, scaling, factor, original, low, high)
    with localcontext() as c:
        c.prec = 60
        want = formula(rot, base, scaling, factor, original, low, high)
        turn = Decimal(2 ** 64)
        for f, w in zip(got, want):
            for p in (1, 524287, 2 ** 31 - 1, -2 ** 31):
                off = (Decimal((p * f) % 2 ** 64) / turn - p * w) % 1   # as the kernel multiplies, modulo a turn
                off = min(abs(off), 1 - abs(off))
                assert off <= abs(p) * (Decimal(2) ** -52 + Decimal(2) ** -65), (p, f)
