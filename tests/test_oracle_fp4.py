"""Pins of the float64 4-bit oracle: exhaustive rounding against exact rationals, and its edge rules."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import fp4
from oracle.formats import E2M1_TABLE, E4M3_TABLE


def _nearest_rational(q, grid):
    best = min(range(len(grid)), key=lambda i: (abs(Fraction(float(grid[i])) - q), i % 2))
    return best


@pytest.mark.parametrize("gs", [np.float32(1), np.float32(2.0 ** -13), np.float32(0.00123)])
def test_nvfp4_codes_are_the_nearest_to_the_exact_quotient(gs):
    rng = np.random.default_rng(1)
    w = (rng.standard_normal((24, 64)) * rng.choice([1e-3, 0.02, 1.0], (24, 1)) * float(gs) * 500).astype(np.float32)
    w[0, :16] = 0
    # exact ties: halves of grid steps times a scale that is hit exactly
    w[1, :16] = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0]) * float(gs)
    codes, sb, g = fp4.quantize(w, "nvfp4", gs)
    assert g == gs
    for r in range(24):
        for b in range(4):
            blk = w[r, b * 16:b * 16 + 16]
            top = Fraction(float(np.abs(blk).max()))
            si = _nearest_rational(min(top / (6 * Fraction(float(gs))), Fraction(448)), E4M3_TABLE[:127])
            assert sb[r, b] == si
            d = Fraction(float(E4M3_TABLE[si])) * Fraction(float(gs))
            for e in range(16):
                c = codes[r, b * 16 + e]
                if d == 0:
                    assert c == 0
                    continue
                q = min(abs(Fraction(float(blk[e]))) / d, Fraction(6))
                assert c % 8 == _nearest_rational(q, E2M1_TABLE[:8])
                assert (c >= 8) == bool(np.signbit(blk[e]))


def test_mxfp4_scales_are_powers_of_two_and_codes_saturate():
    w = np.zeros((5, 32), np.float32)
    w[0, 0], w[0, 1] = 7.9, -1.0           # 2^2 -> scale 2^0: 7.9 saturates at 6
    w[1, 0] = 2.0 ** -140                  # below every scale
    w[2, 3] = np.nan
    w[3, 3], w[3, 4] = -np.inf, 1
    codes, sb, _ = fp4.quantize(w, "mxfp4")
    assert sb[0, 0] == 127 and codes[0, 0] == 7 and codes[0, 1] == 2 + 8
    assert sb[1, 0] == 0 and not codes[1].any()
    assert list(sb[2:4, 0]) == [255, 255] and not codes[2:4].any() and sb[4, 0] == 0
    v = fp4.values(codes, sb, "mxfp4")
    assert np.isnan(v[2:4]).all() and v[0, 0] == 6


def test_nvfp4_global_scale_ignores_what_is_not_finite():
    w = np.full((2, 32), 0.5)
    w[0, 3], w[1, 20] = np.inf, np.nan
    codes, sb, gs = fp4.quantize(w, "nvfp4")
    assert gs == np.float32(0.5 / 2688)
    assert list(sb.reshape(-1) == 0x7F) == [True, False, False, True]
    z = fp4.quantize(np.zeros((2, 16)), "nvfp4")
    assert z[2] == 1 and not z[0].any() and not z[1].any()


def test_pack_round_trip():
    c = np.random.default_rng(0).integers(0, 16, (3, 32)).astype(np.uint8)
    assert np.array_equal(fp4.unpack(fp4.pack(c)), c)
