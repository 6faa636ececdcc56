"""The MXFP4 test reference against direct statements of the format (CPU)."""
import math
from fractions import Fraction

import numpy as np
import pytest

from tests import mx_ref


def test_scale_is_the_largest_power_with_the_maximum_in_the_top_binade():
    # A / 2^e lies in [4, 8): E2M1's largest binade and its overflow to 6
    rng = np.random.default_rng(1)
    for a in np.concatenate([np.exp(rng.uniform(-80, 80, 200)), 2.0 ** np.arange(-100, 100)]):
        e = int(mx_ref.scale_codes(np.array([a]))[0]) - 127
        assert 4 <= Fraction(a) / Fraction(2) ** e < 8


def test_scale_code_limits():
    got = mx_ref.scale_codes(np.array([0.0, 2.0 ** -149, 2.0 ** -125, 2.0 ** -124, 3.4e38, np.inf, np.nan]))
    assert list(got) == [0, 0, 0, 1, 252, 255, 255]


@pytest.mark.parametrize("a,code", [(0, 0), (0.25, 0), (0.2500001, 1), (0.75, 2), (0.7499999, 1), (1.25, 2), (1.75, 4),
                                    (2.5, 4), (2.5000001, 5), (3.5, 6), (5, 6), (5.0000001, 7), (7.99, 7)])
def test_ties_go_to_the_even_code(a, code):
    assert mx_ref.nearest_code(np.array([float(a)]))[0] == code


def test_layouts_by_element():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((131, 200)) * np.exp(rng.standard_normal((131, 1)))
    c, s = mx_ref.quantize(x)
    q, sf = mx_ref.pack_codes(c), mx_ref.pack_scales(s)
    assert q.shape == (131, 128) and sf.shape == (2, 2, 128, 4)
    for r, k in [(0, 0), (1, 33), (130, 199), (128, 150)]:
        v = x[r, k] / 2.0 ** (int(sf[r // 128, k // 128, r % 128, k // 32 % 4]) - 127)
        nib = (q[r, k // 2] >> (4 * (k % 2))) & 15
        g = mx_ref.GRID[nib & 7]
        assert math.copysign(1, v) == (-1 if nib & 8 else 1)
        assert min(abs(abs(v) - m) for m in mx_ref.GRID) == abs(min(abs(v), 8) - g) or abs(v) > 6
    assert not q[:, 100:].any() and not sf[1, :, 3:].any()


def test_representable_values_come_back():
    codes = np.arange(16, dtype=np.uint8).repeat(2)[None, :].repeat(4, 1)
    s = np.full((1, 4), 130, np.uint8)
    v = mx_ref.values(codes, s)
    assert (mx_ref.fake(v) == v).all()
