"""The 4-bit cache's oracle against values worked out by hand, and rotary positions against
complex products and against differences."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import cache4 as c4


def test_codes():
    assert c4.e2m1_values().tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    x = np.array([0, .24, .25, .26, .75, 1.25, 1.75, 2.5, 2.6, 3.5, 5, 5.01, 6, 7, np.inf])
    want = [0, 0, 0, 1, 2, 2, 4, 4, 5, 6, 6, 7, 7, 7, 7]
    assert c4.e2m1_encode(x).tolist() == want
    assert (c4.e2m1_encode(-x) == np.array(want) + 8).all()
    for code, v in enumerate(c4.e2m1_values()):
        assert c4.e2m1_encode(np.array([v]))[0] == code


@pytest.mark.parametrize("amax,e", [(6, 0), (6.01, 1), (3.01, 0), (3, -1), (1, -2), (0.75, -3),
                                    (1e-30, -60), (0, -60), (1e30, 60), (math.inf, 60)])
def test_block_scale(amax, e):
    x = np.zeros(32)
    x[7] = -amax
    assert c4.block_scale(x) == 127 + e
    x[3] = math.nan
    assert c4.block_scale(x) == 255


def test_write_and_read_back():
    rng = np.random.default_rng(1)
    kc, vc = np.zeros((3, 2, 16, 128), np.uint8), np.zeros((3, 2, 128, 16), np.uint8)
    ks, vs = np.zeros((3, 2, 16, 4), np.uint8), np.zeros((3, 2, 4, 16), np.uint8)
    k, v = rng.standard_normal((5, 2, 128)), 100 * rng.standard_normal((5, 2, 128))
    slots = [18, 19, -1, 48, 5]
    cache = c4.cache_write(k, v, slots, kc, vc, ks, vs)
    ko, vo = c4.cache_read(slots, *cache)
    for x, y in ((k, ko), (v, vo)):
        assert not y[2].any() and not y[3].any()
        for t in (0, 1, 4):
            blocks, got = x[t].reshape(-1, 32), y[t].reshape(-1, 32)
            amax = np.abs(blocks).max(1, keepdims=True)
            # a step at most 2 scales wide, a scale at most a third of the largest value
            assert (np.abs(blocks - got) <= amax / 3).all()
            assert (np.abs(got).max(1, keepdims=True) >= amax * 3 / 4).all()
    assert (c4.unpack(c4.pack(cache[0])) == cache[0]).all()


def test_turned():
    rng = np.random.default_rng(2)
    freq = [0.9, 0.01, 3e-5, 0.3]
    turns = [round(Fraction(f) * 2 ** 64 / Fraction(2 * math.pi)) for f in freq]
    x = rng.standard_normal((3, 2, 128))
    pos = [0, 17, 123456]
    for adjacent in (False, True):
        for first in (0, 40):
            y = c4.turned(x, pos, turns, first, adjacent, False, 1.25)
            i = first + np.arange(8)
            a, b = (i[0::2], i[1::2]) if adjacent else (i[:4], i[4:])
            for t, p in enumerate(pos):
                z = (x[t][:, a] + 1j * x[t][:, b]) * 1.25 * np.exp(1j * p * np.array(freq))
                np.testing.assert_allclose(y[t][:, a], z.real, atol=1e-9)
                np.testing.assert_allclose(y[t][:, b], z.imag, atol=1e-9)
            rest = np.setdiff1d(np.arange(128), i)
            assert (y[:, :, rest] == x[:, :, rest]).all()
            # back: the gradient of sum(y * g) is the inverse turn of g
            g = rng.standard_normal(x.shape)
            back = c4.turned(g, pos, turns, first, adjacent, True, 1.25)
            step = 1e-6
            for t, h, d in ((1, 0, first), (2, 1, first + 5), (1, 1, first + 7), (2, 0, 100)):
                up, down = x.copy(), x.copy()
                up[t, h, d] += step
                down[t, h, d] -= step
                diff = ((c4.turned(up, pos, turns, first, adjacent, False, 1.25)
                         - c4.turned(down, pos, turns, first, adjacent, False, 1.25)) * g).sum()
                assert abs(diff / (2 * step) - back[t, h, d]) < 1e-6
