"""The dropout oracle: its generator against published vectors, its mask's
order and share, and its scaling."""

import numpy as np
import pytest

from oracle import dropout as D


@pytest.mark.parametrize("ctr, key, out", [
    ((0, 0, 0, 0), (0, 0), (0x5f6fb709, 0x0d893f64, 0x4f121f81, 0x4f730a48)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x5207ddc2, 0x45165e59, 0x4d8ee751, 0x8c52f662)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0x4dfccaba, 0x190a87f0, 0xc47362ba, 0xb6b5242a)),
])
def test_generator_matches_published_vectors(ctr, key, out):
    got = D.philox4x32([np.array([c]) for c in ctr], key, 7)
    assert tuple(int(g[0]) for g in got) == out


def test_element_order_and_prefix():
    """Element i is field i % 8 of call i / 8, low half of each word first."""
    seed, off = 0x123456789ABCDEF0, 0xFEDCBA9876543210
    full = D.keep(64, 0.5, seed, off)
    for i in range(64):
        g = np.array([i // 8], dtype=np.uint64)
        w = D.philox4x32([g, g * 0, np.array([off & 0xFFFFFFFF]), np.array([off >> 32])],
                         (seed & 0xFFFFFFFF, seed >> 32), 7)
        field = (int(w[(i % 8) // 2][0]) >> (16 * (i % 2))) & 0xFFFF
        assert full[i] == (field >= 32768)
    np.testing.assert_array_equal(D.keep(13, 0.5, seed, off), full[:13])


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9])
def test_kept_share(p):
    """Within 5 standard deviations of a binomial draw; everything for p = 0."""
    n = 1 << 18
    k = D.keep(n, p, 7, 3)
    q = 1 - D.threshold(p) / 65536
    assert abs(k.sum() - n * q) <= 5 * np.sqrt(n * q * (1 - q))
    assert D.scale(p) == pytest.approx(1 / q)


def test_not_kept_is_zero_whatever_it_was():
    x = np.array([np.inf, np.nan, -np.inf, 1.0] * 64)
    k = D.keep(x.size, 0.5, 1, 2)
    y = D.dropout(x, 0.5, 1, 2)
    assert np.all(y[~k] == 0) and 0 < k.sum() < x.size
