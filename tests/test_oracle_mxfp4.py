"""The MXFP4 oracle: the codec against brute force, the linear against the
plain oracle and against differences."""

import numpy as np
import pytest

import oracle
from oracle import dropout as D
from oracle import mxfp4 as MX


def test_codes_are_the_nearest_values_by_brute_force():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((3, 70)) * np.exp(2 * rng.standard_normal((3, 1)))).astype(np.float32)
    packed, scales = MX.quantize(x)
    assert packed.shape == (3, 128) and scales.shape == (1, 3, 8)
    for m in range(3):
        for b in range(8):
            blk = x[m, 32 * b:32 * b + 32].astype(np.float64)
            top = np.abs(blk).max() if blk.size else 0.0
            e = int(np.floor(np.log2(top))) - 2 if top > 0 else -127
            assert scales[0, m, b] == e + 127
            for t in range(32):
                k = 32 * b + t
                code = (packed[m, k // 2] >> (4 * (k % 2))) & 15
                assert code == (MX.encode_value(blk[t] / 2.0 ** e) if t < blk.size else 0)


@pytest.mark.parametrize("y, want", [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6),
                                     (6.0, 7), (7.9, 7), (-0.75, 10), (-0.1, 8)])
def test_ties_and_saturation(y, want):
    x = np.zeros((1, 32), dtype=np.float32)
    x[0, 0], x[0, 1] = 4.0, y          # 4 sets the scale to one (or less than twice that)
    packed, scales = MX.quantize(x)
    assert scales[0, 0, 0] == 127
    assert packed[0, 0] >> 4 == want == MX.encode_value(y)


def test_special_blocks():
    x = np.zeros((1, 256), dtype=np.float32)
    x[0, 32] = np.inf
    x[0, 64] = np.nan
    x[0, 96] = 1e-45
    x[0, 128] = 3e38
    _, s = MX.quantize(x)
    assert list(s[0, 0]) == [0, 255, 255, 0, 252, 0, 0, 0]
    v = MX.values(x)
    assert np.isnan(v[0, 32:96]).all() and not np.isnan(v[0, 96:]).any() and (v[0, :32] == 0).all()


def test_linear_without_dropout_is_the_plain_oracle():
    rng = np.random.default_rng(1)
    X, W, A, B, G = (rng.standard_normal(s) for s in ((5, 64), (7, 64), (3, 64), (7, 3), (5, 7)))
    Y, H = MX.linear_forward(X, X, W, A, B, 6.0)
    Yr, Hr = oracle.forward(X, W, A, B, 6.0)
    np.testing.assert_allclose(Y, Yr, rtol=1e-12, atol=1e-12)
    for a, b in zip(MX.linear_backward(G, X, W, A, B, 6.0, H=H), oracle.backward(G, X, W, A, B, 6.0)):
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-12)


def test_gradients_with_dropout_against_differences():
    """The forward is linear in each of X, A and B, so a central difference is
    exact up to fp64 rounding (about 1e-10 of the terms summed at this step)."""
    rng = np.random.default_rng(2)
    M, N, K, r = 4, 6, 32, 3
    X, W, A, B, G = (rng.standard_normal(s) for s in ((M, K), (N, K), (r, K), (N, r), (M, N)))
    keep, c = D.keep(M * K, 0.3, 11, 5).reshape(M, K), D.scale(0.3)
    f = lambda X, A, B: float((MX.linear_forward(X, X, W, A, B, 6.0, keep, c)[0] * G).sum())
    grads = MX.linear_backward(G, X, W, A, B, 6.0, keep, c)
    ops = [X, A, B]
    for i, g in enumerate(grads):
        for _ in range(6):
            at = tuple(rng.integers(0, n) for n in ops[i].shape)
            v = []
            for h in (1e-3, -1e-3):
                t = [o.copy() for o in ops]
                t[i][at] += h
                v.append(f(*t))
            assert (v[0] - v[1]) / 2e-3 == pytest.approx(g[at], abs=1e-8)
