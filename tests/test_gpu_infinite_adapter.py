"""Infinities in the adapter's path.  Where a factor is held as two bf16 pieces
(the value and its rest), an infinite value or an infinite other factor must give
what the product gives, an infinity of its sign, and not the NaN of inf - inf: Y of
the MXFP4 forward for every row count against the signs of the exact result, dA and
dB of the MXFP4 backward and of the dropout backward against the plain linear's."""

import numpy as np
import pytest
import torch

from bit_nf4_quantized_08_amd import lib, synth
from tests.gpu_util import REL_FRO_TOL, dev, host, rel_fro, say, to_dev

pytestmark = pytest.mark.gpu

INF = float("inf")
BF16_MAX = 2.0 ** 127 * (2 - 2.0 ** -7)


def _inputs(M, N, K, r, seed):
    W = synth.gaussian((N, K), 0.02, synth.SEED_W + seed)
    X = synth.to_bf16(synth.gaussian((M, K), 1.0, synth.SEED_X + seed))
    A = synth.to_bf16(synth.gaussian((r, K), 0.05, synth.SEED_A + seed))
    B = synth.to_bf16(synth.gaussian((N, r), 0.05, synth.SEED_B + seed))
    G = synth.to_bf16(synth.gaussian((M, N), 1.0, synth.SEED_DY + seed))
    return W, X, A, B, G


# K beyond 8192: several workgroups over K; N = 64, K = 4096: tiles cut over K up to 128 rows
@pytest.mark.parametrize("M, N, K", [(1, 64, 320), (4, 128, 1088), (16, 64, 8256), (20, 192, 320), (32, 64, 8256),
                                     (33, 64, 4096), (100, 64, 4096), (100, 128, 320), (300, 64, 4096), (300, 192, 320)])
@pytest.mark.parametrize("kind", ["H", "overflow", "B"])
def test_mx_forward(M, N, K, kind):
    say(f"mx forward, infinite {kind}, M={M} N={N} K={K}")
    r, j0, k0, k1, n0 = 8, 3, 77, 78, 50
    W, X, A, B, _ = _inputs(M, N, K, r, M)
    sign = torch.where(torch.arange(M) % 3 == 1, -1.0, 1.0).to(torch.bfloat16)
    X[:, k0], X[:, k1] = sign, sign
    w = lib.mxfp4_quantize(to_dev(W))
    if kind == "B":
        B[n0, j0] = INF
    else:   # H[:, j0] = sign * inf, or a finite value that rounds to an infinite bf16 one
        A[j0, :] = 0.0
        A[j0, k0], A[j0, k1] = (INF, 0.0) if kind == "H" else (BF16_MAX, 2.0 ** 119)
    Y, H = lib.qlora_mx_linear_fwd(X.to(dev()), w, A.to(dev()), B.to(dev()), float(r), want_H=True)
    got, Hv = host(Y), host(H)
    if kind == "B":
        want = np.where(Hv[:, j0] < 0, -INF, INF)
        assert (Hv[:, j0] != 0).all()
        np.testing.assert_array_equal(got[:, n0], want)
        assert np.isfinite(np.delete(got, n0, axis=1)).all()
    else:
        s = sign.float().numpy()
        assert np.isinf(Hv[:, j0]).all() if kind == "H" else np.isfinite(Hv).all()
        np.testing.assert_array_equal(got, np.sign(s[:, None] * B[:, j0].float().numpy()[None, :]) * np.float32(INF))


def _spoil(kind, X, G, H):
    """One non-finite spot in a backward's inputs."""
    if kind == "H":
        H[2, 3], H[1, 5], H[3, 0] = INF, -INF, 3.4e38   # the last is finite, its bf16 is not
    elif kind == "nan":
        H[2, 3] = float("nan")
    elif kind == "G":
        G[1, 7], G[3, 9] = INF, -INF
    elif kind == "X":
        X[3, 9], X[0, 17] = INF, -INF


@pytest.mark.parametrize("kind", ["H", "nan", "G", "X"])
@pytest.mark.parametrize("r", [8, 40])
@pytest.mark.parametrize("M", [4, 100, 300])
@pytest.mark.parametrize("base", ["mx", "nf4"])
def test_adapter_gradients(base, M, r, kind):
    """dA and dB: infinities, NaN and finite values where the plain backward has them."""
    say(f"{base} backward, infinite {kind}, M={M} r={r}")
    N, K = 192, 320
    W, X, A, B, G = _inputs(M, N, K, r, M + r)
    H = torch.from_numpy(synth.gaussian((M, r), 1.0, 9))
    _spoil(kind, X, G, H)
    X, A, B, G, H = (t.to(dev()) for t in (X, A, B, G, H))
    w = lib.quantize_weight(to_dev(W))
    _, dA0, dB0 = lib.qlora_linear_bwd(G, X, w, A, B, float(r), H=H)
    if base == "mx":
        _, dA, dB = lib.qlora_mx_linear_bwd(G, X, lib.mxfp4_quantize(to_dev(W)), A, B, float(r), H=H)
    else:
        _, dA, dB = lib.qlora_linear_bwd_dropout(G, X, w, A, B, float(r), lib.Dropout(0.0, 1), H=H)
    for name, a, b in (("dA", host(dA), host(dA0)), ("dB", host(dB), host(dB0))):
        np.testing.assert_array_equal(np.isnan(a), np.isnan(b), err_msg=name)
        np.testing.assert_array_equal(np.isinf(a) * np.sign(a), np.isinf(b) * np.sign(b), err_msg=name)
        f = np.isfinite(b)
        assert rel_fro(a[f], b[f]) <= 2 * REL_FRO_TOL   # either is within REL_FRO_TOL of the exact one


@pytest.mark.parametrize("M, N, K", [(16, 8256, 4160), (5, 16448, 4160), (20, 8256, 4160), (32, 512, 4160)])
@pytest.mark.parametrize("kind", ["H", "B"])
@pytest.mark.parametrize("want_H", [True, False])
def test_mx_forward_row_groups(M, N, K, kind, want_H):
    """Two and four groups of weight rows per wave, ranks beyond 32, H returned or not."""
    say(f"mx forward, infinite {kind}, row groups, M={M} N={N} K={K}")
    r, j0, k0, n0 = 40, 37, 77, N - 10
    gen = torch.Generator().manual_seed(M)
    X, A, B, W = (torch.randn(t, generator=gen) for t in ((M, K), (r, K), (N, r), (N, K)))
    X[:, k0] = torch.where(torch.arange(M) % 3 == 1, -1.0, 1.0)
    if kind == "B":
        B[n0, j0] = INF
    else:
        A[j0, :] = 0.0
        A[j0, k0] = INF
    X, A, B = (t.to(torch.bfloat16).to(dev()) for t in (X, A, B))
    res = lib.qlora_mx_linear_fwd(X, lib.mxfp4_quantize(W.to(dev())), A, B, float(r), want_H=want_H)
    got = host(res[0] if want_H else res)
    H = X.double() @ A.double().t()   # the column's sign; sums of 4160 terms of order 1, far from zero in 64 bits
    col = host(torch.sign(H[:, j0])).astype(np.float32)
    if want_H:
        np.testing.assert_array_equal(np.sign(host(res[1])[:, j0]), col)
    if kind == "B":
        np.testing.assert_array_equal(got[:, n0], col * np.float32(INF))
        assert np.isfinite(np.delete(got, n0, axis=1)).all()
    else:
        np.testing.assert_array_equal(got, np.sign(col[:, None] * host(B)[:, j0][None, :]) * np.float32(INF))
