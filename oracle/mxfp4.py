"""MXFP4: E2M1 elements under one power of two per 32, and the linear over it
(TEST INFRASTRUCTURE ONLY).

The format and its conversion are the OCP microscaling formats specification's:
shared exponent floor(log2 max|x|) - 2, elements rounded to nearest even and
saturated.  READINGS: the shared exponent is clamped at -127; a block with an
infinity or a NaN gets the NaN scale and zero codes; rows are padded with zero
blocks to a multiple of 256 columns.
"""

import numpy as np

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def encode_value(y):
    """Code (0..15) of one scaled fp64 value: nearest level, ties to the even code."""
    d = np.abs(LEVELS - min(abs(y), 6.0))
    best = np.flatnonzero(d == d.min())
    c = int(best[0]) if len(best) == 1 else int(best[best % 2 == 0][0])
    return c | (8 if np.signbit(y) else 0)


def quantize(x):
    """(codes uint8[rows, 128 C] packed, scales uint8[C, rows, 8]) of an fp32-valued matrix."""
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    C = -(-cols // 256)
    v = np.zeros((rows, 256 * C), dtype=np.float64)
    v[:, :cols] = x
    v = v.reshape(rows, 8 * C, 32)
    bad = ~np.isfinite(v).all(axis=2)
    top = np.abs(np.where(bad[:, :, None], 0.0, v)).max(axis=2)
    _, e = np.frexp(top)
    e = np.where(top > 0, np.maximum(e - 1 - 2, -127), -127)
    y = np.where(bad[:, :, None], 0.0, v) * np.exp2(-e.astype(np.float64))[:, :, None]
    m = np.minimum(np.abs(y), 6.0)
    # distance to every level; of two equal ones the even code
    d = np.abs(m[..., None] - LEVELS)
    lo = d.argmin(axis=3)
    nxt = np.minimum(lo + 1, 7)
    tie = (nxt != lo) & (np.take_along_axis(d, nxt[..., None], 3)[..., 0] == np.take_along_axis(d, lo[..., None], 3)[..., 0])
    code = np.where(tie & (lo % 2 == 1), nxt, lo) | (np.signbit(y).astype(np.int64) << 3)
    code = code.reshape(rows, 256 * C).astype(np.uint8)
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    byte = np.where(bad, 255, e + 127).astype(np.uint8)
    return packed, np.ascontiguousarray(byte.reshape(rows, C, 8).transpose(1, 0, 2))


def dequant(packed, scales, cols):
    """fp64 values [rows, cols] (NaN under scale byte 255)."""
    packed = np.asarray(packed)
    rows = packed.shape[0]
    code = np.stack((packed & 15, packed >> 4), axis=2).reshape(rows, -1)
    v = np.where(code >= 8, -1.0, 1.0) * LEVELS[code & 7]
    byte = np.asarray(scales).transpose(1, 0, 2).reshape(rows, -1).astype(np.int64)
    unit = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    return (v.reshape(rows, -1, 32) * unit[:, :, None]).reshape(rows, -1)[:, :cols]


def values(x):
    """What x stands for after quantisation, fp64."""
    return dequant(*quantize(x), np.asarray(x).shape[1])


def linear_forward(base_in, X, What, A, B, alpha, keep=None, c=1.0):
    """(Y, H) in fp64: base_in What^T + (alpha/r) H B^T, H = c (keep * X) A^T."""
    Y = np.asarray(base_in, dtype=np.float64) @ np.asarray(What, dtype=np.float64).T
    if A is None:
        return Y, None
    A, B = np.asarray(A, dtype=np.float64), np.asarray(B, dtype=np.float64)
    D = np.asarray(X, dtype=np.float64)
    if keep is not None:
        D = np.where(keep, D, 0.0) * c
    H = D @ A.T
    return Y + (float(alpha) / A.shape[0]) * (H @ B.T), H


def linear_backward(G, X, What, A, B, alpha, keep=None, c=1.0, H=None):
    """(dX, dA, dB) in fp64 of linear_forward, the base input's rounding passing
    the gradient through; H given replaces the recomputed one in dB."""
    G, What = np.asarray(G, dtype=np.float64), np.asarray(What, dtype=np.float64)
    dX = G @ What
    if A is None:
        return dX, None, None
    A, B = np.asarray(A, dtype=np.float64), np.asarray(B, dtype=np.float64)
    D = np.asarray(X, dtype=np.float64)
    k = np.ones(D.shape) if keep is None else keep * c
    D = np.where(k != 0, D, 0.0) * k
    s = float(alpha) / A.shape[0]
    dH = s * (G @ B)
    H = D @ A.T if H is None else np.asarray(H, dtype=np.float64)
    return dX + k * (dH @ A), dH.T @ D, s * (G.T @ H)
