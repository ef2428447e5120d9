"""Counter-based dropout (TEST INFRASTRUCTURE ONLY).

"QLoRA Explained: A 4-Bit Base, NF4, and What It Really Costs", "Turn a LoRA
script into a QLoRA script with one config object": the adapter is configured
with a dropout.  READING: the pages leave the generator open; the mask is taken
from Philox4x32 with 7 rounds (Salmon et al., "Parallel random numbers: as easy
as 1, 2, 3", SC 2011), eight 16-bit fields per call, element i being field i % 8
of call i / 8, kept when the field is at least round(65536 p).
"""

import numpy as np

_M = (0xD2511F53, 0xCD9E8D57)
_W = (0x9E3779B9, 0xBB67AE85)
_LOW = np.uint64(0xFFFFFFFF)


def philox4x32(counter, key, rounds):
    """counter: four arrays of 32-bit words (as uint64), key: two ints -> four arrays."""
    c = [np.asarray(x, dtype=np.uint64) for x in counter]
    k = [int(key[0]), int(key[1])]
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(_M[0]), c[2] * np.uint64(_M[1])
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & _LOW,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & _LOW]
        k = [(k[0] + _W[0]) & 0xFFFFFFFF, (k[1] + _W[1]) & 0xFFFFFFFF]
    return c


def threshold(p):
    return min(65535, int(np.floor(float(np.float32(p)) * 65536.0 + 0.5)))


def scale(p):
    """1 / (1 - p) of the probability the threshold stands for, in fp64."""
    return 65536.0 / (65536.0 - threshold(p))


def keep(n, p, seed, offset):
    """bool[n]: the elements kept."""
    g = np.arange((n + 7) // 8, dtype=np.uint64)
    off = [np.full_like(g, offset & 0xFFFFFFFF), np.full_like(g, offset >> 32)]
    w = philox4x32([g & _LOW, g >> np.uint64(32)] + off, (seed & 0xFFFFFFFF, seed >> 32), 7)
    f = np.stack([h for x in w for h in (x & np.uint64(0xFFFF), x >> np.uint64(16))], axis=1).reshape(-1)[:n]
    return f >= np.uint64(threshold(p))


def dropout(x, p, seed, offset):
    """c x where kept, 0 elsewhere, in fp64 (c rounded to fp32, as the definition has it)."""
    x = np.asarray(x, dtype=np.float64)
    k = keep(x.size, p, seed, offset).reshape(x.shape)
    return np.where(k, x * float(np.float32(scale(p))), 0.0)
