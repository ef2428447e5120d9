"""CPU-only: what the backwards ask for as workspace."""

import ctypes
import os

import pytest

from bit_nf4_quantized_08_amd import lib

pytestmark = pytest.mark.skipif(not os.path.exists(lib.LIB_PATH), reason="library not built")


def up(x, n):
    return -(-x // n) * n


@pytest.mark.parametrize("M", [1, 64, 333, 4096, 16384, 65536, 1 << 20])
@pytest.mark.parametrize("N, K, r", [(64, 64, 8), (512, 3584, 8), (8192, 8192, 64), (28672, 8192, 16)])
def test_mx_backward_asks_for_what_it_writes(M, N, K, r):
    """dH in bf16, two factors in two bf16 pieces, then the larger of the column sums (at most 16 ranges) and the two
    low-rank products (ranges x 128-row blocks below 256 + blocks, at most 16 ranges), and dX's partial products (at
    most 8, where they are below 256 tiles of 64 x 256)."""
    Mp, rp = up(M, 64), up(r, 32)
    rows = 2 * M * rp + 8 * r * Mp
    sums = 16 * 4 * r * (N + K)
    lowrank = 2 * 4 * rp * min(16 * M, M + (1 << 15))
    cuts = 8 * 4 * 256 * 64 * 256
    assert 0 < lib.mx_workspace_size(lib.QN_OP_BWD, M, N, K, r) <= rows + max(sums, lowrank) + cuts + 8 * 256


def test_mx_backward_of_many_rows():
    """65536 rows of 8192 x 8192, r = 64: 75 MB, not gigabytes of ranges that no kernel writes."""
    assert lib.mx_workspace_size(lib.QN_OP_BWD, 65536, 8192, 8192, 64) < 80e6


def plain_backward(M, N, K, r):
    """B^T, dH, dH^T, (s H)^T, the 128-row sums of dB and dA, the low-rank products of dH and H, each rounded up to
    256 bytes."""
    rp, Mp, ranges = up(r, 32), up(M, 64), -(-M // 128)
    splits = lambda k: max(1, min(-(-256 // ranges), 16, k // 256))
    parts = [2 * rp * N, 2 * M * rp, 2 * rp * Mp, 2 * rp * Mp, 4 * ranges * r * N, 4 * ranges * r * K,
             4 * splits(N) * M * rp, 4 * splits(K) * M * rp]
    return sum(up(p, 256) for p in parts)


SHAPES = [(1, 128, 64, 8), (5, 4096, 4096, 16), (64, 512, 512, 1), (512, 4096, 4096, 16), (512, 8192, 8192, 64),
          (2048, 4096, 4096, 16), (4096, 8192, 28672, 64), (333, 512, 3584, 8), (1000, 128, 128, 33)]


@pytest.mark.parametrize("M, N, K, r", SHAPES)
def test_plain_backward_asks_for_its_own_layout(M, N, K, r):
    """QN_OP_BWD is the plain backward's size, whatever the call with dropout would like, and the call takes it."""
    n = plain_backward(M, N, K, r)
    assert lib.workspace_size(lib.QN_OP_BWD, M, N, K, r) == n
    vp, FAKE = ctypes.c_void_p, 0x10000
    w = lib.NF4WeightStruct(FAKE, FAKE, 0, 0, N, K, 0)
    # refused for its alignment, not its size: nothing is launched
    call = lambda size: lib.load().qlora_linear_bwd(vp(FAKE), vp(FAKE), vp(0), M, ctypes.byref(w), vp(FAKE), vp(FAKE), r,
                                                    16.0, vp(FAKE), vp(FAKE), vp(FAKE), vp(FAKE + 16), size, vp(0))
    assert call(n) == 4 and call(n - 1) == 5


@pytest.mark.parametrize("M, N, K, r", SHAPES + [(1, 64, 64, 64), (8, 64, 64, 32), (17, 64, 64, 24), (61, 512, 3584, 24)])
def test_backward_with_dropout_takes_both_sizes(M, N, K, r):
    vp, FAKE = ctypes.c_void_p, 0x10000
    w = lib.NF4WeightStruct(FAKE, FAKE, 0, 0, N, K, 0)
    d = lib.DropoutStruct(0.1, 1, 2, 0)
    call = lambda size: lib.load().qlora_linear_bwd_dropout(
        vp(FAKE), vp(FAKE), vp(0), M, ctypes.byref(w), vp(FAKE), vp(FAKE), r, 16.0, ctypes.byref(d), vp(FAKE), vp(FAKE),
        vp(FAKE), vp(FAKE + 16), size, vp(0))
    for op in (lib.QN_OP_BWD, lib.QN_OP_BWD_DROPOUT):
        assert call(lib.workspace_size(op, M, N, K, r)) == 4
    assert call(16) == 5
    assert lib.workspace_size(lib.QN_OP_BWD_DROPOUT, M, N + 1, K, r) == 0
