"""CPU-only: what the backwards ask for as workspace."""

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
