"""CPU-only: the calls with dropout say that they need one."""

import pytest
import torch

from bit_nf4_quantized_08_amd import lib


def test_dropout_is_required():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="drop is required"):
        lib.dropout(x, None)
    with pytest.raises(ValueError, match="drop is required"):
        lib.qlora_linear_fwd_dropout(x, None, x, x, 1.0, None)
    with pytest.raises(ValueError, match="drop is required"):
        lib.qlora_linear_bwd_dropout(x, x, None, x, x, 1.0, None)
