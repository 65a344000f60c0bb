"""The tensor forms of the 8-bit quantiser on sides whose rounding up to 16 passes an int."""

import pytest
import torch

from dense_fp32_matrix_row_amd import blockfp8

pytestmark = pytest.mark.gpu

LARGEST = (1 << 31) - 1


@pytest.mark.parametrize("transposed", (False, True))
def test_the_longest_row(transposed):
    x = torch.ones(1, LARGEST, dtype=torch.bfloat16, device="cuda")
    x[0, -1] = -2.0
    n = blockfp8.quantize_transposed(x.view(LARGEST, 1)) if transposed else blockfp8.quantize(x)
    assert n.q.shape == (1, LARGEST) and n.s.shape == (1, -(-LARGEST // 128))
    codes = n.q.view(torch.uint8)
    assert codes[0, :128].eq(0x7e).all()  # 448 of 1 / 448
    assert codes[0, -1].item() == 0xfe and codes[0, -127:-1].eq(0x76).all()  # -448, and 224, of 2 / 448
    torch.cuda.empty_cache()
