"""What the low-precision bindings refuse before they touch a GPU."""

import pytest
import torch

from dense_fp32_matrix_row_amd import blockfp8


@pytest.mark.parametrize("kind", (torch.bfloat16, torch.float16, torch.float64))
def test_a_weight_gradient_that_is_not_float32_is_refused(kind):
    q = blockfp8.BlockFp8(torch.zeros(4, 16, dtype=torch.float8_e4m3fn), torch.ones(4, 1))
    with pytest.raises(TypeError, match="dw is float32"):
        blockfp8.linear_backward(torch.zeros(16, 4), q, q, dw=torch.zeros(4, 4, dtype=kind))
