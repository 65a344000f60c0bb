"""The 8-bit product and layer where a factor is not finite, a product of scales
leaves a float's range, an accumulator has another type, or autograd watches."""

import pytest
import torch

from dense_fp32_matrix_row_amd import blockfp8, orthogonal
from tests import lowp_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("alpha", (float("inf"), float("-inf"), float("nan"), 3.0))
def test_an_empty_sum_takes_no_alpha(alpha, kind):
    """K == 0: D is beta C, whatever alpha is."""
    flat = blockfp8.BlockFp8(torch.empty(5, 0, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(5, 0, device="cuda"), 1)
    c = torch.randn(5, 5, device="cuda").to(TYPES[kind])
    assert torch.equal(blockfp8.gemm(flat, flat, c=c, alpha=alpha, beta=2.0), 2 * c)
    assert (blockfp8.gemm(flat, flat, alpha=alpha, out_dtype=TYPES[kind]) == 0).all()
