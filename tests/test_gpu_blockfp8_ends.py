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


@pytest.mark.parametrize("kind", (torch.bfloat16, torch.float16))
def test_a_weight_gradient_that_is_not_float32_is_refused(kind):
    """And nothing is added to it."""
    dy, x = (torch.randn(32, n, device="cuda") for n in (48, 80))
    _, xt = blockfp8.linear_forward(x, blockfp8.quantize(torch.randn(48, 80, device="cuda"), 128))
    wt = blockfp8.quantize_transposed(torch.randn(48, 80, device="cuda"), 128)
    dw = torch.ones(48, 80, dtype=kind, device="cuda")
    with pytest.raises(TypeError, match="dw is float32"):
        blockfp8.linear_backward(dy, xt, wt, dw=dw)
    assert (dw == 1).all()
    assert blockfp8.linear_backward(dy, xt, wt, dw=dw.float())[1].dtype == torch.float32
