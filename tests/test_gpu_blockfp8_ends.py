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


SIZES = [(3, 70, 300), (150, 140, 700), (700, 600, 400), (2049, 2085, 300)]  # small tiles and large ones


def small_operand(rows, K, block_rows, e8m0, size, seed):
    """A quantised matrix of normal values of about `size`: on the GPU, its codes and its scales in 64 bits."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, K, generator=g, dtype=torch.float64) * size).float()
    q, s = ref.quantize(x, block_rows, e8m0)
    wide = torch.zeros(rows, -(-K // 16) * 16)
    wide[:, :K] = q
    sc = s.to(torch.float8_e8m0fnu if e8m0 else torch.float32)
    return blockfp8.BlockFp8(wide.cuda().to(torch.float8_e4m3fn)[:, :K], sc.cuda(), block_rows), q, s


@pytest.mark.parametrize("size", (2.0 ** -50, 2.0 ** -62))
@pytest.mark.parametrize("b_block", (1, 128))
@pytest.mark.parametrize("scale", ("f32", "e8m0"))
@pytest.mark.parametrize("kind", ("f32", "bf16"))
@pytest.mark.parametrize("M,N,K", SIZES)
def test_scales_that_are_small_on_both_sides(M, N, K, kind, scale, b_block, size):
    """Scales of about 2^-57 and 2^-69: their product is a normal float, and a subnormal one of a dozen bits.
    The sums are normal floats in both."""
    e8m0 = scale == "e8m0"
    a, qa, sa = small_operand(M, K, 1, e8m0, size, 1)
    b, qb, sb = small_operand(N, K, b_block, e8m0, size, 2)
    da, db = ref.dequantize(qa, sa, 1), ref.dequantize(qb, sb, b_block)
    want, sizes = da @ db.T, da.abs() @ db.abs().T
    # sums as in float (2^-23 a term of a running sum, at most 128 of a block and the blocks), for bf16 the cut
    # products of the 8-bit instruction (7 of 8 up to 2^-13 of the eighth) and the result's half step
    tol = (K + 4) * 2.0 ** -23 * sizes + 2.0 ** -149
    if kind == "bf16":
        tol = (tol + 7 * 2.0 ** -13 * sizes) * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    if b_block == 128 and (kind == "f32" or not e8m0):  # the scales' product, half a step of 2^-149
        blocks = [qa[:, k:k + 128] @ qb[:, k:k + 128].T for k in range(0, K, 128)]
        tol = tol + 2.0 ** -150 * sum(t.abs() for t in blocks) * (1 + 2.0 ** -8)
    got = blockfp8.gemm(a, b, out_dtype=TYPES[kind]).cpu().double()
    off = (got - want).abs() > tol
    assert not off.any(), f"{off.sum().item()} off, {((got - want).abs() / tol).max().item()} of the tolerance"
