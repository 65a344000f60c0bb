"""Every tile of the block-scaled product, alone and at the edges of larger ones,
against the definition in 64 bits: all kinds of scales and results."""

import functools

import pytest
import torch

from dense_fp32_matrix_row_amd import blockfp8
from tests import lowp_shapes as shapes
from tests.test_gpu_blockfp8 import SCALES, operand, tolerance, values

pytestmark = pytest.mark.gpu


@functools.lru_cache(maxsize=4)
def side(rows, K, scale, seed):
    """A quantised matrix by its block rows, and each one's value in 64 bits on the GPU."""
    out = {}
    for block in (1, 128):
        a, d = operand(rows, K, block, scale, seed)
        out[block] = a, d.cuda()
    return out


def check(size, scale, kind):
    M, N, K = size
    left, right = side(M, K, scale, 31), side(N, K, scale, 32)
    c = values(M, N, kind, 33).cuda()
    for b_block in (1, 128):
        b, db = right[b_block]
        for a_block in (1, 128):
            a, da = left[a_block]
            product, sizes = da @ db.T.contiguous(), (da.abs() @ db.abs().T.contiguous())

            def hold(got, want, alpha, beta_c):
                tol = tolerance_of(sizes, K, scale, kind, want, beta_c, alpha)
                got = got.double()
                past = torch.isinf(got) & (got.sign() == want.sign()) & (want.abs() + tol >= torch.finfo(kind).max)
                off = ~(((got - want).abs() <= tol) | past)
                assert not off.any(), f"{off.sum().item()} values off, first at {torch.nonzero(off)[0].tolist()}"

            hold(blockfp8.gemm(a, b, out_dtype=kind), product, 1.0, torch.zeros_like(product))
            place = c.clone()
            wide = torch.full((M, N + 5), 3.0, dtype=kind, device="cuda")
            want = 0.5 * product - 2 * c.double()
            assert blockfp8.gemm(a, b, c=place, alpha=0.5, beta=-2.0, out=place) is place
            hold(place, want, 0.5, 2 * c.double())
            blockfp8.gemm(a, b, c=c, alpha=0.5, beta=-2.0, out=wide[:, :N])
            assert torch.equal(torch.nan_to_num(wide[:, :N].float()), torch.nan_to_num(place.float()))
            assert (wide[:, N:] == 3).all()


def tolerance_of(sizes, K, scale, kind, want, beta_c, alpha):
    """test_gpu_blockfp8.tolerance, of a sum of magnitudes that is there."""
    one = torch.ones(1, 1, dtype=torch.float64)
    unit = tolerance(one, one, K, scale, kind, torch.zeros(1, 1, dtype=torch.float64), torch.zeros(1, 1), alpha)
    half = torch.finfo(kind).eps / 2
    least = torch.finfo(kind).smallest_normal * torch.finfo(kind).eps
    return unit.item() * sizes + 2.0 ** -23 * (1 + 2 * half) * beta_c.abs() + half * want.abs() + least


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("size", shapes.GEMM_FLOAT)
def test_float_results(size, scale):
    check(size, scale, torch.float32)


@pytest.mark.parametrize("kind", (torch.bfloat16, torch.float16))
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("size", shapes.GEMM_16_BIT)
def test_16_bit_results(size, scale, kind):
    check(size, scale, kind)


@pytest.mark.parametrize("c_type,kind,table", [(blockfp8.F32, torch.float32, shapes.GEMM_FLOAT),
                                               (blockfp8.BF16, torch.bfloat16, shapes.GEMM_16_BIT)])
def test_every_tile_in_a_captured_graph(c_type, kind, table):
    for (M, N, K), launches in table.items():
        a, x = blockfp8.quantize(torch.randn(M, K, device="cuda")), torch.randn(N, K, device="cuda")
        run = lambda: blockfp8.gemm(a, blockfp8.quantize(x, 128), out_dtype=kind)  # noqa: E731
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        for i in range(3):
            x.copy_(torch.randn(N, K, device="cuda") * (i + 1))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, run()), (M, N, K, launches)
