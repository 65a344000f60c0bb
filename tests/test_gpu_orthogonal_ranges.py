"""The orthogonalised update at the ends of its inputs' ranges, against its definition in 64 bits."""

import pytest
import torch

from dense_fp32_matrix_row_amd import orthogonal
from tests import lowp_reference as ref
from tests.test_gpu_orthogonal import far, matrix, tolerance
from tests.test_gpu_orthogonal_tiles import definition

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("steps", (0, 5))
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", [(70, 50), (300, 520), (2, 40, 90)])
def test_norms_past_a_floats_largest(shape, kind, steps):
    """Finite elements whose |G|_F is 2^130 and more."""
    g = (matrix(shape, torch.float64).clamp(-3, 3) * 2.0 ** 126).to(TYPES[kind])
    assert torch.isfinite(g).all() and g.double().flatten(-2).norm(dim=-1).min() > torch.finfo(torch.float32).max
    co = [orthogonal.QUINTIC] * steps
    got = orthogonal.orthogonalize(g.cuda(), steps=steps)
    assert far(got, ref.orthogonalize(g, co, 1e-7)) <= tolerance(co, TYPES[kind])


@pytest.mark.parametrize("steps", (0, 5))
def test_norms_below_a_floats_normal_numbers(steps):
    """Subnormal elements of a few bits, which are exact as they come, and no eps."""
    g = (matrix((70, 50), torch.float64) * 2.0 ** -142).float()
    assert 0 < g.double().norm() < torch.finfo(torch.float32).smallest_normal
    co = [orthogonal.QUINTIC] * steps
    got = orthogonal.orthogonalize(g.cuda(), steps=steps, eps=0.0)
    assert far(got, ref.orthogonalize(g, co, 0.0)) <= tolerance(co, torch.float32)


def test_eps_counts_beside_a_norm_of_its_own_size():
    g = matrix((40, 60), torch.float32) * 2.0 ** -30
    eps = g.double().norm().item()
    co = [orthogonal.QUINTIC] * 3
    got = orthogonal.orthogonalize(g.cuda(), steps=3, eps=eps)
    want = ref.orthogonalize(g, co, torch.tensor(eps).float().item())
    assert far(got, want) <= tolerance(co, torch.float32)


@pytest.mark.parametrize("steps", (0, 1, 5))
@pytest.mark.parametrize("bad", (float("inf"), float("-inf"), float("nan")))
def test_what_an_infinity_or_a_nan_leaves(bad, steps):
    g = matrix((40, 60), torch.float32)
    g[7, 11] = bad
    got = orthogonal.orthogonalize(g.cuda(), steps=steps).cpu()
    if steps == 0 and bad != bad or steps:
        assert torch.isnan(got).all()
    else:
        assert torch.isnan(got[7, 11]) and (got.flatten()[torch.arange(2400) != 7 * 60 + 11] == 0).all()


@pytest.mark.parametrize("steps", (1, 2, 5))
@pytest.mark.parametrize("less", (1e-2, 1e-4, 1e-6, 1e-7))
@pytest.mark.parametrize("which", ("rows", "columns", "both"))
@pytest.mark.parametrize("shape", [(60, 90), (90, 60), (2, 130, 257), (512, 1024), (1100, 300), (900, 900)])
def test_rows_and_columns_much_smaller_than_the_rest_keep_their_bits(shape, which, less, steps):
    """One row and / or column in sixteen smaller by `less`: each row and column within the tolerance of a whole
    matrix, relative to its own norm."""
    g = matrix(shape, torch.float64, seed=7)
    if which != "columns":
        g[..., ::16, :] *= less
    if which != "rows":
        g[..., ::16] *= less
    g = g.float()
    co = [orthogonal.QUINTIC] * steps
    want = definition(g.cuda(), co, 1e-7)
    off = orthogonal.orthogonalize(g.cuda(), steps=steps).double() - want
    for d in (-1, -2):
        far_off = off.norm(dim=d) / want.norm(dim=d)
        assert far_off.max() <= tolerance(co, torch.float32), far_off.max().item()


def test_polynomials_that_leave_the_unit_interval():
    """Singular values grow to 40 on the way: the pairs' ranges follow the polynomials' bounds."""
    g = matrix((70, 90), torch.float32)
    co = [(40.0, 0.0, 0.0), (30.0, -20.0, 1.0), (1e-4, 0.0, 0.0)]
    got = orthogonal.orthogonalize(g.cuda(), steps=3, coefficients=co)
    want = ref.orthogonalize(g, co, 1e-7)
    assert torch.isfinite(got).all()
    s = 40 * torch.linalg.svdvals(g.double() / g.double().norm()).max()
    # the second step's terms of up to 30 s + 20 s^3 + s^5, each with a product's 2^-20, cancel in part
    assert far(got, want) * want.norm() <= 2.0 ** -20 * 3 * (30 * s + 20 * s ** 3 + s ** 5) * 1e-4 * 70 ** 0.5


@pytest.mark.parametrize("shape", [(5, 1 << 20), (1 << 20, 5), (40, 200_003), (200_003, 40), (3, 33, 70_001), (3, 70_001, 33)])
def test_long_sides(shape):
    """Sides of which a block of the norm's pass takes many parts; some rows and columns small."""
    g = torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(8), device="cuda")
    g[..., ::3, :] *= 1e-5
    g[..., ::7] *= 1e-4
    co = [orthogonal.QUINTIC] * 2
    want = definition(g, co, 1e-7)
    off = orthogonal.orthogonalize(g, steps=2).double() - want
    for d in (-1, -2):
        assert (off.norm(dim=d) <= tolerance(co, torch.float32) * want.norm(dim=d)).all()
