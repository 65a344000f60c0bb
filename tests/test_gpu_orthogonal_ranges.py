"""The orthogonalised update at the ends of its inputs' ranges, against its definition in 64 bits."""

import pytest
import torch

from dense_fp32_matrix_row_amd import orthogonal
from tests import lowp_reference as ref
from tests.test_gpu_orthogonal import far, matrix, tolerance

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
