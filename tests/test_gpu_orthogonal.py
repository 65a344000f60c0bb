"""The orthogonalised update on the GPU against its definition in 64 bits."""

import pytest
import torch

from dense_fp32_matrix_row_amd import orthogonal
from tests import lowp_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def matrix(shape, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(kind)


def tolerance(coefficients, kind):
    """Relative, in the 2-norm of the whole.  A step's three products each take
    operands rounded to 22 bits and leave out a term of 2^-22 (together under
    3 x 2^-22 of their size), sum in float, and round the new iterate to 22
    bits: with the factor |b| + |c| that the products carry, under
    2^-20 (1 + |a| + |b| + |c|) of the iterate.  Later steps multiply an error
    by |a| at most where the iterate grows by as much, and by |a| relative to
    it where it does not.  Then the output's half step."""
    err = 2.0 ** -22
    for a, b, c in coefficients:
        err = err * max(1.0, abs(a)) + 2.0 ** -20 * (1 + abs(a) + abs(b) + abs(c)) / max(1.0, abs(a))
    return err + torch.finfo(kind).eps / 2


def far(got, want):
    """The worst matrix's relative distance."""
    d = (got.cpu().double() - want).flatten(-2).norm(dim=-1)
    return (d / want.flatten(-2).norm(dim=-1)).max().item()


SHAPES = [(1, 1), (1, 50), (50, 1), (2, 3), (31, 33), (32, 32), (33, 64), (64, 65), (65, 64), (100, 257), (300, 129), (256, 256),
          (129, 520), (513, 200)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_against_the_definition(shape, kind):
    g = matrix(shape, TYPES[kind], seed=sum(shape))
    co = [orthogonal.QUINTIC] * 5
    got = orthogonal.orthogonalize(g.cuda())
    assert got.dtype == g.dtype and got.shape == g.shape
    assert far(got, ref.orthogonalize(g, co, 1e-7)) <= tolerance(co, TYPES[kind])


@pytest.mark.parametrize("shape", [(1100, 1300), (1500, 1021), (2, 900, 1500), (2100, 2200), (2800, 2750), (640, 4000), (1024, 2049), (3, 50, 1100)])
def test_large_tiles(shape):
    """Enough for each of the large tiles, ragged on both sides."""
    g = matrix(shape, torch.float32, seed=3)
    co = [orthogonal.QUINTIC] * 2
    got = orthogonal.orthogonalize(g.cuda(), steps=2)
    assert far(got, ref.orthogonalize(g, co, 1e-7)) <= tolerance(co, torch.float32)
    # a block of a few rows by itself: an error there would not show in the whole's norm
    want = ref.orthogonalize(g, co, 1e-7)
    d = (got.cpu().double() - want).flatten(0, -2)
    assert (d.norm(dim=-1) <= 4 * tolerance(co, torch.float32) * want.flatten(0, -2).norm(dim=-1)).all()


@pytest.mark.parametrize("steps", (0, 1, 2, 3, 8))
@pytest.mark.parametrize("shape", [(40, 70), (3, 70, 40)])
def test_steps_and_batches(steps, shape):
    g = matrix(shape, torch.float32, seed=steps)
    co = [(1.5 + 0.1 * i, -0.5 - 0.05 * i, 0.02 * i) for i in range(steps)]
    got = orthogonal.orthogonalize(g.cuda(), steps=steps, coefficients=co, eps=1e-3)
    assert far(got, ref.orthogonalize(g, co, 1e-3)) <= tolerance(co, torch.float32)


def test_the_matrices_of_a_batch_are_independent():
    g = matrix((5, 70, 90), torch.float32)
    g[2] = 0
    g[3, 4, 5] = float("nan")
    g[4] *= 1e-20
    got = orthogonal.orthogonalize(g.cuda(), eps=1e-30)
    for i in (0, 1, 4):
        assert torch.equal(got[i], orthogonal.orthogonalize(g[i].cuda(), eps=1e-30))
    assert (got[2] == 0).all() and torch.isnan(got[3]).all() and torch.isfinite(got[[0, 1, 4]]).all()


def test_singular_values_come_to_one():
    """The cubic 1.5 x - 0.5 x^3 drives every singular value to 1 from below: the result is
    semi-orthogonal, X X^T = 1 within what the rounding of a step leaves (2^-18)."""
    u, _, v = torch.linalg.svd(matrix((60, 90), torch.float64), full_matrices=False)
    g = (u * torch.linspace(0.5, 1.0, 60, dtype=torch.float64)) @ v
    x = orthogonal.orthogonalize(g.float().cuda(), steps=20, coefficients=(1.5, -0.5, 0.0)).cpu().double()
    assert (x @ x.T - torch.eye(60, dtype=torch.float64)).abs().max() <= 2.0 ** -18
    assert (x - u @ v).abs().max() <= 2.0 ** -16


def test_large_and_small_magnitudes_do_not_matter():
    g = matrix((70, 50), torch.float32)
    want = orthogonal.orthogonalize(g.cuda(), eps=0.0)
    for scale in (2.0 ** 100, 2.0 ** -100):  # the squares leave float's range, not double's
        got = orthogonal.orthogonalize((g * scale).cuda(), eps=0.0)
        assert far(got, want.cpu().double()) <= 2.0 ** -20


@pytest.mark.parametrize("kind", TYPES)
def test_strides_in_place_and_own_workspace(kind):
    kind = TYPES[kind]
    whole = matrix((3, 45, 99), kind).cuda()
    g = whole[:, 2:42, 5:96]
    want = orthogonal.orthogonalize(g.contiguous())
    ws = torch.full((orthogonal.hip_orthogonalize_workspace(3, 40, 91, 0),), 0xff, dtype=torch.uint8, device="cuda")
    out = torch.full((3, 41, 93), 7.0, dtype=kind, device="cuda")
    assert torch.equal(orthogonal.orthogonalize(g, out=out[:, :40, :91], workspace=ws), want)
    assert (out[:, 40:] == 7).all() and (out[:, :, 91:] == 7).all()
    before = whole.clone()
    assert torch.equal(orthogonal.orthogonalize(g, out=g), want)
    before[:, 2:42, 5:96] = want
    assert torch.equal(whole, before)


def test_refusals_and_empty():
    g = torch.randn(4, 6, device="cuda")
    with pytest.raises(ValueError):
        orthogonal.orthogonalize(g.T)
    with pytest.raises(ValueError):
        orthogonal.orthogonalize(g, coefficients=[(1.0, 0.0, 0.0)])
    with pytest.raises(TypeError):
        orthogonal.orthogonalize(g.double())
    with pytest.raises(ValueError):
        orthogonal.orthogonalize(g, out=torch.empty(6, 4, device="cuda"))
    with pytest.raises(RuntimeError):
        orthogonal.orthogonalize(g, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(RuntimeError):
        orthogonal.orthogonalize(g, eps=-1.0)
    assert orthogonal.orthogonalize(torch.empty(0, 6, device="cuda")).shape == (0, 6)
    assert (orthogonal.orthogonalize(torch.zeros(5, 6, device="cuda")) == 0).all()


def test_large_sizes_in_a_captured_graph():
    """The symmetric products in parts, and the last columns apart."""
    g = torch.randn(1024, 1153, device="cuda")
    orthogonal.orthogonalize(g, steps=2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = orthogonal.orthogonalize(g, steps=2)
    for i in range(3):
        g.copy_(torch.randn(1024, 1153, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = orthogonal.orthogonalize(g, steps=2)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_other_streams_and_captured_graphs():
    g = torch.randn(2, 70, 130, device="cuda")
    want = orthogonal.orthogonalize(g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = orthogonal.orthogonalize(g)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = orthogonal.orthogonalize(g)
    for i in range(4):
        g.copy_(torch.randn(2, 70, 130, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = orthogonal.orthogonalize(g)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
