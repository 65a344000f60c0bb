"""Every tile of the orthogonalised update, joined parts and columns apart, against
the definition in 64 bits: all types, wide and tall."""

import pytest
import torch

from dense_fp32_matrix_row_amd import orthogonal
from tests import lowp_shapes as shapes
from tests.test_gpu_orthogonal import TYPES, tolerance

pytestmark = pytest.mark.gpu


def definition(g, coefficients, eps):
    """lowp_reference.orthogonalize on the GPU, the smaller side iterated."""
    x = g.double()
    x = x / (x.pow(2).sum(dim=(-2, -1), keepdim=True).sqrt() + eps)
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT.contiguous() if tall else x
    for a, b, c in coefficients:
        s = x @ x.mT.contiguous()
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.mT if tall else x


def hold(got, want, tol):
    """The whole of each matrix within tol of its norm, and each row and column within four times its
    own: an error in a few of them would not show in the whole's norm."""
    off = got.double() - want
    assert (off.flatten(-2).norm(dim=-1) <= tol * want.flatten(-2).norm(dim=-1)).all()
    for d in (-1, -2):
        assert (off.norm(dim=d) <= 4 * tol * want.norm(dim=d)).all()


@pytest.mark.parametrize("tall", (False, True))
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("size", shapes.ORTHOGONALIZE)
def test_every_tile(size, kind, tall):
    batch, rows, cols = size
    rows, cols = (cols, rows) if tall else (rows, cols)
    g = torch.randn(batch, rows, cols, generator=torch.Generator("cuda").manual_seed(5), device="cuda").to(TYPES[kind])
    co = [orthogonal.QUINTIC] * 2
    want = definition(g, co, 1e-7)
    out = torch.full((batch, rows, cols + 3), 7.0, dtype=TYPES[kind], device="cuda")
    workspace = torch.full((orthogonal.hip_orthogonalize_workspace(batch, rows, cols, 0) + 256,), 0xff, dtype=torch.uint8,
                           device="cuda")  # NaN wherever something is read before it is written
    orthogonal.orthogonalize(g, steps=2, out=out[:, :, :cols], workspace=workspace[:-256])
    hold(out[:, :, :cols], want, tolerance(co, TYPES[kind]))
    assert (out[:, :, cols:] == 7).all() and (workspace[-256:] == 0xff).all()
    assert torch.equal(orthogonal.orthogonalize(g, steps=2), out[:, :, :cols])


@pytest.mark.parametrize("size", [(1, 1024, 4097), (5, 400, 1537), (1, 900, 900), (1, 4096, 4096)])
def test_joined_parts_and_columns_apart_in_a_captured_graph(size):
    g = torch.randn(*size, device="cuda")
    orthogonal.orthogonalize(g, steps=2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = orthogonal.orthogonalize(g, steps=2)
    for i in range(3):
        g.copy_(torch.randn(*size, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, orthogonal.orthogonalize(g, steps=2))
