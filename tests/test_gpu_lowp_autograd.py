"""The low-precision operators and autograd: results carry no graph, and what is
written in place is seen by it."""

import pytest
import torch

from dense_fp32_matrix_row_amd import blockfp8, orthogonal

pytestmark = pytest.mark.gpu


def test_results_carry_no_graph():
    x = torch.randn(8, 256, device="cuda", requires_grad=True)
    w = blockfp8.quantize(torch.randn(16, 256, device="cuda"), 128)
    y, xt = blockfp8.linear_forward(x, w)
    for t in (y, xt.q, blockfp8.quantize(x).s, orthogonal.orthogonalize(x)):
        assert not t.requires_grad and t.grad_fn is None


def written_by_gemm(t):
    a = blockfp8.quantize(torch.randn(8, 256, device="cuda"))
    b = blockfp8.quantize(torch.randn(16, 256, device="cuda"), 128)
    blockfp8.gemm(a, b, c=t, beta=1.0, out=t)


def written_by_the_layer(t):
    dy, x = torch.randn(32, 8, device="cuda"), torch.randn(32, 16, device="cuda")
    w = torch.randn(8, 16, device="cuda")
    xt = blockfp8.linear_forward(x, blockfp8.quantize(w, 128))[1]
    blockfp8.linear_backward(dy, xt, blockfp8.quantize_transposed(w, 128), dw=t)


def written_by_the_update(t):
    orthogonal.orthogonalize(t, out=t)


@pytest.mark.parametrize("write", (written_by_gemm, written_by_the_layer, written_by_the_update))
def test_a_saved_tensor_that_is_overwritten_is_noticed(write):
    leaf = torch.randn(8, 16, device="cuda", requires_grad=True)
    saved = leaf.exp()  # whose backward reads the result
    before = saved._version
    write(saved)
    assert saved._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        saved.sum().backward()


@pytest.mark.parametrize("write", (written_by_gemm, written_by_the_layer, written_by_the_update))
def test_inference_tensors_are_written_too(write):
    with torch.inference_mode():
        t = torch.ones(8, 16, device="cuda")
        write(t)
        assert not (t == 1).all()
    write(t)
