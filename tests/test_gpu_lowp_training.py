"""The low-precision operators together: a network that trains, and its single-token form."""

import pytest
import torch

from dense_fp32_matrix_row_amd import blockfp8, lowp_training
from tests import lowp_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", ("f32", "e8m0"))
def test_the_loss_falls(scale):
    _, losses = lowp_training.train(steps=60, scale=torch.float32 if scale == "f32" else torch.float8_e8m0fnu)
    assert losses[-1] < losses[0] / 4, losses


def test_one_step_against_the_same_step_in_64_bits():
    """Gradients of both layers, from the operators' definitions on the CPU: the operands are
    quantised the same way, so what is left is the rounding of bf16 activations (2^-8 each way
    through relu's border at most once an element) and of the products."""
    net = lowp_training.Network(200, 130, 70, seed=3)
    g = torch.Generator().manual_seed(4)
    x, dy = torch.randn(100, 200, generator=g).bfloat16(), (torch.randn(100, 70, generator=g) * 1e-2).bfloat16()
    y, saved = net.forward(x.cuda())
    net.backward(dy.cuda(), saved)
    one, two = net.layers
    h = saved[1].cpu()  # the bf16 hidden values that the second layer saw
    deq = lambda v, rows=1: ref.dequantize(*ref.quantize(v, rows, False), rows)  # noqa: E731
    w2 = deq(two.master.cpu(), 128)
    want_y = deq(h) @ w2.T
    assert ((y.cpu().double() - want_y).abs() <= 2.0 ** -8 * want_y.abs() + 2.0 ** -12 * (deq(h).abs() @ w2.abs().T)).all()
    want = deq(dy.T) @ deq(h.T).T
    assert torch.allclose(two.gradient.cpu().double(), want, rtol=0, atol=2.0 ** -18 * (deq(dy.T).abs() @ deq(h.T).abs().T).max().item())
    dh = blockfp8.gemm(blockfp8.quantize(dy.cuda()), two.wt).cpu() * (h > 0)
    want = deq(dh.T) @ deq(x.T).T
    assert torch.allclose(one.gradient.cpu().double(), want, rtol=0, atol=2.0 ** -18 * (deq(dh.T).abs() @ deq(x.T).abs().T).max().item())


def test_tokens_one_by_one_as_together():
    """A token's row is quantised by itself, so the batch it comes in changes only the order of
    a few sums: each bf16 rounding can fall the other way, once in each of two layers."""
    net = lowp_training.Network(256, 384, 130, seed=5)
    x = torch.randn(70, 256, device="cuda").bfloat16()
    together = net.infer(x)
    apart = torch.cat([net.infer(x[i:i + 1]) for i in range(len(x))])
    far = (together.float() - apart.float()).norm() / together.float().norm()
    assert far <= 2.0 ** -7
