"""The gradients' norm and clipping on the GPU against their definitions in 64 bits."""

import pytest
import torch

from dense_fp32_matrix_row_amd import gradients, sgemm
from tests import serving_reference as ref
from tests.serving_reference import HALF, TYPES

pytestmark = pytest.mark.gpu
EPS = 1e-6


def check(tensors, max_norm, eps=EPS):
    """The norm and the clipped tensors, new and in place, against the definition."""
    host = [t.cpu() for t in tensors]
    norm, c = ref.clip(host, max_norm, eps)
    got, out = gradients.clip_grad_norm(tensors, max_norm, eps=eps)
    assert got.dtype == torch.float32 and got.shape == () and abs(got.item() - norm) <= HALF * norm * 1.001 + 2.0 ** -149
    assert torch.equal(got, gradients.grad_norm(tensors))
    for t, o, h in zip(tensors, out, host):
        assert o.dtype == t.dtype and torch.equal(t.cpu(), h)
        if c == 1.0:
            assert torch.equal(o, t)
        else:
            want = h.double() * c
            tol = 2 * HALF * want.abs() * 1.001 + 2.0 ** -149
            ref.close(o, want, tol + (ref.rounding(t.dtype, want.abs() + tol) if t.dtype != torch.float32 else 0))
    by = gradients.clip_by_norm(tensors, got, max_norm, eps=eps)
    # the norm that is given has been rounded to float: c by a half step more
    for o, p in zip(out, by):
        eps_of = torch.finfo(o.dtype).eps
        assert ((o.double() - p.double()).abs() <= (4 * HALF + eps_of) * o.double().abs() + torch.finfo(o.dtype).smallest_normal * eps_of).all()
    place = [torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t) if t.dim() else t.clone() for t in tensors]
    before = [t._version for t in place]
    again, same = gradients.clip_grad_norm(place, max_norm, eps=eps, out=place)
    assert torch.equal(again, got) and same is place
    assert all(torch.equal(o, p) for o, p in zip(out, place)) and all(t._version == v + 1 for t, v in zip(place, before))
    return got, out


def some(shapes, kinds, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * scale * 4.0 ** (i % 5 - 2)).to(TYPES[kinds[i % len(kinds)]]).cuda() for i, s in enumerate(shapes)]


SHAPES = [(1,), (7,), (256, 256), (3, 5, 7), (4095,), (4096,), (4097,), (1, 1), (1023, 65), (16384,), (16385,), (100001,), ()]


@pytest.mark.parametrize("part", (0.25, 4.0))
@pytest.mark.parametrize("kinds", (("f32",), ("bf16",), ("f16",), ("f32", "bf16", "f16")))
def test_against_the_definition(kinds, part):
    tensors = some(SHAPES, kinds)
    norm, _ = ref.clip([t.cpu() for t in tensors], 1.0, EPS)
    check(tensors, norm * part)
    for n in (1, 2, 5):
        for t in (tensors[n - 1:n], tensors[:n]):
            check(t, ref.clip([v.cpu() for v in t], 1.0, EPS)[0] * part)


@pytest.mark.parametrize("count", (55, 56, 57, 63, 64, 65, 113, 200, 4097, 5000))
def test_many_tensors(count):
    """Beside what fits a launch's arguments, and one, two and three rounds of looking for a chunk's tensor."""
    tensors = some([(1 + (i * 37) % 300,) for i in range(count)], ("f32", "bf16"), seed=count)
    check(tensors, 1.0)


@pytest.mark.parametrize("count", (119, 120, 121, 239, 240, 241, 361))
def test_as_many_tensors_as_a_launch_takes(count):
    """A launch's arguments hold 120 of the table's slots, one a dense tensor: beside one, two and three launches' worth."""
    check(some([(1 + (i * 37) % 300,) for i in range(count)], ("f32", "bf16"), seed=count), 1.0)


@pytest.mark.parametrize("strided", (1, 2, 3))
@pytest.mark.parametrize("count", (59, 60, 61, 79, 119, 120, 121, 300, 2100))
def test_many_strided_tensors(count, strided):
    """One of every `strided` tensors is of rows apart, which take two slots: also pairs of them that lie on both
    sides of the 120th, and where a chunk's tensor is looked for in two rounds."""
    g = torch.Generator().manual_seed(count)
    tensors = []
    for i in range(count):
        rows, cols = 2 + i % 7, 1 + (i * 13) % 60
        kind = (torch.float32, torch.bfloat16)[i % 2]
        t = (torch.randn(rows, cols + 3, generator=g) * 4.0 ** (i % 5 - 2)).to(kind).cuda()
        tensors.append(t[:, 1:1 + cols] if i % strided == 0 else t)
    check(tensors, 1.0)


@pytest.mark.parametrize("first", (0, 1))
def test_strided_tensors_of_many_chunks_each(first):
    """Chunks at the begin and the end of each, found in the table of a launch's arguments and in that in memory."""
    for count in (3, 90):
        wide = torch.randn(count, 40, 4200, device="cuda")
        tensors = [w[:, 1:4200 - i % 3] for i, w in enumerate(wide)]
        check(tensors[first:], 2.0)


def test_more_tensors_than_two_rounds_find():
    """64^3 tensors and more: views of one buffer."""
    n = 64 ** 3 + 5
    buffer = torch.randn(2 * n, device="cuda")
    tensors = list(buffer.view(n, 2).unbind(0))
    want = buffer.clone()
    norm, _ = gradients.clip_grad_norm(tensors, 1.0, out=tensors)
    total = want.double().square().sum().sqrt().item()
    assert abs(norm.item() - total) <= HALF * total * 1.001
    c = 1.0 / (total + EPS)
    assert ((buffer.double() - want.double() * c).abs() <= 2 * HALF * want.double().abs() * c * 1.001 + 2.0 ** -149).all()


def test_every_offset_of_the_first_element():
    """Tensors that begin and end anywhere in 16 bytes."""
    for kind in TYPES.values():
        buffer = torch.randn(40000, device="cuda").to(kind)
        for n in (1, 5, 30, 1000, 9000):
            for at in range(9):
                t = [buffer[at:at + n], buffer[20001 + at:20001 + at + n + 3]]
                before = buffer.clone()
                norm, _ = ref.clip([v.cpu() for v in t], 1.0, EPS)
                got, _ = gradients.clip_grad_norm(t, norm / 2, out=t)
                assert abs(got.item() - norm) <= HALF * norm * 1.001
                c = (norm / 2) / (norm + EPS)
                for v, old in ((t[0], before[at:at + n]), (t[1], before[20001 + at:20001 + at + n + 3])):
                    want = old.cpu().double() * c
                    ref.close(v, want, 2 * HALF * want.abs() * 1.001 + ref.rounding(kind, want.abs() * 1.001))
                    v.copy_(old)
                assert torch.equal(buffer, before)


def test_strides_and_layouts():
    base = torch.randn(300, 400, device="cuda")
    wide = torch.randn(50, 9000, device="cuda").bfloat16()
    tensors = [base[:, :57].T, base[:, 60:100], wide[:, 3:8200], torch.randn(5, 6, 7, device="cuda").permute(2, 0, 1),
               torch.randn(4000, 2, device="cuda")[:, 0], torch.randn(30, 20, 8, device="cuda")[:, :, 2:7], base[:, 100:101]]
    check(tensors, 3.0)
    outs = [torch.full((t.shape[0], *t.shape[1:-1], t.shape[-1] + 3), -1.0, device="cuda", dtype=t.dtype)[..., 1:-2] if t.dim() > 1 else
            torch.empty(2 * len(t), device="cuda", dtype=t.dtype)[::2] for t in tensors[1:3] + tensors[4:5]]
    picked = tensors[1:3] + tensors[4:5]
    norm, got = gradients.clip_grad_norm(picked, 3.0, out=outs)
    _, new = gradients.clip_grad_norm(picked, 3.0)
    assert all(a is b for a, b in zip(got, outs)) and all(torch.equal(a, b) for a, b in zip(outs, new))
    assert (outs[0]._base[..., 0] == -1).all() and (outs[0]._base[..., -2:] == -1).all()


def test_two_columns_of_one_matrix_in_place():
    base = torch.randn(100, 64, device="cuda")
    want = base / (base.double().norm() + EPS).float()
    gradients.clip_grad_norm([base[:, :20], base[:, 20:64]], 1.0, out=[base[:, :20], base[:, 20:64]])
    assert torch.allclose(base, want, rtol=1e-6, atol=0)


def test_norms_past_a_floats_range():
    big = torch.full((100,), 3e38, device="cuda")
    norm, out = gradients.clip_grad_norm([big], 1.0)
    assert norm.item() == float("inf") and torch.allclose(out[0], torch.full_like(big, 0.1), rtol=1e-6)
    norm, out = gradients.clip_grad_norm([big[:1]], 1.0)
    assert norm.item() == big[0].item()
    tiny = torch.full((64,), 2.0 ** -140, device="cuda")
    norm, out = gradients.clip_grad_norm([tiny], 2.0 ** -138, eps=0.0)
    assert norm.item() == 2.0 ** -137 and torch.equal(out[0], tiny / 2)


def test_infinities_nans_zeros_and_limits():
    x = torch.randn(1000, device="cuda")
    y = torch.randn(500, device="cuda").bfloat16()
    x[5] = float("inf")
    norm, (a, b) = gradients.clip_grad_norm([x, y], 1.0)
    assert norm.item() == float("inf") and torch.isnan(a[5]) and (a[:5] == 0).all() and (b == 0).all()
    norm, (a, b) = gradients.clip_grad_norm([x, y], float("inf"))
    assert torch.equal(a, x) and torch.equal(b, y)
    x[6] = float("nan")
    for limit in (1.0, float("inf")):
        norm, (a, b) = gradients.clip_grad_norm([x, y], limit)
        assert torch.isnan(norm) and torch.isnan(a).all() and torch.isnan(b).all()
    zero = torch.zeros(100, device="cuda")
    for eps in (0.0, 1e-6):
        for limit in (0.0, 1.0):
            norm, (a,) = gradients.clip_grad_norm([zero], limit, eps=eps)
            assert norm.item() == 0 and (a == 0).all()
    norm, (a,) = gradients.clip_grad_norm([torch.ones(16, device="cuda")], 0.0)
    assert norm.item() == 4 and (a == 0).all()
    norm, (a,) = gradients.clip_grad_norm([torch.ones(16, device="cuda")], 4.0, eps=0.0)  # on the limit
    assert norm.item() == 4 and (a == 1).all()


def test_tensors_without_elements():
    none = torch.empty(0, 5, device="cuda")
    x = torch.ones(4, device="cuda")
    norm, out = gradients.clip_grad_norm([none, x, none], 1.0)
    assert norm.item() == 2 and out[0].shape == (0, 5) and (out[1] < 0.5).all()
    norm, out = gradients.clip_grad_norm([none], 1.0)
    assert norm.item() == 0 and gradients.grad_norm([none, none]).item() == 0
    assert gradients.clip_by_norm([none], norm, 1.0)[0].shape == (0, 5)


def test_the_same_tensor_twice():
    x = torch.ones(8, device="cuda")
    assert gradients.grad_norm([x, x]).item() == 4.0
    norm, out = gradients.clip_grad_norm([x, x], 2.0, eps=0.0)  # new results of each
    assert norm.item() == 4 and all((o == 0.5).all() for o in out)
    for bad in ([x, x], [x[:5], x[4:]]):
        with pytest.raises(sgemm.SgemmError):
            gradients.clip_grad_norm(bad, 2.0, out=bad)
    with pytest.raises(sgemm.SgemmError):
        gradients.clip_grad_norm([x[:4], x[4:]], 2.0, out=[x[4:], x[:4]])  # one's result in the other's gradient
    assert (x == 1).all()


def test_past_two_gigabytes():
    x = torch.randn((1 << 31) + 100_001, device="cuda", dtype=torch.bfloat16)
    y = torch.randn(33000, 65600, device="cuda", dtype=torch.bfloat16)[:, 1:65598]
    want = sum(t.double().square().sum().item() for t in (*x.split(1 << 28), *y.split(4096))) ** 0.5
    norm, (a, b) = gradients.clip_grad_norm([x, y], want / 4)
    assert abs(norm.item() - want) <= HALF * want * 1.001
    c = (want / 4) / (want + EPS)
    for got, old in ((a[-1000:], x[-1000:]), (a[:1000], x[:1000]), (a[(1 << 31) - 50:(1 << 31) + 50], x[(1 << 31) - 50:(1 << 31) + 50]),
                     (b[-1], y[-1]), (b[32800], y[32800])):
        want = old.cpu().double() * c
        ref.close(got, want, 2 * HALF * want.abs() * 1.001 + ref.rounding(torch.bfloat16, want.abs() * 1.001))


@pytest.mark.parametrize("count", (3, 200))
def test_the_same_again_other_streams_and_captured_graphs(count):
    tensors = some([(1 + (i * 3701) % 30000,) for i in range(count)], ("f32", "bf16"), seed=1)
    want = gradients.clip_grad_norm(tensors, 1.0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = gradients.clip_grad_norm(tensors, 1.0)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and all(torch.equal(a, b) for a, b in zip(got[1], want[1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gradients.clip_grad_norm(tensors, 1.0)
    for i in range(3):
        for t in tensors:
            t.copy_(torch.randn(t.shape, device="cuda") * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        want = gradients.clip_grad_norm(tensors, 1.0)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and all(torch.equal(a, b) for a, b in zip(got[1], want[1]))


def test_gradients_of_leaves():
    """As an optimiser's loop calls it: the .grad of parameters, in place."""
    params = [torch.randn(20, 30, device="cuda", requires_grad=True), torch.randn(30, device="cuda", requires_grad=True)]
    sum((p * p * 3).sum() for p in params).backward()
    grads = [p.grad for p in params]
    norm, _ = gradients.clip_grad_norm(grads, 1.0, out=grads)
    total = sum((6 * p.detach().double()).square().sum().item() for p in params) ** 0.5
    assert abs(norm.item() - total) <= 2 * HALF * total * 1.01
    assert all(torch.allclose(p.grad, 6 * p.detach() / (total + EPS), rtol=1e-6, atol=0) for p in params)


def test_refusals_of_the_tensor_forms():
    x = torch.ones(4, 8, device="cuda")
    for bad in (lambda: gradients.grad_norm([x.double()]), lambda: gradients.clip_grad_norm([x, x.int()], 1.0)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: gradients.clip_grad_norm([x], 1.0, out=[x[:2]]), lambda: gradients.clip_grad_norm([x], 1.0, out=[x.half()]),
                lambda: gradients.clip_grad_norm([x], 1.0, out=[torch.ones(8, 4, device="cuda").T]), lambda: gradients.grad_norm([x, x.cpu()]),
                lambda: gradients.grad_norm([x[0].expand(4, 8)]), lambda: gradients.clip_by_norm([x], torch.ones(()), 1.0)):
        with pytest.raises(ValueError):
            bad()


def test_disjoint_pieces_of_one_matrix_in_place():
    """Strided pieces of other heights, strides and widths than their neighbours, none of them overlapping."""
    base = torch.randn(40, 64, device="cuda")
    want = base / (base.double().norm() + EPS).float()
    pieces = [base[:, :4], base[0, 4:64], base[1:, 4:30], base[1::2, 30:50], base[2::2, 30:50], base[1:21, 50:64], base[21:, 50:64]]
    assert sum(p.numel() for p in pieces) == base.numel()
    _, out = gradients.clip_grad_norm(pieces, 1.0, out=pieces)
    assert out is pieces and torch.allclose(base, want, rtol=1e-6, atol=0)
    with pytest.raises(sgemm.SgemmError):
        gradients.clip_grad_norm([base[1::2, 30:50], base[3:5, 49:60]], 1.0, out=[base[1::2, 30:50], base[3:5, 49:60]])


def test_clipping_by_a_norm_that_is_a_gradient_too():
    x = torch.tensor([3.0, 4.0], device="cuda")
    norm = gradients.grad_norm([x])
    out = gradients.clip_by_norm([x, norm], norm, 1.0, eps=0.0)
    assert torch.allclose(out[0], x / 5) and out[1].item() == 1.0 and norm.item() == 5.0
    with pytest.raises(sgemm.SgemmError):
        gradients.clip_by_norm([x, norm], norm, 1.0, out=[x, norm])
