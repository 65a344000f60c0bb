"""Layer norms, clipping and integer weights in the training example: the operators
in a run together, as they are used."""

import pytest
import torch

from dense_fp32_matrix_row_amd import blockfp8, gradients, int8, layernorm, lowp_training
from tests import lowp_reference as low
from tests import serving_reference as ref

pytestmark = pytest.mark.gpu


def norms_with_parameters(net, seed):
    g = torch.Generator().manual_seed(seed)
    for n in net.norms:
        n.weight.copy_(1 + torch.randn(n.weight.shape, generator=g) / 4)
        n.bias.copy_(torch.randn(n.bias.shape, generator=g) / 4)


def test_a_step_with_norms_against_the_same_step_in_64_bits():
    """Each operator's result against its definition on what the operator before it gave: the activations
    are bf16 (2^-8 of a value each way), the weights' gradients float."""
    net = lowp_training.Network(200, 130, 70, seed=3, norm=True)
    norms_with_parameters(net, 5)
    g = torch.Generator().manual_seed(4)
    x, dy = torch.randn(100, 200, generator=g).bfloat16(), (torch.randn(100, 70, generator=g) * 1e-2).bfloat16()
    y, saved = net.forward(x.cuda())
    net.backward(dy.cuda(), saved)
    (one, two), (n1, n2) = net.layers, net.norms
    h = saved[1].cpu()
    deq = lambda v, rows=1: low.dequantize(*low.quantize(v, rows, False), rows)  # noqa: E731
    f1 = ref.layer_norm(x, n1.weight.cpu(), n1.bias.cpu(), 1e-5)
    f2 = ref.layer_norm(h, n2.weight.cpu(), n2.bias.cpu(), 1e-5)
    # what the layers saw of the norms, from the operators themselves
    v = lowp_training.layernorm.layer_norm(x.cuda(), n1.weight, n1.bias).cpu()
    u = lowp_training.layernorm.layer_norm(h.cuda(), n2.weight, n2.bias).cpu()
    ref.close(v, f1["y"], ref.forward_tolerance(f1, torch.bfloat16))
    ref.close(u, f2["y"], ref.forward_tolerance(f2, torch.bfloat16))
    w2 = deq(two.master.cpu(), 128)
    want = deq(u) @ w2.T
    assert ((y.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -12 * (deq(u).abs() @ w2.abs().T)).all()
    want = deq(dy.T) @ deq(u.T).T
    assert torch.allclose(two.gradient.cpu().double(), want, rtol=0, atol=2.0 ** -18 * (deq(dy.T).abs() @ deq(u.T).abs().T).max().item())
    du = blockfp8.gemm(blockfp8.quantize(dy.cuda()), two.wt).cpu()
    dh, dw, db = ref.layer_norm_backward(f2, du)
    tols = ref.backward_tolerance(f2, du, torch.bfloat16, 100)
    ref.close(n2.weight_gradient, dw, tols[1])
    ref.close(n2.bias_gradient, db, tols[2])
    got = lowp_training.layernorm.layer_norm_backward(du.cuda(), h.cuda(), saved[5], n2.weight)[0]
    ref.close(got, dh, tols[0])
    dh = got.cpu() * (h > 0)
    want = deq(dh.T) @ deq(v.T).T
    assert torch.allclose(one.gradient.cpu().double(), want, rtol=0, atol=2.0 ** -18 * (deq(dh.T).abs() @ deq(v.T).abs().T).max().item())
    dv = blockfp8.gemm(blockfp8.quantize(dh.cuda()), one.wt).cpu()
    _, dw, db = ref.layer_norm_backward(f1, dv)
    tols = ref.backward_tolerance(f1, dv, torch.bfloat16, 100)
    ref.close(n1.weight_gradient, dw, tols[1])
    ref.close(n1.bias_gradient, db, tols[2])
    # all gradients clipped together
    grads = net.gradients()
    assert len(grads) == 6
    before = [t.clone() for t in grads]
    norm, c = ref.clip([t.cpu() for t in grads], 1e-3, 1e-6)
    got, _ = gradients.clip_grad_norm(grads, 1e-3, out=grads)
    assert abs(got.item() - norm) <= 2.0 ** -24 * norm * 1.001
    for t, old in zip(grads, before):
        ref.close(t, old.cpu().double() * c, 2.0 ** -23 * old.cpu().double().abs() * c * 1.001 + 2.0 ** -149)


def test_a_training_run_with_all_of_it():
    net, losses = lowp_training.train(steps=5, tokens=64, inputs=96, hidden=130, outputs=33, norm=True, clip=0.05)
    assert len(losses) == 5 and all(loss == loss and loss < float("inf") for loss in losses)
    assert (net.norms[0].weight != 1).any() and (net.norms[1].bias != 0).any()
    again = lowp_training.train(steps=5, tokens=64, inputs=96, hidden=130, outputs=33, norm=True, clip=0.05)[1]
    assert losses == again  # sums in one order
    # a limit far above the norm changes nothing
    plain = lowp_training.train(steps=3, tokens=64, inputs=96, hidden=130, outputs=33)[1]
    assert plain == lowp_training.train(steps=3, tokens=64, inputs=96, hidden=130, outputs=33, clip=1e9)[1]


@pytest.mark.parametrize("norm", (False, True))
def test_served_tokens_against_the_definition(norm):
    """Each layer on what the one before it gave; tokens one by one as together, bit for bit."""
    net = lowp_training.Network(256, 384, 130, seed=5, norm=norm)
    if norm:
        norms_with_parameters(net, 6)
    served = net.serve()
    x = torch.randn(70, 256, device="cuda").bfloat16()
    together = served.infer(x)
    assert torch.equal(together, torch.cat([served.infer(x[i:i + 1]) for i in range(len(x))]))
    v = x
    for k, layer in enumerate(net.layers):
        v = v.relu() if k else v
        if norm:
            f = ref.layer_norm(v.cpu(), net.norms[k].weight.cpu(), net.norms[k].bias.cpu(), 1e-5)
            v = lowp_training.layernorm.layer_norm(v, net.norms[k].weight, net.norms[k].bias)
            ref.close(v, f["y"], ref.forward_tolerance(f, torch.bfloat16))
        want, size = ref.product(*ref.quantize(v.cpu()), *ref.quantize(layer.master.cpu()))
        v = int8.linear(v, served.weights[k])
        ref.close(v, want, ref.product_tolerance(torch.bfloat16, want, size))
    assert torch.equal(v, together)


def test_serving_in_a_captured_graph():
    net = lowp_training.Network(256, 384, 130, seed=7, norm=True)
    served = net.serve()
    x = torch.randn(4, 256, device="cuda").bfloat16()
    served.infer(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = served.infer(x)
    for i in range(3):
        x.copy_(torch.randn(4, 256, device="cuda") * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        want = served.infer(x)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_a_training_step_in_a_captured_graph():
    """Forward, backward, clipping: workspaces and all, replayed on new tokens."""
    net = lowp_training.Network(96, 130, 33, seed=8, norm=True)
    x, dy = torch.randn(64, 96, device="cuda").bfloat16(), torch.randn(64, 33, device="cuda").bfloat16()

    def step():
        for g in net.gradients():
            g.zero_()
        y, saved = net.forward(x)
        net.backward(dy, saved)
        grads = net.gradients()
        norm, _ = gradients.clip_grad_norm(grads, 0.5, out=grads)
        return y, norm
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, norm = step()
    for i in range(3):
        x.copy_(torch.randn(64, 96, device="cuda") * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        got = [y.clone(), norm.clone(), *(g.clone() for g in net.gradients())]
        want = [*step(), *net.gradients()]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_command_runs(capsys):
    lowp_training.main(["--steps", "3", "--norm", "--clip", "0.1", "--serve", "int8"])
    out = capsys.readouterr().out
    assert "loss" in out and "differ by 0.00e+00" in out


def test_host_threads_call_at_once():
    """Each thread on its own stream, with its own tensors: the results of the calls one after another."""
    import threading

    def work(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x, dy = (torch.randn(300 + seed, 520, generator=g, device="cuda").bfloat16() for _ in range(2))
        w = int8.quantize(torch.randn(264, 520, generator=g, device="cuda"))
        scale, shift = (torch.randn(520, generator=g, device="cuda") for _ in range(2))
        grads = [torch.randn(n, generator=g, device="cuda") for n in (seed + 1, 5000, 70000)] * (1 if seed % 2 else 30)

        def calls():
            y, stats = layernorm.layer_norm_forward(x, scale, shift)
            norm, clipped = gradients.clip_grad_norm(grads, 1.0)
            return [y, stats, *layernorm.layer_norm_backward(dy, x, stats, scale), int8.linear(y, w), int8.linear(y[:3], w),
                    gradients.grad_norm(grads), norm, *clipped]
        return calls

    calls = [work(seed) for seed in range(4)]
    expected = [c() for c in calls]
    torch.cuda.synchronize()
    results, failures = [None] * 4, []

    def thread(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                results[i] = [calls[i]() for _ in range(8)]
            stream.synchronize()
        except Exception as e:  # raised where the test sees it
            failures.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures
    for want, runs in zip(expected, results):
        for got in runs:
            assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("norm", (False, True))
def test_a_served_network_stays_as_it_was_served(norm):
    """Training that goes on changes neither the weights nor the norms' parameters of what is served."""
    net = lowp_training.Network(96, 130, 33, seed=9, norm=norm)
    if norm:
        norms_with_parameters(net, 10)
    served = net.serve()
    x = torch.randn(7, 96, device="cuda").bfloat16()
    want = served.infer(x)
    for part in (*net.layers, *net.norms):
        for gradient in ([part.gradient] if hasattr(part, "gradient") else [part.weight_gradient, part.bias_gradient]):
            gradient.copy_(torch.randn(gradient.shape))
        part.update(0.1)
    assert torch.equal(served.infer(x), want)
    assert not torch.equal(net.serve().infer(x), want)
