"""The integer product's, the layer norm's and the gradient clipping's C ABI without
a GPU: exports, refusals before any HIP call, workspace sizes, plans."""

import ctypes
import os
import re

import pytest
import torch

from dense_fp32_matrix_row_amd import gradients, int8, layernorm, sgemm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x1000  # non-NULL, aligned, never dereferenced: errors return first


def declared(header):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(hip_\w+)\s*\(", text)))


@pytest.mark.parametrize("header,module", [("int8.h", int8), ("layernorm.h", layernorm), ("gradients.h", gradients)])
def test_headers_declare_the_bindings_exports(header, module):
    assert declared(header) == sorted(module.EXPORTS)
    lib = module.load()
    for name in module.EXPORTS:
        assert hasattr(lib, name)


def refused(function, what, usual, change, status):
    assert function(*{**usual, **change}.values(), stream=0) == status
    assert "unknown" not in what(status)


QUANTIZE = dict(rows=4, cols=200, X=FAKE, x_type=0, ldx=200, Q=FAKE, ldq=208, S=FAKE)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), -1), (dict(cols=-1), -2), (dict(X=None), -3), (dict(x_type=3), -4), (dict(x_type=-1), -4),
    (dict(ldx=199), -5), (dict(Q=None), -6), (dict(ldq=199), -7), (dict(S=None), -8), (dict(rows=0), 0),
    (dict(cols=0, X=None, Q=None, S=None), 0),
])
def test_quantize_refusals(change, status):
    refused(int8.hip_int8_quantize, int8.hip_int8_quantize_status_string, QUANTIZE, change, status)


GEMM = dict(M=4, N=8, K=200, A=FAKE, lda=208, SA=FAKE, sa_inc=1, B=FAKE, ldb=208, SB=FAKE, sb_inc=1, bias=FAKE,
            bias_type=0, D=FAKE, ldd=8, d_type=0)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), -1), (dict(N=-1), -2), (dict(K=-1), -3), (dict(K=int8.MAX_K + 1, lda=131072, ldb=131072), -3),
    (dict(A=None), -4), (dict(A=FAKE + 8), -4), (dict(lda=192), -5), (dict(lda=204), -5), (dict(lda=int8.MAX_LD + 16), -5),
    (dict(SA=None), -6), (dict(sa_inc=-1), -7), (dict(B=None), -8), (dict(B=FAKE + 1), -8), (dict(ldb=192), -9),
    (dict(ldb=200), -9), (dict(SB=None), -10), (dict(sb_inc=-1), -11), (dict(bias_type=3), -13), (dict(D=None), -14),
    (dict(ldd=7), -15), (dict(d_type=-1), -16), (dict(M=0), 0), (dict(N=0, D=None, ldd=1), 0),
])
def test_gemm_refusals(change, status):
    refused(int8.hip_int8_gemm, int8.hip_int8_gemm_status_string, GEMM, change, status)


LINEAR = dict(tokens=40, inputs=200, outputs=8, X=FAKE, x_type=1, ldx=200, W=FAKE, ldw=208, SW=FAKE, sw_inc=1, bias=FAKE,
              bias_type=0, Y=FAKE, ldy=8, y_type=1, workspace=FAKE, workspace_bytes=40 * (208 + 4))


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), -1), (dict(inputs=-1), -2), (dict(inputs=int8.MAX_K + 1), -2), (dict(outputs=-1), -3),
    (dict(X=None), -4), (dict(x_type=9), -5), (dict(ldx=199), -6), (dict(W=None), -7), (dict(W=FAKE + 4), -7),
    (dict(ldw=204), -8), (dict(SW=None), -9), (dict(sw_inc=-1), -10), (dict(bias_type=5), -12), (dict(Y=None), -13),
    (dict(ldy=7), -14), (dict(y_type=3), -15), (dict(workspace=None), -16), (dict(workspace=FAKE + 8), -16),
    (dict(workspace_bytes=40 * (208 + 4) - 1), -17), (dict(workspace_bytes=-1, tokens=3), -17), (dict(tokens=0), 0), (dict(outputs=0), 0),
])
def test_linear_refusals(change, status):
    refused(int8.hip_int8_linear, int8.hip_int8_linear_status_string, LINEAR, change, status)


def test_linear_workspace_holds_codes_and_scales_of_all_but_few_tokens():
    assert int8.hip_int8_linear_workspace(40, 200) == 40 * (208 + 4) and int8.hip_int8_linear_workspace(0, 5) == 0
    assert int8.hip_int8_linear_workspace(2 ** 31 - 1, int8.MAX_K) == (2 ** 31 - 1) * (131072 + 4)
    assert int8.hip_int8_linear_workspace(40, 513) == 40 * (640 + 4)
    for tokens, inputs in ((1, 1), (1, 16384), (16, 1024), (9, 1017), (5, 2048), (3, 4090)):
        assert int8.hip_int8_linear_workspace(tokens, inputs) == 0
    for tokens, inputs in ((1, 16385), (17, 8), (16, 1025), (9, 1025), (5, 2049), (3, 4097)):
        assert int8.hip_int8_linear_workspace(tokens, inputs) > tokens * inputs
    for tokens in (*range(20), 33):
        for inputs in (0, 1, 8, 1000, 1017, 1024, 1025, 2048, 4097, 8192, 16377, 16384, 16385):
            assert int8.hip_int8_linear_workspace(tokens, inputs) == int8._linear_bytes(tokens, inputs)
    for bad in ((-1, 5), (5, -1), (5, int8.MAX_K + 1)):
        with pytest.raises(sgemm.SgemmError):
            int8.hip_int8_linear_workspace(*bad)


FORWARD = dict(rows=4, cols=8, type=0, X=FAKE, ldx=8, w=FAKE, b=FAKE, w_type=0, eps=1e-5, Y=FAKE, ldy=8, stats=None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), -1), (dict(cols=-1), -2), (dict(type=3), -3), (dict(X=None), -4), (dict(ldx=7), -5), (dict(w_type=3), -8),
    (dict(w_type=1), -8), (dict(type=1, w_type=2), -8), (dict(w=None, w_type=-1), -8), (dict(eps=-1e-9), -9), (dict(eps=float("nan")), -9), (dict(Y=None), -10), (dict(ldy=7), -11),
    (dict(rows=0), 0), (dict(cols=0, X=None, w=None, b=None, w_type=7), 0),
])
def test_layernorm_forward_refusals(change, status):
    refused(layernorm.hip_layernorm_forward, layernorm.hip_layernorm_forward_status_string, FORWARD, change, status)


BACKWARD = dict(rows=400, cols=8, type=0, DY=FAKE, lddy=8, X=FAKE, ldx=8, stats=FAKE, w=FAKE, w_type=0, DX=FAKE, lddx=8, dw=FAKE,
                db=2 * FAKE, accumulate=0, workspace=FAKE, workspace_bytes=1 << 20)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), -1), (dict(cols=-1), -2), (dict(type=-1), -3), (dict(DY=None), -4), (dict(lddy=7), -5), (dict(X=None), -6),
    (dict(ldx=7), -7), (dict(stats=None), -8), (dict(w_type=3), -10), (dict(w_type=1), -10), (dict(lddx=7), -12), (dict(accumulate=2), -15),
    (dict(db=FAKE), -14), (dict(db=FAKE + 28), -14), (dict(dw=FAKE + 28, db=FAKE), -14),
    (dict(workspace=None), -16), (dict(workspace=FAKE + 8), -16), (dict(workspace_bytes=8), -17),
    (dict(cols=0), 0), (dict(rows=0, dw=None, db=None, workspace=None), 0), (dict(DX=None, dw=None, db=None, workspace=None), 0),
])
def test_layernorm_backward_refusals(change, status):
    refused(layernorm.hip_layernorm_backward, layernorm.hip_layernorm_backward_status_string, BACKWARD, change, status)


def test_layernorm_workspace():
    for cols in (1, 512, 513, 4096, 16384, 16385, 2 ** 31 - 1):
        row = 2 * 4 * cols
        few = [layernorm.hip_layernorm_backward_workspace(n, cols) for n in (1, layernorm.FEW)]
        assert few[0] == 0 == few[1] if cols <= 16384 else few[0] == row
        many = layernorm.hip_layernorm_backward_workspace(2 ** 31 - 1, cols)
        assert many % row == 0 and row <= many <= 2048 * row
    for rows in (0, 1, 2, 31, 32, 33, 255, 256, 257, 500, 767, 768, 769, 5000, 100_000, 2 ** 31 - 1):
        for cols in (1, 100, 128, 129, 256, 257, 512, 1000, 2000, 4096, 4097, 8192, 16384, 16385, 100_000):
            need, has = layernorm.hip_layernorm_backward_workspace(rows, cols), layernorm._workspace_bytes(rows, cols)
            assert need <= has <= max(768 * 8 * cols, need)
    assert layernorm.hip_layernorm_backward_workspace(0, 5) == 0 == layernorm.hip_layernorm_backward_workspace(5, 0)
    for bad in ((-1, 5), (5, -1)):
        with pytest.raises(sgemm.SgemmError):
            layernorm.hip_layernorm_backward_workspace(*bad)


def tensors(*each):
    """A ctypes array of hip_gradient; what is not said is a dense tensor of 100 floats in place."""
    out = (gradients.Gradient * max(len(each), 1))()
    for g, change in zip(out, each):
        usual = dict(x=0x10000, y=0x10000, rows=1, cols=100, ldx=100, ldy=100, type=0)
        for name, value in {**usual, **change}.items():
            setattr(g, name, value)
    return out


def clip_call(each, function=gradients.hip_gradient_clip, **change):
    usual = dict(count=len(each), tensors=tensors(*each), max_norm=1.0, eps=1e-6, norm=0x4000, workspace=FAKE, workspace_bytes=1 << 20)
    status = function(*{**usual, **change}.values(), stream=0)
    assert "unknown" not in gradients.hip_gradient_clip_status_string(status)
    return status


@pytest.mark.parametrize("each,status", [
    ([dict(x=None)], -2), ([dict(x=0x10002)], -2), ([dict(y=None)], -2), ([dict(y=0x20002)], -2), ([dict(rows=-1)], -2),
    ([dict(cols=-1)], -2), ([dict(type=3)], -2), ([dict(type=-1)], -2), ([dict(rows=2, ldx=99)], -2), ([dict(rows=2, ldy=99)], -2),
    ([dict(rows=2, ldx=1 << 41)], -2), ([dict(rows=1 << 41)], -2),
    ([dict(rows=1 << 30, cols=1 << 30, ldx=1 << 30, ldy=1 << 30)], -2), ([dict(cols=1 << 40)] * 100, -2),
    # what is written overlaps
    ([{}, {}], -2), ([{}, dict(x=0x10000 + 396, y=0x10000 + 396)], -2), ([dict(y=0x10004)], -2),
    ([dict(y=0x20000), dict(x=0x30000, y=0x20000 + 200)], -2), ([dict(y=0x20000), dict(x=0x20000, y=0x40000)], -2),
    ([dict(rows=3, ldx=200, ldy=200), dict(rows=3, ldx=200, ldy=200, x=0x10000 + 396, y=0x10000 + 396)], -2),
    ([dict(rows=3, ldx=200, ldy=200), dict(rows=3, ldx=300, ldy=300, x=0x10000 + 400, y=0x10000 + 400)], -2),
    ([dict(rows=3, ldx=200, ldy=100)], -2), ([dict(x=0x3f00, y=0x3f00)], -2),  # the norm lies in the last one
])
def test_clip_refuses_bad_tensors(each, status):
    assert clip_call(each) == status


@pytest.mark.parametrize("change,status", [
    (dict(count=-1), -1), (dict(count=gradients.MAX_COUNT + 1), -1), (dict(tensors=None), -2), (dict(max_norm=-1.0), -3),
    (dict(max_norm=float("nan")), -3), (dict(eps=-1.0), -4), (dict(eps=float("inf")), -4), (dict(workspace=None), -6),
    (dict(workspace=FAKE + 16), -6), (dict(workspace_bytes=100), -7),
])
def test_clip_refusals(change, status):
    assert clip_call([{}], **change) == status
    assert clip_call([{}], gradients.hip_gradient_clip_by, **change) == status
    assert clip_call([{}], gradients.hip_gradient_clip_by, norm=None) == -5


@pytest.mark.parametrize("change,status", [
    (dict(count=-1), -1), (dict(tensors=None), -2), (dict(tensors=tensors(dict(x=None))), -2), (dict(norm=None), -3),
    (dict(workspace=None), -4), (dict(workspace=FAKE + 16), -4), (dict(workspace_bytes=100), -5),
])
def test_norm_refusals(change, status):
    usual = dict(count=1, tensors=tensors({}), norm=0x4000, workspace=FAKE, workspace_bytes=1 << 20)
    assert gradients.hip_gradient_norm(*{**usual, **change}.values(), stream=0) == status
    assert "unknown" not in gradients.hip_gradient_norm_status_string(status)


def test_gradient_workspace():
    for count in (0, 1, 59, 60, 61, 200, gradients.MAX_COUNT):
        assert gradients.hip_gradient_workspace(count) == gradients._workspace_bytes(count)
    for count in (-1, gradients.MAX_COUNT + 1):
        with pytest.raises(sgemm.SgemmError):
            gradients.hip_gradient_workspace(count)


def test_gradient_struct_is_the_headers():
    assert ctypes.sizeof(gradients.Gradient) == 7 * 8  # the bindings write it as seven 64-bit numbers


@pytest.mark.parametrize("make,want", [
    (lambda: torch.empty(4, 5, 6), (1, 120, 120)), (lambda: torch.empty(4, 5).T, (1, 20, 20)),
    (lambda: torch.empty(4, 5, 6).permute(2, 0, 1), (1, 120, 120)), (lambda: torch.empty(4, 8)[:, :5], (4, 5, 8)),
    (lambda: torch.empty(3, 4, 8)[:, :, 1:6], (12, 5, 8)), (lambda: torch.empty(8, 4).T[:, ::2], (4, 4, 8)),
    (lambda: torch.empty(()), (1, 1, 1)), (lambda: torch.empty(1, 1, 1), (1, 1, 1)), (lambda: torch.empty(10)[::3], (4, 1, 3)),
    (lambda: torch.empty(6, 8)[::2, :8], (3, 8, 16)),
])
def test_layouts_of_gradients(make, want):
    t = make()
    got = gradients._layout(t, "t")
    assert got == want if want != (4, 4, 8) else got[0] * got[1] == t.numel()
    rows, cols, ld = got
    places = {r * ld + c for r in range(rows) for c in range(cols)}
    flat = torch.arange(1000).as_strided(t.shape, t.stride())
    assert places == set(flat.reshape(-1).tolist()) and rows * cols == t.numel()


@pytest.mark.parametrize("make", [lambda: torch.empty(3, 1).expand(3, 4), lambda: torch.empty(4).expand(3, 4),
                                  lambda: torch.empty(4, 6, 8)[:, :3, :5], lambda: torch.empty(20).as_strided((3, 4), (2, 1))])
def test_layouts_that_are_refused(make):
    with pytest.raises(ValueError):
        gradients._layout(make(), "t")


def test_layouts_of_a_gradient_and_its_out():
    for t, o in ((torch.empty(4, 8)[:, :5], torch.empty(4, 5)), (torch.empty(4, 5), torch.empty(4, 9)[:, 2:7]),
                 (torch.empty(8, 4)[:5].T, torch.empty(9, 4)[2:7].T), (torch.empty(3, 4, 8)[:, :, :5], torch.empty(3, 4, 5)),
                 (torch.empty(20)[::2], torch.empty(10)), (torch.empty(8, 5).T[:, ::2], torch.empty_like(torch.empty(8, 5).T[:, ::2]))):
        rows, cols, ldx, ldy = gradients._pair(t, o)
        places = [[r * ld + c for r in range(rows) for c in range(cols)] for ld in (ldx, ldy)]
        flat = [torch.arange(1000).as_strided(v.shape, v.stride()).reshape(-1).tolist() for v in (t, o)]
        assert dict(zip(*places)) == dict(zip(*flat))
    for t, o in ((torch.empty(4, 5), torch.empty(5, 4).T), (torch.empty(8, 5).T[:, ::2], torch.empty(5, 4))):  # two orders
        with pytest.raises(ValueError):
            gradients._pair(t, o)


def test_bindings_refuse_host_tensors():
    x = torch.zeros(4, 16)
    q = int8.Int8(torch.zeros(4, 16, dtype=torch.int8), torch.ones(4))
    for call in (lambda: int8.quantize(x), lambda: int8.gemm(q, q), lambda: int8.linear(x, q), lambda: layernorm.layer_norm(x),
                 lambda: layernorm.layer_norm_backward(x, x, torch.zeros(3, 4)), lambda: gradients.grad_norm([x]),
                 lambda: gradients.grad_norm([None]), lambda: gradients.clip_grad_norm([x], 1.0), lambda: gradients.clip_by_norm([x], torch.ones(()), 1.0)):
        with pytest.raises(TypeError):
            call()


def test_clipping_refuses_no_tensors_and_bad_limits():
    for call in (lambda: gradients.grad_norm([]), lambda: gradients.clip_grad_norm([], 1.0),
                 lambda: gradients.clip_grad_norm([torch.ones(3)], -1.0), lambda: gradients.clip_grad_norm([torch.ones(3)], float("nan")),
                 lambda: gradients.clip_grad_norm([torch.ones(3)], 1.0, eps=-1e-6),
                 lambda: gradients.clip_grad_norm([torch.ones(3)], 1.0, out=[]),
                 lambda: gradients.clip_by_norm([torch.ones(3)], torch.ones(2), 1.0),
                 lambda: gradients.clip_by_norm([torch.ones(3)], torch.ones((), dtype=torch.float64), 1.0)):
        with pytest.raises(ValueError):
            call()


def _places(t, address, ld):
    """The bytes of a tensor of the array above."""
    size = 4 if t["type"] == 0 else 2
    return {address + r * ld * size + b for r in range(t["rows"]) for b in range(t["cols"] * size)}


def _overlap(each, norm):
    """Whether what a clipping call writes meets anything else that it touches, byte by byte."""
    sets = [({norm + b for b in range(4)}, True)]
    for t in each:
        y = _places(t, t["y"], t["ldy"])
        sets.append((y, True))
        if t["x"] != t["y"] or (t["rows"] > 1 and t["ldx"] != t["ldy"]):  # the strides of one row are not read
            sets.append((_places(t, t["x"], t["ldx"]), False))
    return any(a & b for i, (a, wa) in enumerate(sets) for b, wb in sets[:i] if wa or wb)


def _refused_as_overlapping(each, norm=0x4000):
    """Without a device a call that is not refused gives the launch's error."""
    status = clip_call(each, norm=norm)
    assert status == -2 or status > 0
    return status == -2


without_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that nothing lies at, in calls that are not refused")


@without_gpu
def test_clip_refuses_what_overlaps_and_nothing_else():
    import random
    rng = random.Random(1)
    found = [0, 0]
    for trial in range(6000):
        kind = rng.choice((0, 1))
        size = 2 if kind else 4

        def tensor():
            rows, cols = rng.randint(1, 6), rng.randint(1, 9)
            ldx = cols + rng.choice((0, 1, 3, 7, 16, rng.randint(0, 40)))
            x = 0x10000 + size * rng.randint(0, 60)
            t = dict(x=x, y=x, rows=rows, cols=cols, ldx=ldx, ldy=ldx, type=kind)
            if rng.random() < 0.3:
                t["y"], t["ldy"] = 0x10000 + size * rng.randint(0, 200), cols + rng.randint(0, 20)
            return t
        each = [tensor() for _ in range(rng.choice((2, 2, 2, 3)))]
        norm = rng.choice((0x4000, 0x10000 + 4 * rng.randint(0, 60)))
        want = _overlap(each, norm)
        found[want] += 1
        assert _refused_as_overlapping(each, norm) == want, str((each, norm))
    assert min(found) > 500


@without_gpu
def test_clip_finds_overlaps_of_many_rows():
    """Rows at two strides meet once in a million, or not at all."""
    rows, one = 1 << 20, 0x100000000000
    for lda, ldb, cols in ((1000, 1001, 1), (4099, 4111, 2), (64, 96, 16), (3000, 2000, 400), (1000, 1000, 300), (7, 1 << 20, 3)):
        a = set(range(0, rows * lda, lda))
        for shift in (0, 1, 5, 16, 17, 300, 499, 500, 700, 12345, 100003, 777777):
            b = [shift + i * ldb for i in range(min(rows, 1 << 14))]
            meets = any((at + d) in a for at in b for d in range(1 - cols, cols))
            each = [dict(x=one, y=one, rows=rows, cols=cols, ldx=lda, ldy=lda, type=0),
                    dict(x=one + 4 * shift, y=one + 4 * shift, rows=len(b), cols=cols, ldx=ldb, ldy=ldb, type=0)]
            assert _refused_as_overlapping(each) == meets, (lda, ldb, cols, shift)
            assert _refused_as_overlapping(each[::-1]) == meets


@without_gpu
def test_clipping_by_a_norm_that_is_a_gradient_too():
    """The norm that is given is read: new results of it are no overlap, a result written over it is."""
    into = dict(x=0x10000, y=0x20000)
    for norm, status in ((0x10000, None), (0x10000 + 396, None), (0x20000, -2), (0x20000 + 396, -2), (0x4000, None)):
        got = clip_call([into], gradients.hip_gradient_clip_by, norm=norm)
        assert got == status if status else got > 0
        assert (clip_call([into], norm=norm) == -2) == (norm != 0x4000)
