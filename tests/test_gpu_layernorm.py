"""Layer norm's forward and backward pass on the GPU against the formulas in 64 bits
and against differences."""

import pytest
import torch

from dense_fp32_matrix_row_amd import layernorm
from tests import serving_reference as ref
from tests.serving_reference import TYPES

pytestmark = pytest.mark.gpu

# every shape of rows, both sides of each border, odd ones among them; the last two are read several times
WIDTHS = (1, 2, 7, 63, 512, 513, 1000, 1024, 1025, 2048, 2049, 4096, 4097, 8192, 8193, 16384, 16385, 20001)
EPS = 1e-5


def params(cols, kind, seed):
    g = torch.Generator().manual_seed(seed)
    return (1 + torch.randn(cols, generator=g) / 2).to(kind), torch.randn(cols, generator=g).to(kind)


def check(x, dy, w, b, kind, eps=EPS):
    """Both passes against the formulas; returns what they gave."""
    rows, cols = x.shape
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    f = ref.layer_norm(x, w, b, eps)
    y, stats = layernorm.layer_norm_forward(x.cuda(), cuda(w), cuda(b), eps=eps)
    assert y.dtype == kind and stats.shape == (3, rows)
    ref.close(y, f["y"], ref.forward_tolerance(f, kind))
    assert torch.equal(layernorm.layer_norm(x.cuda(), cuda(w), cuda(b), eps=eps), y)
    dx, dw, db = layernorm.layer_norm_backward(dy.cuda(), x.cuda(), stats, cuda(w))
    for got, want, tol in zip((dx, dw, db), ref.layer_norm_backward(f, dy), ref.backward_tolerance(f, dy, kind, rows)):
        if got is not None:
            ref.close(got, want, tol)
    assert dx.dtype == kind and (w is not None or (dw is None and db is None))
    return y, stats, dx, dw, db


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("cols", WIDTHS)
def test_against_the_formulas(cols, kind):
    for rows in (1, 3, 37):
        x = ref.values(rows, cols, TYPES[kind], seed=rows * 1000 + cols, offset=0.5)
        g = torch.Generator().manual_seed(cols)
        dy = (torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))).to(TYPES[kind])
        w, b = params(cols, torch.float32 if rows == 3 else TYPES[kind], cols)
        check(x, dy, w, b, TYPES[kind])


@pytest.mark.parametrize("rows", (256, 257, 500, 2300, 5001))
@pytest.mark.parametrize("cols", (64, 777, 1500, 3001, 5000, 9000, 17000))
def test_many_rows_share_the_blocks(rows, cols):
    if rows * cols > 3e7:
        rows //= 8
    x = ref.values(rows, cols, torch.float32, seed=cols, offset=-0.25)
    dy = ref.values(rows, cols, torch.float32, seed=cols + 1)
    w, b = params(cols, torch.float32, cols)
    first = check(x, dy, w, b, torch.float32)
    for a, again in zip(first, check(x, dy, w, b, torch.float32)):
        assert torch.equal(a, again)


@pytest.mark.parametrize("cols", (300, 4000, 20000))
def test_rows_far_off_zero_keep_their_differences(cols):
    """Means of a thousand to ten thousand deviations: the mean's rounding to float alone would move h by 10^-4 to 10^-3."""
    x = (ref.values(20, cols, torch.float32, 1) / 64 + torch.linspace(-1e4, 1e4, 20)[:, None]).float()
    w, b = params(cols, torch.float32, 2)
    check(x, ref.values(20, cols, torch.float32, 3), w, b, torch.float32)


@pytest.mark.parametrize("which", ("none", "weight", "bias"))
@pytest.mark.parametrize("cols", (100, 3000, 20000))
def test_without_weight_or_bias(cols, which):
    x, dy = ref.values(11, cols, torch.float32, 4), ref.values(11, cols, torch.float32, 5)
    w, b = params(cols, torch.float32, 6)
    check(x, dy, w if which == "weight" else None, b if which == "bias" else None, torch.float32)


@pytest.mark.parametrize("eps", (0.0, 1e-12, 1.0))
def test_eps(eps):
    x, dy = ref.values(40, 500, torch.float32, 7)[3:], ref.values(37, 500, torch.float32, 8)
    w, b = params(500, torch.float32, 9)
    check(x, dy, w, b, torch.float32, eps)


def test_constant_rows():
    """No differences: y is the bias; dx is what is left of dy w without its mean, over the root of eps."""
    for cols in (5, 1000, 3000, 20000):
        x = torch.full((4, cols), 3.0)
        x[1], x[2] = 0, -1e4
        w, b = params(cols, torch.float32, 10)
        y, stats, *_ = check(x, ref.values(4, cols, torch.float32, 11), w, b, torch.float32)
        assert torch.equal(y.cpu(), b.expand(4, cols))
        assert torch.equal(stats[0].cpu(), x[:, 0]) and (stats[1] == 0).all()


@pytest.mark.parametrize("cols", (300, 1500, 4000, 20000))
def test_infinities_and_nans_stay_in_their_row(cols):
    x, dy = ref.values(40, cols, torch.float32, 12, offset=1.0), ref.values(40, cols, torch.float32, 13)
    clean = layernorm.layer_norm_forward(x.cuda())
    x[7, cols // 2], x[20, 0], x[33, cols - 1] = float("nan"), float("inf"), float("-inf")
    w, b = params(cols, torch.float32, 14)
    y, stats = layernorm.layer_norm_forward(x.cuda())
    dx, dw, db = layernorm.layer_norm_backward(dy.cuda(), x.cuda(), stats, torch.ones(cols, device="cuda"))
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[[7, 20, 33]] = True
    for t in (y, dx):
        assert torch.isnan(t[bad]).all() and torch.isfinite(t[~bad]).all()
    assert torch.equal(y[~bad], clean[0][~bad])
    assert torch.isnan(dw).all() and torch.isfinite(db).all()
    dy[3, 1] = float("inf")  # in the gradient: that row, and that column of db
    _, stats = clean
    x = ref.values(40, cols, torch.float32, 12, offset=1.0)
    dx, dw, db = layernorm.layer_norm_backward(dy.cuda(), x.cuda(), stats, torch.ones(cols, device="cuda"))
    assert torch.isnan(dx[3]).all() or torch.isnan(dx[3]).sum() + torch.isinf(dx[3]).sum() == cols
    others = torch.arange(40, device="cuda") != 3
    assert torch.isfinite(dx[others]).all() and torch.isfinite(db[2:]).all() and db[1] == float("inf")


@pytest.mark.parametrize("rows", (30, 300))
@pytest.mark.parametrize("cols", (297, 1501, 3001, 17001))
@pytest.mark.parametrize("kind", TYPES)
def test_strided_rows_in_place_and_nothing_outside_is_written(kind, cols, rows):
    kind = TYPES[kind]
    big = lambda seed: ref.values(rows, cols + 37, kind, seed)  # noqa: E731
    x, dy = big(15), big(16)
    inside = slice(3, 3 + cols)  # odd base and row stride
    w, b = params(cols, kind, 17)
    y, stats, dx, dw, db = check(x[:, inside].contiguous(), dy[:, inside].contiguous(), w, b, kind)
    gx, gdy = x.cuda(), dy.cuda()
    out = gx.clone()
    got, stats2 = layernorm.layer_norm_forward(out[:, inside], w.cuda(), b.cuda(), eps=EPS, out=out[:, inside])
    assert torch.equal(got, y) and torch.equal(stats, stats2)
    for place in ("dy", "x", "new"):
        a, c = gx.clone(), gdy.clone()
        o = {"dy": c, "x": a, "new": torch.zeros_like(a)}[place]
        res = layernorm.layer_norm_backward(c[:, inside], a[:, inside], stats, w.cuda(), out=o[:, inside])
        assert all(torch.equal(p, q) for p, q in zip(res, (dx, dw, db)))
        before = {"dy": gdy, "x": gx, "new": torch.zeros_like(a)}[place]
        o[:, inside] = before[:, inside]
        assert torch.equal(o, before)
    out[:, inside] = gx[:, inside]
    assert torch.equal(out, gx)


@pytest.mark.parametrize("cols", (200, 2000, 20000))
def test_gradients_are_added_to_what_is_there(cols):
    x, dy = ref.values(300, cols, torch.float32, 18), ref.values(300, cols, torch.float32, 19)
    w, _ = params(cols, torch.float32, 20)
    y, stats, dx, dw, db = check(x, dy, w, None, torch.float32)
    one, two = torch.randn(cols, device="cuda"), torch.randn(cols, device="cuda")
    want = one + dw, two + db
    version = one._version, two._version
    res = layernorm.layer_norm_backward(dy.cuda(), x.cuda(), stats, w.cuda(), dw=one, db=two)
    assert res[1] is one and res[2] is two and torch.equal(one, want[0]) and torch.equal(two, want[1]) and torch.equal(res[0], dx)
    assert (one._version, two._version) == (version[0] + 1, version[1] + 1)
    only = torch.zeros(cols, device="cuda")  # a bias alone
    _, none, got = layernorm.layer_norm_backward(dy.cuda(), x.cuda(), stats, db=only)
    assert none is None and got is only and torch.equal(only, db)


@pytest.mark.parametrize("cols", (6, 700))
def test_gradients_by_differences(cols):
    """The passes are those of one function: differences of sum(dy * y) in 64 bits, a step of each of x, w and b."""
    rows = 3
    g = torch.Generator().manual_seed(21)
    x, dy = torch.randn(rows, cols, generator=g), torch.randn(rows, cols, generator=g)
    w, b = params(cols, torch.float32, 22)
    _, stats = layernorm.layer_norm_forward(x.cuda(), w.cuda(), b.cuda(), eps=EPS)
    grads = layernorm.layer_norm_backward(dy.cuda(), x.cuda(), stats, w.cuda())
    loss = lambda *v: (dy.double() * ref.layer_norm(v[0], v[1], v[2], EPS)["y"]).sum().item()  # noqa: E731
    step = 2.0 ** -12
    f = ref.layer_norm(x, w, b, EPS)
    tols = ref.backward_tolerance(f, dy, torch.float32, rows)
    args = [t.double() for t in (x, w, b)]
    for k in range(3):
        flat, got = args[k].reshape(-1), grads[k].cpu().double().reshape(-1)
        for i in range(0, flat.numel(), max(flat.numel() // 12, 1)):
            old = flat[i].item()
            flat[i] = old + step
            up = loss(*args)
            flat[i] = old - step
            down = loss(*args)
            flat[i] = old
            # third derivatives are below 100 here, the sums in 64 bits off by 1e-12 of their size
            assert abs((up - down) / (2 * step) - got[i]) <= tols[k].reshape(-1)[i] + 100 * step ** 2 + 1e-8


def test_degenerate_sizes():
    w = torch.ones(5, device="cuda")
    none = torch.empty(0, 5, device="cuda")
    y, stats = layernorm.layer_norm_forward(none, w, w)
    assert y.shape == (0, 5) and stats.shape == (3, 0)
    dx, dw, db = layernorm.layer_norm_backward(none, none, stats, w)
    assert dx.shape == (0, 5) and torch.equal(dw, torch.zeros_like(w)) and torch.equal(db, torch.zeros_like(w))
    one, two = torch.ones(5, device="cuda"), torch.ones(5, device="cuda")
    layernorm.layer_norm_backward(none, none, stats, w, dw=one, db=two)
    assert torch.equal(one, w) and torch.equal(two, w)
    flat = torch.empty(5, 0, device="cuda")
    y, stats = layernorm.layer_norm_forward(flat, flat[0], flat[0])
    dx, dw, db = layernorm.layer_norm_backward(flat, flat, stats, flat[0])
    assert y.shape == (5, 0) and dx.shape == (5, 0) and dw.shape == (0,)


def test_past_two_gigabytes_and_the_widest_row():
    rows, cols = 33000, 35000
    x = torch.randn(rows, cols, device="cuda", dtype=torch.bfloat16)
    w, b = params(cols, torch.float32, 23)
    y, stats = layernorm.layer_norm_forward(x, w.cuda(), b.cuda())
    dx, dw, db = layernorm.layer_norm_backward(x, x, stats, w.cuda())
    for at in (slice(0, 2), slice(30677, 30680), slice(rows - 2, rows)):
        f = ref.layer_norm(x[at].cpu(), w, b, EPS)
        ref.close(y[at], f["y"], ref.forward_tolerance(f, torch.bfloat16))
        ref.close(dx[at], ref.layer_norm_backward(f, x[at].cpu())[0], ref.backward_tolerance(f, x[at].cpu(), torch.bfloat16, 4)[0])
    want = x[:, :64].double().sum(dim=0)
    assert ((db[:64].double() - want).abs() <= 2.0 ** -24 * 1000 * x[:, :64].double().abs().sum(dim=0)).all()
    del x, y, dx
    n = (1 << 31) - 1
    x = torch.ones(1, n, device="cuda", dtype=torch.bfloat16)
    x[0, ::2] = -1  # one more of these: the mean is -1 / n
    y, stats = layernorm.layer_norm_forward(x)
    assert abs(stats[0].item() + 1 / n) <= 1e-15 and abs(stats[2].item() - 1 / (1 + EPS) ** 0.5) <= 1e-6
    assert torch.equal(y, x)
    dx, dw, db = layernorm.layer_norm_backward(x, x, stats, torch.ones(1, device="cuda", dtype=torch.bfloat16).expand(n).contiguous())
    assert abs(db[1].item() - 1) <= 1e-7 and abs(dw[-1].item() - 1) <= 1e-5 and dx.abs().max().item() <= 2e-5


def test_other_streams_and_captured_graphs():
    side = torch.cuda.Stream()
    for rows, cols in ((1, 100), (300, 1024), (2000, 3000), (40, 20000)):
        x, dy = torch.randn(rows, cols, device="cuda"), torch.randn(rows, cols, device="cuda")
        w, b = (t.cuda() for t in params(cols, torch.float32, 24))

        def both():
            y, stats = layernorm.layer_norm_forward(x, w, b)
            return y, *layernorm.layer_norm_backward(dy, x, stats, w)
        want = both()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = both()
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = both()
        for i in range(3):
            x.copy_(torch.randn(rows, cols, device="cuda") * (i + 1))
            graph.replay()
            torch.cuda.synchronize()
            want = both()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want)), (rows, cols)


def test_refusals_of_the_tensor_forms():
    x = torch.randn(8, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    _, stats = layernorm.layer_norm_forward(x, w, w)
    for bad in (lambda: layernorm.layer_norm(x.double()), lambda: layernorm.layer_norm(x, w.double()), lambda: layernorm.layer_norm(x, w.cpu()),
                lambda: layernorm.layer_norm(x, w, w.half()), lambda: layernorm.layer_norm_backward(x, x, stats, w, dw=w.half(), db=w)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: layernorm.layer_norm(x.T), lambda: layernorm.layer_norm(x[:1].expand(8, 64)), lambda: layernorm.layer_norm(x, w[:63]),
                lambda: layernorm.layer_norm(x, torch.ones(128, device="cuda")[::2]), lambda: layernorm.layer_norm(x, eps=-1.0),
                lambda: layernorm.layer_norm(x, out=x.half()), lambda: layernorm.layer_norm(x, eps=float("nan")),
                lambda: layernorm.layer_norm_backward(x[:4], x, stats, w), lambda: layernorm.layer_norm_backward(x.half(), x, stats, w),
                lambda: layernorm.layer_norm_backward(x, x, stats[:2], w), lambda: layernorm.layer_norm_backward(x, x, stats, w, dw=w.clone()),
                lambda: layernorm.layer_norm_backward(x, x, stats, w, dw=w[:3], db=w), lambda: layernorm.layer_norm(x[0])):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("rows", (4, 300))
@pytest.mark.parametrize("cols", (5, 100, 512, 1001, 2000, 3001, 4098, 9000, 9001, 20001, 20002))
@pytest.mark.parametrize("kind", ("f32", "bf16"))
def test_large_constant_rows(kind, cols, rows):
    """No differences, whatever the rows' size: h is 0, and the gradients are those of rows of zeros.  -mean rstd,
    what a zero past the row's end would have for h, passes a float's range (2^110 by 10^6)."""
    kind = TYPES[kind]
    x = torch.full((rows, cols), 2.0 ** 110, dtype=kind)
    x[1] = -2.0 ** 110
    dy = ref.values(rows, cols, kind, 30)
    w, b = params(cols, kind, 31)
    zeros = ref.layer_norm(torch.zeros_like(x), w, b, 1e-12)
    y, stats = layernorm.layer_norm_forward(x.cuda(), w.cuda(), b.cuda(), eps=1e-12)
    assert torch.equal(y.cpu(), b.expand(rows, cols))
    got = layernorm.layer_norm_backward(dy.cuda(), x.cuda(), stats, w.cuda())
    tols = ref.backward_tolerance(zeros, dy, kind, rows)
    for g, want, tol in zip(got, ref.layer_norm_backward(zeros, dy), tols):
        ref.close(g, want, tol)


@pytest.mark.parametrize("eps", (0.0, 1e-5))
@pytest.mark.parametrize("power", (-120, -90, -75, -65, -55, 55, 62, 66, 100, 110))
@pytest.mark.parametrize("cols", (3, 100, 200, 512, 700, 1500, 3000, 9001, 20001))
def test_squares_past_a_floats_range(cols, power, eps):
    """Differences whose squares, or the sums of these, a float cannot hold, or not with all its bits."""
    g = torch.Generator().manual_seed(cols)
    x, dy = torch.randn(5, cols, generator=g) * 2.0 ** power, torch.randn(5, cols, generator=g)
    w, b = params(cols, torch.float32, 32)
    check(x, dy, w, b, torch.float32, eps)


@pytest.mark.parametrize("cols", (3, 100, 200, 512, 700, 1500, 3000, 9001, 20001))
def test_large_constant_rows_whose_sum_is_rounded(cols):
    """The mean is some steps off the values, whose squares pass a float's range; its remainder is these steps."""
    for value in (1.1e10, 1.1e20, 1.1e27, 1.3e30, 1.7e33):
        x, dy = torch.full((4, cols), value), ref.values(4, cols, torch.float32, 33)
        w, b = params(cols, torch.float32, 34)
        y, stats = layernorm.layer_norm_forward(x.cuda(), w.cuda(), b.cuda())
        assert torch.equal(y.cpu(), b.expand(4, cols))
        zeros = ref.layer_norm(torch.zeros_like(x), w, b, EPS)
        got = layernorm.layer_norm_backward(dy.cuda(), x.cuda(), stats, w.cuda())
        for v, want, tol in zip(got, ref.layer_norm_backward(zeros, dy), ref.backward_tolerance(zeros, dy, torch.float32, 4)):
            ref.close(v, want, tol)


@pytest.mark.parametrize("cols", (100, 200, 700, 1500, 3000, 9001))
def test_rows_beside_such_a_row_stay_as_they_are(cols):
    x = torch.randn(9, cols, generator=torch.Generator().manual_seed(35)).cuda()
    want = layernorm.layer_norm_forward(x)
    for at, factor in ((2, 2.0 ** 80), (5, 2.0 ** -80), (8, float("inf"))):
        other = x.clone()
        other[at] *= factor
        got = layernorm.layer_norm_forward(other)
        rest = torch.arange(9, device="cuda") != at
        assert torch.equal(got[0][rest], want[0][rest]) and torch.equal(got[1][:, rest], want[1][:, rest])


def test_tokens_without_columns():
    """Results go where they are asked for, and nothing that comes back is left as the memory was."""
    flat, out = torch.empty(300, 0, device="cuda"), torch.empty(300, 0, device="cuda")
    for _ in range(3):
        torch.full((3, 300), float("nan"), device="cuda")  # freed: what the statistics' memory may hold
        y, stats = layernorm.layer_norm_forward(flat, flat[0], flat[0], out=out)
        assert y is out and (stats == 0).all()
    dx, dw, db = layernorm.layer_norm_backward(flat, flat, stats, flat[0], out=out)
    assert dx is out and dw.shape == db.shape == (0,)
    with pytest.raises(ValueError):
        layernorm.layer_norm_backward(flat, flat, stats, flat[0], out=flat[:4])
    one, two = flat[0].clone(), flat[0].clone()
    res = layernorm.layer_norm_backward(flat, flat, stats, flat[0], dw=one, db=two)
    assert res[0].shape == (300, 0) and res[1] is one and res[2] is two
