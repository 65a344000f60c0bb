"""The integer quantiser and product, layer norm and gradient clipping from their
definitions, in 64 bits on the CPU: what the GPU tests compare with.  And how far
float arithmetic may be off them, counted in its half steps."""

import torch

AMAX_FLOOR = 2.0 ** -100
HALF = 2.0 ** -24  # of a float's rounding, relative
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def rounding(kind, size):
    """The most that rounding a number of this size to `kind` moves it."""
    info = torch.finfo(kind)
    return info.eps / 2 * size + info.smallest_normal * info.eps / 2


# ------------------------------------------------------------------ integers

def quantize(x):
    """(codes, scales): whole numbers in 64 bits; rows with an infinity or NaN have NaN and zeros."""
    top = x.double().abs().amax(dim=1)
    bad = ~torch.isfinite(top)
    s = (torch.where(bad, torch.ones_like(top), top.clamp(min=AMAX_FLOOR)) / 127).float().double()
    q = torch.round(x.double() / s[:, None])
    q[bad] = 0
    return q, torch.where(bad, torch.full_like(s, float("nan")), s)


def product(a, sa, b, sb, bias=None):
    """(D, the size of what is rounded on the way): the sum is exact, below 2^53."""
    p = (a.double() @ b.double().T) * sa.double()[:, None] * sb.double()
    return (p if bias is None else p + bias.double()), p.abs()


def product_tolerance(kind, d, p):
    """The sum to float, times one scale, times the other and plus the bias (one rounding), to D's type."""
    off = 2 * HALF * p + HALF * d.abs()
    return off * (1 + 2.0 ** -20) + 2.0 ** -149 * 3 + (rounding(kind, d.abs() + off) if kind != torch.float32 else 0)


# ---------------------------------------------------------------- layer norm

# additions in a row of a float sum over a row (16 of a thread's own, six steps of 64
# lanes, 15 of wavefronts) and the roundings of its terms and of the division
DEPTH = 16 + 6 + 15 + 5


def layer_norm(x, w, b, eps):
    """A dict of the pass's values."""
    x = x.double()
    d = x - x.mean(dim=1, keepdim=True)
    rstd = 1 / torch.sqrt(d.square().mean(dim=1, keepdim=True) + eps)
    h = d * rstd
    one = torch.ones(x.shape[1], dtype=torch.float64)
    w = one if w is None else w.double()
    y = h * w + (0 if b is None else b.double())
    # the mean is off by DEPTH half steps of the differences' mean size (of the values' where they
    # are far off zero, by a half step of a half step); rstd by half of DEPTH and three; x - mean
    # and the product with rstd by three more
    off_mean = HALF * DEPTH * (d.abs().mean(dim=1, keepdim=True) + HALF * DEPTH * x.abs().mean(dim=1, keepdim=True)) * rstd
    off_h = off_mean * 1.01 + HALF * (DEPTH / 2 + 6) * h.abs()
    return dict(mean=x.mean(dim=1), rstd=rstd, h=h, y=y, w=w, off_h=off_h)


def forward_tolerance(f, kind):
    off = f["off_h"] * f["w"].abs() + HALF * (f["y"].abs() + (f["h"] * f["w"]).abs())
    return off + (rounding(kind, f["y"].abs() + off) if kind != torch.float32 else 2.0 ** -149)


def layer_norm_backward(f, dy):
    """(dx, dw, db)."""
    dy, h = dy.double(), f["h"]
    g = dy * f["w"]
    c1, c2 = g.mean(dim=1, keepdim=True), (g * h).mean(dim=1, keepdim=True)
    return f["rstd"] * (g - c1 - h * c2), (dy * h).sum(dim=0), dy.sum(dim=0)


def backward_tolerance(f, dy, kind, rows):
    """Of dx, dw and db; `rows`: additions in a row of dw's and db's sums, at most."""
    dy, h, off_h, w = dy.double(), f["h"], f["off_h"], f["w"]
    g = dy * w
    c2 = (g * h).mean(dim=1, keepdim=True).abs()
    c1 = g.mean(dim=1, keepdim=True).abs()
    off_c1 = HALF * DEPTH * g.abs().mean(dim=1, keepdim=True)
    off_c2 = HALF * DEPTH * (g * h).abs().mean(dim=1, keepdim=True) + (g.abs() * off_h).mean(dim=1, keepdim=True)
    inner = off_c1 + off_c2 * h.abs() + c2 * off_h + HALF * 3 * (g.abs() + c1 + h.abs() * c2)
    dx = f["rstd"] * (g - g.mean(dim=1, keepdim=True) - h * (g * h).mean(dim=1, keepdim=True))
    off = f["rstd"] * inner * 1.01 + HALF * (DEPTH / 2 + 6) * dx.abs()
    off_w = (dy.abs() * off_h).sum(dim=0) + HALF * (rows + 1) * (dy * h).abs().sum(dim=0)
    off_b = HALF * rows * dy.abs().sum(dim=0)
    return off + (rounding(kind, dx.abs() + off) if kind != torch.float32 else 2.0 ** -149), off_w * 1.01 + 2.0 ** -149, off_b * 1.01 + 2.0 ** -149


# ------------------------------------------------------------------ clipping

def clip(tensors, max_norm, eps):
    """(norm, the factor)."""
    total = sum(float(t.double().square().sum()) for t in tensors) ** 0.5
    return total, 1.0 if total + eps <= max_norm else max_norm / (total + eps)


# -------------------------------------------------------------------- checks

def close(got, want, tol):
    """Within tol, NaN to NaN; an infinity where the value, within tol, is past the type's largest."""
    kind, got = got.dtype, got.detach().cpu().double()
    assert got.shape == want.shape
    past = torch.isinf(got) & (got.sign() == want.sign()) & (want.abs() + tol >= torch.finfo(kind).max)
    off = ~(((got - want).abs() <= tol) | past | (torch.isnan(got) & torch.isnan(want)))
    if off.any():
        at = torch.nonzero(off)[0].tolist()
        raise AssertionError(f"{int(off.sum())} of {off.numel()} values off, first at {at}: {got[tuple(at)]} for {want[tuple(at)]}")


def same(got, want):
    """Equal as numbers, NaN to NaN."""
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape
    off = ~((got == want) | (torch.isnan(got) & torch.isnan(want)))
    assert not off.any(), (int(off.sum()), torch.nonzero(off)[:4].tolist())


def values(rows, cols, kind, seed=0, offset=0.0):
    """Values of many sizes, with zeros, a row of zeros and one of tiny ones."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-6, 7, (1, cols), generator=g).float()) + offset
    x[torch.rand(rows, cols, generator=g) < 0.05] = 0
    if rows > 2:
        x[1] = 0
        x[2] *= 1e-6
    return x.to(kind)
