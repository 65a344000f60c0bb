"""The block-scaled 8-bit operators and the orthogonalised update from their
definitions, in 64 bits on the CPU: what the GPU tests compare with."""

import torch

AMAX_FLOOR = 2.0 ** -100
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # the magnitudes, by code
POWERS = torch.tensor([2.0 ** e for e in range(-120, 124)], dtype=torch.float64)


def to_e4m3(t):
    """The value of t's code: nearest, ties to the even code, magnitudes above 448 not expected."""
    borders = (E4M3[:-1] + E4M3[1:]) / 2
    size = t.abs().contiguous()
    k = torch.searchsorted(borders, size)
    tie = size == borders[k.clamp(max=len(borders) - 1)]
    k = k + (tie & (k % 2 == 1))
    return torch.where(torch.isnan(t), t, torch.copysign(E4M3[k.clamp(max=126)], t))


def scales(x, block_rows, e8m0):
    """The scale of each block of block_rows x 128."""
    r, c = x.shape
    R, C = -(-r // block_rows), -(-c // 128)
    pad = torch.zeros(R * block_rows, C * 128, dtype=torch.float64)
    pad[:r, :c] = x.double().abs()
    top = pad.view(R, block_rows, C, 128).amax(dim=(1, 3))
    bad = ~torch.isfinite(top)
    top = torch.where(bad, torch.ones_like(top), top.clamp(min=AMAX_FLOOR))
    s = POWERS[torch.searchsorted(POWERS * 448, top)] if e8m0 else (top / 448).float().double()
    return torch.where(bad, torch.full_like(s, float("nan")), s)


def spread(s, block_rows, rows, cols):
    return s.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def quantize(x, block_rows, e8m0):
    """(values of the codes, scales), both in 64 bits."""
    s = scales(x, block_rows, e8m0)
    return to_e4m3(x.double() / spread(s, block_rows, *x.shape)), s


def dequantize(q, s, block_rows):
    return q.double() * spread(s.double(), block_rows, *q.shape)


def orthogonalize(g, coefficients, eps):
    """Batch of matrices, one (a, b, c) per step."""
    x = g.double()
    x = x / (x.pow(2).sum(dim=(-2, -1), keepdim=True).sqrt() + eps)
    for a, b, c in coefficients:
        s = x @ x.mT
        x = a * x + (b * s + c * (s @ s)) @ x
    return x
