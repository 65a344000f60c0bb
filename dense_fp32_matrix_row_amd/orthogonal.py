"""Orthogonalising a matrix by Newton-Schulz products (ctypes binding of
include/orthogonal.h).

hip_orthogonalize and hip_orthogonalize_workspace carry the C ABI's names;
orthogonalize takes and returns torch device tensors, runs on torch's current
stream of the tensor's device and raises on errors.  Every operation runs in
the library's HIP kernels; there is no fallback.  The result carries no autograd
graph; an `out` counts as modified for autograd.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Sequence

from . import sgemm as _sgemm
from .blockfp8 import current_stream, written

EXPORTS = ("hip_orthogonalize", "hip_orthogonalize_workspace", "hip_orthogonalize_plan",
           "hip_orthogonalize_status_string")

F32, BF16, F16 = 0, 1, 2
MAX_SIZE = 1 << 20
MAX_STEPS = 64
QUINTIC = (3.4445, -4.7750, 2.0315)

class _Product(ctypes.Structure):
    """hip_orthogonalize_product."""
    _fields_ = [(name, ctypes.c_int) for name in ("tile", "parts", "cut", "cut_tile")]


_bound = None


def load():
    """The library with this header's functions declared."""
    global _bound
    lib = _sgemm.load()
    if lib is not _bound:
        i32, i64, f32, vp = ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_void_p
        lib.hip_orthogonalize.restype = i32
        lib.hip_orthogonalize.argtypes = [i32, i32, i32, i32, vp, i32, i64, i32, ctypes.POINTER(f32), f32,
                                          vp, i32, i64, vp, i64, vp]
        lib.hip_orthogonalize_workspace.restype = i32
        lib.hip_orthogonalize_workspace.argtypes = [i32, i32, i32, i32, ctypes.POINTER(i64)]
        lib.hip_orthogonalize_plan.restype = i32
        lib.hip_orthogonalize_plan.argtypes = [i32, i32, i32, ctypes.POINTER(_Product)]
        lib.hip_orthogonalize_status_string.restype = ctypes.c_char_p
        lib.hip_orthogonalize_status_string.argtypes = [i32]
        _bound = lib
    return lib


def hip_orthogonalize_status_string(status) -> str:
    return load().hip_orthogonalize_status_string(int(status)).decode()


def _check(status):
    if status != 0:
        raise _sgemm.SgemmError(status, hip_orthogonalize_status_string(status))


def hip_orthogonalize_workspace(batch, rows, cols, type) -> int:
    """Bytes of workspace of a call (nothing is launched)."""
    out = ctypes.c_longlong()
    _check(load().hip_orthogonalize_workspace(int(batch), int(rows), int(cols), int(type), ctypes.byref(out)))
    return out.value


def hip_orthogonalize_plan(batch, rows, cols) -> list:
    """The tiles of a step's three products (S, P and P X), a dict each (nothing is launched)."""
    products = (_Product * 3)()
    _check(load().hip_orthogonalize_plan(int(batch), int(rows), int(cols), products))
    return [{name: getattr(p, name) for name, _ in _Product._fields_} for p in products]


def hip_orthogonalize(batch, rows, cols, type, G, ldg, stride_g, steps, coefficients, eps, X, ldx, stride_x,
                      workspace, workspace_bytes, stream=None) -> int:
    """X <- the Newton-Schulz iterate of G; `coefficients` is a sequence of
    3 * steps numbers or None.  Returns the status code (0 = enqueued)."""
    co = None
    if coefficients is not None:
        co = (ctypes.c_float * max(len(coefficients), 1))(*coefficients)
        if len(coefficients) < 3 * int(steps):
            raise ValueError(f"{len(coefficients)} coefficients for {steps} steps")
    a = _sgemm._addr
    return int(load().hip_orthogonalize(int(batch), int(rows), int(cols), int(type), a(G), int(ldg), int(stride_g),
                                        int(steps), co, float(eps), a(X), int(ldx), int(stride_x), a(workspace),
                                        int(workspace_bytes), _sgemm._stream(stream)))


def _layout(name, t):
    """(batch, rows, cols, row stride, matrix stride) of a [..., rows, cols] tensor
    whose columns lie side by side and whose leading dimensions are one stride."""
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must have 2 or 3 dimensions")
    batch = 1 if t.dim() == 2 else t.shape[0]
    rows, cols = t.shape[-2:]
    if cols > 1 and rows > 0 and batch > 0 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    ld = t.stride(-2) if rows > 1 else max(cols, 1)
    if rows > 1 and ld < cols:
        raise ValueError(f"{name}'s rows overlap")
    if max(batch, rows, cols, ld) >= 1 << 31:
        raise ValueError(f"{name} has a side or a row stride of 2^31 or more")
    return batch, rows, cols, max(ld, 1), t.stride(0) if batch > 1 else 0


def orthogonalize(g, steps: int = 5, coefficients: Optional[Sequence] = None, eps: float = 1e-7, out=None,
                  workspace=None):
    """The Newton-Schulz iterate of g, or of each matrix of a 3-D g, as a new
    tensor of g's type or in `out` (which may be g).

    `coefficients`: (a, b, c) for every step (default the quintic 3.4445,
    -4.7750, 2.0315), or a sequence of `steps` such triples.  `workspace`: a
    contiguous device tensor of at least hip_orthogonalize_workspace(...)
    bytes to use instead of a new one."""
    import torch
    types = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
    if not g.is_cuda:
        raise TypeError("g must live on the GPU")
    if g.dtype not in types:
        raise TypeError(f"g is float32, bfloat16 or float16, not {g.dtype}")
    batch, rows, cols, ldg, stride_g = _layout("g", g)
    co = list(QUINTIC if coefficients is None else coefficients)
    if len(co) == 3 and not any(hasattr(v, "__len__") for v in co):
        co = [co] * steps
    if len(co) != steps or any(len(v) != 3 for v in co):
        raise ValueError("coefficients are (a, b, c), or one such triple for each step")
    flat = [float(x) for v in co for x in v]
    device = g.device
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return orthogonalize(g, steps, co, eps, out, workspace)
    new = out is None
    if new:
        out = torch.empty(g.shape, dtype=g.dtype, device=device)
    if out.shape != g.shape or out.dtype != g.dtype or out.device != device:
        raise ValueError(f"out is {tuple(out.shape)} {out.dtype}, not {tuple(g.shape)} {g.dtype}")
    _, _, _, ldx, stride_x = _layout("out", out)
    kind = types[g.dtype]
    if workspace is None:
        workspace = torch.empty(max(hip_orthogonalize_workspace(batch, rows, cols, kind), 1), dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous and on g's device")
    _check(hip_orthogonalize(batch, rows, cols, kind, g, ldg, stride_g, steps, flat, eps, out, ldx, stride_x, workspace,
                             workspace.numel() * workspace.element_size(), current_stream(device.index)))
    if not new:
        written(out)
    return out
