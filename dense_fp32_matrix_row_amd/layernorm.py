"""Layer norm's forward and backward pass (ctypes binding of include/layernorm.h).

hip_layernorm_forward and hip_layernorm_backward carry the C ABI's names and
argument order and return its status codes.  layer_norm, layer_norm_forward and
layer_norm_backward take and return torch device tensors, run on torch's current
stream of the tensors' device and raise on errors.  Every operation runs in the
library's HIP kernels; there is no fallback.  Results carry no autograd graph: the
gradients are layer_norm_backward's.  A tensor that is written in place (out, dw,
db) counts as modified for autograd.
"""

from __future__ import annotations

import ctypes

from . import sgemm as _sgemm
from .blockfp8 import _call, _matrix, _same_device, _types, written

EXPORTS = ("hip_layernorm_forward", "hip_layernorm_backward", "hip_layernorm_backward_workspace",
           "hip_layernorm_forward_status_string", "hip_layernorm_backward_status_string")

F32, BF16, F16 = 0, 1, 2
FEW = 256  # HIP_LAYERNORM_FEW

_bound = None


def load():
    """The library with this header's functions declared."""
    global _bound
    lib = _sgemm.load()
    if lib is not _bound:
        i32, i64, f32, vp = ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_void_p
        lib.hip_layernorm_forward.restype = i32
        lib.hip_layernorm_forward.argtypes = [i32, i32, i32, vp, i32, vp, vp, i32, f32, vp, i32, vp, vp]
        lib.hip_layernorm_backward.restype = i32
        lib.hip_layernorm_backward.argtypes = [i32, i32, i32, vp, i32, vp, i32, vp, vp, i32, vp, i32, vp, vp, i32, vp, i64, vp]
        lib.hip_layernorm_backward_workspace.restype = i32
        lib.hip_layernorm_backward_workspace.argtypes = [i32, i32, ctypes.POINTER(i64)]
        for name in EXPORTS[-2:]:
            getattr(lib, name).restype = ctypes.c_char_p
            getattr(lib, name).argtypes = [i32]
        _bound = lib
    return lib


def hip_layernorm_forward(rows, cols, type, X, ldx, w, b, w_type, eps, Y, ldy, stats, stream=None) -> int:
    """Y <- the layer norm of X's rows; returns the status code (0 = enqueued)."""
    a, s = _sgemm._addr, _sgemm._stream
    return int(load().hip_layernorm_forward(int(rows), int(cols), int(type), a(X), int(ldx), a(w), a(b), int(w_type),
                                            float(eps), a(Y), int(ldy), a(stats), s(stream)))


def hip_layernorm_backward(rows, cols, type, DY, lddy, X, ldx, stats, w, w_type, DX, lddx, dw, db, accumulate, workspace,
                           workspace_bytes, stream=None) -> int:
    """The gradients by X, w and b; returns the status code."""
    a, s = _sgemm._addr, _sgemm._stream
    return int(load().hip_layernorm_backward(int(rows), int(cols), int(type), a(DY), int(lddy), a(X), int(ldx), a(stats),
                                             a(w), int(w_type), a(DX), int(lddx), a(dw), a(db), int(accumulate),
                                             a(workspace), int(workspace_bytes), s(stream)))


def hip_layernorm_backward_workspace(rows, cols) -> int:
    """Bytes of workspace of a call (nothing is launched)."""
    out = ctypes.c_longlong()
    rc = load().hip_layernorm_backward_workspace(int(rows), int(cols), ctypes.byref(out))
    if rc != 0:
        raise _sgemm.SgemmError(rc, hip_layernorm_backward_status_string(rc))
    return out.value


def hip_layernorm_forward_status_string(status) -> str:
    return load().hip_layernorm_forward_status_string(int(status)).decode()


def hip_layernorm_backward_status_string(status) -> str:
    return load().hip_layernorm_backward_status_string(int(status)).decode()


def _tokens(name, x):
    """(rows, columns, row stride, type) of tokens."""
    rows, cols, ld = _matrix(name, x)
    kind = _types().get(x.dtype)
    if kind is None:
        raise TypeError(f"{name} is float32, bfloat16 or float16, not {x.dtype}")
    return rows, cols, ld, kind


def _like(name, t, x):
    """The row stride of a tensor of x's shape and type."""
    if t.shape != x.shape or t.dtype != x.dtype:
        raise ValueError(f"{name} is {tuple(t.shape)} {t.dtype}, not {tuple(x.shape)} {x.dtype}")
    return _matrix(name, t)[2]


def _vector(name, v, cols, dtype=None):
    if not v.is_cuda:
        raise TypeError(f"{name} must live on the GPU")
    if tuple(v.shape) != (cols,):
        raise ValueError(f"{name} is {tuple(v.shape)}, not {(cols,)}")
    if cols > 1 and v.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and v.dtype != dtype:
        raise TypeError(f"{name} is {dtype}, not {v.dtype}")


def _params(weight, bias, cols, x):
    """(addresses of both, their type)."""
    first = weight if weight is not None else bias
    if first is None:
        return None, None, F32
    for name, v in (("weight", weight), ("bias", bias)):
        if v is not None:
            _vector(name, v, cols)
            if v.dtype != first.dtype:
                raise TypeError(f"weight and bias of two types: {weight.dtype} and {bias.dtype}")
    kind = _types().get(first.dtype)
    if kind is None or kind != F32 and first.dtype != x.dtype:
        raise TypeError(f"weight and bias are float32 or of x's type, not {first.dtype}")
    return weight.data_ptr() if weight is not None else None, bias.data_ptr() if bias is not None else None, kind


def _forward(x, weight, bias, eps, out, keep):
    import torch
    rows, cols, ldx, kind = _tokens("x", x)
    w, b, w_type = _params(weight, bias, cols, x)
    if not eps >= 0:
        raise ValueError(f"eps is {eps}, not 0 or more")
    _same_device(x, weight, bias, out)
    device = x.device
    if out is None:
        y, ldy = torch.empty((rows, cols), dtype=x.dtype, device=device), max(cols, 1)
    else:
        y, ldy = out, _like("out", out, x)
    stats = (torch.empty if cols else torch.zeros)((3, rows), dtype=torch.float32, device=device) if keep else None
    _call(device, load().hip_layernorm_forward, hip_layernorm_forward_status_string, rows, cols, kind, x.data_ptr(), ldx,
          w, b, w_type, eps, y.data_ptr(), ldy, stats.data_ptr() if keep else None)
    if out is not None:
        written(out)
    return y, stats


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out=None):
    """The layer norm of tokens x (T x I, rows may be strided) over their last
    dimension, as a new tensor of x's type or in `out` (which may be x).  weight and
    bias: I numbers, float32 or of x's type, or None."""
    return _forward(x, weight, bias, eps, out, False)[0]


def layer_norm_forward(x, weight=None, bias=None, eps: float = 1e-5, out=None):
    """layer_norm(...), and the rows' statistics, which layer_norm_backward takes
    (float32, 3 x T: the means, what their rounding left over, and 1 / the deviations;
    zeros without columns)."""
    return _forward(x, weight, bias, eps, out, True)


def _workspace_bytes(rows, cols) -> int:
    """At least hip_layernorm_backward_workspace, without a call: a part a row, 768 at most,
    none of few rows."""
    if rows <= FEW and cols <= 16384:
        return 0
    if cols > 16384:
        return hip_layernorm_backward_workspace(rows, cols)
    return min(rows, 768) * 8 * cols


def layer_norm_backward(dy, x, stats, weight=None, dw=None, db=None, out=None):
    """The gradients of layer_norm_forward: dx (of x's type, a new tensor or in `out`,
    which may be dy or x), dw and db.

    dw and db are float32, new tensors, or added to the tensors given, in place (which
    must not overlap each other, nor the weight).  Without a weight, and without dw and
    db to add to, both are None."""
    import torch
    rows, cols, ldx, kind = _tokens("x", x)
    lddy = _like("dy", dy, x)
    w, _, w_type = _params(weight, None, cols, x)
    if tuple(stats.shape) != (3, rows) or stats.dtype != torch.float32 or not stats.is_contiguous():
        raise ValueError(f"stats are {tuple(stats.shape)} {stats.dtype}, not {(3, rows)} torch.float32, contiguous")
    given = dw is not None, db is not None
    if given[0] != given[1] and weight is not None:
        raise ValueError("dw and db to add to are given both or neither")
    for name, v in (("dw", dw), ("db", db)):
        if v is not None:
            _vector(name, v, cols, torch.float32)
    _same_device(x, dy, stats, weight, dw, db, out)
    device = x.device
    add = any(given)
    if weight is not None and not add:
        dw, db = (torch.empty(cols, dtype=torch.float32, device=device) for _ in range(2))
    if out is None:
        dx, lddx = torch.empty((rows, cols), dtype=x.dtype, device=device), max(cols, 1)
    else:
        dx, lddx = out, _like("out", out, x)
    bytes = _workspace_bytes(rows, cols) if dw is not None or db is not None else 0
    workspace = torch.empty(bytes, dtype=torch.uint8, device=device) if bytes else None
    _call(device, load().hip_layernorm_backward, hip_layernorm_backward_status_string, rows, cols, kind, dy.data_ptr(), lddy,
          x.data_ptr(), ldx, stats.data_ptr(), w, w_type, dx.data_ptr(), lddx,
          dw.data_ptr() if dw is not None else None, db.data_ptr() if db is not None else None, int(add),
          workspace.data_ptr() if bytes else None, bytes)
    for t, there in ((out, out is not None), (dw, given[0]), (db, given[1])):
        if there:
            written(t)
    return dx, dw, db
