"""The global norm of many gradients, and clipping by it (ctypes binding of
include/gradients.h).

hip_gradient_norm, hip_gradient_clip and hip_gradient_clip_by carry the C ABI's names
and argument order and return its status codes; their tensors are a ctypes array of
hip_gradient.  grad_norm, clip_grad_norm and clip_by_norm take and return torch
device tensors, run on torch's current stream of the tensors' device and raise on
errors.  Every operation runs in the library's HIP kernels; there is no fallback.
Results carry no autograd graph; tensors that are written in place count as modified
for autograd.
"""

from __future__ import annotations

import array
import ctypes
import operator

from . import sgemm as _sgemm
from .blockfp8 import _call, _types, written

EXPORTS = ("hip_gradient_norm", "hip_gradient_clip", "hip_gradient_clip_by", "hip_gradient_workspace",
           "hip_gradient_norm_status_string", "hip_gradient_clip_status_string")

F32, BF16, F16 = 0, 1, 2
MAX_COUNT = 1 << 20  # HIP_GRADIENT_MAX_COUNT


class Gradient(ctypes.Structure):
    """hip_gradient."""
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p)] + [(name, ctypes.c_longlong) for name in (
        "rows", "cols", "ldx", "ldy", "type")]


_bound = None


def load():
    """The library with this header's functions declared."""
    global _bound
    lib = _sgemm.load()
    if lib is not _bound:
        i32, i64, f64, vp = ctypes.c_int, ctypes.c_longlong, ctypes.c_double, ctypes.c_void_p
        lib.hip_gradient_norm.restype = i32
        lib.hip_gradient_norm.argtypes = [i32, vp, vp, vp, i64, vp]
        for name in ("hip_gradient_clip", "hip_gradient_clip_by"):
            getattr(lib, name).restype = i32
            getattr(lib, name).argtypes = [i32, vp, f64, f64, vp, vp, i64, vp]
        lib.hip_gradient_workspace.restype = i32
        lib.hip_gradient_workspace.argtypes = [i32, ctypes.POINTER(i64)]
        for name in EXPORTS[-2:]:
            getattr(lib, name).restype = ctypes.c_char_p
            getattr(lib, name).argtypes = [i32]
        _bound = lib
    return lib


def hip_gradient_norm(count, tensors, norm, workspace, workspace_bytes, stream=None) -> int:
    """norm <- the tensors' norm; returns the status code (0 = enqueued)."""
    a, s = _sgemm._addr, _sgemm._stream
    return int(load().hip_gradient_norm(int(count), tensors, a(norm), a(workspace), int(workspace_bytes), s(stream)))


def hip_gradient_clip(count, tensors, max_norm, eps, norm, workspace, workspace_bytes, stream=None) -> int:
    """norm <- the tensors' norm, y <- c x; returns the status code."""
    a, s = _sgemm._addr, _sgemm._stream
    return int(load().hip_gradient_clip(int(count), tensors, float(max_norm), float(eps), a(norm), a(workspace),
                                        int(workspace_bytes), s(stream)))


def hip_gradient_clip_by(count, tensors, max_norm, eps, norm, workspace, workspace_bytes, stream=None) -> int:
    """y <- c x by the norm given; returns the status code."""
    a, s = _sgemm._addr, _sgemm._stream
    return int(load().hip_gradient_clip_by(int(count), tensors, float(max_norm), float(eps), a(norm), a(workspace),
                                           int(workspace_bytes), s(stream)))


def hip_gradient_workspace(count) -> int:
    """Bytes of workspace of a call (nothing is launched)."""
    out = ctypes.c_longlong()
    rc = load().hip_gradient_workspace(int(count), ctypes.byref(out))
    if rc != 0:
        raise _sgemm.SgemmError(rc, hip_gradient_norm_status_string(rc))
    return out.value


def hip_gradient_norm_status_string(status) -> str:
    return load().hip_gradient_norm_status_string(int(status)).decode()


def hip_gradient_clip_status_string(status) -> str:
    return load().hip_gradient_clip_status_string(int(status)).decode()


def _layout(t, what):
    """(rows, cols, row stride) of a tensor that is rows of neighbours at one stride."""
    sizes = [(n, s) for n, s in zip(t.shape, t.stride()) if n != 1]
    sizes.sort(key=lambda e: -e[1])  # any order of the dimensions: every element once is all that counts
    cols = 1
    while sizes and sizes[-1][1] == cols:
        cols *= sizes.pop()[0]
    if not sizes:
        return 1, cols, cols
    rows, ld = sizes.pop()
    while sizes and sizes[-1][1] == ld * rows:
        rows *= sizes.pop()[0]
    if sizes or ld < cols:
        raise ValueError(f"{what} of sizes {tuple(t.shape)} and strides {t.stride()} is not dense, nor rows of neighbours "
                         "at one stride")
    return rows, cols, ld


def _describe(tensors, outs):
    """(device, an array with seven numbers a tensor, as hip_gradient has them)."""
    from torch import Tensor
    types = _types()
    try:
        kinds = [types.get(t.dtype) for t in tensors]
    except AttributeError:  # the gradient of a parameter that has none, as a rule
        other = next(t for t in tensors if not isinstance(t, Tensor))
        raise TypeError(f"gradients are tensors, not {type(other).__name__}") from None
    device = tensors[0].device
    index = tensors[0].get_device()
    if index < 0:
        raise TypeError("gradients must live on the GPU")
    if None in kinds:
        raise TypeError(f"gradients are float32, bfloat16 or float16, not {tensors[kinds.index(None)].dtype}")
    places = list(map(Tensor.get_device, tensors))
    if places.count(index) != len(places):
        raise ValueError(f"tensors on {device} and {next(t for t, at in zip(tensors, places) if at != index).device}")
    if outs is not None:
        for t, o in zip(tensors, outs):
            if o.shape != t.shape or o.dtype != t.dtype:
                raise ValueError(f"out is {tuple(o.shape)} {o.dtype}, not {tuple(t.shape)} {t.dtype}")
            if o.get_device() != index:
                raise ValueError(f"tensors on {device} and {o.device}")
    n = len(tensors)
    x = array.array("q", map(Tensor.data_ptr, tensors))
    out = array.array("q", bytes(56 * n))
    out[0::7] = x
    out[1::7] = x if outs is None else array.array("q", map(Tensor.data_ptr, outs))
    out[2::7] = array.array("q", [1]) * n
    out[3::7] = array.array("q", map(Tensor.numel, tensors))
    out[6::7] = array.array("q", kinds)
    dense = list(map(Tensor.is_contiguous, tensors))
    if outs is not None:
        dense = list(map(operator.and_, dense, map(Tensor.is_contiguous, outs)))
    if False in dense:  # rows, columns and strides of the others
        for i in (i for i, flat in enumerate(dense) if not flat):
            t, o = tensors[i], None if outs is None else outs[i]
            if t.numel():
                rows, cols, ldx, ldy = _pair(t, t if o is None else o)
                out[7 * i + 2:7 * i + 6] = array.array("q", (rows, cols, ldx, ldy))
    return device, out


def _pair(t, o):
    """(rows, cols, strides of both) of a gradient and another tensor for its result."""
    if t.stride() == o.stride():
        rows, cols, ld = _layout(t, "a gradient")
        return rows, cols, ld, ld
    # elements correspond by their places in both: the dimensions in the gradient's order
    order = sorted((d for d in range(t.dim()) if t.shape[d] != 1), key=lambda d: -t.stride(d))
    shape = [t.shape[d] for d in order]
    if t.stride(order[-1]) != 1 or o.stride(order[-1]) != 1:
        shape.append(1)  # rows of one element
    cols, strides = shape[-1], []
    for v in (t, o):
        outer = [(v.shape[d], v.stride(d)) for d in order][:len(shape) - 1]
        ld = outer[-1][1] if outer else cols
        if any(s != n * r for (_, s), (n, r) in zip(outer, outer[1:])) or ld < cols:
            raise ValueError(f"a gradient and its out, of strides {t.stride()} and {o.stride()}, are not rows of neighbours "
                             "in one order, each at one stride")
        strides.append(ld)
    return t.numel() // cols, cols, *strides


def _workspace_bytes(count) -> int:
    """hip_gradient_workspace without a call."""
    return 16384 + (64 * count if count > 60 else 0)


def _run(function, what, device, described, *args):
    """A call with the tensors, a workspace and torch's current stream."""
    import torch
    count = len(described) // 7
    bytes = _workspace_bytes(count)
    workspace = torch.empty(bytes, dtype=torch.uint8, device=device)
    _call(device, function, what, count, described.buffer_info()[0], *args, workspace.data_ptr(), bytes)


def _outs(tensors, out):
    """(where the results go, those of them that count as modified)."""
    import torch
    if out is None:
        new = [torch.empty_like(t) for t in tensors]
        return new, ()
    out = tensors if out is tensors else list(out)
    if len(out) != len(tensors):
        raise ValueError(f"{len(out)} tensors in out, {len(tensors)} gradients")
    return out, out


def _written(tensors):
    import torch
    if not tensors:
        return
    try:
        torch.autograd.graph.increment_version(tensors)
    except RuntimeError:  # inference tensors have no version to advance
        for t in tensors:
            written(t)


def _list(tensors):
    tensors = tensors if isinstance(tensors, list) else list(tensors)
    if len(tensors) > MAX_COUNT:
        raise ValueError(f"{len(tensors)} tensors, at most {MAX_COUNT}")
    return tensors


def _limits(max_norm, eps):
    if not max_norm >= 0:
        raise ValueError(f"max_norm is {max_norm}, not 0 or more")
    if not 0 <= eps < float("inf"):
        raise ValueError(f"eps is {eps}, not 0 or more")


def grad_norm(tensors):
    """The 2-norm of all elements of the tensors (any shapes, dense or rows of
    neighbours at one stride, float32, bfloat16 and float16 mixed, one device), as a
    0-dimensional float32 tensor.  A tensor that is given twice counts twice."""
    import torch
    tensors = _list(tensors)
    if not tensors:
        raise ValueError("no tensors")
    device, described = _describe(tensors, None)
    norm = torch.empty((), dtype=torch.float32, device=device)
    _run(load().hip_gradient_norm, hip_gradient_norm_status_string, device, described, norm.data_ptr())
    return norm


def clip_grad_norm(tensors, max_norm: float, eps: float = 1e-6, out=None):
    """(the norm, as grad_norm gives it, and the tensors times min(1, max_norm / (norm +
    eps))).  The results are new tensors, or `out`'s: as many tensors of the same shapes
    and types, which may be the gradients themselves (`out=tensors` clips in place, and
    writes nothing while the norm is within the limit).  No two of the results may share
    memory, nor one with another's gradient: such a call is refused."""
    import torch
    tensors = _list(tensors)
    _limits(max_norm, eps)
    if not tensors:
        raise ValueError("no tensors")
    outs, modified = _outs(tensors, out)
    device, described = _describe(tensors, None if outs is tensors else outs)
    norm = torch.empty((), dtype=torch.float32, device=device)
    _run(load().hip_gradient_clip, hip_gradient_clip_status_string, device, described, max_norm, eps, norm.data_ptr())
    _written(modified)
    return norm, outs


def clip_by_norm(tensors, norm, max_norm: float, eps: float = 1e-6, out=None):
    """clip_grad_norm's tensors by a norm that is there (one float32 number on the
    tensors' device): grad_norm's, or the root of several ranks' summed squares."""
    import torch
    tensors = _list(tensors)
    _limits(max_norm, eps)
    if not tensors:
        raise ValueError("no tensors")
    if norm.dtype != torch.float32 or norm.numel() != 1:
        raise ValueError(f"norm is {tuple(norm.shape)} {norm.dtype}, not one torch.float32")
    outs, modified = _outs(tensors, out)
    device, described = _describe(tensors, None if outs is tensors else outs)
    if norm.device != device:
        raise ValueError(f"tensors on {device} and {norm.device}")
    _run(load().hip_gradient_clip_by, hip_gradient_clip_status_string, device, described, max_norm, eps, norm.data_ptr())
    _written(modified)
    return outs
