"""8-bit block-scaled products (ctypes binding of include/blockfp8.h): the
quantiser, the product, and a linear layer's forward and backward made of them.

hip_fp8_quantize and hip_fp8_gemm carry the C ABI's names and argument order
and return its status codes; matrix and stream arguments are as in `sgemm`.
quantize, quantize_transposed, quantize_both, gemm, linear_forward and
linear_backward take and return torch device tensors, run on torch's current
stream of the tensors' device and raise on errors.  Every operation runs in the
library's HIP kernels; there is no fallback.

Results carry no autograd graph, also those of tensors that require gradients:
a layer's gradients are linear_backward's.  A tensor that is written in place
(out, dw) counts as modified for autograd.
"""

from __future__ import annotations

import ctypes
import dataclasses
from typing import Tuple

from . import sgemm as _sgemm

EXPORTS = ("hip_fp8_quantize", "hip_fp8_gemm", "hip_fp8_gemm_plan", "hip_fp8_quantize_status_string",
           "hip_fp8_gemm_status_string")

F32, BF16, F16 = 0, 1, 2
SCALE_F32, SCALE_E8M0 = 0, 1
BLOCK = 128
MAX_LD = 1 << 23
MAX_LAUNCHES = 3  # HIP_FP8_GEMM_MAX_LAUNCHES

class _Launch(ctypes.Structure):
    """hip_fp8_gemm_launch."""
    _fields_ = [(name, ctypes.c_int) for name in ("tile_m", "tile_n", "row0", "col0", "rows", "cols", "skip_rows",
                                                  "skip_cols", "threads")] + [("workgroups", ctypes.c_longlong)]


_bound = None


def load():
    """The library with this header's functions declared."""
    global _bound
    lib = _sgemm.load()
    if lib is not _bound:
        i32, i64, f32, vp = ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_void_p
        lib.hip_fp8_quantize.restype = i32
        lib.hip_fp8_quantize.argtypes = [i32, i32, vp, i32, i32, i32, i32, vp, i32, vp, i64, i64,
                                         vp, i32, vp, i64, i64, vp]
        lib.hip_fp8_gemm.restype = i32
        lib.hip_fp8_gemm.argtypes = [i32, i32, i32, f32, vp, i32, vp, i64, i64, i32,
                                     vp, i32, vp, i64, i64, i32, i32, f32, vp, i32, vp, i32, i32, vp]
        lib.hip_fp8_gemm_plan.restype = i32
        lib.hip_fp8_gemm_plan.argtypes = [i32, i32, i32, i32, ctypes.POINTER(_Launch), ctypes.POINTER(i32)]
        for name in ("hip_fp8_quantize_status_string", "hip_fp8_gemm_status_string"):
            getattr(lib, name).restype = ctypes.c_char_p
            getattr(lib, name).argtypes = [i32]
        _bound = lib
    return lib


def hip_fp8_quantize(rows, cols, X, x_type, ldx, block_rows, scale_type, Q, ldq, S, s_row, s_col,
                     QT, ldqt, ST, st_row, st_col, stream=None) -> int:
    """Codes and scales of X and / or of its transpose; returns the status code (0 = enqueued)."""
    a, s = _sgemm._addr, _sgemm._stream
    return int(load().hip_fp8_quantize(int(rows), int(cols), a(X), int(x_type), int(ldx), int(block_rows),
                                       int(scale_type), a(Q), int(ldq), a(S), int(s_row), int(s_col),
                                       a(QT), int(ldqt), a(ST), int(st_row), int(st_col), s(stream)))


def hip_fp8_gemm(M, N, K, alpha, A, lda, SA, sa_row, sa_col, a_block_rows, B, ldb, SB, sb_row, sb_col,
                 b_block_rows, scale_type, beta, C, ldc, D, ldd, c_type, stream=None) -> int:
    """D <- alpha*A@B^T + beta*C of quantised A and B; returns the status code."""
    a, s = _sgemm._addr, _sgemm._stream
    return int(load().hip_fp8_gemm(int(M), int(N), int(K), float(alpha), a(A), int(lda), a(SA), int(sa_row),
                                   int(sa_col), int(a_block_rows), a(B), int(ldb), a(SB), int(sb_row),
                                   int(sb_col), int(b_block_rows), int(scale_type), float(beta), a(C),
                                   int(ldc), a(D), int(ldd), int(c_type), s(stream)))


def hip_fp8_gemm_plan(M, N, K, c_type) -> list:
    """What hip_fp8_gemm enqueues for a shape, a dict a launch (nothing is launched)."""
    launches, count = (_Launch * MAX_LAUNCHES)(), ctypes.c_int()
    rc = load().hip_fp8_gemm_plan(int(M), int(N), int(K), int(c_type), launches, ctypes.byref(count))
    if rc != 0:
        raise _sgemm.SgemmError(rc, hip_fp8_gemm_status_string(rc))
    return [{name: getattr(launch, name) for name, _ in _Launch._fields_} for launch in launches[:count.value]]


def hip_fp8_quantize_status_string(status) -> str:
    return load().hip_fp8_quantize_status_string(int(status)).decode()


def hip_fp8_gemm_status_string(status) -> str:
    return load().hip_fp8_gemm_status_string(int(status)).decode()


@dataclasses.dataclass(frozen=True)
class BlockFp8:
    """A quantised matrix: q, its e4m3 codes (rows x cols, columns side by
    side), and s, a scale for each block of block_rows x 128 (float32, or
    float8_e8m0fnu for powers of two)."""

    q: "torch.Tensor"  # noqa: F821
    s: "torch.Tensor"  # noqa: F821
    block_rows: int = 1

    @property
    def shape(self):
        return self.q.shape


_TYPES = None    # of matrices that are not quantised
_SCALES = None
_CODES = None    # of quantised ones


def _tables():
    """The type codes by torch's dtypes, and the dtypes of codes (torch is imported on first use)."""
    global _TYPES, _SCALES, _CODES
    if _TYPES is None:
        import torch
        _SCALES = {torch.float32: SCALE_F32, torch.float8_e8m0fnu: SCALE_E8M0}
        _CODES = (torch.float8_e4m3fn, torch.uint8)
        _TYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
    return _TYPES, _SCALES, _CODES


def _types():
    return _tables()[0]


def _scale_type(dtype) -> int:
    kind = _tables()[1].get(dtype)
    if kind is None:
        raise TypeError(f"scales are float32 or float8_e8m0fnu, not {dtype}")
    return kind


def _ceil(a, b):
    return -(-a // b)


def _matrix(name, t):
    """(rows, columns, row stride) of a 2-D view whose columns lie side by side."""
    if not t.is_cuda:
        raise TypeError(f"{name} must live on the GPU")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D row-major view with unit column stride")
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and cols > 1 and rows > 0:
        raise ValueError(f"{name} must be a 2-D row-major view with unit column stride")
    if rows >= 1 << 31 or cols >= 1 << 31:
        raise ValueError(f"{name} has a side of 2^31 or more")
    if rows <= 1:
        return rows, cols, max(cols, 1)
    if ld < cols:
        raise ValueError(f"{name}'s rows overlap")
    if ld >= 1 << 31:
        raise ValueError(f"{name}'s row stride is 2^31 or more")
    return rows, cols, max(ld, 1)


def _same_device(first, *others):
    device = first.get_device()
    for t in others:
        if t is not None and t.get_device() != device:
            raise ValueError(f"tensors on {first.device} and {t.device}")


def current_stream(index: int) -> int:
    """The handle of torch's current stream of a device (what
    torch.cuda.current_stream(index).cuda_stream is, in a twelfth of its 1.1 us
    where torch has the short way)."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _call(device, function, what, *args):
    """The C function with torch's current stream of the device as its last
    argument, the device current; raises on errors."""
    import torch
    index = device.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _call(device, function, what, *args)
    status = function(*args, current_stream(index))
    if status != 0:
        raise _sgemm.SgemmError(status, what(status))


def written(t):
    """Tells autograd that t has been written to, as torch's own in-place operations
    do, so that a graph that saved it notices."""
    import torch
    if not t.is_inference():  # these have no version to advance
        torch.autograd.graph.increment_version(t)


def _empty(rows, cols, block_rows, scale, device):
    """Room for a quantised matrix: rows of a multiple of 16 bytes, the scales
    of one block column side by side.  And the row stride."""
    import torch
    ld = max(_ceil(cols, 16) * 16, 16)
    if ld >= 1 << 31:  # more than a stride can be, and than a product takes
        ld = cols
    q = torch.empty((rows, ld), dtype=torch.float8_e4m3fn, device=device)
    if ld != cols:
        q = q[:, :cols]
    r = _ceil(rows, block_rows)
    return BlockFp8(q, torch.empty_strided((r, _ceil(cols, BLOCK)), (1, r), dtype=scale, device=device), block_rows), ld


def _quantize(x, block_rows, scale, as_is, transposed):
    import torch
    rows, cols, ldx = _matrix("x", x)
    x_type = _types().get(x.dtype)
    if x_type is None:
        raise TypeError(f"x is float32, bfloat16 or float16, not {x.dtype}")
    if block_rows not in (1, BLOCK):
        raise ValueError(f"block_rows is 1 or 128, not {block_rows}")
    scale = torch.float32 if scale is None else scale
    kind = _scale_type(scale)
    device = x.device
    n, ldn = _empty(rows, cols, block_rows, scale, device) if as_is else (None, 0)
    t, ldt = _empty(cols, rows, block_rows, scale, device) if transposed else (None, 0)
    if rows and cols:
        args = []
        for o, ld in ((n, ldn), (t, ldt)):
            args += [o.q.data_ptr(), ld, o.s.data_ptr(), *o.s.stride()] if o is not None else [None, 0, None, 0, 0]
        _call(device, load().hip_fp8_quantize, hip_fp8_quantize_status_string,
              rows, cols, x.data_ptr(), x_type, ldx, block_rows, kind, *args)
    return n, t


def quantize(x, block_rows: int = 1, scale=None) -> BlockFp8:
    """x (2-D, rows may be strided) in blocks of block_rows x 128; `scale` is
    torch.float32 (default) or torch.float8_e8m0fnu."""
    return _quantize(x, block_rows, scale, True, False)[0]


def quantize_transposed(x, block_rows: int = 1, scale=None) -> BlockFp8:
    """x's transpose, in blocks of block_rows x 128 of the transpose."""
    return _quantize(x, block_rows, scale, False, True)[1]


def quantize_both(x, block_rows: int = 1, scale=None) -> Tuple[BlockFp8, BlockFp8]:
    """quantize(x) and quantize_transposed(x) from one read of x."""
    return _quantize(x, block_rows, scale, True, True)


def _operand(name, o):
    """(rows, K, the C function's arguments) of a quantised matrix."""
    q, s, block_rows = o.q, o.s, o.block_rows
    rows, K, ld = _matrix(name, q)
    if q.dtype not in _tables()[2]:
        raise TypeError(f"{name}'s codes are float8_e4m3fn (or its bytes as uint8), not {q.dtype}")
    if rows <= 1 or K == 0:
        ld = max(_ceil(ld, 16) * 16, 16)
    if block_rows not in (1, BLOCK):
        raise ValueError(f"{name}'s block_rows is 1 or 128, not {block_rows}")
    if tuple(s.shape) != (_ceil(rows, block_rows), _ceil(K, BLOCK)):
        raise ValueError(f"{name}'s scales are {tuple(s.shape)}, not {(_ceil(rows, block_rows), _ceil(K, BLOCK))}")
    if not s.is_cuda:
        raise TypeError(f"{name}'s scales must live on the GPU")
    if K % 16 and rows and ld % 16 == 0:  # the last row is read up to a multiple of 16 bytes
        if q.storage_offset() + (rows - 1) * ld + _ceil(K, 16) * 16 > q.untyped_storage().nbytes():
            raise ValueError(f"{name}'s storage ends within the last row's padding to a multiple of 16 bytes")
    return rows, K, (q.data_ptr(), ld, s.data_ptr(), *s.stride(), block_rows)


def gemm(a: BlockFp8, b: BlockFp8, c=None, alpha: float = 1.0, beta: float = 0.0, out=None, out_dtype=None):
    """alpha * a @ b^T + beta * c as a new tensor, or in `out` (which may be c).

    The result's type is out's, c's, or out_dtype (default bfloat16).  The sums of
    a 16-bit result cut products 13 bits below the largest of eight neighbours;
    who wants a float's sums takes a float32 result and rounds it."""
    import torch
    M, K, left = _operand("a", a)
    N, L, right = _operand("b", b)
    if L != K:
        raise ValueError(f"shape mismatch: a {(M, K)}, b {(N, L)}")
    scale = a.s.dtype
    if scale != b.s.dtype:
        raise TypeError(f"scales of two types: {scale} and {b.s.dtype}")
    kind = _scale_type(scale)
    if beta == 0.0:
        c = None
    elif c is None:
        raise ValueError("beta is not 0 but there is no c")
    dtype = out.dtype if out is not None else c.dtype if c is not None else out_dtype or torch.bfloat16
    c_type = _types().get(dtype)
    if c_type is None:
        raise TypeError(f"the result is float32, bfloat16 or float16, not {dtype}")
    if out_dtype is not None and out_dtype != dtype:
        raise TypeError(f"out_dtype is {out_dtype}, but the result is {dtype}")
    for name, t in (("c", c), ("out", out)):
        if t is not None and (tuple(t.shape) != (M, N) or t.dtype != dtype):
            raise ValueError(f"{name} is {tuple(t.shape)} {t.dtype}, not {(M, N)} {dtype}")
    _same_device(a.q, a.s, b.q, b.s, c, out)
    device = a.q.device
    new = out is None
    if new:
        out = torch.empty((M, N), dtype=dtype, device=device)
        ldd = max(N, 1)
    else:
        ldd = _matrix("out", out)[2]
    from_c, ldc = (c.data_ptr(), _matrix("c", c)[2]) if c is not None else (None, 0)
    _call(device, load().hip_fp8_gemm, hip_fp8_gemm_status_string, M, N, K, alpha, *left, *right, kind, beta,
          from_c, ldc, out.data_ptr(), ldd, c_type)
    if not new:
        written(out)
    return out


def linear_forward(x, w: BlockFp8, out_dtype=None):
    """y = x w^T of tokens x (T x I) and a quantised weight w (O x I).

    Returns y (T x O, of x's type by default) and x^T quantised (I x T), which
    linear_backward takes.  x is read once."""
    xq, xt = quantize_both(x, 1, w.s.dtype)
    return gemm(xq, w, out_dtype=out_dtype or x.dtype), xt


def linear_backward(dy, xt: BlockFp8, wt: BlockFp8, dw=None, out_dtype=None):
    """The gradients of linear_forward: dx = dy w (T x I) and dw = dy^T x (O x I).

    dy: T x O; xt: x^T as linear_forward returned it; wt: w^T quantised (I x O).
    dx has dy's type by default.  dw is float32, a new tensor, or added to the
    tensor given, in place (float32 too: sums that grow over many calls lose what
    a 16-bit type cuts off in each)."""
    import torch
    if dw is not None and dw.dtype != torch.float32:
        raise TypeError(f"dw is float32, not {dw.dtype}")
    dyq, dyt = quantize_both(dy, 1, wt.s.dtype)
    dx = gemm(dyq, wt, out_dtype=out_dtype or dy.dtype)
    if dw is None:
        return dx, gemm(dyt, xt, out_dtype=torch.float32)
    return dx, gemm(dyt, xt, c=dw, beta=1.0, out=dw)
