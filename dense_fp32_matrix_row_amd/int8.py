"""Products of 8-bit integers with a scale for each token and each channel (ctypes
binding of include/int8.h): the quantiser, the product, and a linear layer as it
is served, made of both.

hip_int8_quantize, hip_int8_gemm and hip_int8_linear carry the C ABI's names and
argument order and return its status codes; matrix and stream arguments are as in
`sgemm`.  quantize, gemm and linear take and return torch device tensors, run on
torch's current stream of the tensors' device and raise on errors.  Every
operation runs in the library's HIP kernels; there is no fallback.  Results carry
no autograd graph; an `out` counts as modified for autograd.
"""

from __future__ import annotations

import ctypes
import dataclasses

from . import sgemm as _sgemm
from .blockfp8 import _call, _matrix, _same_device, _types, written

EXPORTS = ("hip_int8_quantize", "hip_int8_gemm", "hip_int8_gemm_plan", "hip_int8_linear", "hip_int8_linear_workspace",
           "hip_int8_quantize_status_string", "hip_int8_gemm_status_string", "hip_int8_linear_status_string")

F32, BF16, F16 = 0, 1, 2
MAX_K = 131071   # HIP_INT8_MAX_K
MAX_LD = 1 << 23
MAX_LAUNCHES = 3  # HIP_INT8_GEMM_MAX_LAUNCHES
AMAX_FLOOR = 2.0 ** -100


class _Launch(ctypes.Structure):
    """hip_int8_gemm_launch."""
    _fields_ = [(name, ctypes.c_int) for name in ("tile_m", "tile_n", "row0", "col0", "rows", "cols", "skip_rows",
                                                  "skip_cols", "threads")] + [("workgroups", ctypes.c_longlong)]


_bound = None


def load():
    """The library with this header's functions declared."""
    global _bound
    lib = _sgemm.load()
    if lib is not _bound:
        i32, i64, vp = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p
        lib.hip_int8_quantize.restype = i32
        lib.hip_int8_quantize.argtypes = [i32, i32, vp, i32, i32, vp, i32, vp, vp]
        lib.hip_int8_gemm.restype = i32
        lib.hip_int8_gemm.argtypes = [i32, i32, i32, vp, i32, vp, i64, vp, i32, vp, i64, vp, i32, vp, i32, i32, vp]
        lib.hip_int8_gemm_plan.restype = i32
        lib.hip_int8_gemm_plan.argtypes = [i32, i32, i32, ctypes.POINTER(_Launch), ctypes.POINTER(i32)]
        lib.hip_int8_linear.restype = i32
        lib.hip_int8_linear.argtypes = [i32, i32, i32, vp, i32, i32, vp, i32, vp, i64, vp, i32, vp, i32, i32, vp, i64, vp]
        lib.hip_int8_linear_workspace.restype = i32
        lib.hip_int8_linear_workspace.argtypes = [i32, i32, ctypes.POINTER(i64)]
        for name in EXPORTS[-3:]:
            getattr(lib, name).restype = ctypes.c_char_p
            getattr(lib, name).argtypes = [i32]
        _bound = lib
    return lib


def hip_int8_quantize(rows, cols, X, x_type, ldx, Q, ldq, S, stream=None) -> int:
    """Codes and scales of X's rows; returns the status code (0 = enqueued)."""
    a, s = _sgemm._addr, _sgemm._stream
    return int(load().hip_int8_quantize(int(rows), int(cols), a(X), int(x_type), int(ldx), a(Q), int(ldq), a(S), s(stream)))


def hip_int8_gemm(M, N, K, A, lda, SA, sa_inc, B, ldb, SB, sb_inc, bias, bias_type, D, ldd, d_type, stream=None) -> int:
    """D <- A@B^T + bias of quantised A and B; returns the status code."""
    a, s = _sgemm._addr, _sgemm._stream
    return int(load().hip_int8_gemm(int(M), int(N), int(K), a(A), int(lda), a(SA), int(sa_inc), a(B), int(ldb), a(SB),
                                    int(sb_inc), a(bias), int(bias_type), a(D), int(ldd), int(d_type), s(stream)))


def hip_int8_gemm_plan(M, N, K) -> list:
    """What hip_int8_gemm enqueues for a shape, a dict a launch (nothing is launched)."""
    launches, count = (_Launch * MAX_LAUNCHES)(), ctypes.c_int()
    rc = load().hip_int8_gemm_plan(int(M), int(N), int(K), launches, ctypes.byref(count))
    if rc != 0:
        raise _sgemm.SgemmError(rc, hip_int8_gemm_status_string(rc))
    return [{name: getattr(launch, name) for name, _ in _Launch._fields_} for launch in launches[:count.value]]


def hip_int8_linear(tokens, inputs, outputs, X, x_type, ldx, W, ldw, SW, sw_inc, bias, bias_type, Y, ldy, y_type,
                    workspace, workspace_bytes, stream=None) -> int:
    """Y <- X@W^T + bias, X quantised on the way; returns the status code."""
    a, s = _sgemm._addr, _sgemm._stream
    return int(load().hip_int8_linear(int(tokens), int(inputs), int(outputs), a(X), int(x_type), int(ldx), a(W), int(ldw),
                                      a(SW), int(sw_inc), a(bias), int(bias_type), a(Y), int(ldy), int(y_type),
                                      a(workspace), int(workspace_bytes), s(stream)))


def hip_int8_linear_workspace(tokens, inputs) -> int:
    """Bytes of workspace of a call (nothing is launched)."""
    out = ctypes.c_longlong()
    rc = load().hip_int8_linear_workspace(int(tokens), int(inputs), ctypes.byref(out))
    if rc != 0:
        raise _sgemm.SgemmError(rc, hip_int8_linear_status_string(rc))
    return out.value


def hip_int8_quantize_status_string(status) -> str:
    return load().hip_int8_quantize_status_string(int(status)).decode()


def hip_int8_gemm_status_string(status) -> str:
    return load().hip_int8_gemm_status_string(int(status)).decode()


def hip_int8_linear_status_string(status) -> str:
    return load().hip_int8_linear_status_string(int(status)).decode()


@dataclasses.dataclass(frozen=True)
class Int8:
    """A quantised matrix: q, its codes (rows x cols, int8, columns side by side,
    rows of a multiple of 16 bytes for a product, best of 128), and s, a float32 scale
    for each row."""

    q: "torch.Tensor"  # noqa: F821
    s: "torch.Tensor"  # noqa: F821

    @property
    def shape(self):
        return self.q.shape


def _type(name, dtype) -> int:
    kind = _types().get(dtype)
    if kind is None:
        raise TypeError(f"{name} is float32, bfloat16 or float16, not {dtype}")
    return kind


def _stride(K) -> int:
    """What a product reads of a row, in bytes."""
    return max(-(-K // 16) * 16, 16)


def _row(K) -> int:
    """The rows that quantize makes, in bytes: long ones in whole cache lines, of which
    a product's loads then take one each (4096 x 4096 x 4097 70 -> 62 us)."""
    return -(-K // 128) * 128 if K >= 512 else _stride(K)


def quantize(x) -> Int8:
    """x (2-D, rows may be strided) with a scale for each row."""
    import torch
    rows, cols, ldx = _matrix("x", x)
    x_type = _type("x", x.dtype)
    device = x.device
    ld = _row(cols)
    if ld >= 1 << 31:  # more than a stride can be, and than a product takes
        ld = cols
    q = torch.empty((rows, ld), dtype=torch.int8, device=device)
    if ld != cols:
        q = q[:, :cols]
    s = torch.empty(rows, dtype=torch.float32, device=device)
    if cols:
        _call(device, load().hip_int8_quantize, hip_int8_quantize_status_string,
              rows, cols, x.data_ptr(), x_type, ldx, q.data_ptr(), ld, s.data_ptr())
    else:  # what a row of zeros has
        s.fill_(AMAX_FLOOR / 127)
    return Int8(q, s)


_kinds = None  # int8, float32 (torch is imported on first use)


def _operand(name, o):
    """(rows, K, the C function's arguments) of a quantised matrix."""
    global _kinds
    if _kinds is None:
        import torch
        _kinds = torch.int8, torch.float32
    q, s = o.q, o.s
    rows, K, ld = _matrix(name, q)
    if q.dtype != _kinds[0]:
        raise TypeError(f"{name}'s codes are int8, not {q.dtype}")
    if s.dtype != _kinds[1]:
        raise TypeError(f"{name}'s scales are float32, not {s.dtype}")
    if not s.is_cuda:
        raise TypeError(f"{name}'s scales must live on the GPU")
    if s.dim() != 1 or s.shape[0] != rows:
        raise ValueError(f"{name}'s scales are {tuple(s.shape)}, not {(rows,)}")
    if rows <= 1 or K == 0:
        ld = _stride(max(K, ld))
    if K % 16 and rows and ld % 16 == 0:  # the last row is read up to a multiple of 16 bytes
        if q.storage_offset() + (rows - 1) * ld + _stride(K) > q.untyped_storage().nbytes():
            raise ValueError(f"{name}'s storage ends within the last row's padding to a multiple of 16 bytes")
    return rows, K, (q.data_ptr(), ld, s.data_ptr(), s.stride(0) if rows > 1 else 1)


def _bias(bias, N):
    """(address, type) of a bias, or of none."""
    if bias is None:
        return None, 0
    if not bias.is_cuda:
        raise TypeError("bias must live on the GPU")
    kind = _type("bias", bias.dtype)
    if tuple(bias.shape) != (N,):
        raise ValueError(f"bias is {tuple(bias.shape)}, not {(N,)}")
    if N > 1 and bias.stride(0) != 1:
        raise ValueError("bias must be contiguous")
    return bias.data_ptr(), kind


def _result(out, out_dtype, default, M, N, device):
    """(result, its type, row stride): `out`, or a new tensor."""
    import torch
    dtype = out.dtype if out is not None else out_dtype or default
    kind = _type("the result", dtype)
    if out is None:
        return torch.empty((M, N), dtype=dtype, device=device), kind, max(N, 1)
    if out_dtype is not None and out_dtype != dtype:
        raise TypeError(f"out_dtype is {out_dtype}, but the result is {dtype}")
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out is {tuple(out.shape)}, not {(M, N)}")
    return out, kind, _matrix("out", out)[2]


def gemm(a: Int8, b: Int8, bias=None, out=None, out_dtype=None):
    """a @ b^T (+ bias, a number for each column) as a new tensor, or in `out`, which
    must not overlap the operands.  The result's type is out's, or out_dtype
    (default bfloat16)."""
    import torch
    M, K, left = _operand("a", a)
    N, L, right = _operand("b", b)
    if L != K:
        raise ValueError(f"shape mismatch: a {(M, K)}, b {(N, L)}")
    bias_at, bias_type = _bias(bias, N)
    _same_device(a.q, a.s, b.q, b.s, bias, out)
    device = a.q.device
    d, d_type, ldd = _result(out, out_dtype, torch.bfloat16, M, N, device)
    _call(device, load().hip_int8_gemm, hip_int8_gemm_status_string, M, N, K, *left, *right, bias_at, bias_type,
          d.data_ptr(), ldd, d_type)
    if out is not None:
        written(out)
    return d


def _linear_bytes(T, I) -> int:
    """hip_int8_linear_workspace without a call: few tokens need none."""
    if T <= 16 and (1 << (T - 1).bit_length() if T > 1 else T) * (-(-I // 8) * 8) <= 16384 or I == 0:
        return 0
    return T * (_row(I) + 4)


def linear(x, w: Int8, bias=None, out=None, out_dtype=None):
    """x w^T (+ bias) of tokens x (T x I, rows may be strided) and a quantised weight w
    (O x I): gemm(quantize(x), w, bias), bit for bit, in one call.  The result has
    x's type by default, or out's (which must not overlap what is read) or out_dtype."""
    import torch
    T, I, ldx = _matrix("x", x)
    x_type = _type("x", x.dtype)
    O, L, right = _operand("w", w)
    if L != I:
        raise ValueError(f"shape mismatch: x {(T, I)}, w {(O, L)}")
    bias_at, bias_type = _bias(bias, O)
    _same_device(x, w.q, w.s, bias, out)
    device = x.device
    y, y_type, ldy = _result(out, out_dtype, x.dtype, T, O, device)
    bytes = _linear_bytes(T, I)
    workspace = torch.empty(bytes, dtype=torch.uint8, device=device) if bytes else None
    _call(device, load().hip_int8_linear, hip_int8_linear_status_string, T, I, O, x.data_ptr(), x_type, ldx, *right,
          bias_at, bias_type, y.data_ptr(), ldy, y_type, workspace.data_ptr() if bytes else None, bytes)
    if out is not None:
        written(out)
    return y
