"""The 8-bit products' and the orthogonalised update's C ABI without a GPU:
exports, refusals before any HIP call, workspace sizes, and the reference that
the GPU tests compare with."""

import os
import re

import pytest
import torch

from dense_fp32_matrix_row_amd import blockfp8, orthogonal, sgemm
from tests import lowp_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x1000  # non-NULL, aligned, never dereferenced: errors return first


def declared(header):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(hip_\w+)\s*\(", text)))


@pytest.mark.parametrize("header,module", [("blockfp8.h", blockfp8), ("orthogonal.h", orthogonal)])
def test_headers_declare_the_bindings_exports(header, module):
    assert declared(header) == sorted(module.EXPORTS)
    lib = module.load()
    for name in module.EXPORTS:
        assert hasattr(lib, name)


QUANTIZE = dict(rows=4, cols=200, X=FAKE, x_type=0, ldx=200, block_rows=1, scale_type=0, Q=FAKE, ldq=208, S=FAKE,
                s_row=1, s_col=4, QT=FAKE, ldqt=16, ST=FAKE, st_row=1, st_col=200)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), -1), (dict(cols=-1), -2), (dict(X=None), -3), (dict(x_type=3), -4), (dict(x_type=-1), -4),
    (dict(ldx=199), -5), (dict(block_rows=2), -6), (dict(block_rows=0), -6), (dict(scale_type=2), -7),
    (dict(Q=None, S=None, QT=None, ST=None), -8), (dict(Q=None), -8), (dict(ldq=199), -9), (dict(S=None), -10),
    (dict(s_row=-1), -11), (dict(s_col=-1), -12), (dict(QT=None), -13), (dict(ldqt=3), -14), (dict(ST=None), -15),
    (dict(st_row=-1), -16), (dict(st_col=-1), -17),
    (dict(rows=0), 0), (dict(cols=0, ldx=1, X=None), 0),
])
def test_quantize_refusals(change, status):
    assert blockfp8.hip_fp8_quantize(*{**QUANTIZE, **change}.values(), stream=0) == status
    assert "unknown" not in blockfp8.hip_fp8_quantize_status_string(status)


GEMM = dict(M=4, N=8, K=200, alpha=1.0, A=FAKE, lda=208, SA=FAKE, sa_row=1, sa_col=4, a_block_rows=1,
            B=FAKE, ldb=208, SB=FAKE, sb_row=1, sb_col=8, b_block_rows=128, scale_type=0, beta=1.0, C=FAKE, ldc=8,
            D=FAKE, ldd=8, c_type=0)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), -1), (dict(N=-1), -2), (dict(K=-1), -3), (dict(A=None), -5), (dict(A=FAKE + 8), -5),
    (dict(lda=192), -6), (dict(lda=204), -6), (dict(lda=blockfp8.MAX_LD + 16), -6), (dict(SA=None), -7),
    (dict(sa_row=-1), -8), (dict(sa_col=-1), -9), (dict(a_block_rows=64), -10), (dict(B=None), -11),
    (dict(B=FAKE + 1), -11), (dict(ldb=192), -12), (dict(ldb=200), -12), (dict(SB=None), -13), (dict(sb_row=-1), -14),
    (dict(sb_col=-1), -15), (dict(b_block_rows=0), -16), (dict(scale_type=-1), -17), (dict(C=None), -19),
    (dict(ldc=7), -20), (dict(D=None), -21), (dict(ldd=7), -22), (dict(c_type=9), -23),
    (dict(M=0), 0), (dict(N=0, D=None, C=None), 0),
])
def test_gemm_refusals(change, status):
    assert blockfp8.hip_fp8_gemm(*{**GEMM, **change}.values(), stream=0) == status
    assert "unknown" not in blockfp8.hip_fp8_gemm_status_string(status)


ORTHOGONALIZE = dict(batch=2, rows=4, cols=8, type=0, G=FAKE, ldg=8, stride_g=32, steps=1,
                     coefficients=(1.5, -0.5, 0.0), eps=0.0, X=FAKE, ldx=8, stride_x=32, workspace=FAKE,
                     workspace_bytes=1 << 30)


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), -1), (dict(batch=65536), -1), (dict(rows=-1), -2), (dict(rows=orthogonal.MAX_SIZE + 1), -2),
    (dict(cols=-1), -3), (dict(cols=orthogonal.MAX_SIZE + 1), -3), (dict(type=5), -4), (dict(G=None), -5),
    (dict(ldg=7), -6), (dict(stride_g=-1), -7), (dict(steps=-1), -8),
    (dict(steps=65, coefficients=(0.0,) * 195), -8), (dict(coefficients=None), -9), (dict(eps=-1.0), -10),
    (dict(eps=float("nan")), -10), (dict(X=None), -11), (dict(ldx=7), -12), (dict(stride_x=31), -13),
    (dict(workspace=None), -14), (dict(workspace=FAKE + 128), -14), (dict(workspace_bytes=100), -15),
    (dict(batch=0), 0), (dict(rows=0), 0), (dict(cols=0, G=None), 0),
])
def test_orthogonalize_refusals(change, status):
    assert orthogonal.hip_orthogonalize(*{**ORTHOGONALIZE, **change}.values(), stream=0) == status
    assert "unknown" not in orthogonal.hip_orthogonalize_status_string(status)


def test_orthogonalize_workspace_grows_with_the_batch_and_holds_the_iterate():
    one = orthogonal.hip_orthogonalize_workspace(1, 100, 300, 0)
    assert one >= 3 * 100 * 300 * 4 + 2 * 100 * 100 * 4
    assert orthogonal.hip_orthogonalize_workspace(1, 300, 100, 0) == one
    assert orthogonal.hip_orthogonalize_workspace(4, 100, 300, 0) > 3 * one
    for batch, rows, cols in ((0, 4, 4), (3, 0, 4), (3, 4, 0)):  # nothing to hold
        assert orthogonal.hip_orthogonalize_workspace(batch, rows, cols, 0) >= 0
    with pytest.raises(sgemm.SgemmError):
        orthogonal.hip_orthogonalize_workspace(-1, 4, 4, 0)


def test_bindings_refuse_host_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        blockfp8.quantize(x)
    with pytest.raises(TypeError):
        orthogonal.orthogonalize(x)
    q = blockfp8.BlockFp8(torch.zeros(4, 16, dtype=torch.float8_e4m3fn), torch.ones(4, 1))
    with pytest.raises(TypeError):
        blockfp8.gemm(q, q)


def test_reference_rounds_to_e4m3_as_the_type_does():
    # every float that torch's own cast rounds; the cast is to nearest even
    x = torch.cat([torch.randn(20000) * 10 ** torch.empty(20000).uniform_(-4, 2), torch.arange(-448.0, 449.0)])
    x = x.clamp(-448, 448)
    assert torch.equal(ref.to_e4m3(x.double()), x.to(torch.float8_e4m3fn).double())


def test_reference_scales_leave_nothing_above_448():
    x = torch.randn(130, 300, dtype=torch.float64).float()
    for rows in (1, 128):
        s = ref.scales(x, rows, True)
        t = (x.double() / ref.spread(s, rows, *x.shape)).abs()
        assert t.max() <= 448 and torch.equal(torch.exp2(torch.log2(s).round()), s)
        s = ref.scales(x, rows, False)
        assert (x.double() / ref.spread(s, rows, *x.shape)).abs().max() <= 448 * (1 + 2.0 ** -23)
