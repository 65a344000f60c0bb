"""The 8-bit operators on sides of 2^31 - 1, where an index and a tile's width
added pass an int: the last elements are right and nothing past them is touched."""

import pytest
import torch

from dense_fp32_matrix_row_amd import blockfp8
from tests import lowp_reference as ref

pytestmark = pytest.mark.gpu

LARGEST = (1 << 31) - 1
END = LARGEST // 128 * 128 - 128  # where the last whole block of 128 begins; a partial one follows
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("block_rows", (1, 128))
@pytest.mark.parametrize("kind", TYPES)
def test_quantize_the_widest_row(kind, block_rows):
    g = torch.Generator().manual_seed(1)
    x = torch.ones(LARGEST + 64, dtype=TYPES[kind], device="cuda")
    x[LARGEST:] = float("nan")  # read by mistake, it would make the last block NaN
    last = torch.randn(LARGEST - END, generator=g).to(TYPES[kind])
    x[END:LARGEST] = last.cuda()
    q = torch.full((LARGEST + 64,), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.empty(-(-LARGEST // 128), device="cuda")
    assert blockfp8.hip_fp8_quantize(1, LARGEST, x, blockfp8._types()[x.dtype], LARGEST, block_rows, 0, q, LARGEST, s, 1, 1,
                                     None, 0, None, 0, 0) == 0
    want, ws = ref.quantize(last[None], 1, False)
    assert torch.equal(q[END:LARGEST].view(torch.float8_e4m3fn).cpu().double(), want[0])
    assert torch.equal(s[-2:].cpu().double(), ws[0])
    assert (q[LARGEST:] == 0x55).all()
    assert (q[:256] == 0x7e).all() and (s[:2].double() == torch.tensor(1 / 448, device="cuda").float().double()).all()


@pytest.mark.parametrize("side", ("rows", "columns"))
@pytest.mark.parametrize("kind", TYPES)
def test_gemm_the_longest_and_the_widest_result(kind, side):
    """D of 2^31 - 1 rows (columns) and one column (row), in place over C.  Codes are small whole numbers under
    scales of 1, so every sum is exact; bf16 holds whole numbers up to 256."""
    K = 16
    g = torch.Generator().manual_seed(2)
    long = torch.full((LARGEST, K), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    last = torch.randint(-3, 4, (LARGEST - END, K), generator=g).float()
    long[END:] = last.to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    one = torch.randint(-3, 4, (1, K), generator=g).float()
    short = one.to(torch.float8_e4m3fn).cuda()
    d = torch.full((LARGEST + 64,), 5.0, dtype=TYPES[kind], device="cuda")
    s_long, s_short = torch.ones(-(-LARGEST // 128), device="cuda"), torch.ones(1, device="cuda")
    a, b = (long, K, s_long, 1, 1, 128), (short, K, s_short, 1, 1, 128)
    c_type = blockfp8._types()[d.dtype]
    M, N = (LARGEST, 1) if side == "rows" else (1, LARGEST)
    if side == "columns":
        a, b = b, a
    assert blockfp8.hip_fp8_gemm(M, N, K, 1.0, *a, *b, 0, 1.0, d, N, d, N, c_type) == 0
    want = (last.double() @ one.double().T)[:, 0] + 5
    assert torch.equal(d[END:LARGEST].cpu().double(), want)
    assert (d[LARGEST:] == 5).all()
    assert (d[:512] == one.sum().item() + 5).all()
