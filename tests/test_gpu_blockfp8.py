"""The 8-bit block-scaled quantiser, product and linear layer on the GPU against
their definitions in 64 bits."""

import pytest
import torch

from dense_fp32_matrix_row_amd import blockfp8
from tests import lowp_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SCALES = {"f32": torch.float32, "e8m0": torch.float8_e8m0fnu}


def values(rows, cols, kind, seed=0):
    """Values of many sizes, with zeros, a row of zeros and a block of tiny ones."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-6, 7, (1, cols), generator=g).float())
    x[torch.rand(rows, cols, generator=g) < 0.05] = 0
    if rows > 2:
        x[1] = 0
        x[2] *= 1e-6
    return x.to(kind)


def same(got, want):
    """Equal as numbers, NaN to NaN."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = torch.isnan(want) | (got == want)
    assert ok.all(), (ok.logical_not().sum().item(), torch.nonzero(~ok)[:4].tolist())


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("block_rows", (1, 128))
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 129), (128, 128), (127, 7), (130, 300), (257, 640), (16, 1024)])
def test_quantize_equals_the_definition(rows, cols, kind, block_rows, scale):
    x = values(rows, cols, TYPES[kind], seed=rows * 1000 + cols)
    d = x.cuda()
    n, t = blockfp8.quantize_both(d, block_rows, SCALES[scale])
    for got, want in ((n, x), (t, x.T)):
        q, s = ref.quantize(want, block_rows, scale == "e8m0")
        same(got.q, q)
        same(got.s, s)
    alone = blockfp8.quantize(d, block_rows, SCALES[scale])
    across = blockfp8.quantize_transposed(d, block_rows, SCALES[scale])
    for a, b in ((alone, n), (across, t)):
        assert torch.equal(a.q.view(torch.uint8), b.q.view(torch.uint8))
        assert torch.equal(a.s.float(), b.s.float())


@pytest.mark.parametrize("scale", SCALES)
def test_quantize_borders_between_codes(scale):
    """Quotients that lie on, and one float step beside, every border between two codes, for several scales."""
    borders = (ref.E4M3[:-1] + ref.E4M3[1:]) / 2
    rows = []
    for top in (448.0, 7.0, 5.1234567, 3.3e-5, 1.9999999, 2.0 ** -90):
        s = ref.scales(torch.tensor([[top]], dtype=torch.float32), 1, scale == "e8m0").item()
        b = (borders * s).float()
        x = torch.cat([b, torch.nextafter(b, torch.full_like(b, 1e30)), torch.nextafter(b, torch.zeros_like(b))])
        x = x[x.abs() <= top]
        x = torch.cat([x, -x])
        for i in range(0, len(x), 127):
            part = torch.zeros(128)
            part[0] = top
            part[1:1 + len(x[i:i + 127])] = x[i:i + 127]
            rows.append(part)
    x = torch.stack(rows)
    q, s = ref.quantize(x, 1, scale == "e8m0")
    n, t = blockfp8.quantize(x.cuda(), 1, SCALES[scale]), blockfp8.quantize_transposed(x.T.contiguous().cuda(), 1, SCALES[scale])
    for got in (n, t):
        same(got.q, q)
        same(got.s, s)


@pytest.mark.parametrize("kind", ("bf16", "f16"))
def test_quantize_every_quotient_of_16_bit_mantissas(kind):
    """With 16-bit elements 448 x / a is exactly a border again and again: every mantissa of bf16 (a
    sample of f16's) over every largest one, at sizes down to the subnormal codes."""
    kind = TYPES[kind]
    bits = 7 if kind == torch.bfloat16 else 10
    m = torch.arange(2 ** bits) if bits == 7 else torch.arange(0, 2 ** bits, 7)
    tops = (1 + m / 2.0 ** bits).repeat_interleave(3) * 4.0
    rows = []
    for shift in (0, 1, 3, 9, 11, 13, 15, 17):
        x = torch.zeros(len(tops), 128)
        x[:, 0] = tops
        pick = torch.arange(len(m)).view(-1)[:126] if bits == 7 else torch.arange(len(m))
        for part in range(3):
            chosen = (1 + m[(pick + part * 53) % len(m)][:127] / 2.0 ** bits) * 2.0 ** (1 - shift)
            x[part::3, 1:1 + len(chosen)] = chosen * (1 - 2 * (part % 2))
        rows.append(x)
    x = torch.cat(rows).to(kind)
    for block_rows in (1,):
        q, s = ref.quantize(x, block_rows, False)
        n, t = blockfp8.quantize(x.cuda(), block_rows), blockfp8.quantize_transposed(x.T.contiguous().cuda(), block_rows)
        for got in (n, t):
            same(got.q, q)
            same(got.s, s)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("block_rows", (1, 128))
def test_quantize_infinities_and_nans_stay_visible(block_rows, scale):
    x = values(260, 300, torch.float32)
    x[3, 140], x[200, 5], x[259, 299] = float("inf"), float("nan"), float("-inf")
    n, t = blockfp8.quantize_both(x.cuda(), block_rows, SCALES[scale])
    for got, want in ((n, x), (t, x.T)):
        q, s = ref.quantize(want, block_rows, scale == "e8m0")
        same(got.s, s)
        same(got.q, q)


@pytest.mark.parametrize("kind", TYPES)
def test_quantize_extreme_magnitudes(kind):
    kind = TYPES[kind]
    info = torch.finfo(kind)
    x = torch.zeros(6, 256, dtype=kind)
    x[0, :4] = torch.tensor([info.max, -info.max, info.max / 2, 1.0], dtype=kind)
    x[1, :3] = torch.tensor([info.tiny, -info.tiny, 0], dtype=kind)
    x[2, :2] = torch.tensor([info.smallest_normal / 4, 0], dtype=kind)
    x[3] = -0.0
    x[4] = 1.0
    for scale in SCALES:
        n = blockfp8.quantize(x.cuda(), 1, SCALES[scale])
        q, s = ref.quantize(x, 1, scale == "e8m0")
        same(n.q, q)
        same(n.s, s)


@pytest.mark.parametrize("kind", TYPES)
def test_quantize_strided_rows_and_nothing_outside_is_written(kind):
    x = values(70, 333, TYPES[kind]).cuda()[:, 3:300]  # odd base and row stride
    rows, cols = x.shape
    q = torch.full((rows + 2, 320), 0x55, dtype=torch.uint8, device="cuda")
    qt = torch.full((cols + 2, 80), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((rows + 1, 7), -1.0, device="cuda")  # row-major scales, padded
    st = torch.full((cols + 1, 5), -1.0, device="cuda")
    code = blockfp8.hip_fp8_quantize(rows, cols, x, blockfp8._types()[x.dtype], x.stride(0), 1, 0,
                                     q[1:], 320, s, 7, 1, qt[1:], 80, st, 5, 1)
    assert code == 0
    want, ws = ref.quantize(x.cpu(), 1, False)
    same(q[1:-1, :cols].view(torch.float8_e4m3fn), want)
    same(s[:rows, :3], ws)
    want, ws = ref.quantize(x.cpu().T, 1, False)
    same(qt[1:-1, :rows].view(torch.float8_e4m3fn), want)
    same(st[:cols, :1], ws)
    for whole, inner in ((q, (slice(1, -1), slice(0, cols))), (qt, (slice(1, -1), slice(0, rows)))):
        whole[inner] = 0x55
        assert (whole == 0x55).all()
    for whole, inner in ((s, (slice(0, rows), slice(0, 3))), (st, (slice(0, cols), slice(0, 1)))):
        whole[inner] = -1.0
        assert (whole == -1.0).all()


def operand(rows, K, block_rows, scale, seed, ld=None, fill=0x7f, major="column"):
    """A quantised matrix on the GPU whose row padding is NaN codes, and its value in 64 bits."""
    x = values(rows, K, torch.float32, seed)
    q, s = ref.quantize(x, block_rows, scale == "e8m0")
    ld = -(-K // 16) * 16 if ld is None else ld
    wide = torch.full((rows, ld), fill, dtype=torch.uint8)
    wide[:, :K] = q.to(torch.float8_e4m3fn).view(torch.uint8)
    sc = s.to(SCALES[scale])
    raw = sc.view(torch.uint8) if scale == "e8m0" else sc
    raw = raw.cuda().T.contiguous().T if major == "column" else raw.cuda()
    sc = raw.view(SCALES[scale]) if scale == "e8m0" else raw
    return blockfp8.BlockFp8(wide.cuda().view(torch.float8_e4m3fn)[:, :K], sc, block_rows), ref.dequantize(q, s, block_rows)


def tolerance(a, b, K, scale, out, want, c=0.0, alpha=1.0):
    """The sum's terms are exact products; the matrix cores may cut instead of
    round (2^-23 a term of the running sum).  For 16-bit outputs seven of eight
    neighbouring products may each lose up to 2^-13 of the eighth besides.  Blocks of 128 summed alone and
    added take 128 + 2 K / 128 of those, one running sum K; then the scaling by
    alpha, the addition of beta C and the rounding to the output's type."""
    size = abs(alpha) * (a.abs() @ b.abs().T)
    steps = (128 + 2 * -(-K // 128) if scale == "f32" else K) + 4
    bound = steps * 2.0 ** -23 * size + 2.0 ** -23 * abs(c)
    if out != torch.float32:
        bound = bound + 7 * 2.0 ** -13 * size
    half = torch.finfo(out).eps / 2
    least = torch.finfo(out).smallest_normal * torch.finfo(out).eps
    return bound * (1 + 2 * half) + half * want.abs() + least


def close(got, want, tol):
    """Within tol; an infinity where the value, within tol, is past the type's largest."""
    kind, got = got.dtype, got.cpu().double()
    past = torch.isinf(got) & (got.sign() == want.sign()) & (want.abs() + tol >= torch.finfo(kind).max)
    off = ~(((got - want).abs() <= tol) | past)
    assert not off.any(), f"{off.sum().item()} values off, first at {torch.nonzero(off)[0].tolist()}"


SHAPES = [(1, 1, 1), (1, 64, 128), (1, 300, 1000), (2, 17, 16), (16, 130, 257), (33, 65, 127), (64, 64, 129), (65, 128, 512),
          (128, 128, 128), (100, 513, 640), (257, 300, 1040), (300, 1, 400), (513, 129, 2050)]


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("a_block,b_block", [(1, 128), (1, 1), (128, 128), (128, 1)])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_against_the_definition(M, N, K, a_block, b_block, scale):
    a, da = operand(M, K, a_block, scale, 1)
    b, db = operand(N, K, b_block, scale, 2)
    want = da @ db.T
    out = torch.full((M, N + 3), float("nan"), device="cuda")
    blockfp8.gemm(a, b, out=out[:, :N])
    assert torch.isnan(out[:, N:]).all()
    close(out[:, :N], want, tolerance(da, db, K, scale, torch.float32, want))


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("b_block", (1, 128))
@pytest.mark.parametrize("kind", ("bf16", "f32"))
@pytest.mark.parametrize("K", (1, 128, 200, 384, 505, 640, 1023))
def test_gemm_large_tiles(K, kind, b_block, scale):
    """Enough rows and columns for the large tiles, ragged on both sides; one to eight steps along K."""
    M, N = 2049, 2085
    a, da = operand(M, K, 1, scale, 13)
    b, db = operand(N, K, b_block, scale, 14)
    c = values(M, N, TYPES[kind], 15)
    want = da @ db.T
    tol = tolerance(da, db, K, scale, TYPES[kind], want)
    close(blockfp8.gemm(a, b, out_dtype=TYPES[kind]), want, tol)
    want = 0.5 * want - c.double()
    close(blockfp8.gemm(a, b, c=c.cuda(), alpha=0.5, beta=-1.0), want, tolerance(da, db, K, scale, TYPES[kind], want, c.double(), 0.5))


def sampled(rows, seed):
    """Rows at both ends, beside multiples of the tiles' sizes, and some between."""
    g = torch.Generator().manual_seed(seed)
    at = {0, 1, 127, 128, 255, 256, rows - 257, rows - 2, rows - 1, *torch.randint(0, rows, (40,), generator=g).tolist()}
    return torch.tensor(sorted(r for r in at if 0 <= r < rows))


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("b_block", (1, 128))
@pytest.mark.parametrize("kind", ("bf16", "f32"))
@pytest.mark.parametrize("M,N,K", [(4090, 4090, 400), (4090, 3900, 513), (4097, 4097, 1290), (4097, 2048, 1000), (2048, 4097, 900),
                                   (4100, 4200, 1600)])
def test_gemm_largest_tiles_and_ragged_edges_apart(M, N, K, kind, b_block, scale):
    """Sizes whose last rows and columns are computed apart, and the largest tiles: rows and columns of D by sample."""
    a, da = operand(M, K, 1, scale, 16)
    b, db = operand(N, K, b_block, scale, 17)
    c = values(M, N, TYPES[kind], 18)
    got = blockfp8.gemm(a, b, c=c.cuda(), alpha=1.0, beta=0.5).cpu()
    r, n = sampled(M, 1), sampled(N, 2)
    for left, right, part, ci in ((da[r], db, got[r], c[r]), (da, db[n], got[:, n], c[:, n])):
        want = left @ right.T + 0.5 * ci.double()
        close(part, want, tolerance(left, right, K, scale, TYPES[kind], want, 0.5 * ci.double()))
    assert torch.equal(got, blockfp8.gemm(a, b, c=c.cuda(), alpha=1.0, beta=0.5).cpu())  # the same again


@pytest.mark.parametrize("kind", ("bf16", "f32"))
@pytest.mark.parametrize("scale", SCALES)
def test_gemm_large_tiles_scales_of_any_layout_and_kind(scale, kind):
    """Row-major scales with padding, and the ends of the scales' ranges, against the small tiles'
    results for the same rows (whole numbers under powers of two: all sums are exact)."""
    M, N, K = 2300, 2100, 700
    g = torch.Generator().manual_seed(19)
    ops = []
    for rows in (M, N):
        q = torch.randint(-4, 5, (rows, 704), generator=g).float()
        q[:, K:] = float("nan")
        s = torch.exp2(torch.randint(-3, 4, (rows, 9), generator=g).float())
        if rows == M:
            s[5], s[7, 2], s[11] = 2.0 ** -127, float("nan"), 2.0 ** 100
        else:
            s[6] = 2.0 ** 126
        raw = s.to(SCALES[scale]).view(torch.uint8).cuda() if scale == "e8m0" else s.cuda()
        raw = raw.view(SCALES[scale]) if scale == "e8m0" else raw
        ops.append(blockfp8.BlockFp8(q.to(torch.float8_e4m3fn).cuda()[:, :K], raw[:, :6], 1))
    got = blockfp8.gemm(*ops, out_dtype=TYPES[kind])
    part = [blockfp8.BlockFp8(o.q[:40], o.s[:40], 1) for o in ops]
    few = blockfp8.gemm(*part, out_dtype=TYPES[kind])
    # Column 6 passes float's range, but for row 5: an infinity or, where two parts of a sum overflow with
    # opposite signs, a NaN, as the sum's order has it.
    past = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    past[:, 6] = True
    past[5, 6] = past[7, 6] = False
    shown = got.masked_fill(past, 0)
    assert torch.equal(torch.nan_to_num(shown[:40, :40], nan=-7.0),
                       torch.nan_to_num(few.masked_fill(past[:40, :40], 0), nan=-7.0))
    assert torch.isnan(got[7]).all() and not torch.isnan(shown[:7]).any()
    want = (ops[0].q[:5].cpu().double() * ops[0].s[:5].cpu().double().repeat_interleave(128, 1)[:, :K]) @ (
        ops[1].q.cpu().double() * ops[1].s.cpu().double().repeat_interleave(128, 1)[:, :K]).T
    exact = torch.arange(N) != 6
    assert torch.equal(got[:5].cpu()[:, exact], want[:, exact].to(TYPES[kind]))


@pytest.mark.parametrize("M", (3, 600))
def test_gemm_operands_past_two_gigabytes(M):
    """A's offsets pass 2^31 bytes; the last rows are checked."""
    K, rows = 65600, 33000
    g = torch.Generator(device="cuda").manual_seed(20)
    q = torch.randint(0, 0x78, (rows, K), generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.rand(-(-K // 128), rows, generator=g, device="cuda").T + 0.5
    a = blockfp8.BlockFp8(q, s, 1)
    b = blockfp8.BlockFp8(q[:M], s[:M], 1)
    got = blockfp8.gemm(a, b, out_dtype=torch.float32)
    at = torch.tensor([0, 16384, 32760, rows - 1])
    da = a.q[at.cuda()].cpu().double() * a.s[at.cuda()].cpu().double().repeat_interleave(128, 1)[:, :K]
    db = b.q.cpu().double() * b.s.cpu().double().repeat_interleave(128, 1)[:, :K]
    want = da @ db.T
    close(got[at.cuda()], want, tolerance(da, db, K, "f32", torch.float32, want))


def test_quantize_past_two_gigabytes():
    rows, cols = 33000, 65600
    g = torch.Generator(device="cuda").manual_seed(21)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)
    n, t = blockfp8.quantize_both(x)
    for r0 in (0, 32768, rows - 232):  # whole blocks of 128 rows, and the last ones
        part = x[r0 // 128 * 128:][:256, cols - 200:].cpu()
        q, s = ref.quantize(x[r0 // 128 * 128:][:256, cols // 128 * 128 - 128:].cpu(), 1, False)
        same(n.q[r0 // 128 * 128:][:256, cols // 128 * 128 - 128:], q)
        q, s = ref.quantize(part.T, 1, False)
        same(t.q[cols - 200:, r0 // 128 * 128:][:, :256], q)


def test_products_of_every_size_in_a_captured_graph():
    """One launch, several, and both in turn."""
    sizes = [(1, 300, 500), (200, 140, 512), (700, 900, 300), (2100, 2100, 300), (4097, 2048, 1000)]
    for M, N, K in sizes:
        a = blockfp8.quantize(torch.randn(M, K, device="cuda"))
        x = torch.randn(N, K, device="cuda")
        run = lambda: blockfp8.gemm(a, blockfp8.quantize(x, 128), out_dtype=torch.float32)  # noqa: E731
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        for i in range(3):
            x.copy_(torch.randn(N, K, device="cuda") * (i + 1))
            graph.replay()
            torch.cuda.synchronize()
            want = run()
            torch.cuda.synchronize()
            assert torch.equal(got, want), (M, N, K)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("alpha,beta", [(1.0, 0.0), (0.5, 1.0), (-2.0, 3.0), (1.0, -1.0)])
def test_gemm_types_and_scaling(alpha, beta, kind, scale):
    kind = TYPES[kind]
    for M, N, K in ((3, 70, 200), (130, 67, 300), (257, 300, 1040)):
        a, da = operand(M, K, 1, scale, 3)
        b, db = operand(N, K, 128, scale, 4)
        c = values(M, N, kind, 5)
        want = alpha * (da @ db.T) + beta * c.double()
        got = blockfp8.gemm(a, b, c=c.cuda(), alpha=alpha, beta=beta, out_dtype=kind)
        assert got.dtype == kind
        close(got, want, tolerance(da, db, K, scale, kind, want, beta * c.double(), alpha))
        place = c.cuda()
        assert torch.equal(blockfp8.gemm(a, b, c=place, alpha=alpha, beta=beta, out=place), got)


@pytest.mark.parametrize("scale", SCALES)
def test_gemm_whole_numbers_are_exact(scale):
    """Codes that are small whole numbers under scales of 1 and 2: every partial sum is exact."""
    M, N, K = 200, 190, 700
    g = torch.Generator().manual_seed(7)
    q = [torch.randint(-8, 9, (r, K), generator=g).float() for r in (M, N)]
    s = [torch.randint(0, 2, (r, 6), generator=g).float() + 1 for r in (M, N)]
    ops = []
    for qi, si in zip(q, s):
        wide = torch.zeros(qi.shape[0], 704)
        wide[:, :K] = qi
        ops.append(blockfp8.BlockFp8(wide.cuda().to(torch.float8_e4m3fn)[:, :K], si.cuda().to(SCALES[scale]), 1))
    want = ref.dequantize(q[0], s[0], 1) @ ref.dequantize(q[1], s[1], 1).T
    assert torch.equal(blockfp8.gemm(*ops, out_dtype=torch.float32).cpu().double(), want)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("M", (1, 200))
def test_gemm_scales_of_any_layout_and_wide_rows(M, scale):
    N, K = 150, 333
    a, da = operand(M, K, 1, scale, 8, ld=512, major="row")
    b, db = operand(N, K, 1, scale, 9, ld=400, major="row")
    a2, _ = operand(M, K, 1, scale, 8)
    b2, _ = operand(N, K, 1, scale, 9)
    got = blockfp8.gemm(a, b, out_dtype=torch.float32)
    assert torch.equal(got, blockfp8.gemm(a2, b2, out_dtype=torch.float32))
    assert ((got.cpu().double() - da @ db.T).abs() <= tolerance(da, db, K, scale, torch.float32, da @ db.T)).all()


@pytest.mark.parametrize("scale", SCALES)
def test_gemm_nan_stays_in_its_row_and_column(scale):
    M, N, K = 150, 140, 300
    x, y = values(M, K, torch.float32, 10), values(N, K, torch.float32, 11)
    x[17, 150], y[33, 5] = float("nan"), float("inf")
    a, b = blockfp8.quantize(x.cuda(), 1, SCALES[scale]), blockfp8.quantize(y.cuda(), 1, SCALES[scale])
    bad = torch.isnan(blockfp8.gemm(a, b, out_dtype=torch.float32).cpu())
    want = torch.zeros(M, N, dtype=torch.bool)
    want[17], want[:, 33] = True, True
    assert torch.equal(bad, want)


def test_gemm_degenerate_sizes():
    a, _ = operand(4, 128, 1, "f32", 12)
    none = blockfp8.BlockFp8(torch.empty(0, 128, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(0, 1, device="cuda"), 1)
    assert blockfp8.gemm(none, a).shape == (0, 4) and blockfp8.gemm(a, none).shape == (4, 0)
    c = torch.randn(4, 4, device="cuda")
    bad = blockfp8.BlockFp8(a.q, torch.full_like(a.s, float("nan")), 1)
    assert torch.equal(blockfp8.gemm(bad, bad, c=c, alpha=0.0, beta=2.0), 2 * c)  # neither operand is read
    flat = blockfp8.BlockFp8(torch.empty(4, 0, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(4, 0, device="cuda"), 1)
    assert torch.equal(blockfp8.gemm(flat, flat, c=c, beta=-1.0), -c)
    assert torch.equal(blockfp8.gemm(flat, flat, out_dtype=torch.float32), torch.zeros_like(c))
    e = blockfp8.quantize(torch.empty(0, 5, device="cuda"))
    assert e.q.shape == (0, 5)


def test_refusals_of_the_tensor_forms():
    x = torch.randn(8, 256, device="cuda")
    a = blockfp8.quantize(x)
    with pytest.raises(ValueError):
        blockfp8.quantize(x.T)  # columns apart
    with pytest.raises(ValueError):
        blockfp8.quantize(x[:1].expand(8, 256))  # rows overlap
    with pytest.raises(TypeError):
        blockfp8.quantize(x.double())
    with pytest.raises(TypeError):
        blockfp8.quantize(x, scale=torch.bfloat16)
    with pytest.raises(ValueError):
        blockfp8.quantize(x, block_rows=64)
    with pytest.raises(ValueError):
        blockfp8.gemm(a, blockfp8.quantize(x[:, :128]))
    with pytest.raises(TypeError):
        blockfp8.gemm(a, blockfp8.quantize(x, scale=torch.float8_e8m0fnu))
    with pytest.raises(ValueError):
        blockfp8.gemm(a, a, beta=1.0)
    with pytest.raises(ValueError):
        blockfp8.gemm(a, a, out=torch.empty(8, 9, device="cuda"))
    with pytest.raises(ValueError):
        blockfp8.gemm(blockfp8.BlockFp8(a.q, a.s[:4], 1), a)
    odd = torch.zeros(4 * 200, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).view(4, 200)
    with pytest.raises(RuntimeError):  # rows of 200 bytes
        blockfp8.gemm(blockfp8.BlockFp8(odd, torch.ones(4, 2, device="cuda"), 1), blockfp8.BlockFp8(odd, torch.ones(4, 2, device="cuda"), 1))


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("T,I,O", [(5, 130, 70), (200, 300, 257)])
def test_linear_layer_and_its_gradients(T, I, O, scale):
    e8m0 = scale == "e8m0"
    x, dy = values(T, I, torch.bfloat16, 20), values(T, O, torch.bfloat16, 21)
    w = values(O, I, torch.float32, 22)
    wn, wt = blockfp8.quantize_both(w.cuda(), 128, SCALES[scale])
    y, xt = blockfp8.linear_forward(x.cuda(), wn, out_dtype=torch.float32)
    dx, dw = blockfp8.linear_backward(dy.cuda(), xt, wt, out_dtype=torch.float32)
    deq = lambda v, rows: ref.dequantize(*ref.quantize(v, rows, e8m0), rows)  # noqa: E731
    xq, wq, dyq = deq(x, 1), deq(w, 128), deq(dy, 1)
    xtq, dytq = deq(x.T, 1), deq(dy.T, 1)
    for got, left, right, K in ((y, xq, wq, I), (dx, dyq, wq.T, O), (dw, dytq, xtq, T)):
        want = left @ right.T
        close(got, want, tolerance(left, right, K, scale, torch.float32, want))
    # the gradients are those of sum(dy * y), but for the operands' rounding: by differences of that sum
    step = 1.0 / 16
    loss = lambda xv, wv: (dyq * (xv @ wv.T)).sum()  # noqa: E731
    d = torch.zeros_like(xq)
    d[T // 2, I // 2] = step
    diff = (loss(xq + d, wq) - loss(xq - d, wq)) / (2 * step)
    assert abs(diff - dx.cpu().double()[T // 2, I // 2]) <= tolerance(dyq, wq.T, O, scale, torch.float32, dyq @ wq)[T // 2, I // 2] + 1e-9 * abs(diff) + 1e-6
    # accumulated into a gradient that is there
    acc = torch.randn(O, I, device="cuda")
    want = acc.cpu().double() + dytq @ xtq.T
    _, dw2 = blockfp8.linear_backward(dy.cuda(), xt, wt, dw=acc)
    assert dw2 is acc
    assert ((acc.cpu().double() - want).abs() <= tolerance(dytq, xtq, T, scale, torch.float32, want, want.abs() + 1)).all()


def test_other_streams_and_captured_graphs():
    x = torch.randn(200, 512, device="cuda")
    w = torch.randn(140, 512, device="cuda")
    want = blockfp8.gemm(blockfp8.quantize(x), blockfp8.quantize(w, 128), out_dtype=torch.float32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = blockfp8.gemm(blockfp8.quantize(x), blockfp8.quantize(w, 128), out_dtype=torch.float32)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = blockfp8.gemm(blockfp8.quantize(x), blockfp8.quantize(w, 128), out_dtype=torch.float32)
    for i in range(4):
        x.copy_(torch.randn(200, 512, device="cuda") * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        want = blockfp8.gemm(blockfp8.quantize(x), blockfp8.quantize(w, 128), out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", (torch.float8_e5m2, torch.float8_e4m3fnuz, torch.int8))
def test_codes_of_another_type_are_refused(dtype):
    a = blockfp8.quantize(torch.ones(4, 128, device="cuda"))
    other = blockfp8.BlockFp8(a.q.view(dtype), a.s, 1)
    for pair in ((a, other), (other, a)):
        with pytest.raises(TypeError, match="codes"):
            blockfp8.gemm(*pair)
    same = blockfp8.BlockFp8(a.q.view(torch.uint8), a.s, 1)
    assert torch.equal(blockfp8.gemm(same, same), blockfp8.gemm(a, a))
