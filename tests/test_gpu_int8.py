"""The integer quantiser, product and linear layer on the GPU against their
definitions in 64 bits."""

import pytest
import torch

from dense_fp32_matrix_row_amd import int8
from tests import serving_reference as ref
from tests import serving_shapes as shapes
from tests.serving_reference import TYPES

pytestmark = pytest.mark.gpu

WIDTHS = (1, 7, 8, 65, 511, 512, 513, 1024, 1025, 2047, 2049, 4096, 4097, 8193, 16384, 16385, 20001)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("cols", WIDTHS)
def test_quantize_equals_the_definition(cols, kind):
    for rows in (1, 3, 6, 37):
        x = ref.values(rows, cols, TYPES[kind], seed=rows * 1000 + cols)
        got = int8.quantize(x.cuda())
        q, s = ref.quantize(x)
        ref.same(got.q, q)
        ref.same(got.s, s)
        assert got.q.dtype == torch.int8 and got.shape == (rows, cols)


def test_quantize_borders_between_codes():
    """Quotients that lie on, and one float step beside, every border between two codes, for several scales."""
    borders = torch.arange(127, dtype=torch.float64) + 0.5
    rows = []
    for top in (127.0, 254.0, 7.0, 5.1234567, 3.3e-5, 1.9999999, 2.0 ** -90, 1e30, 127 * 2.0 ** -100, 3.0e38):
        s = ref.quantize(torch.tensor([[top]], dtype=torch.float32))[1].item()
        b = (borders * s).float()
        x = torch.cat([b, torch.nextafter(b, torch.full_like(b, float("inf"))), torch.nextafter(b, torch.zeros_like(b))])
        x = x[x.abs() <= top]
        row = torch.zeros(1000)
        row[0] = top
        row[1:1 + 2 * len(x)] = torch.cat([x, -x])
        rows.append(row)
    x = torch.stack(rows)
    q, s = ref.quantize(x)
    got = int8.quantize(x.cuda())
    ref.same(got.q, q)
    ref.same(got.s, s)


@pytest.mark.parametrize("kind", ("bf16", "f16"))
def test_quantize_every_quotient_of_16_bit_mantissas(kind):
    """With 16-bit elements 127 x / a is exactly a border again and again: every bf16 mantissa (a sample of f16's)
    over every largest one."""
    bits, kind = (7, torch.bfloat16) if kind == "bf16" else (10, torch.float16)
    m = torch.arange(0, 2 ** bits, 1 if bits == 7 else 5)
    tops = 1 + m / 2.0 ** bits
    x = torch.zeros(len(tops), 1 + 8 * len(m))
    x[:, 0] = 2 * tops
    for shift in range(8):
        part = (1 + m / 2.0 ** bits) * 2.0 ** -shift
        x[:, 1 + shift * len(m):1 + (shift + 1) * len(m)] = part * (-1) ** shift
    x = x.to(kind)
    q, s = ref.quantize(x)
    got = int8.quantize(x.cuda())
    ref.same(got.q, q)
    ref.same(got.s, s)


@pytest.mark.parametrize("cols", (300, 3000, 20000))
@pytest.mark.parametrize("kind", TYPES)
def test_quantize_infinities_nans_and_extremes(kind, cols):
    kind = TYPES[kind]
    info = torch.finfo(kind)
    x = ref.values(9, cols, kind, 5)
    x[0, 140], x[3, 5], x[4, 299], x[5] = float("inf"), float("nan"), float("-inf"), 0
    x[6, :4] = torch.tensor([info.max, -info.max, info.max / 2, 1.0], dtype=kind)
    x[7] = 0
    x[7, :2] = torch.tensor([info.tiny, -info.tiny / 4], dtype=kind)
    x[8] = -0.0
    got = int8.quantize(x.cuda())
    q, s = ref.quantize(x)
    ref.same(got.q, q)
    ref.same(got.s, s)


@pytest.mark.parametrize("cols", (297, 5000, 20000))
@pytest.mark.parametrize("kind", TYPES)
def test_quantize_strided_rows_and_nothing_outside_is_written(kind, cols):
    x = ref.values(70, cols + 36, TYPES[kind]).cuda()[:, 3:3 + cols]  # odd base and row stride
    ld = cols + 23
    q = torch.full((72, ld), 0x55, dtype=torch.int8, device="cuda")
    s = torch.full((72,), -1.0, device="cuda")
    code = int8.hip_int8_quantize(70, cols, x, {"f32": 0, "bf16": 1, "f16": 2}[kind], x.stride(0), q[1:], ld, s[1:])
    assert code == 0
    want, scales = ref.quantize(x.cpu())
    ref.same(q[1:-1, :cols], want)
    ref.same(s[1:-1], scales)
    q[1:-1, :cols] = 0x55
    assert (q == 0x55).all() and s[0] == -1 and s[-1] == -1


def test_quantize_more_rows_than_a_launch_has_blocks():
    rows = 4 * (1 << 23) + 5
    x = torch.ones(rows, 1, device="cuda", dtype=torch.bfloat16)
    x[-3:] = -254.0
    got = int8.quantize(x)
    assert (got.q[:-3] == 127).all() and (got.q[-3:] == -127).all()
    assert (got.s[-3:] == 2.0).all() and torch.equal(got.s[:-3], (torch.ones(rows - 3, device="cuda") / 127))


def operand(rows, K, seed, ld=None, fill=0x7f, low=-128):
    """A quantised matrix on the GPU whose row padding is not zero, and its parts on the CPU."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(low, 128, (rows, K), generator=g, dtype=torch.int8)
    s = torch.exp2(torch.randint(-9, 3, (rows,), generator=g).float()) * (1 + torch.rand(rows, generator=g))
    wide = torch.full((rows, -(-K // 16) * 16 if ld is None else ld), fill, dtype=torch.int8)
    wide[:, :K] = q
    return int8.Int8(wide.cuda()[:, :K], s.cuda()), q, s


SHAPES = [(1, 1, 1), (1, 64, 128), (1, 300, 1000), (2, 17, 16), (16, 130, 257), (33, 65, 127), (64, 64, 129), (65, 128, 512),
          (128, 128, 128), (100, 513, 640), (257, 300, 1040), (300, 1, 400), (513, 129, 2050), (5, 9, 20000)]


@pytest.mark.parametrize("bias", (None, *TYPES))
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_against_the_definition(M, N, K, kind, bias):
    a, qa, sa = operand(M, K, 1)
    b, qb, sb = operand(N, K, 2)
    c = None if bias is None else ref.values(1, N, TYPES[bias], 3)[0]
    want, size = ref.product(qa, sa, qb, sb, c)
    out = torch.full((M, N + 3), float("nan"), device="cuda", dtype=TYPES[kind])
    got = int8.gemm(a, b, bias=None if c is None else c.cuda(), out=out[:, :N])
    assert torch.isnan(out[:, N:]).all()
    ref.close(got, want, ref.product_tolerance(TYPES[kind], want, size))


@pytest.mark.parametrize("kind", ("f32", "bf16"))
@pytest.mark.parametrize("size", shapes.INT8)
def test_gemm_every_tile_and_edge(size, kind):
    M, N, K = size
    a, qa, sa = operand(M, K, 4)
    b, qb, sb = operand(N, K, 5)
    c = ref.values(1, N, torch.float32, 6)[0]
    got = int8.gemm(a, b, bias=c.cuda(), out_dtype=TYPES[kind])
    # every element, from exact sums (below 2^53) on the GPU
    p = (a.q.double() @ b.q.double().T.contiguous()) * sa.cuda().double()[:, None] * sb.cuda().double()
    want = p + c.cuda().double()
    tol = ref.product_tolerance(TYPES[kind], want, p.abs())
    off = (got.double() - want).abs() > tol
    assert not off.any(), torch.nonzero(off)[:4].tolist()
    assert torch.equal(got, int8.gemm(a, b, bias=c.cuda(), out_dtype=TYPES[kind]))


@pytest.mark.parametrize("K", (1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 384, 505, 640, 1023))
def test_gemm_large_tiles_and_ragged_k(K):
    """Whole sums, which have to be equal: scales of 1 and sums below 2^24."""
    for M, N in ((2049, 2085), (600, 4100)):
        g = torch.Generator(device="cuda").manual_seed(K)
        ld = -(-K // 16) * 16 + 16
        q = [torch.randint(-128, 128, (r, ld), generator=g, device="cuda", dtype=torch.int8) for r in (M, N)]
        one = [torch.ones(r, device="cuda") for r in (M, N)]
        got = int8.gemm(int8.Int8(q[0][:, :K], one[0]), int8.Int8(q[1][:, :K], one[1]), out_dtype=torch.float32)
        assert torch.equal(got.double(), q[0][:, :K].double() @ q[1][:, :K].double().T.contiguous())


@pytest.mark.parametrize("M,N", [(3, 5), (300, 300), (2100, 2100)])
def test_gemm_longest_sums(M, N):
    """131071 products of -128 by -128, the most that 32 bits hold, and of -128 by 127."""
    K = int8.MAX_K
    a = torch.full((M, 131072), -128, dtype=torch.int8, device="cuda")
    b = torch.full((N, 131072), -128, dtype=torch.int8, device="cuda")
    b[1] = 127
    one = [torch.ones(r, device="cuda") for r in (M, N)]
    got = int8.gemm(int8.Int8(a[:, :K], one[0]), int8.Int8(b[:, :K], one[1]), out_dtype=torch.float32)
    want = torch.full((N,), 16384.0 * K, dtype=torch.float64)
    want[1] = -128.0 * 127 * K
    assert torch.equal(got.cpu(), want.float().expand(M, N))
    wide = int8.Int8(torch.zeros(2, 131088, dtype=torch.int8, device="cuda")[:, :K + 1], torch.ones(2, device="cuda"))
    with pytest.raises(RuntimeError):
        int8.gemm(wide, wide)


@pytest.mark.parametrize("M", (1, 200, 2100))
def test_gemm_strided_scales_wide_rows_and_one_scale_for_all(M):
    N, K = 2150, 333
    a, qa, sa = operand(M, K, 8, ld=512)
    b, qb, sb = operand(N, K, 9, ld=400)
    every = lambda s: s.repeat_interleave(3)[::3]  # noqa: E731  strided
    got = int8.gemm(int8.Int8(a.q, every(a.s)), int8.Int8(b.q, every(b.s)), out_dtype=torch.float32)
    assert torch.equal(got, int8.gemm(a, b, out_dtype=torch.float32))
    d, size = ref.product(qa, sa, qb, sb)
    ref.close(got, d, ref.product_tolerance(torch.float32, d, size))
    one = torch.full((1,), 0.75, device="cuda")
    got = int8.gemm(int8.Int8(a.q, one.expand(M)), int8.Int8(b.q, one.expand(N)), out_dtype=torch.float32)
    d, size = ref.product(qa, torch.full((M,), 0.75), qb, torch.full((N,), 0.75))
    ref.close(got, d, ref.product_tolerance(torch.float32, d, size))


@pytest.mark.parametrize("M,N", [(50, 40), (2100, 2100)])
def test_gemm_scales_of_every_kind_stay_in_their_row_and_column(M, N):
    K = 260
    a, qa, sa = operand(M, K, 10)
    b, qb, sb = operand(N, K, 11)
    sa[3], sa[5], sa[7], sb[9], sb[11], sb[13] = float("nan"), float("inf"), -2.0, float("nan"), 0.0, 1e-40
    sa[6], sb[6] = 1e20, 1e25  # past a float's range together
    got = int8.gemm(int8.Int8(a.q, sa.cuda()), int8.Int8(b.q, sb.cuda()), out_dtype=torch.float32)
    d, size = ref.product(qa, sa, qb, sb)
    tol = ref.product_tolerance(torch.float32, d, size)
    ref.close(got, d, torch.nan_to_num(tol, nan=0.0, posinf=0.0))  # infinities and, times 0, NaN: as they are


def test_gemm_degenerate_sizes():
    a, _, _ = operand(4, 128, 12)
    none = int8.Int8(torch.empty(0, 128, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"))
    assert int8.gemm(none, a).shape == (0, 4) and int8.gemm(a, none).shape == (4, 0)
    flat = int8.quantize(torch.empty(4, 0, device="cuda"))
    assert flat.q.shape == (4, 0) and torch.equal(flat.s, torch.full((4,), 2.0 ** -100 / 127, device="cuda"))
    bias = torch.randn(5, device="cuda")
    five = int8.Int8(torch.empty(5, 0, dtype=torch.int8, device="cuda"), torch.full((5,), float("nan"), device="cuda"))
    assert torch.equal(int8.gemm(flat, five, bias=bias, out_dtype=torch.float32), bias.expand(4, 5))  # the scales are not read
    assert torch.equal(int8.gemm(flat, five, out_dtype=torch.bfloat16), torch.zeros(4, 5, device="cuda", dtype=torch.bfloat16))
    assert int8.quantize(torch.empty(0, 5, device="cuda")).q.shape == (0, 5)
    w = int8.quantize(torch.randn(6, 32, device="cuda"))
    assert int8.linear(torch.empty(0, 32, device="cuda"), w).shape == (0, 6)
    assert torch.equal(int8.linear(torch.empty(3, 0, device="cuda"), five, bias=bias), bias.expand(3, 5))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,I,O", [(1, 130, 70), (5, 512, 300), (200, 300, 257), (33, 4097, 65), (1, 17000, 20), (2100, 400, 2100),
                                   # few tokens in one launch, and just more than that
                                   (1, 1, 1), (1, 16384, 33), (1, 16377, 16), (2, 8192, 50), (3, 4091, 17), (4, 4096, 100), (7, 1999, 31),
                                   (8, 2048, 16), (9, 1000, 40), (16, 1024, 300), (16, 1025, 300), (15, 127, 5), (17, 128, 40), (2, 129, 4100)])
def test_linear_layer(T, I, O, kind):
    x = ref.values(T, I + 5, TYPES[kind], 20)[:, 2:-3]  # rows apart, odd
    w = ref.values(O, I, torch.float32, 21)
    bias = ref.values(1, O, TYPES[kind], 22)[0]
    wq = int8.quantize(w.cuda())
    got = int8.linear(x.cuda(), wq, bias=bias.cuda())
    assert got.dtype == TYPES[kind]
    assert torch.equal(got, int8.gemm(int8.quantize(x.cuda()), wq, bias=bias.cuda(), out_dtype=TYPES[kind]))
    want, size = ref.product(*ref.quantize(x), *ref.quantize(w), bias)
    ref.close(got, want, ref.product_tolerance(TYPES[kind], want, size))
    for out_type in TYPES.values():
        place = torch.empty(T, O + 4, device="cuda", dtype=out_type)[:, 1:-3]
        assert int8.linear(x.cuda(), wq, out=place) is place
        assert torch.equal(place, int8.linear(x.cuda(), wq, out_dtype=out_type))


@pytest.mark.parametrize("T", (40, 16, 5))
@pytest.mark.parametrize("kind", TYPES)
def test_linear_nan_stays_in_its_token(kind, T):
    x = ref.values(T, 300, TYPES[kind], 23)
    x[T - 3, 150], x[1, 3] = float("nan"), float("inf")
    y = int8.linear(x.cuda(), int8.quantize(torch.randn(70, 300, device="cuda")))
    bad = torch.isnan(y).cpu()
    assert bad[T - 3].all() and bad[1].all() and bad.sum() == 2 * 70


def test_linear_few_tokens_and_more_outputs_than_a_launch_has_tiles():
    """Blocks that take several tiles; and rows of a weight past 2^31 bytes."""
    w = torch.randint(-128, 128, (70001, 1024), device="cuda", dtype=torch.int8)
    s = torch.rand(70001, device="cuda") + 0.5
    for T in (1, 16):
        x = ref.values(T, 1000, torch.bfloat16, 27)
        y = int8.linear(x.cuda(), int8.Int8(w[:, :1000], s), out_dtype=torch.float32)
        want, size = ref.product(*ref.quantize(x), w[:, :1000].cpu(), s.cpu())
        ref.close(y, want, ref.product_tolerance(torch.float32, want, size))
    wide = torch.randint(-128, 128, (140000, 16384), device="cuda", dtype=torch.int8)
    s = torch.rand(140000, device="cuda") + 0.5
    x = ref.values(1, 16384, torch.bfloat16, 28)
    y = int8.linear(x.cuda(), int8.Int8(wide, s), out_dtype=torch.float32)
    at = torch.tensor([0, 131071, 131072, 139999], device="cuda")
    want, size = ref.product(*ref.quantize(x), wide[at].cpu(), s[at].cpu())
    ref.close(y[:, at], want, ref.product_tolerance(torch.float32, want, size))


@pytest.mark.parametrize("M", (3, 600))
def test_gemm_operands_past_two_gigabytes(M):
    """A's offsets pass 2^31 bytes; rows by sample."""
    K, rows = 65600, 33000
    g = torch.Generator(device="cuda").manual_seed(24)
    q = torch.randint(-128, 128, (rows, K), generator=g, device="cuda", dtype=torch.int8)
    s = torch.rand(rows, generator=g, device="cuda") + 0.5
    got = int8.gemm(int8.Int8(q, s), int8.Int8(q[:M], s[:M]), out_dtype=torch.float32)
    at = torch.tensor([0, 16384, 32760, rows - 1], device="cuda")
    want, size = ref.product(q[at].cpu(), s[at].cpu(), q[:M].cpu(), s[:M].cpu())
    ref.close(got[at], want, ref.product_tolerance(torch.float32, want, size))


def test_gemm_result_past_two_gigabytes():
    M, N, K = 40000, 33000, 48
    a, qa, sa = operand(M, K, 25)
    b, qb, sb = operand(N, K, 26)
    got = int8.gemm(a, b)
    for at in (slice(0, 3), slice(32767, 32770), slice(M - 2, M)):
        want, size = ref.product(qa[at], sa[at], qb, sb)
        ref.close(got[at], want, ref.product_tolerance(torch.bfloat16, want, size))


def test_quantize_past_two_gigabytes_and_the_widest_row():
    x = torch.randn(33000, 65600, device="cuda", dtype=torch.bfloat16)
    got = int8.quantize(x)
    for at in (slice(0, 2), slice(16383, 16386), slice(32998, 33000)):
        q, s = ref.quantize(x[at].cpu())
        ref.same(got.q[at], q)
        ref.same(got.s[at], s)
    del x, got
    n = (1 << 31) - 1
    x = torch.ones(1, n, device="cuda", dtype=torch.bfloat16)
    x[0, -1] = -254.0
    got = int8.quantize(x)
    assert got.s.item() == 2.0 and got.q[0, -1] == -127
    assert (got.q[0, :-1] == 0).all()  # 1/2 goes to the even code


def test_other_streams_and_captured_graphs():
    sizes = [(1, 300, 500), (200, 140, 512), (700, 900, 300), (2100, 2100, 300), (4097, 2048, 1000)]
    side = torch.cuda.Stream()
    for M, N, K in sizes:
        x = torch.randn(M, K, device="cuda")
        w = int8.quantize(torch.randn(N, K, device="cuda"))
        want = int8.linear(x, w)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = int8.linear(x, w)
        side.synchronize()
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = int8.linear(x, w)
            again = int8.gemm(int8.quantize(x), w, out_dtype=torch.float32)
        for i in range(3):
            x.copy_(torch.randn(M, K, device="cuda") * (i + 1))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, again)
            want = int8.linear(x, w)
            torch.cuda.synchronize()
            assert torch.equal(got, want), (M, N, K)


def test_refusals_of_the_tensor_forms():
    x = torch.randn(8, 256, device="cuda")
    a = int8.quantize(x)
    for bad in (lambda: int8.quantize(x.double()), lambda: int8.gemm(int8.Int8(a.q.view(torch.uint8), a.s), a),
                lambda: int8.gemm(int8.Int8(a.q, a.s.double()), a), lambda: int8.gemm(a, a, out_dtype=torch.float64),
                lambda: int8.gemm(a, a, bias=torch.ones(8, device="cuda", dtype=torch.float64)), lambda: int8.linear(x.double(), a),
                lambda: int8.gemm(a, a, out=torch.empty(8, 8, device="cuda"), out_dtype=torch.bfloat16),
                lambda: int8.gemm(a, a, bias=torch.ones(8)), lambda: int8.gemm(int8.Int8(a.q, a.s.cpu()), a)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: int8.quantize(x.T), lambda: int8.quantize(x[:1].expand(8, 256)), lambda: int8.gemm(a, int8.quantize(x[:, :128])),
                lambda: int8.gemm(int8.Int8(a.q, a.s[:4]), a), lambda: int8.gemm(a, a, out=torch.empty(8, 9, device="cuda")),
                lambda: int8.gemm(a, a, bias=torch.ones(7, device="cuda")), lambda: int8.gemm(a, a, bias=torch.ones(16, device="cuda")[::2]),
                lambda: int8.linear(x[:, :128], a), lambda: int8.quantize(x[0])):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros(4 * 200, dtype=torch.int8, device="cuda").view(4, 200)
    with pytest.raises(RuntimeError):  # rows of 200 bytes
        int8.gemm(int8.Int8(odd, torch.ones(4, device="cuda")), int8.Int8(odd, torch.ones(4, device="cuda")))
    short = torch.zeros(4 * 208 - 8, dtype=torch.int8, device="cuda").as_strided((4, 200), (208, 1))
    with pytest.raises(ValueError):  # the last row's padding is not there
        int8.gemm(int8.Int8(short, torch.ones(4, device="cuda")), a)


def test_out_counts_as_modified():
    a = int8.quantize(torch.randn(4, 64, device="cuda"))
    out = torch.zeros(4, 4, device="cuda")
    before = out._version
    int8.gemm(a, a, out=out)
    int8.linear(torch.randn(4, 64, device="cuda"), a, out=out)
    assert out._version == before + 2


@pytest.mark.parametrize("cols,per_block", ((1, 16), (8, 16), (200, 8), (1025, 1)))
def test_quantize_rows_of_a_blocks_second_turn(cols, per_block):
    """A launch has at most 2^31 threads, 256 a block here: `per_block` rows of the shape that takes these widths
    are a block's at a time, and the rows from per_block * 2^23 on a second turn's."""
    first = per_block << 23
    rows = first + 5
    x = torch.zeros(rows, cols, device="cuda", dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(cols)
    some = (torch.randn(40, cols, generator=g) * 3).bfloat16()
    places = torch.cat([torch.arange(10), torch.arange(first // 2, first // 2 + 10), torch.arange(rows - 20, rows)])
    x[places.cuda()] = some.cuda()
    q = torch.full((rows, cols), 0x55, dtype=torch.int8, device="cuda")
    s = torch.full((rows,), -1.0, device="cuda")
    assert int8.hip_int8_quantize(rows, cols, x, int8.BF16, cols, q, cols, s) == 0
    want, scales = ref.quantize(some)
    ref.same(q[places.cuda()], want)
    ref.same(s[places.cuda()], scales)
    others = torch.ones(rows, dtype=torch.bool, device="cuda")
    others[places.cuda()] = False
    for at in range(0, rows, 1 << 24):  # rows of zeros
        here = others[at:at + (1 << 24)]
        assert not q[at:at + (1 << 24)][here].any()
        assert (s[at:at + (1 << 24)][here] == torch.tensor(int8.AMAX_FLOOR / 127, dtype=torch.float32)).all()
