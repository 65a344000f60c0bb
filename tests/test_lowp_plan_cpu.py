"""Which kernels the 8-bit product and the orthogonalised update take for a shape,
decided on the host."""

import pytest

from dense_fp32_matrix_row_amd import blockfp8, orthogonal, sgemm
from tests import lowp_shapes as shapes

LIMIT = 1 << 31  # work-items a launch takes
LARGEST = (1 << 31) - 1

SHAPES = [(1, 1, 1), (1, 4096, 4096), (300, 500, 0), (700, 700, 700), (2049, 2085, 640), (4097, 4097, 4097), (4100, 4200, 1600),
          (4097, 2048, 1000), (2048, 4097, 900), (8192, 8192, 8192), (100_000, 70_001, 300),
          (LARGEST, 1, 16), (1, LARGEST, 16), (LARGEST, 16, 1 << 23), (LARGEST - 300, 3, 128), (3, LARGEST - 127, 128),
          (LARGEST, 1, 0)]


@pytest.mark.parametrize("c_type", (blockfp8.F32, blockfp8.BF16, blockfp8.F16))
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_launches_cover_the_result_once_and_fit_a_launch(M, N, K, c_type):
    plan = blockfp8.hip_fp8_gemm_plan(M, N, K, c_type)
    assert 1 <= len(plan) <= blockfp8.MAX_LAUNCHES
    area = 0
    for p in plan:
        assert 0 < p["workgroups"] and p["workgroups"] * p["threads"] <= LIMIT
        assert p["row0"] >= 0 and p["row0"] + p["rows"] <= M and p["col0"] >= 0 and p["col0"] + p["cols"] <= N
        assert p["row0"] % 128 == 0 and p["col0"] % 128 == 0  # a block of scales begins there
        skip = p["skip_rows"] * p["skip_cols"]
        assert skip == 0 or p["skip_rows"] % p["tile_m"] == 0 == p["skip_cols"] % p["tile_n"]
        area += p["rows"] * p["cols"] - skip
    assert area == M * N
    # pieces are disjoint: with the right area, it is enough that no two share a corner or cover one another
    parts = [(p["row0"], p["col0"], p["row0"] + p["rows"], p["col0"] + p["cols"]) for p in plan if not p["skip_rows"]]
    for i, a in enumerate(parts):
        for b in parts[:i]:
            assert a[0] >= b[2] or b[0] >= a[2] or a[1] >= b[3] or b[1] >= a[3]


def test_plan_refusals_and_nothing_to_do():
    for args, status in (((-1, 1, 1, 0), -1), ((1, -1, 1, 0), -2), ((1, 1, -1, 0), -3), ((1, 1, 1, 3), -23)):
        with pytest.raises(sgemm.SgemmError) as e:
            blockfp8.hip_fp8_gemm_plan(*args)
        assert e.value.status == status
    assert blockfp8.hip_fp8_gemm_plan(0, 5, 5, 0) == [] == blockfp8.hip_fp8_gemm_plan(5, 0, 5, 0)


@pytest.mark.parametrize("table,c_types,tiles", [
    (shapes.GEMM_FLOAT, (blockfp8.F32,), {(16, 16), (32, 32), (64, 64), (128, 128)}),
    (shapes.GEMM_16_BIT, (blockfp8.BF16, blockfp8.F16), {(16, 16), (32, 32), (64, 64), (256, 128), (256, 256)}),
])
def test_the_gpu_tests_sizes_reach_every_tile_of_the_product(table, c_types, tiles):
    keys = ("tile_m", "tile_n", "row0", "col0", "skip_rows", "skip_cols")
    for size, launches in table.items():
        for c_type in c_types:
            assert [tuple(p[k] for k in keys) for p in blockfp8.hip_fp8_gemm_plan(*size, c_type)] == launches, size
    alone = {p[0][:2] for p in table.values() if len(p) == 1}
    assert alone == tiles
    edges = {(q[:2], "both" if q[4] else "right" if q[3] else "low") for p in table.values() for q in p[1:]}
    small = {(16, 16), (32, 32), (64, 64)}
    assert {t for t, _ in edges} == small and {side for _, side in edges} == {"both", "right", "low"}


def test_the_gpu_tests_sizes_reach_every_tile_of_the_update():
    for size, products in shapes.ORTHOGONALIZE.items():
        assert [tuple(p.values()) for p in orthogonal.hip_orthogonalize_plan(*size)] == products, size
        batch, rows, cols = size  # a tall matrix is iterated as its transpose
        assert [tuple(p.values()) for p in orthogonal.hip_orthogonalize_plan(batch, cols, rows)] == products, size
    for i in range(3):
        assert {p[i][0] for p in shapes.ORTHOGONALIZE.values()} == {32, 64, 128, 192, 256}
    for i in range(2):
        assert any(p[i][1] > 1 for p in shapes.ORTHOGONALIZE.values())
    assert {p[2][3] for p in shapes.ORTHOGONALIZE.values()} == {0, 32, 64, 128}
    assert {p[2][0] for p in shapes.ORTHOGONALIZE.values() if p[2][2]} == {128, 192, 256}


def test_update_plan_refusals_and_nothing_to_do():
    for size, status in (((-1, 4, 4), -1), ((65536, 4, 4), -1), ((1, -1, 4), -2), ((1, 4, orthogonal.MAX_SIZE + 1), -3)):
        with pytest.raises(sgemm.SgemmError) as e:
            orthogonal.hip_orthogonalize_plan(*size)
        assert e.value.status == status
    for size in ((0, 4, 4), (1, 0, 4), (1, 4, 0)):
        assert all(v == 0 for p in orthogonal.hip_orthogonalize_plan(*size) for v in p.values())
