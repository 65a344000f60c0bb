"""The integer product's plans and its large tiles' assembly loops without a GPU."""

import os

import pytest

from dense_fp32_matrix_row_amd import int8, sgemm
from tests import serving_shapes as shapes
from tests.test_nt_loop_cpu import CSRC, gen_nt_loop, run, walk

LIMIT = 1 << 31  # work-items a launch takes
LARGEST = (1 << 31) - 1


def test_committed_text_is_the_generators():
    with open(os.path.join(CSRC, "int8_loop.inc")) as f:
        assert f.read() == gen_nt_loop.generate(gen_nt_loop.INT8_LOOPS)


@pytest.mark.parametrize("args", gen_nt_loop.INT8_LOOPS)
def test_registers_of_reads_under_way_are_not_touched(args):
    loop = gen_nt_loop.Loop(*args)
    assert loop.registers <= 240
    lines = loop.text()
    at = {line[5:-4]: n for n, line in enumerate(lines) if line.startswith(".L")}
    back = lines.index("s_branch .Lnt_turn_%=")
    turn, until = lines[at["turn"] + 1:at["check"]], lines[at["check"] + 1:back]
    last = lines[at["next"] + 1:lines.index("s_branch .Lnt_last_%=")]
    for end, stop in (("whole", at["masked"]), ("masked", len(lines))):
        walk(2 * (turn + until) + turn + last + lines[at[end] + 1:stop])
    body = turn + until
    assert sum(line == "s_barrier" for line in body) == loop.positions  # one a step
    for n, line in enumerate(lines):
        if line == "s_barrier":
            assert lines[n - 1].startswith("s_waitcnt vmcnt(") and lines[n - 1].endswith("lgkmcnt(0)")
    loads = [(body[n - 2], line) for n, line in enumerate(body) if "load" in line]
    assert len(loads) == loop.positions * loop.loads
    assert all(loads.count(x) == loop.positions // loop.stages for x in loads)


@pytest.mark.parametrize("args", gen_nt_loop.INT8_LOOPS)
def test_every_step_is_loaded_in_order_and_has_arrived(args):
    loop = gen_nt_loop.Loop(*args)
    for n in range(1, 4 * loop.positions + 3):
        first, issued, barriers, matrix = run(gen_nt_loop.Loop(*args), n)
        assert matrix == n * loop.mt * loop.nt * 2  # two products of 64 along K
        assert len(barriers) == n
        for step in range(n):
            mine = issued[step * loop.loads:(step + 1) * loop.loads]
            assert len(mine) == loop.loads and barriers[step] >= (step + 1) * loop.loads
            assert mine == [((first + step) % loop.stages, False)] * loop.loads
        assert all(zero for _, zero in issued[n * loop.loads:])


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 4096, 4096), (700, 700, 700), (2049, 2085, 640), (4097, 4097, 4097), (8192, 8192, 8192),
                                   (4100, 4200, 1600), (100_000, 70_001, 300), (LARGEST, 1, 16), (1, LARGEST, 16),
                                   (LARGEST, 16, int8.MAX_K), (LARGEST - 300, 3, 128), (3, LARGEST - 127, 128)])
def test_launches_cover_the_result_once_and_fit_a_launch(M, N, K):
    plan = int8.hip_int8_gemm_plan(M, N, K)
    assert 1 <= len(plan) <= int8.MAX_LAUNCHES
    area = 0
    for p in plan:
        assert 0 < p["workgroups"] and p["workgroups"] * p["threads"] <= LIMIT
        assert p["row0"] >= 0 and p["row0"] + p["rows"] <= M and p["col0"] >= 0 and p["col0"] + p["cols"] <= N
        skip = p["skip_rows"] * p["skip_cols"]
        assert skip == 0 or p["skip_rows"] % p["tile_m"] == 0 == p["skip_cols"] % p["tile_n"]
        area += p["rows"] * p["cols"] - skip
    assert area == M * N
    parts = [(p["row0"], p["col0"], p["row0"] + p["rows"], p["col0"] + p["cols"]) for p in plan if not p["skip_rows"]]
    for i, a in enumerate(parts):
        for b in parts[:i]:
            assert a[0] >= b[2] or b[0] >= a[2] or a[1] >= b[3] or b[1] >= a[3]


def test_plan_refusals_and_nothing_to_do():
    for args, status in (((-1, 1, 1), -1), ((1, -1, 1), -2), ((1, 1, -1), -3), ((1, 1, int8.MAX_K + 1), -3)):
        with pytest.raises(sgemm.SgemmError) as e:
            int8.hip_int8_gemm_plan(*args)
        assert e.value.status == status
    for size in ((0, 5, 5), (5, 0, 5), (5, 5, 0)):
        assert int8.hip_int8_gemm_plan(*size) == []


def test_the_gpu_tests_sizes_reach_every_tile():
    keys = ("tile_m", "tile_n", "row0", "col0", "skip_rows", "skip_cols")
    for size, launches in shapes.INT8.items():
        assert [tuple(p[k] for k in keys) for p in int8.hip_int8_gemm_plan(*size)] == launches, size
    assert {p[0][:2] for p in shapes.INT8.values() if len(p) == 1} == set(shapes.INT8_TILES)
    edges = {"both" if q[4] else "right" if q[3] else "low" for p in shapes.INT8.values() for q in p[1:]}
    assert edges == {"both", "right", "low"}


def test_the_quantiser_has_no_kernel_that_no_width_takes():
    """Rows of fewer than eight columns have kernels of their own, of the narrowest shape alone, for three types."""
    import re
    with open(sgemm.LIBRARY, "rb") as f:
        names = set(re.findall(rb"k_rowsILb0ENS_8RowShapeILi(\d+)ELi(\d+)ELi\d+EEE([a-zA-Z0-9_]*?)EEv", f.read()))
    assert {(lanes, chunks) for lanes, chunks, _ in names} == {(b"16", b"1")} and len(names) == 3
