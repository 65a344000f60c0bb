"""The large tiles' assembly loops without a GPU: the committed text is what the
generator writes, and every LDS read of it is waited for before its use."""

import os
import re
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_fp32_matrix_row_amd", "csrc")
sys.path.insert(0, CSRC)
import gen_nt_loop  # noqa: E402


def test_committed_text_is_the_generators():
    with open(os.path.join(CSRC, "nt_loop.inc")) as f:
        assert f.read() == gen_nt_loop.generate()


def registers(text):
    out = set()
    for a, b in re.findall(r"\bv\[(\d+):(\d+)\]", text):
        out |= set(range(int(a), int(b) + 1))
    return out | {int(n) for n in re.findall(r"\bv(\d+)\b", text)}


def walk(lines):
    """One pass over straight text: the reads under way at each use."""
    under_way = []
    for n, line in enumerate(lines):
        op, _, rest = line.partition(" ")
        if op == "s_waitcnt":
            m = re.search(r"lgkmcnt\((\d+)\)", rest)
            if m:
                left = int(m.group(1))
                under_way = under_way[len(under_way) - left:] if left else []
            continue
        touched = registers(rest)
        for r in under_way:
            assert not (touched & r), (n, line)
        if op.startswith("ds_read"):
            under_way.append(registers(rest.split(",")[0]))
            under_way = under_way[-15:] if len(under_way) > 15 else under_way


@pytest.mark.parametrize("args", gen_nt_loop.LOOPS)
def test_registers_of_reads_under_way_are_not_touched(args):
    loop = gen_nt_loop.Loop(*args)
    assert loop.registers <= 256
    lines = loop.text()
    at = {line[:-1]: n for n, line in enumerate(lines) if line.startswith(".L")}
    begin, end = at[".Lnt_loop_%="], next(n for n, line in enumerate(lines) if line.startswith("s_cbranch_scc1 .Lnt_loop"))
    body = lines[begin + 1:end]
    walk(body + body + lines[end + 1:at.get(".Lnt_masked_%=", len(lines))])
    # one barrier a step, met by all loads: two steps a turn
    assert sum(line == "s_barrier" for line in body) == 2
    for n, line in enumerate(lines):
        if line == "s_barrier":
            assert lines[n - 1] == "s_waitcnt vmcnt(0) lgkmcnt(0)"
    # the loads of a turn: two whole steps' into each stage, each once
    loads = [(lines[n - 2], line) for n, line in enumerate(lines) if begin < n < end and "load" in line and line.endswith("lds")]
    loads += [("scales", n) for n, line in enumerate(body) if "load" in line and not line.endswith("offen lds")]
    assert len(loads) == 2 * loop.loads and len(set(loads)) == len(loads)
