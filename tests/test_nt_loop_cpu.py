"""The large tiles' assembly loops without a GPU: the committed text is what the
generator writes; replayed, every step's loads go to its stage and have arrived
at its barrier, and no register that an LDS read is on its way to is touched."""

import os
import re
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_fp32_matrix_row_amd", "csrc", "lowp")
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
    assert loop.registers <= 240
    lines = loop.text()
    at = {line[5:-4]: n for n, line in enumerate(lines) if line.startswith(".L")}
    back = lines.index("s_branch .Lnt_turn_%=")
    turn, until = lines[at["turn"] + 1:at["check"]], lines[at["check"] + 1:back]
    last = lines[at["next"] + 1:lines.index("s_branch .Lnt_last_%=")]
    for end in [e for e in ("whole", "masked") if e in at]:
        stop = at["masked"] if end == "whole" and "masked" in at else len(lines)
        walk(2 * (turn + until) + turn + last + lines[at[end] + 1:stop])
    body = turn + until
    # one barrier a step, met by the loads that the next step needs
    assert sum(line == "s_barrier" for line in body) == loop.positions
    for n, line in enumerate(lines):
        if line == "s_barrier":
            assert lines[n - 1].startswith("s_waitcnt vmcnt(") and lines[n - 1].endswith("lgkmcnt(0)")
    # a turn's loads: every part of every stage as often
    loads = [(body[n - 2], line) for n, line in enumerate(body) if "load" in line and line.endswith("lds")]
    loads += [(line, line) for line in body if "load" in line and not line.endswith("lds")]
    assert len(loads) == loop.positions * loop.loads
    assert all(loads.count(x) == loop.positions // loop.stages for x in loads)


def run(loop, n):
    """Replays the scalar control flow for n steps: the stages that are loaded and
    read, in order, and how many loads may be under way at each barrier."""
    lines = loop.text()
    at = {line[:-1]: k for k, line in enumerate(lines) if line.startswith(".L")}
    u = loop.positions
    first = (u - n % u) % u
    regs = {"%[first]": first, "%[turns]": (n - 1) // u - (first == u - 1), "%[left]": n, "%[single]": int(n == 1), "%[partial]": 0}
    val = lambda t: regs[t] if t in regs else int(t, 0)  # noqa: E731
    scc, k, steps, barriers, matrix, zero = 0, 0, 0, [], 0, False
    issued, arrived = [], 0  # the stage of each load, in order; how many have come
    while k < len(lines):
        op, _, rest = lines[k].partition(" ")
        args = [x.strip() for x in rest.split(",")]
        if op == "s_cmp_eq_u32":
            scc = val(args[0]) == val(args[1])
        elif op == "s_cmp_lg_u32" and args[0] in regs:
            scc = val(args[0]) != val(args[1])
        elif op == "s_cmp_gt_i32":
            zero = not val(args[0]) > val(args[1])
        elif op == "s_bitcmp1_b32":
            scc = bool(val(args[0]) >> val(args[1]) & 1)
        elif op == "s_sub_u32" and args[0] in regs:
            regs[args[0]] -= val(args[2])
        elif op == "s_branch" or (op == "s_cbranch_scc1" and scc):
            k = at[rest]
            continue
        elif "load" in op:
            if rest.endswith("lds"):
                m0 = int(lines[k - 2].split(",")[2])
                scales = m0 >= loop.stages * loop.stride
                stage = (m0 - loop.stages * loop.stride) // loop.scale_stage if scales else m0 // loop.stride
            else:
                stage = int(args[0][1:]) - loop.sv
            issued.append((stage, zero))
        elif op == "s_waitcnt" and "vmcnt" in rest:
            arrived = max(arrived, len(issued) - int(rest[6:rest.index(")")]))
        elif op == "s_barrier":
            barriers.append(arrived)
        elif op.startswith("v_mfma"):
            matrix += 1
        k += 1
    return first, issued, barriers, matrix


@pytest.mark.parametrize("args", gen_nt_loop.LOOPS)
def test_every_step_is_loaded_in_order_and_has_arrived(args):
    loop = gen_nt_loop.Loop(*args)
    per = loop.mt * loop.nt * {"p": 3, "w": 4}.get(loop.kind[0], 1)
    for n in range(1, 4 * loop.positions + 3):
        first, issued, barriers, matrix = run(gen_nt_loop.Loop(*args), n)
        assert matrix == n * per
        # a barrier before each step, behind which its loads have come
        assert len(barriers) == n
        for step in range(n):
            mine = issued[step * loop.loads:(step + 1) * loop.loads]
            assert len(mine) == loop.loads and barriers[step] >= (step + 1) * loop.loads
            assert mine == [((first + step) % loop.stages, False)] * loop.loads
        assert all(zero for _, zero in issued[n * loop.loads:])
