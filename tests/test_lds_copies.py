"""Wait states before the copies from memory straight into LDS, read from the gfx950 assembly the
compiler writes (no GPU needed).

Those copies are written as inline assembly, which the compiler's own pass for such waits does not look
into.  gfx9 needs one wait state between a scalar write of m0, which holds a copy's LDS address, and
the copy, and five between a vector instruction's write of a scalar register and a memory instruction that
reads it (the copy's descriptor and offset).  Every instruction counts as one state, s_nop n as n + 1."""

import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from tests.test_kernel_resources import CSRC, ROOT, _hipcc

SOURCES = ("ns_gemm.hip", "linear_grad.hip", "peaks.hip", "attention.hip", "attention_dq.hip", "attention_dkv.hip")


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    cc, out = _hipcc(), tmp_path_factory.mktemp("asm")

    def compiled(src):
        to = str(out / (src + ".s"))
        subprocess.run([cc, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                        "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-x", "hip",
                        "--cuda-device-only", "-S", os.path.join(CSRC, src), "-o", to], check=True, capture_output=True)
        return open(to).read()

    with cf.ThreadPoolExecutor(max_workers=min(6, os.cpu_count() or 1)) as ex:
        return dict(zip(SOURCES, ex.map(compiled, SOURCES)))


def _program(text):
    """(instructions, their predecessors) of a listing."""
    ins, labels = [], {}
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        m = re.match(r"([.\w$@]+):", line)
        if m:
            labels[m.group(1)] = len(ins)
        elif re.match(r"[a-z]\w+(\s|$)", line) and not line.startswith("."):
            ins.append(line)
    before = [[] for _ in ins]
    for i, line in enumerate(ins):
        op = line.split()[0]
        if op.startswith(("s_branch", "s_cbranch")):
            to = labels.get(line.split()[1])
            if to is not None and to < len(ins):
                before[to].append(i)
        if i + 1 < len(ins) and op not in ("s_branch", "s_endpgm", "s_setpc_b64"):
            before[i + 1].append(i)
    return ins, before


def _registers(operand):
    """Scalar registers that an operand names."""
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.fullmatch(r"s(\d+)", operand)
    return {int(m.group(1))} if m else set()


def _operands(line):
    return [x.strip() for x in line.split(None, 1)[1].split(",")] if " " in line or "\t" in line else []


def _written(line):
    """Scalar registers a vector instruction writes (its first operand, or a carry behind a vector one)."""
    if not line.startswith("v_"):
        return set()
    ops = _operands(line)
    got = _registers(ops[0])
    if re.match(r"v_(\w+_co_|div_scale|mad_[iu]64)", line) and len(ops) > 1:
        got |= _registers(ops[1])
    return got


def _too_soon(ins, before):
    """The copies into LDS that follow too soon, and how many copies there are."""
    found, copies = [], 0
    for i, line in enumerate(ins):
        if not (line.startswith(("buffer_load", "global_load")) and re.search(r"\blds\b", line)):
            continue
        copies += 1
        reads = set()
        for x in _operands(line):
            for word in x.split():
                reads |= _registers(word)
        best = {}
        ahead = [(p, 0) for p in before[i]]
        while ahead:
            at, states = ahead.pop()
            if states >= 5 or best.get(at, 9) <= states:
                continue
            best[at] = states
            one = ins[at]
            if states < 1 and re.match(r"s_\w+\s+m0\b", one):
                found.append((one, line))
            if _written(one) & reads:
                found.append((one, line))
            m = re.match(r"s_nop (\d+)", one)
            states += int(m.group(1)) + 1 if m else 1
            ahead += [(p, states) for p in before[at]]
    return found, copies


def test_the_search_finds_what_it_looks_for():
    text = "f:\n s_mov_b32 m0, s2\n%s buffer_load_dwordx4 v1, s[4:7], 0 offen lds\n s_endpgm\n"
    assert len(_too_soon(*_program(text % ""))[0]) == 1
    assert _too_soon(*_program(text % " s_nop 0\n")) == ([], 1)
    lane = "f:\n v_readfirstlane_b32 s6, v0\n s_cbranch_scc1 .L1\n s_branch .L2\n.L1:\n s_nop %d\n" \
           "buffer_load_dword v1, s[4:7], 0 offen lds\n.L2:\n s_endpgm\n"
    assert len(_too_soon(*_program(lane % 2))[0]) == 1
    assert _too_soon(*_program(lane % 3)) == ([], 1)


@pytest.mark.parametrize("src", SOURCES)
def test_copies_into_lds_wait_for_their_registers(listings, src):
    found, copies = _too_soon(*_program(listings[src]))
    assert copies > 0
    assert not found, (src, len(found), copies, found[:3])
