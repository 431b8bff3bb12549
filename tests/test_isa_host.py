"""The built library's own gfx950 code, disassembled: what the hardware leaves to the program
where the compiler does not look, inside inline assembly.

  * An SGPR written by a vector instruction may be read by a memory instruction after five
    wait states (an instruction is one, s_nop N is N + 1), and m0 written by a scalar one by a
    load into LDS after one.
  * LDS accesses of 16 bytes are aligned to 16.
  * The innermost loops with matrix instructions keep their registers: at most 3 accesses to
    scratch memory in one (more measured 7 to 17% of a product).

Walks back from every memory instruction over all ways that lead to it."""

import os
import re
import shutil
import subprocess

import pytest

import w4a16_gemm_amd as w4

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"

pytestmark = pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="llvm-objdump is not available")

LINE = re.compile(r"^\t(\S+)\s*(.*?)\s*// ([0-9A-F]{12}): ")
HEAD = re.compile(r"^(?:[0-9a-f]+ )?<(\w+)>:$")
TARGET = re.compile(r"<(\w+)\+0x([0-9a-f]+)>")
SGPR = re.compile(r"\bs(?:\[(\d+):(\d+)\]|(\d+)\b)|\b(vcc|m0)\b")
TWO_RESULTS = re.compile(r"_co_|^v_div_scale|^v_mad_[ui]64")
VMEM = ("buffer_", "global_", "scratch_", "flat_")


def scalars(operands):
    regs = set()
    for lo, hi, one, name in SGPR.findall(operands):
        if name:
            regs.add(name)
        else:
            regs.update(range(int(lo or one), int(hi or one) + 1))
    return regs


def kernels(text):
    """{kernel: [(mnemonic, operands, address, branch target or None)]}"""
    found, name, rows = {}, None, None
    for line in text.splitlines():
        m = LINE.match(line)
        if m and rows is not None:
            op, operands, address = m.groups()
            target = TARGET.search(line) if op.startswith(("s_cbranch", "s_branch")) else None
            rows.append((op, operands, int(address, 16), target and int(target.group(2), 16)))
        else:
            h = HEAD.match(line)
            if h:
                name, rows = h.group(1), []
                found[name] = rows
    return found


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    """Kernels of the built library, by name."""
    w4.lib()
    from w4a16_gemm_amd import build
    folder = tmp_path_factory.mktemp("isa")
    copy = folder / "lib.so"
    shutil.copy(build.LIB, copy)
    subprocess.run([OBJDUMP, "--offloading", str(copy)], check=True, capture_output=True, cwd=folder)
    found = {}
    for image in sorted(folder.glob("*gfx950*")):
        text = subprocess.run([OBJDUMP, "-d", str(image)], check=True, capture_output=True, text=True).stdout
        found.update(kernels(text))
    assert sum(len(rows) for rows in found.values()) > 100000
    return found


def predecessors(rows):
    """Indexes that come before each instruction, by fall-through or branch."""
    start = rows[0][2] if rows else 0
    at = {address - start: i for i, (_, _, address, _) in enumerate(rows)}
    before = [[i - 1] if i and rows[i - 1][0] not in ("s_branch", "s_endpgm", "s_setpc_b64") else [] for i in range(len(rows))]
    for i, row in enumerate(rows):
        if row[3] is not None and row[3] in at:
            before[at[row[3]]].append(i)
    return before


def written_by_vector(row):
    op, operands = row[0], row[1]
    if not op.startswith("v_"):
        return set()
    parts = operands.split(", ")
    return scalars(", ".join(parts[:2] if TWO_RESULTS.search(op) else parts[:1]))


def too_soon(rows, before, i, regs, writes, states):
    """An instruction that writes one of regs, fewer than `states` wait states before i."""
    todo, seen = [(p, 0) for p in before[i]], set()
    while todo:
        j, passed = todo.pop()
        if passed >= states or (j, passed) in seen:
            continue
        seen.add((j, passed))
        if writes(rows[j]) & regs:
            return j
        op, operands = rows[j][:2]
        passed += int(operands) + 1 if op == "s_nop" else 1
        todo.extend((p, passed) for p in before[j])
    return None


def report(name, rows, j, i):
    return f"{name}:\n" + "\n".join(f"    {rows[k][0]} {rows[k][1]}" for k in ([*range(j, i + 1)] if j < i else [j, i]))


def hazards(name, rows):
    before = predecessors(rows)
    for i, (op, operands, _, _) in enumerate(rows):
        if not op.startswith(VMEM):
            continue
        regs = scalars(operands)
        if regs:
            j = too_soon(rows, before, i, regs, written_by_vector, 5)
            if j is not None:
                yield report(name, rows, j, i)
        if operands.endswith(" lds") or "_lds_" in op:
            j = too_soon(rows, before, i, {"m0"},
                         lambda row: scalars(row[1].split(", ")[0]) if row[0].startswith("s_") else set(), 1)
            if j is not None:
                yield report(name, rows, j, i)


def test_scalar_operands_of_memory_instructions_have_settled(library):
    assert any(" lds" in operands or "_lds_" in op for rows in library.values() for op, operands, _, _ in rows)
    found = [h for name, rows in library.items() for h in hazards(name, rows)]
    assert not found, f"{len(found)} of them, the first:\n" + "\n".join(found[:3])


def test_16_byte_accesses_of_lds_are_aligned(library):
    """What an instruction adds to its address keeps the address's own alignment."""
    found = {}
    for name, rows in library.items():
        for op, operands, _, _ in rows:
            if re.fullmatch(r"ds_(read|write)_b128", op):
                offset = re.search(r"offset:(\d+)", operands)
                if offset and int(offset.group(1)) % 16:
                    found.setdefault(name, f"{op} {operands}")
    assert not found, found


def inner_products(rows):
    """(first, last) instruction of the innermost loops with matrix instructions."""
    at = {row[2] - rows[0][2]: i for i, row in enumerate(rows)}
    loops = [(at[row[3]], i) for i, row in enumerate(rows) if row[3] in at and at[row[3]] <= i]
    loops = [(a, b) for a, b in loops if any(row[0].startswith("v_mfma") for row in rows[a:b])]
    return [(a, b) for a, b in loops if not any((c, d) != (a, b) and a <= c and d <= b for c, d in loops)]


def test_products_keep_their_registers(library):
    found, seen = {}, 0
    for name, rows in library.items():
        for a, b in inner_products(rows):
            seen += 1
            count = sum(row[0].startswith("scratch_") for row in rows[a:b])
            if count > 3:
                found[name] = max(count, found.get(name, 0))
    assert seen > 100
    assert not found, found


SAMPLE = """
<kernel>:
\tv_readfirstlane_b32 s3, v2                                 // 000000000100: 7E060502
\ts_mov_b32 m0, s1                                           // 000000000104: BEFC0001
\ts_nop {nop}                                                    // 000000000108: BF800000
\tbuffer_load_dwordx4 v20, s[8:11], s3 offen lds             // 00000000010C: E05D1000 03020014
\ts_cbranch_scc1 65533                                       // 000000000114: BF85FFFD <kernel+0xc>
\ts_endpgm                                                   // 000000000118: BF810000
"""


@pytest.mark.parametrize("nop,found", [(0, 1), (2, 1), (3, 0), (4, 0)])
def test_the_walk_finds_what_it_looks_for(nop, found):
    (name, rows), = kernels(SAMPLE.format(nop=nop)).items()
    assert len(list(hazards(name, rows))) == found


def test_the_walk_follows_branches():
    """The write lies behind the read, one step before the jump back to it."""
    text = SAMPLE.format(nop=4).replace("\ts_cbranch_scc1",
                                        "\tv_readlane_b32 s9, v2, 1                  // 000000000112: D2890009\n\ts_cbranch_scc1")
    (name, rows), = kernels(text).items()
    assert len(list(hazards(name, rows))) == 1
