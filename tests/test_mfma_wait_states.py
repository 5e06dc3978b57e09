"""Wait states behind the matrix instructions that are written in inline assembly
(csrc/attention.hip), read from the disassembly of the built device code.

The compiler keeps the distances that the hardware asks for behind its own matrix
instructions but does not look into assembly. Checked along every path of the pipelined
attention kernels, branches included, behind each of them (eight passes):
  - 12 wait states before anything but a matrix instruction touches its result, or a
    matrix instruction reads it as an operand or as part of another accumulator;
  - 8 before anything but a matrix instruction writes the accumulator it started from.
A matrix instruction that goes on with the same accumulator needs none. And before each:
  - 2 behind a vector instruction that writes an operand of it."""

import os
import re
import shutil
import subprocess

import pytest

import int8_gemm_amd as cr

OBJDUMP = next((p for p in ("/opt/rocm/llvm/bin/llvm-objdump", shutil.which("llvm-objdump"))
                if p and os.path.exists(p)), None)
RESULT, STARTED, OPERAND = 12, 8, 2


def registers(operand):
    """The vector registers an operand names, as (file, number)."""
    found = set()
    for m in re.finditer(r"\b([va])(\d+)\b|\b([va])\[(\d+):(\d+)\]", operand):
        if m[1]:
            found.add((m[1], int(m[2])))
        else:
            found |= {(m[3], n) for n in range(int(m[4]), int(m[5]) + 1)}
    return found


class Instruction:
    def __init__(self, line):
        text, _, note = line.partition("//")
        self.text = text.strip()
        self.op, _, rest = self.text.partition(" ")
        self.args = [a.strip() for a in re.split(r",(?![^\[]*\])", rest)] if rest else []
        self.address = int(note.split(":")[0], 16)
        target = re.search(r"<\S+\+0x([0-9a-f]+)>", note)
        self.target = int(target[1], 16) if target and "branch" in self.op else None
        self.mfma = self.op.startswith("v_mfma")
        self.regs = [registers(a) for a in self.args]
        self.states = int(self.args[0], 0) + 1 if self.op == "s_nop" else 1
        # a store has no result; other instructions write their first operand
        stores = "store" in self.op or self.op.startswith("ds_write")
        self.writes = self.regs[0] if self.regs and not stores else set()
        self.touches = set().union(*self.regs) if self.regs else set()


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if OBJDUMP is None:
        pytest.skip("no llvm-objdump")
    if not os.path.exists(cr.library_path()):
        from int8_gemm_amd import _build
        _build.build()
    where = tmp_path_factory.mktemp("code")
    lib = shutil.copy(cr.library_path(), where / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", str(lib)], check=True, capture_output=True, cwd=where)
    found = {}
    for obj in sorted(where.glob("*gfx950*")):
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(obj)], check=True,
                              capture_output=True, text=True).stdout
        lines = None
        for line in text.splitlines():
            start = re.match(r"[0-9a-f]+ <(.+)>:", line)
            if start:
                lines = found.setdefault(start[1], []) if "attention_wide" in start[1] else None
            elif lines is not None and "//" in line:
                lines.append(Instruction(line))
    return found


def paths(code, at, states):
    """Instructions within `states` wait states behind code[at], on every path, with the
    states that lie between."""
    index = {c.address - code[0].address: i for i, c in enumerate(code)}
    seen, todo = {}, [(at + 1, 0)]
    while todo:
        i, gone = todo.pop()
        if gone >= states or i >= len(code) or seen.get(i, states) <= gone:
            continue
        seen[i] = gone
        c = code[i]
        yield c, gone
        if c.op in ("s_endpgm", "s_setpc_b64"):
            continue
        if c.target is not None:
            todo.append((index[c.target], gone + 1))
            if c.op == "s_branch":
                continue
        todo.append((i + 1, gone + c.states))


def test_matrix_results_are_waited_for(kernels):
    assert len(kernels) >= 4
    seen, bad = 0, []
    for name, code in kernels.items():
        for i, c in enumerate(code):
            near = code[i + 1:i + 1 + OPERAND]
            if c.op.startswith("v_") and not c.mfma and any(d.mfma or d.target for d in near):
                for d, gone in paths(code, i, OPERAND):
                    if d.mfma and c.writes & set().union(*d.regs[1:4]):
                        bad.append((name, gone, c.text, d.text))
            if not c.mfma:
                continue
            seen += 1
            result, start = c.regs[0], c.regs[3]
            for d, gone in paths(code, i, RESULT):
                if d.mfma:
                    operands = d.regs[1] | d.regs[2]
                    if d.regs[3] != result:
                        operands = operands | d.regs[3]
                    if operands & result:
                        bad.append((name, gone, c.text, d.text))
                elif d.touches & result:
                    bad.append((name, gone, c.text, d.text))
                elif gone < STARTED and d.writes & start:
                    bad.append((name, gone, c.text, d.text))
    assert seen > 500
    assert not bad, f"{len(bad)}: {bad[:3]}"


def test_the_check_finds_what_it_looks_for():
    def code(*lines):
        return [Instruction(f"\t{t}  // {4 * i:012X}: {n}") for i, (t, n) in enumerate(lines)]
    mfma = ("v_mfma_f32_32x32x16_bf16 a[0:15], v[0:3], v[4:7], a[0:15]", "")
    near = code(mfma, ("s_nop 10", ""), ("v_accvgpr_read_b32 v9, a15", ""))
    got = [(d.text, gone) for d, gone in paths(near, 0, RESULT)]
    assert got == [("s_nop 10", 0), ("v_accvgpr_read_b32 v9, a15", 11)]
    assert near[2].touches & near[0].regs[0] == {("a", 15)}
    far = code(mfma, ("s_nop 11", ""), ("v_accvgpr_read_b32 v9, a15", ""))
    assert [d.op for d, _ in paths(far, 0, RESULT)] == ["s_nop"]
    back = code(("v_mov_b32_e32 v1, a3", ""), mfma, ("s_cbranch_scc1 -3", "BF <k+0x0>"),
                ("s_endpgm", ""))
    assert "v_mov_b32_e32" in [d.op for d, _ in paths(back, 1, RESULT)]
