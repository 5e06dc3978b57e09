"""Wait states of the built device code, read from its disassembly.

The compiler keeps the distances that the hardware asks for between its own
instructions but does not look into blocks of inline assembly, which the
global -> LDS copies are written in (csrc/lds_copy.h). Checked along the
straight-line order of every kernel:
  - a scalar write of M0, then a copy to LDS: one wait state;
  - a vector instruction's write of an SGPR, then a memory access that reads
    it: five."""

import os
import re
import shutil
import subprocess

import pytest

import int8_gemm_amd as cr

OBJDUMP = next((p for p in ("/opt/rocm/llvm/bin/llvm-objdump", shutil.which("llvm-objdump"))
                if p and os.path.exists(p)), None)


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """The instructions of each device function of the library."""
    if OBJDUMP is None:
        pytest.skip("no llvm-objdump")
    if not os.path.exists(cr.library_path()):
        from int8_gemm_amd import _build
        _build.build()
    where = tmp_path_factory.mktemp("code")
    lib = shutil.copy(cr.library_path(), where / "lib.so")
    # device objects are written beside the file
    subprocess.run([OBJDUMP, "--offloading", str(lib)], check=True, capture_output=True,
                   cwd=where)
    found = {}
    for i, obj in enumerate(sorted(where.glob("*gfx950*"))):
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(obj)], check=True,
                              capture_output=True, text=True).stdout
        lines = None
        for line in text.splitlines():
            start = re.match(r"[0-9a-f]+ <(.+)>:", line)
            line = line.split("//")[0].strip()
            if start:
                lines = found.setdefault((i, start.group(1)), [])
            elif lines is not None and line:
                lines.append(line)
    assert len(found) > 50
    return found


def split(line):
    """(mnemonic, operands) of an instruction."""
    op, _, rest = line.partition(" ")
    return op, [a.strip() for a in rest.split(",")]


def before(lines, at, states):
    """The instructions less than `states` wait states before lines[at]."""
    for line in reversed(lines[:at]):
        op, args = split(line)
        if states <= 0 or op in ("s_endpgm", "s_branch", "s_setpc_b64"):
            return
        yield op, args
        states -= int(args[0]) + 1 if op == "s_nop" else 1


def sgprs(operand):
    """The numbers of the SGPRs that an operand names."""
    found = set()
    for m in re.finditer(r"\bs(\d+)\b|\bs\[(\d+):(\d+)\]", operand):
        found |= {int(m[1])} if m[1] else set(range(int(m[2]), int(m[3]) + 1))
    return found


def copies(lines):
    return [i for i, line in enumerate(lines) if split(line)[0].startswith("global_load_lds")]


def test_copies_wait_for_m0(kernels):
    seen, bad = 0, []
    for (_, name), lines in kernels.items():
        for i in copies(lines):
            seen += 1
            for op, args in before(lines, i, 1):
                if op.startswith("s_") and args[0] == "m0":
                    bad.append((name, lines[i - 1], lines[i]))
    assert seen > 100
    assert not bad, f"{len(bad)} of {seen}: {bad[0]}"


def test_accesses_wait_for_sgprs_that_vector_instructions_write(kernels):
    seen, bad = 0, []
    for (_, name), lines in kernels.items():
        for i, line in enumerate(lines):
            op, args = split(line)
            if not re.match(r"(global|flat|buffer|scratch)_", op):
                continue
            read = set().union(*(sgprs(a) for a in args))
            seen += bool(read)
            for was, to in before(lines, i, 5) if read else ():
                if was.startswith("s_"):
                    # a scalar write since, which waits for the vector one by itself
                    read = read - sgprs(to[0])
                # results: the first operand, or the first two (carries)
                elif was.startswith("v_") and \
                        sgprs(to[0] + " " + (to[1] if "_co_" in was else "")) & read:
                    bad.append((name, was, to, line))
    assert seen > 100
    assert not bad, f"{len(bad)} of {seen}: {bad[0]}"
