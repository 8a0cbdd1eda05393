"""Wait states in front of exchanges between lanes, in the library as it was built.

A vector instruction's result may be taken from another lane (by a swap of rows or
halves, or a DPP operand) two wait states after it was written, no earlier.  The
compiler keeps that distance for the instructions it chose, but does not look into
inline assembly, so the machine code itself is read here."""
import re
import shutil
import subprocess
import os

import pytest

import mamba_ssd_chunked_02_amd as ssd

WAIT_STATES = 2
OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
REGISTERS = re.compile(r"\bv(?:(\d+)|\[(\d+):(\d+)\])")


def registers(operand):
    m = REGISTERS.search(operand)
    if not m:
        return set()
    if m.group(1):
        return {int(m.group(1))}
    return set(range(int(m.group(2)), int(m.group(3)) + 1))


def early_exchanges(lines):
    """(exchanges, those too near behind the write of what they take) of a listing."""
    seen, early = 0, []
    written = []  # wait states behind it, registers, instruction: of the last vector instructions
    function = "?"
    for line in lines:
        if line.endswith(">:"):
            function, written = line.split("<")[-1][:-2], []
            continue
        text = line.split("//")[0].strip()
        if not text or not line.startswith("\t"):
            continue
        name, _, rest = text.partition(" ")
        if name in ("s_endpgm", "s_branch"):  # what follows is reached from elsewhere
            written = []
            continue
        operands = rest.split(",")
        swap = name.startswith(("v_permlane16_swap", "v_permlane32_swap"))
        taken = set()
        if swap:
            taken = registers(operands[0]) | registers(operands[1])
        elif "_dpp" in name:  # the first source; comparisons and the like have another place for their result
            taken = registers(operands[1])
        if taken:
            seen += 1
            for states, regs, what in written:
                if regs & taken and states < WAIT_STATES:
                    early.append("%s: %s, %d behind %s" % (function, text, states, what))
        states = int(rest.split()[0], 0) + 1 if name == "s_nop" else 1
        written = [(s + states, regs, what) for s, regs, what in written if s + states < WAIT_STATES]
        if name.startswith("v_"):
            to = registers(operands[0])
            if swap or name.startswith("v_swap"):
                to |= registers(operands[1])
            written.append((0, to, text))
    return seen, early


def test_reader():
    """The reader finds what it is to find, in a listing written by hand."""
    def one(*body):
        return early_exchanges(["0 <f>:"] + ["\t%s // 00: 00" % b for b in body])
    swap = "v_permlane32_swap_b32_e32 v2, v5"
    fma = "v_fma_f32 v5, v1, v1, v1"
    assert one(fma, "s_nop 1", swap) == (1, [])
    assert one(fma, "v_mov_b32_e32 v9, 0", "s_nop 0", swap) == (1, [])
    assert len(one(fma, swap)[1]) == 1
    assert len(one(fma, "v_mov_b32_e32 v9, 0", swap)[1]) == 1
    assert len(one("v_pk_mul_f32 v[4:5], v[0:1], v[0:1]", "s_nop 0", swap)[1]) == 1
    assert len(one(swap, "v_permlane16_swap_b32_e32 v5, v7")[1]) == 1
    assert one(fma, "s_branch 12", swap) == (1, [])
    dpp = "v_add_f32_dpp v1, v5, v3 row_mirror row_mask:0xf bank_mask:0xf"
    assert len(one(fma, dpp)[1]) == 1 and one("v_mov_b32_e32 v3, 0", dpp) == (1, [])


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no disassembler")
def test_the_library(tmp_path):
    library = str(tmp_path / "lib.so")
    if not os.path.exists(ssd.library_path()):
        pytest.skip("the library is not built")
    shutil.copy(ssd.library_path(), library)
    subprocess.run([OBJDUMP, "--offloading", library], check=True, capture_output=True, cwd=tmp_path)
    seen, early = 0, []
    for f in sorted(os.listdir(tmp_path)):
        if "gfx950" not in f:
            continue
        r = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(tmp_path / f)], check=True, capture_output=True,
                           text=True)
        n, e = early_exchanges(r.stdout.splitlines())
        seen += n
        early += e
    assert seen > 1000
    assert not early, "%d of %d:\n%s" % (len(early), seen, "\n".join(early[:40]))
