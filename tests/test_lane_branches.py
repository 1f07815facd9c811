"""The built kernels bring lanes back from a branch before they copy registers.

Where lanes of a wave part at a branch, the block in which they meet begins with the instruction that sets the mask of live
lanes back.  The compiler has put copies of registers before it (from the lower half of the register file to the upper,
where a kernel needs more than 256): a wave that jumps to the block with no lane live copies nothing, and reads what was
there before later on.  One build of the attention of many fp32 rows lost addresses that way and read outside its memory.
The kernels have no lane branches while their operands are in registers; here the disassembled library is searched."""
import os
import subprocess

import pytest

from rank_sgmv_bgmv_amd import build
from test_matrix_waits import OBJDUMP, kernels, listing

VECTOR = ("v_", "ds_", "global_", "buffer_", "flat_", "scratch_")
SCALAR = ("v_readlane", "v_writelane", "v_readfirstlane")  # of all lanes, live or not


def lost(kernel):
    """Vector instructions of a block that is jumped to with no lane live, before the one that brings the lanes back."""
    found = []
    for to in sorted({kernel.next[i][1] for i, (name, _) in enumerate(kernel.ins) if name == "s_cbranch_execz"}):
        before = []
        for name, rest in kernel.ins[to:]:
            if name.startswith("s_or") and "exec" in (name + rest):
                found += before
                break
            if name.startswith(("s_branch", "s_cbranch", "s_endpgm")) or rest.startswith("exec"):
                break
            if name.startswith(VECTOR) and not name.startswith(SCALAR):
                before.append(f"{name} {rest}")
    return found


def test_the_reading_itself():
    copy, back = "v_accvgpr_write_b32 a1, v1", "s_or_b64 exec, exec, s[0:1]"
    part = ["s_and_saveexec_b64 s[0:1], vcc", "s_cbranch_execz 1", "v_mov_b32_e32 v0, 0"]
    assert lost(listing(*part, copy, back, "s_endpgm")) == [copy]
    assert lost(listing(*part, "s_mov_b32 s4, s5", "v_readlane_b32 s6, v9, 3", back, copy, "s_endpgm")) == []


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="needs the disassembler of the compiler that built the library")
def test_lanes_are_back_before_registers_are_copied(tmp_path):
    if not os.path.exists(build.LIB):
        build.build()
    copy = tmp_path / "lib.so"
    copy.write_bytes(open(build.LIB, "rb").read())
    subprocess.run([OBJDUMP, "--offloading", copy.name], cwd=tmp_path, check=True, capture_output=True)
    branches, early = 0, {}
    for part in sorted(tmp_path.glob("*gfx950")):
        text = subprocess.run([OBJDUMP, "-d", str(part)], check=True, capture_output=True, text=True).stdout
        for name, kernel in kernels(text):
            branches += sum(i[0] == "s_cbranch_execz" for i in kernel.ins)
            if found := lost(kernel):
                early[name] = found
    assert branches > 100
    assert not early, early
