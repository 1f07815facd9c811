"""The built kernels leave a matrix instruction the time it needs before its result is read or overwritten.

The hardware does not wait by itself: between a matrix instruction of N passes and another instruction than a product that
adds to the same registers, the program has to have N + 4 wait states (N + 3 for 2 passes; one an instruction, s_nop k is
k + 1).  The compiler puts them in, but has missed ways through a branch that is taken.  Here every way through the
disassembled kernels of the library is followed from each matrix instruction on."""
import os
import re
import subprocess

import pytest

from rank_sgmv_bgmv_amd import build

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"

# passes of 4 clocks
PASSES = {"v_mfma_f32_16x16x16_bf16": 4, "v_mfma_f32_16x16x32_bf16": 4, "v_mfma_f32_16x16x32_f16": 4,
          "v_mfma_i32_16x16x64_i8": 4, "v_mfma_f32_32x32x16_f16": 8, "v_mfma_f32_32x32x16_bf16": 8}


def registers(text):
    found = set()
    for kind, lo, hi, one in re.findall(r"\b([av])(?:\[(\d+):(\d+)\]|(\d+)\b)", text):
        found.update((kind, r) for r in range(int(lo or one), int(hi or one) + 1))
    return found


class Kernel:
    """Instructions (name, operands) and where each may go on."""

    def __init__(self, lines):
        self.ins, at = [], {}
        for address, text in lines:
            at[address] = len(self.ins)
            name, _, rest = text.partition(" ")
            self.ins.append((name, rest))
        self.next = []
        for i, ((address, _), (name, rest)) in enumerate(zip(lines, self.ins)):
            on = [i + 1] if i + 1 < len(lines) else []
            if name.startswith(("s_branch", "s_cbranch")):
                word = int(rest.split()[0], 0)  # in words of 4 bytes, from the next instruction on
                to = at[address + 4 + 4 * (word - 65536 if word >= 32768 else word)]
                on = [to] if name == "s_branch" else on + [to]
            elif name in ("s_endpgm", "s_setpc_b64"):
                on = []
            self.next.append(on)

    def early(self):
        """(product, instruction, wait states between them) where there are too few."""
        found = {}
        vector = [registers(rest) if name.startswith(("v_", "ds_", "global_", "buffer_", "flat_", "scratch_")) else set()
                  for name, rest in self.ins]
        for i, (name, rest) in enumerate(self.ins):
            if not name.startswith("v_mfma"):
                continue
            passes = PASSES[name]
            need, result = passes + 4, registers(rest.split(",")[0])
            least, ways = {}, [(j, 0) for j in self.next[i]]
            while ways:
                j, states = ways.pop()
                other, operands = self.ins[j]
                if other.startswith("v_mfma"):
                    states = max(states, passes)  # it begins when the first has left the matrix unit's first stage
                if states >= need or least.get(j, need) <= states:
                    continue
                least[j] = states
                if other.startswith("v_mfma"):
                    d, a, b = (registers(x) for x in operands.split(",")[:3])
                    hit = bool((a | b) & result)
                    if not hit and d == result:
                        continue  # from there on it is that product's result
                else:
                    hit = bool(vector[j] & result)
                if hit:
                    found[i, j] = min(states, found.get((i, j), need))
                    continue
                took = int(operands.split()[0], 0) + 1 if other == "s_nop" else 1
                ways += [(k, states + took) for k in self.next[j]]
        return [(" ".join(self.ins[i]), " ".join(self.ins[j]), states) for (i, j), states in sorted(found.items())]


def kernels(disassembly):
    name, lines = None, []
    for line in disassembly.splitlines():
        head = re.match(r"^[0-9a-f]+ <(\S+)>:", line)
        if head:
            if name:
                yield name, Kernel(lines)
            name, lines = head.group(1), []
        elif name and (m := re.match(r"^\t(\S.*?)\s*// ([0-9A-F]+):", line)):
            lines.append((int(m.group(2), 16), m.group(1)))
    if name:
        yield name, Kernel(lines)


def listing(*instructions):
    return Kernel([(4 * i, text) for i, text in enumerate(instructions)])


def test_the_reading_itself():
    """A result read too early, in a row and through a branch that is taken, and one that is not."""
    product = "v_mfma_f32_16x16x32_f16 a[0:3], v[0:3], v[4:7], a[0:3]"
    read = "v_accvgpr_read_b32 v9, a2"
    assert listing(product, "s_nop 6", read, "s_endpgm").early() == [(product, read, 7)]
    assert listing(product, "s_nop 7", read, "s_endpgm").early() == []
    other = "v_mfma_f32_16x16x32_f16 a[4:7], v[0:3], v[4:7], a[4:7]"
    skipped = listing(product, "s_cbranch_vccnz 2", other, "s_nop 4", read, "s_endpgm")
    assert skipped.early() == [(product, read, 1)]
    assert listing(product, other, "s_cbranch_vccnz 0", "s_nop 4", read, "s_endpgm").early() == []
    assert listing(product, "v_mfma_f32_16x16x32_f16 a[0:3], v[0:3], v[4:7], a[0:3]", "s_nop 7", read, "s_endpgm").early() == []
    assert len(listing(product, "v_mfma_f32_16x16x32_f16 a[4:7], a[0:3], v[4:7], 0", "s_endpgm").early()) == 1


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="needs the disassembler of the compiler that built the library")
def test_results_of_products_are_waited_for(tmp_path):
    if not os.path.exists(build.LIB):
        build.build()
    copy = tmp_path / "lib.so"
    copy.write_bytes(open(build.LIB, "rb").read())
    subprocess.run([OBJDUMP, "--offloading", copy.name], cwd=tmp_path, check=True, capture_output=True)
    products, early = 0, {}
    for part in sorted(tmp_path.glob("*gfx950")):
        text = subprocess.run([OBJDUMP, "-d", str(part)], check=True, capture_output=True, text=True).stdout
        for name, kernel in kernels(text):
            products += sum(i[0].startswith("v_mfma") for i in kernel.ins)
            if found := kernel.early():
                early[name] = found
    assert products > 1000
    assert not early, early
