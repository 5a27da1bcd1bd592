"""Wait states in the built device code (CPU only: reads the disassembly of the
library).  The compiler puts the waits a gfx950 hazard needs between its own
instructions, and none inside or before inline assembly, so the sources have to
keep to them there:
  * a scalar write of m0 and a load into LDS that uses it: 1;
  * a vector write of a scalar register and a memory instruction that reads it: 5;
  * a matrix product and any other instruction that reads or writes its result:
    12 (8 passes: the 16-bit 32x32x16 products) or 20 (16 passes: FP8 32x32x64)."""
import os
import re
import shutil
import subprocess

import pytest

from delayed_scaling_amd import LIB_PATH

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
_REG = re.compile(r"\b([sva])(?:(\d+)\b|\[(\d+):(\d+)\])")
_TARGET = re.compile(r"<[^>]*\+0x([0-9a-f]+)>|<([^>+]+)>")


def registers(text):
    """Every register an operand text names, as (file, number)."""
    out = set()
    for f, one, lo, hi in _REG.findall(text):
        out.update((f, n) for n in (range(int(one), int(one) + 1) if one else range(int(lo), int(hi) + 1)))
    if "vcc" in text:
        out.update((("s", 106), ("s", 107)))
    if re.search(r"\bm0\b", text):
        out.add(("s", 124))
    return out


class Function:
    """One function's instructions: (mnemonic, operands) in order, and the places
    an instruction can be followed by."""

    def __init__(self, name, start):
        self.name, self.start, self.ops, self.at, self.jump = name, start, [], {}, {}

    def add(self, address, op, operands, target):
        self.at[address] = len(self.ops)
        if target is not None:
            self.jump[len(self.ops)] = target
        self.ops.append((op, operands))

    def after(self, i):
        op = self.ops[i][0]
        out = []
        if i in self.jump and self.jump[i] in self.at:
            out.append(self.at[self.jump[i]])
        if op not in ("s_branch", "s_endpgm", "s_setpc_b64") and i + 1 < len(self.ops):
            out.append(i + 1)
        return out

    def within(self, i, states):
        """Instructions that can issue fewer than `states` wait states after i."""
        best, todo = {}, [(n, 0) for n in self.after(i)]
        while todo:
            n, waited = todo.pop()
            if waited >= states or best.get(n, states) <= waited:
                continue
            best[n] = waited
            op, operands = self.ops[n]
            step = int(operands, 0) + 1 if op == "s_nop" else 1
            todo += [(m, waited + step) for m in self.after(n)]
        return best

    def text(self, i):
        return " ".join(self.ops[i])


def functions(tmp):
    """The functions of every gfx950 code object in the library."""
    shutil.copy(LIB_PATH, os.path.join(tmp, "lib.so"))
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp, check=True, capture_output=True)
    objects = [f for f in sorted(os.listdir(tmp)) if f.endswith("gfx950")]
    assert objects
    for obj in objects:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--mcpu=gfx950", obj], cwd=tmp, check=True,
                              capture_output=True, text=True).stdout
        f = None
        for line in text.splitlines():
            if line.startswith("\t") and "//" in line:
                body, _, note = line.partition("//")
                op, _, operands = body.strip().partition(" ")
                target = None
                if op.startswith(("s_branch", "s_cbranch")):
                    m = _TARGET.search(note) or _TARGET.search(operands)
                    target = f.start + (int(m.group(1), 16) if m.group(1) else 0) if m else None
                f.add(int(note.strip().split(":")[0], 16), op, operands.strip(), target)
            elif line.endswith(">:"):
                if f is not None:
                    yield f
                address, name = line[:-1].split(" ", 1)
                f = Function(name.strip("<>"), int(address, 16))
        if f is not None:
            yield f


MEMORY = ("buffer_", "global_", "flat_", "scratch_", "ds_")


def destination(operands):
    return operands.split(",", 1)[0]


def hazards(f):
    for i, (op, operands) in enumerate(f.ops):
        if op.startswith("s_") and destination(operands) == "m0":
            for n in f.within(i, 1):
                if f.ops[n][0].startswith("buffer_load") and f.ops[n][1].endswith(" lds"):
                    yield "m0", i, n
        elif op.startswith(("v_readfirstlane", "v_readlane")) or (op.startswith("v_cmp") and operands[0] in "sv"):
            written = {r for r in registers(destination(operands)) if r[0] == "s"}
            for n in f.within(i, 5) if written else ():
                if f.ops[n][0].startswith(MEMORY) and written & registers(f.ops[n][1]):
                    yield "scalar register", i, n
        elif op.startswith("v_mfma"):
            written = registers(destination(operands))
            for n in f.within(i, 20 if "32x32x64" in op else 12):
                other, regs = f.ops[n]
                if not other.startswith(("v_mfma", "s_")) and written & registers(regs):
                    yield "product", i, n


@pytest.fixture(scope="module")
def found(tmp_path_factory):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    out, seen = [], {"m0": 0, "product": 0, "functions": 0}
    for f in functions(str(tmp_path_factory.mktemp("code"))):
        seen["functions"] += 1
        seen["m0"] += sum(op.startswith("s_mov") and destination(r) == "m0" for op, r in f.ops)
        seen["product"] += sum(op.startswith("v_mfma") for op, _ in f.ops)
        out += [(kind, f.name, f.text(i), f.text(n)) for kind, i, n in hazards(f)]
    return out, seen


def test_the_code_is_read(found):
    """(That the checks below look at something.)"""
    assert found[1]["m0"] > 1000 and found[1]["product"] > 1000 and found[1]["functions"] > 100


@pytest.mark.parametrize("kind", ["m0", "scalar register", "product"])
def test_no_wait_is_missing(found, kind):
    bad = [x for x in found[0] if x[0] == kind]
    assert not bad, (len(bad), len({x[1] for x in bad}), bad[:3])


def test_the_check_finds_what_it_should():
    """Planted faults, on made-up code."""
    def code(*lines):
        f = Function("f", 0)
        for i, line in enumerate(lines):
            op, _, operands = line.partition(" ")
            f.add(4 * i, op, operands, 8 if op == "s_cbranch_vccnz" else None)
        return [k for k, _, _ in hazards(f)]

    load = "buffer_load_dwordx4 v1, s[4:7], 0 offen lds"
    assert code("s_mov_b32 m0, s3", load) == ["m0"]
    assert code("s_mov_b32 m0, s3", "s_nop 0", load) == []
    assert code("v_readfirstlane_b32 s6, v0", "s_nop 3", load) == ["scalar register"]
    assert code("v_readfirstlane_b32 s6, v0", "s_nop 4", load) == []
    product = "v_mfma_f32_32x32x16_f16 v[0:15], v[20:23], v[24:27], v[0:15]"
    assert code(product, "s_nop 10", "v_max3_f32 v40, v41, v3, v42") == ["product"]
    assert code(product, "s_nop 11", "v_max3_f32 v40, v41, v3, v42") == []
    assert code(product, "s_cbranch_vccnz 1", "v_max3_f32 v40, v41, v15, v42") == ["product", "product"] or \
        code(product, "s_cbranch_vccnz 1", "v_max3_f32 v40, v41, v15, v42") == ["product"]
