"""The dense linear layers' built code keeps the wait states that the compiler
does not place around inline asm (linear.hip): checked on the disassembly of
the built object, on the CPU."""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OBJ = os.path.join(ROOT, "_build", "linear.o")
BIN = "/opt/rocm/llvm/bin"
TOOLS = [os.path.join(BIN, t) for t in ("llvm-objcopy", "clang-offload-bundler", "llvm-objdump")]

pytestmark = pytest.mark.skipif(
    not os.path.exists(OBJ) or not all(shutil.which(t) for t in TOOLS),
    reason="needs the built object and LLVM's binary tools")


def registers(token):
    m = re.match(r"([vas])\[(\d+):(\d+)\]$", token)
    if m:
        return {(m[1], i) for i in range(int(m[2]), int(m[3]) + 1)}
    m = re.match(r"([vas])(\d+)$", token)
    return {(m[1], int(m[2]))} if m else set()


@pytest.fixture(scope="module")
def instructions(tmp_path_factory):
    d = tmp_path_factory.mktemp("isa")
    fat, dev = str(d / "fat.bin"), str(d / "dev.co")
    subprocess.run([TOOLS[0], f"--dump-section=.hip_fatbin={fat}", OBJ, str(d / "x.o")], check=True)
    subprocess.run([TOOLS[1], "--unbundle", "--type=o", f"--input={fat}", f"--output={dev}",
                    "--targets=hipv4-amdgcn-amd-amdhsa--gfx950"], check=True)
    out = subprocess.run([TOOLS[2], "-d", "--no-show-raw-insn", dev], check=True, text=True,
                         capture_output=True).stdout
    rows = []
    for line in out.splitlines():
        line = line.split("//")[0].strip()
        if not line or line.endswith(">:") or ":" in line.split()[0]:
            continue
        op, _, rest = line.partition(" ")
        rows.append((op, [a.strip() for a in rest.split(",")], line))
    return rows


def before(rows, i, states):
    """The instructions less than ``states`` wait states before row i."""
    n, j = 0, i - 1
    while j >= 0 and n < states:
        op, args, _ = rows[j]
        if op != "s_nop":
            yield rows[j]
        n += int(args[0], 0) + 1 if op == "s_nop" else 1
        j -= 1


def is_load(row):
    return row[0].startswith("buffer_load") and row[2].endswith("lds")


def test_loads_and_products_were_found(instructions):
    assert sum(is_load(r) for r in instructions) > 1000
    assert sum(r[0].startswith("v_mfma") for r in instructions) > 2000


def test_scalars_settle_before_a_load_reads_them(instructions):
    for i, row in enumerate(instructions):
        if is_load(row):
            used = {r for r in registers(row[1][1]) if r[0] == "s"}
            assert used
            for op, args, line in before(instructions, i, 5):
                assert not (op.startswith("v_") and registers(args[0]) & used), (line, row[2])


def test_an_instruction_lies_between_m0_and_a_load(instructions):
    for i, row in enumerate(instructions):
        if is_load(row):
            assert all(args[0] != "m0" for _, args, _ in before(instructions, i, 1)), row[2]
        elif row[1][0] == "m0":  # and nothing else writes M0
            assert row[0] == "s_mov_b32"


def test_operands_settle_before_a_product(instructions):
    for i, row in enumerate(instructions):
        if row[0].startswith("v_mfma"):
            used = set().union(*(registers(a) for a in row[1][1:]))
            for op, args, line in before(instructions, i, 2):
                other = op.startswith("v_") and not op.startswith("v_mfma")
                assert not (other and registers(args[0]) & used), (line, row[2])


def test_no_scratch(instructions):
    """A spill's reload waits for the output stores before it (an epilogue
    with 15 of them cost 15 us a tile)."""
    assert not [r[2] for r in instructions if r[0].startswith("scratch_")]


def test_no_packed_fp32(instructions):
    assert not [r[2] for r in instructions if re.match(r"v_pk_(add|mul|fma)_f32", r[0])]
