"""The tile engine in the objects beside the dense layers' (products grouped by
expert, 8-bit integers): the same checks of wait states, spills and packed fp32
on their disassembly, and that each is the present source's."""

import os
import subprocess

import pytest

import test_linear_isa as isa
from sparse_input_gemv_amd.build import BUILD, SOURCES, source_hash
from test_linear_isa import (pytestmark, test_an_instruction_lies_between_m0_and_a_load,  # noqa: F401
                             test_no_packed_fp32, test_no_scratch, test_operands_settle_before_a_product,
                             test_scalars_settle_before_a_load_reads_them)
from test_linear_isa_sums import test_sums_settle_before_they_are_used  # noqa: F401

ENGINES = [s for s in ("grouped.hip", "grouped_backward.hip", "int8.hip") if s in SOURCES]


@pytest.fixture(scope="module", params=ENGINES)
def instructions(request, tmp_path_factory):
    d = tmp_path_factory.mktemp("isa")
    fat, dev = str(d / "fat.bin"), str(d / "dev.co")
    obj = os.path.join(BUILD, request.param.replace(".hip", ".o"))
    subprocess.run([isa.TOOLS[0], f"--dump-section=.hip_fatbin={fat}", obj, str(d / "x.o")], check=True)
    subprocess.run([isa.TOOLS[1], "--unbundle", "--type=o", f"--input={fat}", f"--output={dev}",
                    "--targets=hipv4-amdgcn-amd-amdhsa--gfx950"], check=True)
    out = subprocess.run([isa.TOOLS[2], "-d", "--no-show-raw-insn", dev], check=True, text=True,
                         capture_output=True).stdout
    rows = []
    for line in out.splitlines():
        line = line.split("//")[0].strip()
        if not line or line.endswith(">:") or ":" in line.split()[0]:
            continue
        op, _, rest = line.partition(" ")
        rows.append((op, [a.strip() for a in rest.split(",")], line))
    return rows


def test_the_engine_was_found(instructions):
    assert sum(isa.is_load(r) for r in instructions) > 200
    assert sum(r[0].startswith("v_mfma") for r in instructions) > 200


@pytest.mark.parametrize("src", ENGINES)
def test_the_objects_are_the_present_sources(src):
    path = os.path.join(BUILD, src.replace(".hip", ".o.src"))
    assert os.path.exists(path) and open(path).read() == source_hash(src), "build again"
