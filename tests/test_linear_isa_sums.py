"""The dense linear layers' built code waits after the last product before
anything else touches a sum, and is the code of the present source."""

import os
import re

import pytest

from sparse_input_gemv_amd.build import BUILD, source_hash
from test_linear_isa import instructions, pytestmark  # noqa: F401

STATES = 18  # a product's result after which any other instruction may name it (linear.hip)
REG = re.compile(r"\b([va])(?:(\d+)|\[(\d+):(\d+)\])(?![\w\[])")


def named(line):
    out = set()
    for kind, one, lo, hi in REG.findall(line):
        out |= {(kind, i) for i in (range(int(lo), int(hi) + 1) if lo else (int(one),))}
    return out


def early_uses(rows, states=STATES):
    """(product, other) pairs less than ``states`` wait states apart where the
    other names the product's sum and is not the same sum's next product."""
    found, pending = [], []  # (states passed, registers, line)
    for op, args, line in rows:
        if op in ("s_branch", "s_endpgm", "s_setpc_b64"):
            pending = []
            continue
        names = named(line)
        product = op.startswith("v_mfma")
        for _, regs, by in pending:
            own = product and named(args[0]) == regs and not any(named(a) & regs for a in args[1:3])
            if names & regs and not own:
                found.append((by, line))
        n = int(args[0], 0) + 1 if op == "s_nop" else 1
        pending = [(k + n, r, by) for k, r, by in pending if k + n < states]
        if product:
            pending.append((0, named(args[0]), line))
    return found


def row(line):
    op, _, rest = line.partition(" ")
    return op, [a.strip() for a in rest.split(",")], line


def test_the_scan_finds_an_early_use():
    product = "v_mfma_f32_16x16x32_f16 a[0:3], v[8:11], v[12:15], a[0:3]"
    other = "v_mfma_f32_16x16x32_f16 a[4:7], v[8:11], v[12:15], a[4:7]"
    read, late = "v_accvgpr_read_b32 v1, a2", ["s_nop 15", "s_nop 7"]
    use = lambda *lines: early_uses([row(v) for v in lines])  # noqa: E731
    assert use(product, read) == use(product, other, "s_nop 14", read) == [(product, read)]
    assert use(product, "v_accvgpr_write_b32 a0, 0") and use(product, "v_accvgpr_mov_b32 a9, a3")
    assert not use(product, product, other, product)
    assert not use(product, *late, read) and not use(product, "v_accvgpr_read_b32 v1, a4")
    assert not use(product, "v_add_u32_e32 v2, v0, v1")


def test_sums_settle_before_they_are_used(instructions):  # noqa: F811
    assert early_uses(instructions) == []


def test_the_object_is_the_present_source():
    src = os.path.join(BUILD, "linear.o.src")
    assert os.path.exists(src) and open(src).read() == source_hash("linear.hip"), "build again"
