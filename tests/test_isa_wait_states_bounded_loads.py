"""Wait states around the loads to LDS through buffer descriptors, along every path that leads to one.

The same two faults as in test_isa_wait_states_across_branches: a word of the descriptor that a vector instruction wrote
fewer than 5 wait states before, and M0 written directly before, or by a vector instruction.
"""
import os
import subprocess

import pytest

from test_isa_wait_states import OBJDUMP, device_code
from test_isa_wait_states_across_branches import functions, listing, scan


def bounded(body):
    """The function with its buffer loads to LDS under the name that ``scan`` looks for, and no others."""
    out = []
    for address, instruction, target in body:
        op, _, rest = instruction.partition(" ")
        if op.startswith("buffer_load") and rest.split()[-1] == "lds":
            op = "buffer_load_lds_" + op
        elif "_load_lds_" in op:
            op = "other_load"
        out.append((address, op + " " + rest if rest else op, target))
    return out


def test_scan_sees_both_faults():
    load = "buffer_load_dwordx4 v2, s[4:7], 0 offen lds"
    assert scan(bounded(listing("v_readlane_b32 s6, v1, 3", "s_nop 0", load)))[1]
    assert scan(bounded(listing("v_readfirstlane_b32 s4, v1", "s_nop 4", load))) == (1, [])
    assert scan(bounded(listing("v_readfirstlane_b32 s8, v1", load))) == (1, [])
    assert scan(bounded(listing("s_mov_b32 m0, s1", load)))[1]
    assert scan(bounded(listing("buffer_load_dwordx4 v[2:5], v6, s[4:7], 0 offen"))) == (0, [])
    loop = ["s_nop 7", load, "v_readlane_b32 s7, v1, 0", "s_cbranch_scc1 65533 -> 1", "s_endpgm"]
    assert scan(bounded(listing(*loop)))[1]


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_every_path_to_a_bounded_load_of_the_built_library(tmp_path):
    total = 0
    for i, code in enumerate(device_code()):
        path = tmp_path / f"{i}.co"
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(path)], capture_output=True, text=True,
                              check=True).stdout
        for body in functions(text.splitlines()):
            loads, bad = scan(bounded(body))
            total += loads
            assert not bad, f"{len(bad)} of {loads} loads, e.g. {bad[:3]}"
    assert total >= 8 * 4 * 2   # eight kernels, a stage of four loads where they begin and in a step
