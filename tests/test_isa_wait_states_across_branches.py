"""Wait states around the inline-asm loads of the built library, along every path that leads to one.

The linear scan of test_isa_wait_states starts anew at each function; a path through a branch, such as a loop's
back edge, brings other instructions before a load than those printed above it.  Here every load to LDS is followed
backwards through all its predecessors for the same two faults, and M0 must come from a scalar instruction (one
wait state), never from a vector instruction, which would need more.
"""
import collections
import os
import re
import subprocess

import pytest

from test_isa_wait_states import OBJDUMP, device_code, registers

FUNCTION = re.compile(r"^[0-9a-f]+ <(.*)>:$")
LINE = re.compile(r"^\s+(\S.*?)\s*//\s*([0-9A-F]+):(.*)$")
TARGET = re.compile(r"<[^>+]*(?:\+0x([0-9a-f]+))?>")


def functions(lines):
    """Lists of (address, instruction, branch target or None)."""
    out = []
    for line in lines:
        if FUNCTION.match(line):
            out.append([])
        elif (m := LINE.match(line)) and out:
            target = TARGET.search(m.group(3)) if m.group(1).startswith(("s_branch", "s_cbranch")) else None
            start = out[-1][0][0] if out[-1] else int(m.group(2), 16)
            out[-1].append((int(m.group(2), 16), m.group(1),
                            start + int(target.group(1) or "0", 16) if target else None))
    return out


def split(instruction):
    op, _, rest = instruction.partition(" ")
    return op, [a.strip() for a in re.split(r",\s*(?![^\[]*\])", rest)]


def scan(body):
    """(loads to LDS, violations) of one function."""
    at = {address: i for i, (address, _, _) in enumerate(body)}
    before = collections.defaultdict(list)
    for i, (_, instruction, target) in enumerate(body):
        op = instruction.split()[0]
        if op.startswith(("s_branch", "s_cbranch")):
            before[at[target]].append(i)
        if not op.startswith(("s_branch", "s_endpgm")) and i + 1 < len(body):
            before[i + 1].append(i)
    loads, bad = 0, []
    for i, (_, instruction, _) in enumerate(body):
        op, args = split(instruction)
        if "_load_lds_" not in op:
            continue
        loads += 1
        used = set().union(*(registers(a.split()[0]) for a in args if a))
        seen, stack = set(), [(p, 0) for p in before[i]]
        while stack:
            j, gap = stack.pop()
            if gap >= 5 or (j, gap) in seen:
                continue
            seen.add((j, gap))
            op, args = split(body[j][1])
            vector = op.startswith(("v_readfirstlane", "v_readlane", "v_cmp"))
            if (vector and registers(args[0]) & used) or (args[0] == "m0" and (vector or gap < 1)):
                bad.append((body[j][1], instruction, gap))
            states = int(args[0], 0) + 1 if op == "s_nop" else 1
            stack += [(p, gap + states) for p in before[j]]
    return loads, bad


def listing(*instructions):
    """A function of 4-byte instructions; "-> n" after a branch names its target by number."""
    lines = ["0000000000001000 <f>:"]
    for i, text in enumerate(instructions):
        op, _, target = text.partition(" -> ")
        lines.append(f"\t{op}  // {0x1000 + 4 * i:012X}:" + (f" <f+0x{4 * int(target):x}>" if target else ""))
    return functions(lines)[0]


def test_scan_follows_a_back_edge():
    load = "global_load_lds_dwordx4 v2, s[4:5]"
    loop = ["s_nop 7", load, "v_readfirstlane_b32 s4, v1", "s_cbranch_scc1 65533 -> 1", "s_endpgm"]
    assert ("v_readfirstlane_b32 s4, v1", load, 1) in scan(listing(*loop))[1]
    loop[2:3] = ["v_readfirstlane_b32 s4, v1", "s_nop 3"]
    assert scan(listing(*loop)) == (1, [])
    assert scan(listing("s_mov_b32 m0, s1", load))[1] and not scan(listing("s_mov_b32 m0, s1", "s_nop 0", load))[1]
    assert scan(listing("v_readfirstlane_b32 m0, v1", "s_nop 0", load))[1]


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_every_path_to_a_load_of_the_built_library(tmp_path):
    total = 0
    for i, code in enumerate(device_code()):
        path = tmp_path / f"{i}.co"
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(path)], capture_output=True, text=True,
                              check=True).stdout
        for body in functions(text.splitlines()):
            loads, bad = scan(body)
            total += loads
            assert not bad, f"{len(bad)} of {loads} loads, e.g. {bad[:3]}"
    assert total > 500
