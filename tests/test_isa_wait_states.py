"""Wait states around the inline-asm loads of the built library.

The compiler inserts the wait states the hardware asks for around its own
instructions, but not around inline asm.  For every load to LDS of the GEMM kernels
this scans the disassembly of this library's own code for

* a scalar register of the load's address that a vector instruction (v_readfirstlane,
  v_readlane, a compare) wrote fewer than 5 wait states before: the load would
  use an old address;
* M0 written by a scalar instruction directly before.
"""
import os
import re
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "moe_fp8_gemm_amd", "libdgfp8.so")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def device_code():
    """The gfx950 code objects bundled in the library."""
    data = open(LIB, "rb").read()
    at = data.find(MAGIC)
    while at >= 0:
        count, = struct.unpack_from("<Q", data, at + len(MAGIC))
        p = at + len(MAGIC) + 8
        for _ in range(count):
            off, size, n = struct.unpack_from("<QQQ", data, p)
            name = data[p + 24:p + 24 + n]
            p += 24 + n
            if b"gfx950" in name and size:
                yield data[at + off:at + off + size]
        at = data.find(MAGIC, at + 1)


def registers(arg):
    m = re.match(r"s\[(\d+):(\d+)\]$", arg)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.match(r"s(\d+)$", arg)
    return {int(m.group(1))} if m else {-1} if arg == "vcc" else set()


def scan(lines):
    """(loads to LDS, violations) of a disassembly."""
    loads, bad, recent = 0, [], []      # recent: (wait states it stands for, SGPRs a vector instruction wrote, writes M0)
    for line in lines:
        line = line.split("//")[0].strip()
        if not line or line.endswith(":"):
            if line.endswith(">:"):
                recent = []
            continue
        op, _, rest = line.partition(" ")
        args = [a.strip() for a in re.split(r",\s*(?![^\[]*\])", rest)]
        if "_load_lds_" in op:
            loads += 1
            used = set().union(*(registers(a.split()[0]) for a in args if a))
            gap = 0
            for states, wrote, m0 in reversed(recent):
                if gap >= 5:
                    break
                if wrote & used or (m0 and gap < 1):
                    bad.append(line)
                    break
                gap += states
        wrote = registers(args[0]) if op.startswith(("v_readfirstlane", "v_readlane", "v_cmp")) else set()
        states = int(rest, 0) + 1 if op == "s_nop" else 1
        recent = (recent + [(states, wrote, op.startswith("s_") and args[0] == "m0")])[-8:]
    return loads, bad


def test_scan_sees_both_faults():
    assert scan(["v_readfirstlane_b32 s4, v1", "s_nop 0", "global_load_lds_dwordx4 v2, s[4:5]"])[1]
    assert scan(["s_mov_b32 m0, s1", "global_load_lds_dword v[2:3], off"])[1]
    assert scan(["v_readfirstlane_b32 s4, v1", "s_nop 4", "s_mov_b32 m0, s1", "s_nop 0",
                 "global_load_lds_dwordx4 v2, s[4:5]"]) == (1, [])


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_loads_to_lds_of_the_built_library(tmp_path):
    total = 0
    for i, code in enumerate(device_code()):
        path = tmp_path / f"{i}.co"
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(path)], capture_output=True, text=True,
                              check=True).stdout
        loads, bad = scan(text.splitlines())
        total += loads
        assert not bad, f"{len(bad)} of {loads} loads, e.g. {bad[:3]}"
    assert total > 500
