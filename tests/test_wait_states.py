"""Wait states of the built kernels' direct loads into LDS (no GPU).

The instruction set asks the program, not the hardware, for two distances in
front of such a load: one wait state after a scalar instruction wrote m0, which
holds the LDS address, and five after a vector instruction wrote a scalar
register that the load reads.  The compiler keeps them for the loads it issues
itself; those issued from inline assembly are checked here, in the code as it
was built."""
import os
import re
import shutil
import subprocess

import pytest

from qat_nvfp4_quantize_amd import build

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def _written(operands):
    """Scalar registers in an instruction's first operand."""
    return _scalars(operands.split(",")[0])


def _scalars(text):
    out = set()
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        out.update(range(int(a), int(b) + 1))
    out.update(int(a) for a in re.findall(r"\bs(\d+)\b", text))
    return out


def too_close(lines):
    """(line number, text) of each direct load to LDS that comes too early.  A
    branch between two instructions counts as what it is, one wait state, so the
    order of the text is the shortest distance."""
    code = []
    for n, line in enumerate(lines):
        line = line.split("//")[0].strip()
        if line and not line.endswith(":"):
            op, _, rest = line.partition(" ")
            code.append((n, op, rest))
    bad, seen = [], 0
    for i, (n, op, rest) in enumerate(code):
        if not ("load_lds_" in op or (op.startswith("buffer_load") and re.search(r"\blds\b", rest))):
            continue
        seen += 1
        reads = _scalars(rest)
        apart = 0
        for _, before, operands in reversed(code[max(0, i - 5):i]):
            to = operands.split(",")[0].strip()
            if apart < 1 and before.startswith("s_") and to == "m0":
                bad.append((n, op + " " + rest))
            if before.startswith("v_readlane") or before.startswith("v_readfirstlane") or before.startswith("v_cmp"):
                if _written(operands) & reads:
                    bad.append((n, op + " " + rest))
            apart += 1 + (int(operands, 0) if before == "s_nop" else 0)
            if apart >= 5:
                break
    return bad, seen


def test_the_check_sees_what_it_looks_for():
    load = "global_load_lds_dwordx4 v[2:3], off"
    assert too_close(["s_mov_b32 m0, s4", load])[0] and too_close(["s_add_u32 m0, s4, s5 // 0x1", "L:", load])[0]
    assert too_close(["s_mov_b32 m0, s4", "s_nop 0", load]) == ([], 1)
    assert too_close(["s_mov_b32 m0, s4", "v_add_u32_e32 v0, v1, v2", load]) == ([], 1)
    load = "buffer_load_dwordx4 v5, s[8:11], 0 offen lds"
    assert too_close(["v_readfirstlane_b32 s9, v1", "s_nop 3", load])[0]
    assert too_close(["v_readfirstlane_b32 s9, v1", "s_nop 4", load]) == ([], 1)
    assert too_close(["v_readfirstlane_b32 s12, v1", load]) == ([], 1)
    assert too_close(["s_mov_b32 m0, s4", "buffer_load_dwordx4 v[0:3], v5, s[8:11], 0 offen"]) == ([], 0)


def test_direct_loads_keep_their_distance(tmp_path):
    if not os.path.exists(build.LIB) or not os.path.exists(OBJDUMP):
        pytest.skip("libnvq.so not built, or no disassembler")
    lib = shutil.copy(build.LIB, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, cwd=tmp_path)
    codes = sorted(f for f in os.listdir(tmp_path) if f.endswith("gfx950"))
    assert codes
    total = 0
    for f in codes:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", f], check=True, capture_output=True,
                              text=True, cwd=tmp_path).stdout
        bad, seen = too_close(text.splitlines())
        assert not bad, (f, len(bad), "of", seen, bad[:3])
        total += seen
    assert total > 100  # the dense products' and the grouped products' alone
