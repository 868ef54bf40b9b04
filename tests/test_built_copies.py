"""The built kernels' copies into LDS, which are written in assembly: the compiler does
not look into that for hazards. A scalar register that a vector instruction wrote (a lane
read back, also that of a spilled register) is valid for a memory instruction five wait
states later, so none of a copy's may be written closer to it."""
import os
import re
import subprocess

import pytest

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "token_dispatch_mb_amd", "libmoebal.so")
OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
WAIT = 5
# vector instructions with a scalar result, in their first operand, or in their second
FIRST = re.compile(r"v_readfirstlane_b32|v_readlane_b32|v_cmp")
SECOND = re.compile(r"v_div_scale|v_mad_u64|v_mad_i64|v_(add|sub|addc|subb|subrev|subbrev)_co")


def scalars(text):
    found = set()
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        found |= set(range(int(a), int(b) + 1))
    return found | {int(a) for a in re.findall(r"\bs(\d+)\b", text)} | set(
        re.findall(r"\b(m0|vcc)\b", text))


def close_writes(lines):
    """The number of copies, and those with a register written too close before."""
    copies, close, before = 0, [], []  # (wait states, scalar registers written)
    for line in lines:
        text = line.split("//")[0].strip()
        if not re.match(r"[a-z]\w* ?", text) or text.endswith(":"):
            continue
        name, _, operands = text.partition(" ")
        if name.startswith("buffer_load") and operands.split()[-1] == "lds":
            copies += 1
            need, waited = scalars(operands) | {"m0"}, 0
            for states, written in reversed(before):
                if waited >= WAIT:
                    break
                if written & need:
                    close.append(text)
                    break
                waited += states
        parts, written = operands.split(","), set()
        if FIRST.match(name):
            written = scalars(parts[0])
        elif SECOND.match(name) and len(parts) > 1:
            written = scalars(parts[1])
        states = int(operands, 0) + 1 if name == "s_nop" else 1
        before = (before + [(states, written)])[-2 * WAIT:]
    return copies, close


@pytest.mark.parametrize("between,found", [
    ([], 1), (["v_mov_b32_e32 v1, v2"], 1), (["s_nop 3"], 1), (["s_nop 4"], 0),
    (["v_mov_b32_e32 v1, v2"] * 4, 1), (["v_mov_b32_e32 v1, v2"] * 5, 0),
])
@pytest.mark.parametrize("write", [
    "v_readlane_b32 s6, v255, 3", "v_readfirstlane_b32 s62, v8", "v_cmp_gt_i32_e64 s[4:5], v1, v2",
    "v_add_co_u32_e64 v1, s[6:7], v2, v3", "v_readfirstlane_b32 m0, v8",
])
def test_a_close_write_is_found(write, between, found):
    copy = "buffer_load_dwordx4 v8, s[4:7], s62 offen lds"
    code = ["\t%s   // 000000003C80: BEC00022" % t for t in [write, *between, copy]]
    assert (close_writes(code)[0], len(close_writes(code)[1])) == (1, found)
    other = "v_readlane_b32 s9, v255, 3"
    assert close_writes([other, copy]) == (1, [])


@pytest.mark.skipif(not os.path.exists(LIB), reason="the library is not built")
@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no disassembler")
def test_no_close_write_in_the_library(tmp_path):
    os.symlink(LIB, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True,
                   capture_output=True, timeout=60)
    parts = sorted(f for f in os.listdir(tmp_path) if f.endswith("gfx950"))
    assert parts
    copies = 0
    for part in parts:
        code = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", part], cwd=tmp_path, check=True,
                              capture_output=True, text=True, timeout=60).stdout
        n, close = close_writes(code.splitlines())
        copies += n
        assert not close, close[:5]
    assert copies > 1000  # the tiles of the 4-bit and 16-bit products
