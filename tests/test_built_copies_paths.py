"""The built kernels' copies into LDS once more, along every way that leads to them:
a write before a branch to the copy, backwards too, or before a jump too far for one, is
as close as the instructions that run in between. And a copy does not wait by itself
where its buffer has waited for all copies of a stage."""
import os
import re
import subprocess

import pytest

from .test_built_copies import FIRST, LIB, OBJDUMP, SECOND, WAIT, scalars


def instructions(lines):
    """[(address, name, operands, branch target or None, function)]"""
    out, start, function = [], 0, None
    for line in lines:
        head = re.match(r"([0-9a-f]+) <(\S+)>:", line)
        if head:
            start, function = int(head[1], 16), head[2]
            continue
        m = re.match(r"\s+(\S+)\s*(.*?)\s*// ([0-9A-F]+):(.*)", line)
        if not m:
            continue
        to = re.search(r"<\S+?(?:\+0x([0-9a-f]+))?>", m[4]) if "branch" in m[1] else None
        out.append((int(m[3], 16), m[1], m[2], start + int(to[1] or "0", 16) if to else None, function))
    return out


def far_target(code, i):
    """Where `s_setpc_b64` goes: s_getpc_b64, and a constant added to it, before it."""
    lo = int(re.match(r"s\[(\d+):", code[i][2])[1])
    add = None
    for j in range(i - 1, max(i - 8, -1), -1):
        _, name, operands, _, _ = code[j]
        if name == "s_add_u32" and operands.startswith(f"s{lo}, s{lo}, "):
            add = int(operands.split(",")[2], 0)
        if name == "s_getpc_b64" and operands.startswith(f"s[{lo}:") and add is not None:
            return code[j + 1][0] + (add - (1 << 32) if add >> 31 else add)
    raise AssertionError(f"a jump to where? {code[i]}")


def before(code):
    """For each instruction, those that may run right before it."""
    at = {c[0]: i for i, c in enumerate(code)}
    prev = [[] for _ in code]
    for i, (_, name, _, target, function) in enumerate(code):
        if name == "s_setpc_b64":
            target = far_target(code, i)
        if target is not None:
            prev[at[target]].append(i)
        if name not in ("s_branch", "s_setpc_b64", "s_endpgm") and i + 1 < len(code) and (
                code[i + 1][4] == function):
            prev[i + 1].append(i)
    return prev


def written(name, operands):
    parts = operands.split(",")
    if FIRST.match(name):
        return scalars(parts[0])
    return scalars(parts[1]) if SECOND.match(name) and len(parts) > 1 else set()


def copies(code):
    return [i for i, c in enumerate(code)
            if c[1].startswith("buffer_load") and c[2].split()[-1] == "lds"]


def close_writes(code):
    """Copies with a register of theirs written too close before, on some way to them."""
    prev, close = before(code), []
    for i in copies(code):
        need, ways, seen = scalars(code[i][2]) | {"m0"}, [(p, 0) for p in prev[i]], {}
        while ways:
            j, waited = ways.pop()
            if waited >= WAIT or seen.get(j, WAIT) <= waited:
                continue
            seen[j] = waited
            _, name, operands, _, _ = code[j]
            if written(name, operands) & need:
                close.append((code[i][:3], code[j][:3]))
                break
            states = int(operands, 0) + 1 if name == "s_nop" else 1
            ways += [(p, waited + states) for p in prev[j]]
    return close


def listing(*texts):
    """A listing of 4-byte instructions at 0x100; `text -> n` branches to the n-th."""
    lines = ["0000000000000100 <f>:"]
    for i, text in enumerate(texts):
        text, _, to = text.partition(" -> ")
        lines.append("\t%s // %012X: BF820000%s" % (text, 0x100 + 4 * i,
                                                    " <f+0x%x>" % (4 * int(to)) if to else ""))
    return instructions(lines)


COPY, WRITE, IDLE = "buffer_load_dwordx4 v8, s[4:7], s62 offen lds", "v_readlane_b32 s6, v255, 3", "v_mov_b32_e32 v1, v2"


@pytest.mark.parametrize("code,found", [
    ([WRITE, COPY], 1), ([WRITE, "s_nop 4", COPY], 0),
    ([COPY, *[IDLE] * 5, WRITE, "s_cbranch_scc1 65500 -> 0"], 1),  # backwards
    ([COPY, WRITE, *[IDLE] * 5, "s_cbranch_scc1 65500 -> 0"], 0),
    ([WRITE, "s_branch 6 -> 8", *[IDLE] * 6, COPY], 1),  # over the wait
    ([WRITE, "s_branch 6 -> 3", IDLE, *[IDLE] * 5, COPY], 0),
    # a far jump: from the third instruction on, 0x18 bytes to the one before the copy
    ([WRITE, "s_getpc_b64 s[98:99]", "s_add_u32 s98, s98, 0x18", "s_addc_u32 s99, s99, 0",
      "s_setpc_b64 s[98:99]", *[IDLE] * 4, COPY], 0),
    ([WRITE, "s_getpc_b64 s[98:99]", "s_add_u32 s98, s98, 0x1c", "s_addc_u32 s99, s99, 0",
      "s_setpc_b64 s[98:99]", *[IDLE] * 4, COPY], 1),
    (["s_nop 4", "s_getpc_b64 s[98:99]", "s_add_u32 s98, s98, 0x1c", WRITE, "s_setpc_b64 s[98:99]",
      *[IDLE] * 4, COPY], 1),
    ([WRITE, "s_endpgm", COPY], 0),
])
def test_close_writes_are_found_along_the_ways(code, found):
    code = listing(*code)
    assert len(copies(code)) == 1 and len(close_writes(code)) == found


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    if not os.path.exists(LIB) or not os.path.exists(OBJDUMP):
        pytest.skip("the library is not built, or no disassembler")
    at = tmp_path_factory.mktemp("parts")
    os.symlink(LIB, at / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=at, check=True, capture_output=True,
                   timeout=60)
    parts = [f for f in os.listdir(at) if f.endswith("gfx950")]
    code = [subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", p], cwd=at, check=True,
                           capture_output=True, text=True, timeout=60).stdout for p in parts]
    return [instructions(c.splitlines()) for c in code]


def test_no_close_write_on_any_way(library):
    n = 0
    for code in library:
        n += len(copies(code))
        close = close_writes(code)
        assert not close, close[:3]
    assert n > 1000


def test_copies_of_rows_do_not_wait_one_by_one(library):
    """Of a kernel's copies, those with a wait of their own right before them: the two
    of the 4-bit products' scales, in each of the places that they are unrolled to."""
    for code in library:
        by_kernel = {}
        for i in copies(code):
            by_kernel.setdefault(code[i][4], []).append(
                code[i - 1][1] == "s_nop" and int(code[i - 1][2], 0) >= 4)
        for kernel, waits in by_kernel.items():
            assert sum(waits) <= len(waits) // 4, (kernel, sum(waits), len(waits))
