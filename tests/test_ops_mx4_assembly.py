"""What the compiler cannot guard around the inline assembly of the 4-bit products: descriptors and
m0 are old enough when a load into LDS reads them, a matrix instruction's operands when
it reads those, the sums in the accumulation registers are left alone until they are
ready, and the stores that a wait lets go on are as many as it counts.  This compiles the
kernels and looks."""
import os
import re
import subprocess

import pytest

from test_ops_assembly import CSRC, _flags, _instructions
from test_ops_assembly_hazards import _before, _registers, _written


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("asm") / "mx4.s")
    subprocess.run(["hipcc", *_flags(), "-S", "--offload-device-only", os.path.join(CSRC, "mx4.hip"), "-o", out],
                   check=True, stderr=subprocess.DEVNULL)
    found = re.findall(r"^(_ZN\w*(?:product|held)_kernel\w*):(.*?)^\.Lfunc_end", open(out).read(), re.S | re.M)
    assert len(found) >= 6
    return [(name, *_instructions(text)) for name, text in found]


def test_descriptors_are_old_enough(kernels):
    """Vector memory reads a scalar that a vector instruction wrote five wait states before
    at the least."""
    for name, code, labels in kernels:
        loads = [i for i, c in enumerate(code) if c.startswith("buffer_load") and " lds" in c]
        assert len(loads) >= 6, name
        for i in loads:
            reads = _registers(code[i], "s")
            assert reads, code[i]
            for c in _before(code, labels, i, 5):
                if c.startswith("v_"):
                    assert not _registers(_written(c), "s") & reads, (name, c, code[i])


def test_m0_is_old_enough(kernels):
    """A load into LDS takes m0 one wait state after it is written, and no other instruction
    writes or reads it meanwhile."""
    for name, code, _ in kernels:
        for i, c in enumerate(code):
            if c.startswith("buffer_load") and " lds" in c:
                assert re.match(r"s_nop\s+", code[i - 1]) and re.match(r"s_mov_b32 m0,", code[i - 2]), (name, code[i - 2:i])
            elif re.search(r"\bm0\b", c):
                assert re.match(r"s_mov_b32 m0,", c) and " lds" in code[i + 2], (name, c)


def test_operands_are_old_enough(kernels):
    """A matrix instruction reads a vector register that a vector instruction other than a
    matrix one wrote two wait states before at the least."""
    for name, code, labels in kernels:
        for i, c in enumerate(code):
            if not c.startswith("v_mfma"):
                continue
            operands = c.split(None, 1)[1].split(",", 1)[1]
            v, a = _registers(operands, "v"), _registers(operands, "a")
            for b in _before(code, labels, i, 2):
                if b.startswith("v_") and not b.startswith("v_mfma"):
                    to = _written(b)
                    assert not (_registers(to, "v") & v or _registers(to, "a") & a), (name, b, c)


def test_sums_are_left_alone_until_they_are_ready(kernels):
    """On every path from a matrix instruction to the wait that follows, accumulation
    registers appear in matrix instructions only."""
    held = [k for k in kernels if "held_kernel" in k[0]]
    assert len(held) == 3
    for name, code, labels in held:
        todo = [i for i, c in enumerate(code) if c.startswith("v_mfma")]
        assert len(todo) == 256, name
        seen = set()
        while todo:
            i = todo.pop()
            if i in seen:
                continue
            seen.add(i)
            c = code[i]
            if c.startswith("s_nop 15"):
                continue
            assert not c.startswith("s_endpgm"), name
            if not c.startswith("v_mfma"):
                assert not re.search(r"\ba(\[\d+:\d+\]|\d+)\b", c) and "scratch" not in c, (name, c)
            to = re.match(r"s_c?branch\w*\s+(\S+)", c)
            if to:
                todo.append(labels[to.group(1)])
            if not c.startswith("s_branch"):
                todo.append(i + 1)


def test_a_whole_tiles_stores_are_as_many_as_are_left_under_way(kernels):
    """The first wait after a whole tile lets its stores go on by their number: 32 of 16 bytes in
    16-bit types, streamed or not; in fp32 63 of its 64 (there the ragged tile has as many)."""
    for name, code, _ in [k for k in kernels if "held_kernel" in k[0]]:
        wide = [c for c in code if c.startswith("global_store_dwordx4")]
        waits = [c for c in code if re.match(r"s_waitcnt vmcnt\((32|63)\)", c)]
        if "held_kernelILi0E" in name:
            assert len(wide) == 128 and any("63" in c for c in waits), name
        else:
            streamed = [c for c in wide if re.search(r"\bnt\b", c)]
            assert len(streamed) == 32 and len(wide) == 64 and any("32" in c for c in waits), name
        assert not any(c.startswith("scratch_") for c in code), name
