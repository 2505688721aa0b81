"""The matrix products keep their sums in the accumulation registers by inline
assembly, whose results the compiler takes as ready at once.  That is sound only
where nothing but matrix instructions touches those registers until the wait that
ends the loop's body.  This compiles the kernels and looks."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sharded_optimizer_step_zero_amd", "csrc")


def _flags():
    import importlib.util
    spec = importlib.util.spec_from_file_location("_zs_build_flags", os.path.join(CSRC, "..", "_build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m.HIPCC_FLAGS


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("asm") / "xent.s")
    subprocess.run(["hipcc", *_flags(), "-S", "--offload-device-only", os.path.join(CSRC, "xent.hip"), "-o", out],
                   check=True, stderr=subprocess.DEVNULL)
    return open(out).read()


def _instructions(text):
    """(instructions, index of each label)"""
    code, labels = [], {}
    for line in text.split("\n"):
        line = line.split(";")[0].strip()
        if re.match(r"^[.\w$]+:$", line):
            labels[line[:-1]] = len(code)
        elif line and not line.startswith("."):
            code.append(line)
    return code, labels


def test_sums_are_left_alone_until_they_are_ready(assembly):
    """On every path from a matrix instruction to the wait that follows, accumulation
    registers appear in matrix instructions only."""
    kernels = re.findall(r"^(_ZN\w*gemm_kernel\w*):(.*?\ts_endpgm)", assembly, re.S | re.M)
    assert len(kernels) >= 14
    for name, text in kernels:
        code, labels = _instructions(text)
        todo = [i for i, c in enumerate(code) if c.startswith("v_mfma")]
        assert len(todo) >= 16, name
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
