"""What the compiler cannot guard around the inline assembly of the matrix products: m0 is
named as overwritten, a buffer descriptor's scalars are old enough when a load reads them,
and a matrix instruction's operands when it reads those.  This reads the source and the
assembly made from it."""
import os
import re

import pytest

from test_ops_assembly import CSRC, _instructions, assembly  # noqa: F401  (a fixture)


def _asm_statements(src):
    """Each asm statement of a source, string and operands."""
    out = []
    for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(", src):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(src[i], 0)
            i += 1
        out.append(src[m.end():i - 1])
    return out


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".hip", ".h", ".cpp"))))
def test_m0_is_named_as_overwritten(name):
    for text in _asm_statements(open(os.path.join(CSRC, name)).read()):
        if re.search(r"\bs_mov_b32 m0\b", text):
            assert re.search(r':[^:]*"m0"[^:]*$', text), text


def _registers(text, kind):
    """The numbers of all s, v or a registers named in the text."""
    out = set()
    for a, b in re.findall(rf"\b{kind}\[(\d+):(\d+)\]", text):
        out.update(range(int(a), int(b) + 1))
    out.update(int(a) for a in re.findall(rf"\b{kind}(\d+)\b", text))
    return out


def _kernels(text):
    found = re.findall(r"^(_ZN\w*gemm_kernel\w*):(.*?)^\.Lfunc_end", text, re.S | re.M)
    assert len(found) >= 14
    return found


def _before(code, labels, i, states):
    """Instructions that can come fewer than `states` wait states before instruction i, on
    any path."""
    into = {}
    for k, c in enumerate(code):
        m = re.match(r"s_c?branch\w*\s+(\S+)", c)
        if m:
            into.setdefault(labels[m.group(1)], []).append(k)
    todo, seen = [(i, 0)], {}
    while todo:
        at, age = todo.pop()
        if seen.get(at, 1 << 30) <= age or age >= states:
            continue
        seen[at] = age
        sources = list(into.get(at, []))
        if at > 0 and not re.match(r"s_branch\b|s_endpgm", code[at - 1]):
            sources.append(at - 1)
        for k in sources:
            if age < states:
                yield code[k]
            m = re.match(r"s_nop\s+(\S+)", code[k])
            todo.append((k, age + (int(m.group(1), 0) + 1 if m else 1)))


def _written(c):
    """The destination operand's text of an instruction."""
    return c.split(None, 1)[1].split(",")[0] if " " in c or "\t" in c else ""


def test_descriptors_are_old_enough(assembly):  # noqa: F811
    """Vector memory reads a scalar that a vector instruction wrote five wait states before
    at the least."""
    for name, text in _kernels(assembly):
        code, labels = _instructions(text)
        loads = [i for i, c in enumerate(code) if c.startswith("buffer_load") and " lds" in c]
        assert len(loads) >= 6, name
        for i in loads:
            reads = _registers(code[i], "s")
            assert reads, code[i]
            for c in _before(code, labels, i, 5):
                if c.startswith("v_"):
                    assert not _registers(_written(c), "s") & reads, (name, c, code[i])


def test_m0_is_old_enough(assembly):  # noqa: F811
    """A load into LDS takes m0 one wait state after it is written, and no other instruction
    writes or reads it meanwhile."""
    for name, text in _kernels(assembly):
        code, _ = _instructions(text)
        for i, c in enumerate(code):
            if c.startswith("buffer_load") and " lds" in c:
                assert re.match(r"s_nop\s+", code[i - 1]) and re.match(r"s_mov_b32 m0,", code[i - 2]), (name, code[i - 2:i])
            elif re.search(r"\bm0\b", c):
                assert re.match(r"s_mov_b32 m0,", c) and " lds" in code[i + 2], (name, c)


def test_operands_are_old_enough(assembly):  # noqa: F811
    """A matrix instruction reads a vector register that a vector instruction other than a
    matrix one wrote two wait states before at the least."""
    for name, text in _kernels(assembly):
        code, labels = _instructions(text)
        for i, c in enumerate(code):
            if not c.startswith("v_mfma"):
                continue
            operands = c.split(None, 1)[1].split(",", 1)[1]
            v, a = _registers(operands, "v"), _registers(operands, "a")
            for b in _before(code, labels, i, 2):
                if b.startswith("v_") and not b.startswith("v_mfma"):
                    to = _written(b)
                    assert not (_registers(to, "v") & v or _registers(to, "a") & a), (name, b, c)
