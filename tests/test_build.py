"""The build of the product library: what it passes on, and what a failing source leaves."""
import importlib.util
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def builder(tmp_path, monkeypatch):
    """The build module with sources of its own (plain C++, for the host compiler), and the
    commands that it ran."""
    spec = importlib.util.spec_from_file_location(
        "_zs_build_test", os.path.join(ROOT, "sharded_optimizer_step_zero_amd", "_build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    (tmp_path / "a.cpp").write_text("int a() { return 1; }\n")
    (tmp_path / "b.cpp").write_text("int b() { return 2; }\n")
    (tmp_path / "bad.cpp").write_text("int c( { return 3; }\n")
    # takes seconds to compile
    (tmp_path / "slow.cpp").write_text("#include <regex>\n#include <iostream>\n#include <algorithm>\n" + "".join(
        f"bool f{i}(const std::string& s) {{ return std::regex_match(s, std::regex(\"{i}+\")); }}\n" for i in range(60)))
    m.LIB = str(tmp_path / "lib.so")
    m.HOST_SOURCES = []
    m.SOURCES = [str(tmp_path / "a.cpp"), str(tmp_path / "b.cpp")]
    m.started, m.commands = [], []
    popen, run = subprocess.Popen, subprocess.run

    class Recorded(popen):
        def __init__(self, cmd, *a, **k):
            super().__init__(cmd, *a, **k)
            m.started.append(self)
            m.commands.append(list(cmd))
    monkeypatch.setattr(subprocess, "Popen", Recorded)
    yield m
    monkeypatch.setattr(subprocess, "Popen", popen)
    monkeypatch.setattr(subprocess, "run", run)


def test_flags_reach_every_compiler_and_the_linker(builder):
    builder.build(extra_flags=["-DEXTRA=1"])
    assert os.path.exists(builder.LIB)
    assert len(builder.commands) == 3 and all("-DEXTRA=1" in c for c in builder.commands)
    assert "-shared" in builder.commands[-1]


def test_a_failing_source_leaves_nothing_running(builder, tmp_path):
    builder.SOURCES = [str(tmp_path / f) for f in ("bad.cpp", "slow.cpp", "a.cpp")]
    with pytest.raises(subprocess.CalledProcessError) as e:
        builder.build()
    assert any(c.endswith("bad.cpp") for c in e.value.cmd)
    assert len(builder.started) == 3 and all(p.returncode is not None for p in builder.started)
    assert not os.path.exists(builder.LIB) and not os.path.exists(builder.LIB + ".tmp")
