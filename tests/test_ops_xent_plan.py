"""Which tiles and pieces a cross entropy call takes, from the rules' own source compiled for
the host: the GPU tests' cases reach every path that they are there for."""
import ctypes
import os
import subprocess

import pytest

from test_gpu_ops_xent_tiles import CASES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sharded_optimizer_step_zero_amd", "csrc")
SOURCE = """
#include "xent_plan.h"
extern "C" void query(int64_t tokens, int64_t vocab, int64_t width, int backward, int64_t* out) {
  const zs::ops::xent::Plan p =
      zs::ops::xent::plan((void*)4096, width, (void*)4096, width, tokens, vocab, width, backward != 0);
  const int64_t v[] = {p.small, p.small_h, p.small_w, p.piece, p.splits, p.copy_w, p.copy_h, (int64_t)p.total};
  for (int i = 0; i < 8; i++) out[i] = v[i];
}
"""
NAMES = ["small", "small_h", "small_w", "piece", "splits", "copy_w", "copy_h", "total"]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("plan")
    (tmp / "q.cpp").write_text(SOURCE)
    lib = str(tmp / "q.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-I", CSRC,
                    str(tmp / "q.cpp"), "-o", lib], check=True)
    query = ctypes.CDLL(lib).query
    i64 = ctypes.c_int64

    def ask(tokens, vocab, width, backward):
        out = (i64 * 8)()
        query(i64(tokens), i64(vocab), i64(width), int(backward), out)
        return dict(zip(NAMES, out))
    return ask


@pytest.mark.parametrize("shape", CASES)
def test_cases_take_their_paths(plan, shape):
    want, (tokens, vocab, width) = CASES[shape], shape
    p = plan(*shape, True)
    p["pieces"] = -(-vocab // p["piece"])
    p["last"] = vocab - (p["pieces"] - 1) * p["piece"]
    assert {k: p[k] for k in want} == want
    assert plan(*shape, False)["small"] == want["small"]  # the loss's product too


def test_every_path_has_a_case(plan):
    """Both tiles of every product, one piece and several, whole and copied weights, one part
    of k and several; both tiles of the logits and large ones of grad_weight with more than
    three steps of 64 along k and a ragged last one."""
    for key in ("small", "small_h", "small_w"):
        assert {v[key] for v in CASES.values()} == {0, 1}, key
    assert {v["pieces"] for v in CASES.values()} == {1, 2} and {v["copy_w"] for v in CASES.values()} == {0, 1}
    assert {v["splits"] > 1 for v in CASES.values()} == {False, True}

    def ragged(k):
        return k > 192 and k % 64 != 0
    for small in (0, 1):
        assert any(v["small"] == small and ragged(s[2]) for s, v in CASES.items())
    assert any(not v["small_w"] and ragged(s[0]) for s, v in CASES.items())


def test_the_workspace_is_the_plan(plan):
    from sharded_optimizer_step_zero_amd import ops
    for shape in CASES:
        tokens, vocab, width = shape
        for backward in (0, 1):
            assert ops.zs_xent_workspace_bytes(4096, width, 4096, width, tokens, vocab, width, backward) == \
                plan(*shape, backward)["total"]
