"""The rows per thread of the single-token state update, from the library's own rule
compiled for the host (CPU): the cases of tests/test_gpu_step_rows.py have the rows that
they are there for, and leave a remainder."""
import ctypes
import os
import shutil
import subprocess

import pytest

from tests.step_rows_cases import CASES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
#include "ssd_step_rule.h"
extern "C" int rows(long b, long h, long p, int n) { return ssd::step_rows(b, h, p, n); }
extern "C" int lanes(int n) { return ssd::step_lpr(n); }
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("rule")
    (d / "rule.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "state_space_model_ssd_amd", "csrc"), str(d / "rule.cpp"),
                    "-o", str(d / "rule.so")], check=True)
    so = ctypes.CDLL(str(d / "rule.so"))
    so.rows.argtypes = [ctypes.c_long] * 3 + [ctypes.c_int]
    return so


@pytest.mark.parametrize("name", sorted(CASES))
def test_cases_have_their_rows(rule, name):
    rows, (batch, H, P, N) = CASES[name][0], CASES[name][1][:4]
    assert rule.rows(batch, H, P, N) == rows
    lanes = rule.lanes(N)
    threads = 256
    while threads > 64 and threads // 2 * rows >= P * lanes:
        threads //= 2
    assert P % (threads // lanes * rows) != 0 or N % 4 != 0 or lanes * 4 != N


def test_every_count_of_rows_is_covered(rule):
    assert {c[0] for c in CASES.values()} == {2, 4}
    assert rule.rows(1, 24, 64, 128) == 1 and rule.rows(10 ** 4, 10 ** 3, 64, 3) == 1
    assert [rule.lanes(n) for n in (1, 2, 3, 4, 5, 16, 17, 127, 128, 129, 255, 256)] == \
        [1, 2, 4, 1, 2, 4, 8, 32, 32, 64, 64, 64]
