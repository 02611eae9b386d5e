"""Chunk counts of a packed batch, added as the plan adds them (the library's own rule compiled for
the host, CPU): lengths that run back and forth, 0 to all tokens and back, never pass the chunks that
there is room for, also where their plain sum does not fit 32 bits."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
#include "ssd_plan_rule.h"
extern "C" int add(int a, int b, int most) { return ssd::add_chunks(a, b, most); }
"""


@pytest.fixture(scope="module")
def add(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "rule.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "state_space_model_ssd_amd", "csrc"), str(d / "rule.cpp"),
                    "-o", str(d / "rule.so")], check=True)
    return ctypes.CDLL(str(d / "rule.so")).add


def test_one_sum(add):
    most = 2 ** 24 + 5
    for a, b, want in ((0, 0, 0), (3, 4, 7), (most, 0, most), (0, most, most), (most, most, most),
                       (most - 1, 1, most), (most - 2, 1, most - 1), (1, most - 1, most)):
        assert add(a, b, most) == want, (a, b)
    assert add(0, 0, 0) == 0


@pytest.mark.parametrize("tokens", [2 ** 30 - 1, 10 ** 6, 130])
@pytest.mark.parametrize("nseq", [3, 256, 300, 1000])
@pytest.mark.parametrize("kind", ["back and forth", "rising"])
def test_prefixes(add, tokens, nseq, kind):
    """Waves of 64 sequences, four waves at a time, as plan_seq_kernel does."""
    L = 64
    if kind == "rising":
        cu = np.sort(np.random.default_rng(1).integers(0, tokens + 1, nseq + 1))
    else:
        cu = np.arange(nseq + 1) % 2 * tokens
    begin = np.clip(cu[:-1], 0, tokens)
    counts = (np.maximum(np.clip(cu[1:], 0, tokens), begin) - begin + L - 1) // L
    most = int(min((tokens + nseq * (L - 1)) // L, tokens))
    got, carry = [], 0
    for base in range(0, nseq, 256):
        c = np.zeros(256, np.int64)
        c[:len(counts[base:base + 256])] = np.minimum(counts[base:base + 256], most)
        totals = []
        for w in range(4):
            v = [int(x) for x in c[64 * w:64 * w + 64]]
            off = 1
            while off < 64:
                v = [add(v[i], v[i - off], most) if i >= off else v[i] for i in range(64)]
                off *= 2
            before = carry
            for t in totals:
                before = add(before, t, most)
            got += [before if i == 0 else add(before, v[i - 1], most) for i in range(64)]
            totals.append(v[63])
        for t in totals:
            carry = add(carry, t, most)
    want = np.minimum(np.concatenate(([0], np.cumsum(counts))), most)
    assert got[:nseq] + [carry] == want.tolist()
    if kind == "back and forth" and nseq > 256 and tokens > 2 ** 29:
        assert counts.sum() >= 2 ** 31
