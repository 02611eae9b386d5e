"""How long sequences of the gated delta rule are cut: the library's own rule compiled for the host
(CPU), against the estimate made of the chains themselves, one by one."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
#include "ssd_delta_cut.h"
extern "C" int best(const int* n, int seqs, int least, int H, int P, int N, int block, int cus) {
  ssd::DeltaCut c;
  c.least = least;
  ssd::DeltaCut::Sums v = {};
  int chunks = 0;
  for (int i = 0; i < seqs; ++i) {
    v.add(c, n[i], 1);
    chunks += n[i];
  }
  return ssd::DeltaCut::best(c, v, chunks, H, P, N, block, cus);
}
extern "C" void segment(const int* first, int n, int length, int slot, int* out) {
  ssd::DeltaCut::segment(n, length, slot, [&](int i) { return first[i]; }, out[0], out[1]);
}
extern "C" void cut(int n, int length, int* out) { ssd::DeltaCut::cut(n, length, out[0], out[1]); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("cut")
    (d / "rule.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "state_space_model_ssd_amd", "csrc"), str(d / "rule.cpp"),
                    "-o", str(d / "rule.so")], check=True)
    return ctypes.CDLL(str(d / "rule.so"))


def segments(lib, n, length):
    out = (ctypes.c_int * 2)()
    lib.cut(n, length, out)
    parts, per = out
    return [min(per, n - i * per) for i in range(parts)]


def best(lib, n, least, *sizes):
    return lib.best((ctypes.c_int * len(n))(*n), len(n), least, *sizes)


def estimates(lib, n, least, H, P, N, block, cus):
    """Steps of no cutting (0) and of each length."""
    rows, unit = -(-P // block) * H, -(-N // block) * H
    work = lambda chains, r: sum(chains) * r  # noqa: E731
    every = work(n, rows) // cus
    steps = {0: max(max(n), every)}
    for i in range(6):
        L = least << i
        if max(n) < 2 * L:
            continue
        cut = [segments(lib, c, L) for c in n]
        zeros = [s for segs in cut for s in segs[:-1]]
        units = [s for segs in cut for s in segs[1:-1]]
        chain = max(s for segs in cut for s in segs)
        steps[L] = max((work(zeros, rows) + work(units, unit)) // cus, L) + max(every, chain) + max(n) // L + 6
    return steps


@pytest.mark.parametrize("least", [1, 16, 50])
def test_segments_cover_the_sequence(lib, least):
    for n in list(range(300)) + [1000, 4097]:
        s = segments(lib, n, least)
        assert sum(s) == n and max(s) <= (least if n >= 2 * least else max(n, 1)) and (n == 0 or min(s) > 0)
        assert len(s) <= n // least + 1


def test_lengths_are_those_of_the_least_estimate(lib):
    r = random.Random(5)
    seen = set()
    for _ in range(2000):
        n = [int(2 ** r.uniform(0, 8)) for _ in range(r.randint(1, 64))]
        sizes = (r.choice((1, 2, 4, 8, 16, 32)), r.choice((16, 64, 128)), r.choice((32, 64, 128)), r.choice((32, 64)), 256)
        steps = estimates(lib, n, 16, *sizes)
        got = best(lib, n, 16, *sizes)
        assert steps[got] == min(steps.values()), (n, sizes, got, steps)
        seen.add(got)
    assert {0, 16, 32, 64} <= seen


def test_sequences_that_stay_whole_count(lib):
    """A sequence of 47 chunks is not cut into segments of 32, so with these the second pass takes
    47 steps: segments of 16 are shorter."""
    assert best(lib, [47, 141], 16, 16, 64, 128, 32, 256) == 16


def test_every_segment_has_a_slot(lib):
    """The sequences' first segments in the first slots, in order, so that where nothing is cut the
    workgroups without work are behind all others; every other one in a slot of its own."""
    r = random.Random(6)
    for _ in range(300):
        n = [r.choice((0, 1, r.randint(0, 40), r.randint(0, 300))) for _ in range(r.randint(1, 64))]
        first = [sum(n[:i]) for i in range(len(n))]
        least = r.choice((1, 16, 20))
        length = r.choice((0, least, 2 * least, 4 * least))
        arr, out, seen = (ctypes.c_int * len(n))(*first), (ctypes.c_int * 2)(), []
        for slot in range(len(n) + (sum(n) + r.randint(0, 5)) // least):
            lib.segment(arr, len(n), length, slot, out)
            seq, part = out
            if part < len(segments(lib, n[seq], length)):
                seen.append((seq, part))
                assert (part == 0) == (slot < len(n))
        assert seen[:len(n)] == [(i, 0) for i in range(len(n))] and len(set(seen)) == len(seen)
        assert len(seen) == sum(len(segments(lib, c, length)) for c in n)
