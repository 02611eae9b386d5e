"""Buffers of one call that share memory (CPU only: refused before anything reaches a
device; the comparison itself against every byte of small layouts)."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from state_space_model_ssd_amd import binding as b
from tests.test_layer_host import BAD, conv, lib, norm, step  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
#include "ssd_span.h"
extern "C" int overlap(const unsigned long* v) {
  return ssd::overlap({v[0], v[1], v[2], v[3]}, {v[4], v[5], v[6], v[7]});
}
extern "C" unsigned long capped(unsigned long a, unsigned long b) { return ssd::capped(a, b); }
"""


@pytest.fixture(scope="module")
def span(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("span")
    (d / "span.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "state_space_model_ssd_amd", "csrc"), str(d / "span.cpp"),
                    "-o", str(d / "span.so")], check=True)
    so = ctypes.CDLL(str(d / "span.so"))
    so.capped.restype = ctypes.c_ulong
    so.capped.argtypes = [ctypes.c_ulong] * 2
    return so


def bytes_of(at, row, rows, stride):
    return {at + i * stride + k for i in range(rows) for k in range(row)}


def test_overlap_against_every_byte(span):
    rnd = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(60000):
        v = []
        stride = rnd.randint(1, 12)                 # rows of both have it, or are contiguous
        for _ in range(2):
            row = rnd.randint(1, 12)
            s = stride if rnd.random() < 0.7 and row <= stride else row
            v += [100 + rnd.randint(0, 60), row, rnd.randint(1, 6), s]
        shared = bool(bytes_of(*v[:4]) & bytes_of(*v[4:]))
        one = [v[2] == 1 or v[3] == v[1], v[6] == 1 or v[7] == v[5]]
        got = bool(span.overlap((ctypes.c_ulong * 8)(*v)))
        if one[0] or one[1] or v[3] == v[7]:
            assert got == shared, v
            seen[shared] += 1
        else:
            assert got or not shared, v
    assert min(seen.values()) > 5000


def test_overlap_of_nothing_and_of_huge_sizes(span):
    f = lambda *v: span.overlap((ctypes.c_ulong * 8)(*v))  # noqa: E731
    assert not f(0, 8, 1, 8, 0, 8, 1, 8)            # null
    assert not f(100, 0, 1, 0, 100, 8, 1, 8)        # empty
    assert not f(100, 8, 0, 8, 100, 8, 1, 8)
    assert span.capped(2 ** 31, 2 ** 31) == 2 ** 62 and span.capped(2 ** 40, 2 ** 40) == 2 ** 62
    assert span.capped(0, 5) == span.capped(5, 0) == 0 and span.capped(3, 7) == 21
    assert f(2 ** 47, 2 ** 62, 1, 2 ** 62, 2 ** 56, 4, 1, 4)


def ptrs(n):
    """n addresses far apart."""
    return [(i + 1) << 40 for i in range(n)]


def test_conv_forward_refuses_shared_memory(lib):  # noqa: F811
    # xbc, weight, bias, initial states, cu, out x, out b, out c, final states
    p = conv(batch=1, nseq=2)
    for i, j in ((3, 8), (0, 5), (0, 6), (0, 7), (5, 6), (6, 7), (5, 8), (1, 5), (2, 7), (4, 8)):
        a = ptrs(9)
        a[j] = a[i]
        assert lib.ssd_conv_fwd(ctypes.byref(p), *a, None) == BAD, (i, j)
    a = ptrs(9)
    a[5] = a[0] + 96 * 100 * 2 - 2                  # the last element only
    assert lib.ssd_conv_fwd(ctypes.byref(p), *a, None) == BAD


def test_conv_backward_refuses_shared_memory(lib):  # noqa: F811
    # xbc, weight, bias, init, cu, dout x, b, c, dfinal, dx, dweight, dbias, dinit, workspace
    p = conv(batch=1, nseq=2)
    for i, j in ((0, 9), (5, 9), (8, 12), (3, 12), (1, 10), (2, 11), (9, 13), (10, 13), (0, 13), (12, 9)):
        a = ptrs(14)
        a[j] = a[i]
        assert lib.ssd_conv_bwd(ctypes.byref(p), *a, 1 << 30, None) == BAD, (i, j)
    # columns of one wider tensor that overlap: in_stride 200, dx 95 channels behind x
    q = conv(batch=1, nseq=2, in_stride=200, din_stride=200)
    a = ptrs(14)
    a[9] = a[0] + 2 * 95
    assert lib.ssd_conv_bwd(ctypes.byref(q), *a, 1 << 30, None) == BAD
    a[9] = a[0] + 2 * 105                           # its row's end reaches the next row of x
    assert lib.ssd_conv_bwd(ctypes.byref(q), *a, 1 << 30, None) == BAD


def test_steps_refuse_shared_memory(lib):  # noqa: F811
    # xbc, weight, bias, states | slots, out x, out b, out c
    p = conv(seqlen=1)
    for i, j in ((0, 3), (3, 5), (0, 5), (5, 6), (4, 7), (1, 3)):
        a = ptrs(8)
        a[j] = a[i]
        assert lib.ssd_conv_step(ctypes.byref(p), *a[:4], 2, *a[4:], None) == BAD, (i, j)
    # x, dt, dt_bias, A, B, C, D, states, slots, out
    for i, j in ((0, 9), (1, 9), (4, 7), (7, 9), (3, 7), (8, 9)):
        a = ptrs(10)
        a[j] = a[i]
        assert lib.ssd_step(ctypes.byref(step()), *a, None) == BAD, (i, j)
    a = ptrs(10)                                    # B behind x in a row, out inside the row
    a[9] = a[0] + 2 * 512
    a[4] = a[9]
    assert lib.ssd_step(ctypes.byref(step(x_stride=2000, b_stride=2000)), *a, None) == BAD


def test_block_norm_refuses_shared_memory(lib):  # noqa: F811
    # x, residual, gate, post, scale, pre, out, residual out
    p = norm(residual_dtype=b.SSD_BF16)
    for i, j in ((0, 7), (1, 6), (2, 6), (2, 7), (5, 6), (6, 7), (3, 7)):
        a = ptrs(8)
        a[j] = a[i]
        assert lib.ssd_block_norm_fwd(ctypes.byref(p), *a, None) == BAD, (i, j)
    for i, j in ((0, 6), (1, 7)):                   # in place, but shifted
        a = ptrs(8)
        a[j] = a[i] + 2
        assert lib.ssd_block_norm_fwd(ctypes.byref(p), *a, None) == BAD, (i, j)
    a = ptrs(8)                                     # an fp32 stream over the bf16 rows
    a[1] = a[6] = a[0]
    assert lib.ssd_block_norm_fwd(ctypes.byref(norm()), *a, None) == BAD
    # x, residual, gate, post, scale, pre, dout, dh, dx, dres, dgate, dpost, dscale, dpre, ws
    for i, j in ((0, 8), (6, 8), (7, 9), (8, 9), (8, 10), (2, 10), (11, 12), (5, 13), (8, 14), (0, 14)):
        a = ptrs(15)
        a[j] = a[i]
        assert lib.ssd_block_norm_bwd(ctypes.byref(p), *a, 1 << 30, None) == BAD, (i, j)
