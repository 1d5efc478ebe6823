"""Rows that are turned into rows they overlap: the arithmetic (csrc/gdpa_cache_index.h, compiled for the host) against every
pair of rows, and the calls that gdpa_rope refuses for it."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from jagged_attention_recommender_gb300 import build as gbuild
from tests.test_cache_cpu import A, INV
from tests.test_history_cpu import refused, rope

HOST = r"""
#include "gdpa_cache_index.h"
extern "C" int overlap(long long apart, long long xs, long long ys, long long len, long long T) {
  return gdpa::rows_overlap(apart, xs, ys, len, T);
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    gbuild.build()
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    d = tmp_path_factory.mktemp("rows_overlap")
    src, so = d / "host.cpp", d / "host.so"
    src.write_text(HOST)
    subprocess.check_call([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", gbuild.CSRC, str(src), "-o", str(so)])
    lib = ctypes.CDLL(str(so))
    lib.overlap.argtypes = [ctypes.c_longlong] * 5
    return lib


def test_every_place_of_small_rows(host):
    for T in (1, 2, 3, 7):
        for length in (1, 3, 4):
            for xs in (4, 5, 8, 9):
                for ys in (4, 5, 7, 8, 16):
                    x = np.arange(T) * xs
                    for apart in range(-T * ys - 10, T * xs + 11):
                        y = apart + np.arange(T) * ys
                        want = bool((np.abs(x[:, None] - y[None]) < length).any())
                        assert bool(host.overlap(apart, xs, ys, length, T)) == want, (T, length, xs, ys, apart)


def test_rows_far_apart(host):
    big = 1 << 40
    assert not host.overlap(big, 12288, 8192, 8192, 1 << 21) and not host.overlap(-big, 12288, 8192, 8192, 1 << 21)
    # every row and every second row of one buffer, in columns of their own
    assert not host.overlap(512, 1024, 2048, 512, 1 << 20) and host.overlap(512, 1024, 2048, 513, 1 << 20)
    # the last row of x ends at 2^20 1024 - 512
    assert host.overlap((1 << 30) - 513, 1024, 512, 512, 1 << 20) and not host.overlap((1 << 30) - 512, 1024, 512, 512, 1 << 20)


@pytest.mark.parametrize("kw", [
    dict(y=A + 512, x_stride=512), dict(y=A + 1024 * 3 + 256, x_stride=512, y_stride=264),   # rows of x from A on, 512 elements apart
    dict(y=A - 3 * 528, y_stride=264), dict(y=A - 2 * 1024, y_stride=1024, x_stride=512),
    dict(y=A + 16, x_stride=1 << 20, T=1), dict(y=A + 16, y_stride=1 << 20),
])
def test_rope_refuses_rows_of_other_strides_that_overlap(host, kw):
    refused(rope, INV, **kw)
