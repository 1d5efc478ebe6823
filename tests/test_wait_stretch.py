"""How long the roles of the kernel for many rows wait for one another (csrc/gdpa_cache_order.h, compiled for the host): at
least as long as the largest calls take them."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

from jagged_attention_recommender_gb300 import build as gbuild

HOST = r"""
#include "gdpa_cache_order.h"
extern "C" unsigned long long stretch(long long rows, long long sequences) { return gdpa::wait_stretch(rows, sequences); }
"""


@pytest.fixture(scope="module")
def stretch(tmp_path_factory):
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    d = tmp_path_factory.mktemp("wait_stretch")
    src, so = d / "host.cpp", d / "host.so"
    src.write_text(HOST)
    subprocess.check_call([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", gbuild.CSRC, str(src), "-o", str(so)])
    f = ctypes.CDLL(str(so)).stretch
    f.argtypes, f.restype = [ctypes.c_longlong] * 2, ctypes.c_ulonglong
    return f


def test_ordinary_calls_wait_no_longer(stretch):
    assert stretch(1, 1) == stretch(1 << 20, 1 << 20) == 1


@pytest.mark.parametrize("rows", [1, 2 ** 27, 2 ** 31 - 257])
@pytest.mark.parametrize("sequences", [1, 2 ** 26, 2 ** 28, 2 ** 31 - 4098])
def test_the_largest_calls_have_the_time_they_take(stretch, rows, sequences):
    """At 4 s a unit; an item's rows take 2^-27 s each, a sequence without rows 610 ns / 32."""
    assert 4 * stretch(rows, sequences) >= 1.5 * (rows * 2.0 ** -27 + sequences * 610e-9 / 32)
