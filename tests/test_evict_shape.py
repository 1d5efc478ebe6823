"""How an eviction's choice is launched (csrc/gdpa_cache_index.h, compiled for the host): with clusters that the device
places, and a part of the tokens for each CTA that holds them all."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

from jagged_attention_recommender_gb300 import build as gbuild

HOST = r"""
#include "gdpa_cache_index.h"
extern "C" void shape(long long heads, long long most, int sms, int widest, long long* out) {
  const gdpa::ChooseShape c = gdpa::choose_shape(heads, most, sms, widest);
  out[0] = c.ctas, out[1] = c.threads, out[2] = c.part;
}
extern "C" int every() { return gdpa::kEveryCluster; }
extern "C" int most() { return gdpa::kMostCluster; }
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    d = tmp_path_factory.mktemp("evict_shape")
    src, so = d / "host.cpp", d / "host.so"
    src.write_text(HOST)
    subprocess.check_call([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", gbuild.CSRC, str(src), "-o", str(so)])
    return ctypes.CDLL(str(so))


def shape(host, heads, most, sms, widest):
    out = (ctypes.c_longlong * 3)()
    host.shape(ctypes.c_longlong(heads), ctypes.c_longlong(most), sms, widest, out)
    return tuple(out)


@pytest.mark.parametrize("sms", [14, 76, 152])
def test_clusters_are_no_wider_than_the_device_places(host, sms):
    for widest in (host.every(), host.most()):
        for heads in (1, 2, 4, 9, 77, 152, 303, 304, 1 << 20, (1 << 31) * 100):
            for most in (16, 17, 2048, 4096, 8192, 131072, 400003, 2 ** 31 - 16):
                ctas, threads, part = shape(host, heads, most, sms, widest)
                assert 1 <= ctas <= widest and ctas & (ctas - 1) == 0 and threads in (256, 1024)
                assert part % 4 == 0 and part * ctas >= most and (ctas == 1 or heads * ctas <= sms)
                # a sequence that is as long as the table or shorter: every CTA's part of it
                for length in (1, most // 2, most):
                    assert ((length + ctas - 1) // ctas + 3) // 4 * 4 <= part


def test_a_device_that_places_eight(host):
    """Two histories of 131 072 tokens with 2 heads each: 16 CTAs a head, or 8 with twice the tokens."""
    assert host.every() == 8
    assert shape(host, 4, 131072, 152, host.most()) == (16, 1024, 8192)
    assert shape(host, 4, 131072, 152, host.every()) == (8, 1024, 16384)
