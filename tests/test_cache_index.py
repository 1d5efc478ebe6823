"""The paged cache's index arithmetic (csrc/gdpa_cache_index.h), compiled for the host as plain C++."""
from __future__ import annotations

import ctypes
import fractions
import os
import shutil
import subprocess

import numpy as np
import pytest

from jagged_attention_recommender_gb300 import build as gbuild

HOST = r"""
#include "gdpa_cache_index.h"
#include <algorithm>
using namespace gdpa;

// the lookups of gdpa_cache.cuh: by halves, and by 32 lanes of a warp
static int find_one(const int* off, int B, int r) {
  int lo = 0, hi = B;
  while (lo < hi) { const int mid = (lo + hi) >> 1; if (off[mid + 1] > r) hi = mid; else lo = mid + 1; }
  return lo;
}
static int find_warp(const int* off, int B, int r) {
  int lo = 0, hi = B;
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    int n = 0;
    while (n < 32 && off[std::min(lo + step * (n + 1), hi)] <= r) ++n;
    lo = std::min(lo + step * n, hi);
    if (n < 32) hi = std::min(lo + step - 1, hi);
  }
  return lo;
}

// The owners of every group of `rows` rows, as the append kernel finds them: {row, cnt, pos, b, tab} each.  Returns how
// many there are; *bad counts the rows that flag the launch.
extern "C" int owners(const int* off, const int* lens, int T, int B, long long most, int rows, int* out, int* bad) {
  int found = 0;
  *bad = 0;
  for (int g0 = 0; g0 < T; g0 += rows) {
    const int b0 = find_warp(off, B, g0);
    int tab = 0;
    for (int lane = 0; lane < rows && g0 + lane < T; ++lane) {
      const int r = g0 + lane;
      int b = b0;
      for (int i = 0; i < 32; ++i) b += (b0 + i < B ? off[b0 + i + 1] : 0x7fffffff) <= r;
      if (b == b0 + 32) b = find_one(off, B, r);
      if (b >= B) continue;
      const OwnedRows o = owned_rows(cache_sequence(off[b], off[b + 1], lens[b], T, most), r);
      *bad += o.bad;
      tab += o.cnt;
      if (o.cnt == 0) continue;
      if (tab > rows + kCacheBlock - 1) { ++*bad; continue; }
      const int v[6] = {r, o.cnt, o.pos, b, tab - o.cnt, g0};
      std::copy(v, v + 6, out + 6 * found++);
    }
  }
  return found;
}

extern "C" unsigned long long turn(double f) { return turn_fraction(f); }
extern "C" int first(int pos, int window) { return first_key(pos, window); }
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    d = tmp_path_factory.mktemp("cache_index")
    src, so = d / "host.cpp", d / "host.so"
    src.write_text(HOST)
    subprocess.check_call([cxx, "-std=c++17", "-O1", "-fwrapv", "-Wall", "-Werror", "-shared", "-fPIC", "-I", gbuild.CSRC,
                           str(src), "-o", str(so)])
    lib = ctypes.CDLL(str(so))
    lib.turn.argtypes, lib.turn.restype = [ctypes.c_double], ctypes.c_uint64
    return lib


def owners(host, off, lens, T, most, rows):
    off, lens = np.asarray(off, np.int32), np.asarray(lens, np.int32)
    out = np.zeros((T + 1, 6), np.int32)
    bad = ctypes.c_int(0)
    n = host.owners(off.ctypes.data_as(ctypes.c_void_p), lens.ctypes.data_as(ctypes.c_void_p), T, len(lens),
                    ctypes.c_longlong(most), rows, out.ctypes.data_as(ctypes.c_void_p), ctypes.byref(bad))
    return out[:n], bad.value


def check_inside(got, off, lens, T, most, rows):
    for r, cnt, pos, b, tab, g0 in got.tolist():
        what = (off, lens, rows, r, cnt, pos, b, tab)
        assert 1 <= cnt <= 16 and pos % 16 + cnt <= 16, what
        assert 0 <= off[b] <= r and r + cnt <= off[b + 1] <= T, what          # rows of the sequence
        assert 0 <= pos and pos + cnt <= lens[b] <= most, what                # positions in the page table
        assert 0 <= tab and tab + cnt <= rows + 15, what                      # room in the table of angles
    for g0 in np.unique(got[:, 5]):
        assert (got[:, 5] == g0).sum() <= 16


def test_decreasing_offsets_leave_every_owner_inside(host):
    off, lens, most = [0, 24, 2, 3, 13, 39], [43, 853, 353, 535, 360], 64 * 16
    got, bad = owners(host, off, lens, 39, most, 16)
    check_inside(got, off, lens, 39, most, 16)
    assert bad > 0


@pytest.mark.parametrize("seed", range(40))
def test_any_offsets_leave_every_owner_inside(host, seed):
    rng = np.random.default_rng(seed)
    for _ in range(50):
        B, T = int(rng.integers(1, 90)), int(rng.integers(1, 200))
        off = np.sort(rng.integers(0, T + 1, B + 1))
        off[0] = 0
        for _ in range(int(rng.integers(0, 6))):  # spoilt places
            off[rng.integers(0, B + 1)] = rng.choice([0, T, -1, T + 1, -2 ** 31, 2 ** 31 - 1, int(rng.integers(0, T + 1))])
        most = 16 * int(rng.integers(1, 70))
        lens = rng.integers(0, most + 1, B)
        lens[rng.random(B) < 0.1] = rng.choice([-1, most + 1, -2 ** 31, 2 ** 31 - 1])
        rows = int(rng.choice([1, 2, 4, 8, 16]))
        got, _ = owners(host, off, lens, T, most, rows)
        check_inside(got, off.tolist(), lens.tolist(), T, most, rows)


@pytest.mark.parametrize("seed", range(20))
@pytest.mark.parametrize("rows", [1, 4, 16])
def test_right_offsets_give_every_row_to_one_owner(host, seed, rows):
    rng = np.random.default_rng(100 + seed)
    new = rng.integers(0, [2, 4, 40][seed % 3], int(rng.integers(1, 120)))
    off = np.concatenate([[0], np.cumsum(new)])
    T = int(off[-1]) + int(rng.integers(0, 5))  # rows behind the last sequence
    if T == 0:
        return
    lens = new + rng.integers(0, 60, len(new))
    got, bad = owners(host, off, lens, T, 128, rows)
    check_inside(got, off.tolist(), lens.tolist(), T, 128, rows)
    assert bad == 0
    times = np.zeros(T, int)
    for r, cnt, pos, b, _, _ in got.tolist():
        times[r:r + cnt] += 1
        assert pos == lens[b] - new[b] + r - off[b]
    assert (times[:off[-1]] == 1).all() and (times[off[-1]:] == 0).all()


def test_a_window_s_first_key(host):
    ends = [-2 ** 31 + 256, -2 ** 31 + 300, -5, -1, 0, 1, 2, 6, 7, 2 ** 20, 2 ** 31 - 17]
    for pos in ends:
        for window in (0, 1, 2, 6, 7, 8, 2 ** 20, 2 ** 31 - 4, 2 ** 31 - 1):
            assert host.first(pos, window) == (max(0, pos - window + 1) if window else 0), (pos, window)


def two_pi(digits=60):
    """2 pi as a fraction, by Machin's formula in whole numbers."""
    def arctan_of_one_over(n):
        term = total = 10 ** (digits + 10) // n
        k = 1
        while term:
            term //= -n * n
            k += 2
            total += term // k
        return total
    return fractions.Fraction(8 * (4 * arctan_of_one_over(5) - arctan_of_one_over(239)), 10 ** (digits + 10))


def test_fractions_of_a_turn(host):
    """Off by one unit of 2^-64 at most, so that an angle is right to 2^-32 turns (and the unit below it) wherever a
    position lies."""
    circle = two_pi()
    freqs = list(10000.0 ** (-np.arange(0, 128, 2) / 128)) + list(5e5 ** (-np.arange(0, 64, 2) / 64))
    freqs += [0.0, 5e-324, 1e-300, 2.0 ** -70, 1e-12, 1.0, np.pi, 2 * np.pi, 100.0, 12345.678, 2.0 ** 30, 1e11]
    for f in freqs:
        for x in (f, -f):
            exact = fractions.Fraction(x) / circle
            got = host.turn(x)
            units = (fractions.Fraction(got) - exact * 2 ** 64) % 2 ** 64
            assert min(units, 2 ** 64 - units) <= 1, (x, float(units))
            for pos in (1, 131071, 2 ** 24 + 1, 2 ** 31 - 17):
                angle = (pos * got % 2 ** 64 >> 32) / fractions.Fraction(2 ** 32)
                off = (angle - exact * pos) % 1
                assert min(off, 1 - off) <= fractions.Fraction(3, 2) / 2 ** 32, (x, pos)
