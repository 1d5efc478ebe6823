"""The order in which the kernel of the stored keys' weight brings a CTA's items (csrc/gdpa_cache_order.h), compiled for the
host: a model of the roles that read the items' ring, one thread each, in which every wait has to end."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from jagged_attention_recommender_gb300 import build as gbuild

HOST = r"""
#include "gdpa_cache_order.h"
#include <chrono>
#include <condition_variable>
#include <mutex>
#include <thread>
#include <vector>
using namespace gdpa;

// A ring of `places` records that `readers` warps read, each in order.  A sums warp that has read an item that some row
// sees reads on once the item's copies are there; the copies find two items' notes of room.
struct Model {
  std::mutex m;
  std::condition_variable changed;
  const unsigned char* chunks;  // of an item: 0 no row sees it
  int items, places, readers;
  std::vector<int> read;        // records that each reader has read
  int written = 0, brought = 0, summed = 0;  // brought, summed: items that some row sees
  bool given_up = false;

  template <class F>
  bool wait(std::unique_lock<std::mutex>& l, const F& f) {
    if (!changed.wait_for(l, std::chrono::seconds(10), [&]() { return given_up || f(); })) given_up = true;
    changed.notify_all();
    return !given_up;
  }
  // Record i (items: no more), once it is written.
  bool next(int reader, int& i) {
    std::unique_lock<std::mutex> l(m);
    if (!wait(l, [&]() { return written > read[reader]; })) return false;
    i = read[reader]++;
    changed.notify_all();
    return i < items;
  }
  void find() {
    for (int i = 0; i <= items; ++i) {
      std::unique_lock<std::mutex> l(m);
      if (!wait(l, [&]() {
            for (int r : read)
              if (r < i - places + 1) return false;
            return true;
          }))
        return;
      written = i + 1;
      changed.notify_all();
    }
  }
  void sum(int reader) {
    int i, mine = 0;
    while (next(reader, i)) {
      if (!chunks[i]) continue;
      ++mine;
      std::unique_lock<std::mutex> l(m);
      if (!wait(l, [&]() { return brought >= mine; })) return;
      if (reader == 1) summed = mine;
      changed.notify_all();
    }
  }
  // Returns the items that were brought, in `out`.
  int copy(int* out) {
    int i = -1, looked = -1, item = -1, n = 0;
    bring_in_order([&]() { return next(0, i); }, [&]() { return chunks[i] != 0; }, [&]() { looked = i; }, [&]() { item = looked; },
                   [&]() {
                     std::unique_lock<std::mutex> l(m);
                     if (!wait(l, [&]() { return brought < summed + 2; })) return false;
                     out[n++] = item;
                     ++brought;
                     changed.notify_all();
                     return true;
                   });
    return n;
  }
};

extern "C" int run(const unsigned char* chunks, int items, int places, int readers, int* out) {
  Model a;
  a.chunks = chunks, a.items = items, a.places = places, a.readers = readers;
  a.read.assign(readers, 0);
  std::vector<std::thread> t;
  t.emplace_back([&]() { a.find(); });
  for (int r = 1; r < readers; ++r) t.emplace_back([&a, r]() { a.sum(r); });
  const int n = a.copy(out);
  for (auto& x : t) x.join();
  return a.given_up ? -1 : n;
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    d = tmp_path_factory.mktemp("cache_order")
    src, so = d / "host.cpp", d / "host.so"
    src.write_text(HOST)
    subprocess.check_call([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-pthread", "-I", gbuild.CSRC,
                           str(src), "-o", str(so)])
    return ctypes.CDLL(str(so))


def bring(host, chunks, readers=3, places=4):
    chunks = np.ascontiguousarray(chunks, np.uint8)
    out = np.full(len(chunks) + 1, -1, np.int32)
    n = host.run(chunks.ctypes.data_as(ctypes.c_void_p), len(chunks), places, readers, out.ctypes.data_as(ctypes.c_void_p))
    assert n >= 0, "a role waits for ever"
    assert np.array_equal(out[:n], np.flatnonzero(chunks))


@pytest.mark.parametrize("gap", [0, 1, 2, 3, 4, 5, 6, 9, 40])
def test_items_that_no_row_sees_between_those_that_rows_see(host, gap):
    for lead in (0, 1, 7):
        bring(host, [0] * lead + ([1] + [0] * gap) * 5 + [1])
        bring(host, [0] * lead + ([1, 1, 1] + [0] * gap) * 5)


@pytest.mark.parametrize("chunks", [[], [0], [1], [0] * 30, [1] * 30, [0] * 9 + [1], [1] + [0] * 9])
def test_few_items_and_none(host, chunks):
    bring(host, chunks)


@pytest.mark.parametrize("seed", range(12))
def test_any_order(host, seed):
    rng = np.random.default_rng(seed)
    bring(host, rng.random(int(rng.integers(1, 150))) < rng.choice([0.05, 0.2, 0.6]), readers=int(rng.integers(2, 6)))


def windowed_items(lens, new, H, window, ctas, cta):
    """Whether any row sees the items of a CTA, in its order: items of 256 keys, head by head, taken there and back."""
    seen = []
    for n, rows in zip(lens, new):
        k0 = np.arange(0, n, 256)
        first = np.maximum(n - rows - window + 1, 0)
        seen += list(np.tile(k0 + 255 >= first, H))
    at, back, got = cta, False, []
    while at < len(seen):
        got.append(seen[at])
        back = not back
        at += 2 * (ctas - 1 - cta if back else cta) + 1
    return got


@pytest.mark.parametrize("lens,rows,H,window", [([6000] * 64, 100, 8, 512), ([131072] * 2, 128, 8, 4096), ([24000] * 4, 100, 8, 300)])
def test_windows_over_many_items(host, lens, rows, H, window):
    """Calls whose windows leave long runs of items unseen, as the CTAs of a GPU of 152 SMs meet them."""
    for cta in (0, 1, 75, 151):
        bring(host, windowed_items(lens, [rows] * len(lens), H, window, 152, cta))
