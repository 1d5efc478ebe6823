"""Offsets, lengths, page tables and places that no 32-bit word can lie at are refused by every entry point of the cache,
before any CUDA call."""
from __future__ import annotations

import pytest

from jagged_attention_recommender_gb300 import build as gbuild
from tests import test_cache_cpu as cache
from tests import test_history_cpu as hist
from tests.test_cache_cpu import A, INV, Desc


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("call,names", [
    (lambda **kw: cache.append(Desc(), **kw), ["offsets", "kv_lens", "page_table"]),
    (lambda **kw: cache.fwd(Desc(), **kw), ["offsets", "kv_lens", "page_table", "lse"]),
    (hist.weights, ["offsets", "kv_lens", "page_table", "lse"]),
    (hist.evict, ["kv_lens", "page_table", "new_table", "kept", "new_lens"]),
    (hist.rope, ["offsets", "first"]),
], ids=["append", "fwd", "weights", "evict", "rope"])
def test_words_that_are_not_aligned_are_refused(call, names, off):
    for name in names:
        hist.refused(call, INV, **{name: 3 * A + off})
