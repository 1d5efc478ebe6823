"""Refusals of the paged cache at the ends of its 32-bit counts (all before any CUDA call)."""
from __future__ import annotations

import pytest

from jagged_attention_recommender_gb300 import build as gbuild
from jagged_attention_recommender_gb300 import gdpa
from tests.test_cache_cpu import UNS, Desc, append, fwd


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()
    yield


@pytest.mark.parametrize("kw", [dict(T=2 ** 31 - 1), dict(T=2 ** 31 - 256), dict(B=2 ** 31 - 1), dict(B=2 ** 31 - 4097)])
def test_counts_near_the_end_of_32_bits_are_refused(kw):
    # (the lookups step up to 32 rows, the schedule up to a block's share of sequences, past the last one)
    kw = dict(kw, Hq=2, q_stride=256)
    for call in (append, fwd):
        with pytest.raises(gdpa.GdpaError) as e:
            call(Desc(), **dict(kw, offsets=None))
        assert e.value.code == UNS
