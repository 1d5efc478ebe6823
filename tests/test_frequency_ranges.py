"""gdpa_rope_freqs at the ends of its ranges."""
from __future__ import annotations

import numpy as np
import pytest

from jagged_attention_recommender_gb300 import build as gbuild
from jagged_attention_recommender_gb300 import gdpa
from tests import history_ref as hist
from tests.test_cache_cpu import UNS
from tests.test_history_cpu import refused


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()


@pytest.mark.parametrize("rot,base,factor", [(16, 1e4, 1e300), (64, 1e300, 1e10), (128, 1e308, 2.0), (16, 1.7e308, 1.5)])
def test_a_stretched_base_that_64_bits_do_not_hold_is_refused(rot, base, factor):
    """(Its pairs but the first would stand still.)"""
    refused(gdpa.gdpa_rope_freqs, UNS, rot, base, gdpa.GDPA_ROPE_SCALE_BASE, factor)


@pytest.mark.parametrize("rot,base,factor", [(16, 1e4, 1e200), (64, 1e300, 100.0), (128, 1.0 + 2.0 ** -52, 1.0)])
@pytest.mark.parametrize("scaling", range(4))
def test_far_bases_and_factors(rot, base, factor, scaling):
    f, m = gdpa.gdpa_rope_freqs(rot, base, scaling, factor, 4096)
    with np.errstate(divide="ignore"):
        want, wm = hist.frequencies(rot, base, scaling, factor, 4096)
    # (base^x with ln(base) x up to 1000: its own error is 2^-53 of that)
    assert np.isfinite(f).all() and (f > 0).all() and np.allclose(f, want, rtol=1e-12, atol=0) and abs(m - wm) <= 2.0 ** -23 * wm
