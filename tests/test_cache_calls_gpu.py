"""Calls of the paged cache that programs may make and that the other GPU tests leave out: offsets, windows, pages and
values at the ends of what the documentation allows."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from jagged_attention_recommender_gb300 import build as gbuild
from jagged_attention_recommender_gb300 import gdpa
from tests import cache_ref as ref
from tests.test_cache_gpu import Dev, check_append, check_fwd, host, inv_freq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()
    yield


def test_append_with_decreasing_offsets_stays_inside():
    """Rows that the lookup gives to a sequence that does not hold them are left out and the launch is flagged."""
    H, D, P, T = 2, 64, 16, 39
    x = ref.make(60, 4, H, D, P, [T], [T], [0], spare=70)
    x.lens, x.new = [43, 853, 353, 535, 360], [0] * 5
    x.offsets = np.array([0, 24, 2, 3, 13, 39], np.int32)
    pages = x.k_codes.shape[0]
    x.table = np.arange(5 * 64, dtype=np.int32).reshape(5, 64) % (pages - 4)  # the last four pages are nobody's
    d = Dev(x, inv_freq(D))
    before = [host(t).copy() for t in (d.k_codes, d.v_codes, d.k_sf, d.v_sf)]
    d.append()
    assert gdpa.gdpa_device_status() == gdpa.GDPA_ERR_INVALID_ARG
    for t, was in zip((d.k_codes, d.v_codes, d.k_sf, d.v_sf), before):
        np.testing.assert_array_equal(host(t)[-4:], was[-4:])
    x = ref.make(61, 4, H, D, P, [40, 20], [3, 20], [37, 0])  # the next call is right
    d = Dev(x, inv_freq(D))
    d.append()
    check_append(x, d, inv_freq(D), False)


FEW_MANY = [(4, 1), (64, 2)]  # six rows of one: the kernel for few rows (24) and for many (192)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", FEW_MANY)
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 4, 2 ** 30, 7, 6])
def test_a_window_of_any_size_with_more_rows_than_tokens(D, heads, window):
    """Rows in front of the first token have negative positions: a window near 2^31 in front of them is still one."""
    x = ref.make(62, *heads, D, 16, [2, 3, 40], [5, 6, 4])
    d = Dev(x, pad=1)
    d.fwd(window=window)
    check_fwd(x, d, True, window)
