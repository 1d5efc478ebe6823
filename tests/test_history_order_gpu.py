"""The weight that stored keys receive from many rows where a CTA has many items of keys: with long runs of them that no row
sees between those that rows see (tests/test_history_order.py has the order), and with stages that are filled time and again."""
from __future__ import annotations

import numpy as np
import pytest

from tests import cache_ref as ref
from tests.test_history_gpu import check_weights, run_weights, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,D,P,lens,rows,window", [
    (4, 128, 64, [12000] * 8, 70, 300),
    (3, 64, 16, [6000, 20000, 17000, 3000, 12000, 11111] * 2, 130, 100),
])
@pytest.mark.parametrize("in_place,with_in,decay", [(True, True, 0.5), (False, True, 1.0), (False, False, 1.0)])
def test_weights_through_windows_far_shorter_than_the_histories(H, D, P, lens, rows, window, in_place, with_in, decay):
    x = ref.make(window, H, H, D, P, lens, [rows] * len(lens))
    check_weights(x, 1, window, decay=decay, in_place=in_place, with_in=with_in)


def test_weights_of_some_sequences_through_windows():
    """Sequences all of whose keys are seen beside such whose keys mostly are not."""
    lens = [200, 15000, 300, 31, 15000, 15000, 400, 14000] * 2
    x = ref.make(3, 6, 3, 128, 32, lens, [min(n, 90) for n in lens])
    check_weights(x, 1, 128, decay=0.25)


@pytest.mark.parametrize("H,D,rows", [(2, 64, 130), (3, 128, 70)])
@pytest.mark.parametrize("with_in", [False, True])
def test_weights_of_many_tiles_on_pages_of_their_own(H, D, rows, with_in):
    """Every block of a tile lies on a page of its own, and a CTA's stages are filled anew for many tiles: each key's weight
    arrives in its own slot, time and again."""
    x = ref.make(D + rows, H, H, D, 16, [9000, 16, 30001, 20000, 129, 255], [rows, 16, 3, rows, rows, 1])
    lse = np.float64(np.float32(ref.attend(x, 1, 0, float(np.float32(D ** -0.5)))[1]))
    first = check_weights(x, 1, 0, with_in=with_in, lse=lse, max_q=rows)
    w_in = np.random.default_rng(0).exponential(0.2, x.k_codes.shape[:3])  # (those of check_weights)
    for _ in range(10):
        assert (run_weights(x, 1, 0, 1.0, w_in, lse, with_in=with_in, max_q=rows) == first).all()
    status()
