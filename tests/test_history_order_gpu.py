"""The weight that stored keys receive from many rows through windows far shorter than the histories: a CTA has many items of
keys, and long runs of them that no row sees lie between those that rows see (tests/test_history_order.py has the order)."""
from __future__ import annotations

import pytest

from tests import cache_ref as ref
from tests.test_history_gpu import check_weights

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
