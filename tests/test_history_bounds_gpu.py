"""Offsets out of range: the sequences that they spoil get nothing, the others what they should, and nothing else is
written."""
from __future__ import annotations

import numpy as np
import pytest

from jagged_attention_recommender_gb300 import gdpa
from tests import cache_ref as ref
from tests import history_ref as hist
from tests.test_history_gpu import SENTINEL, run_weights, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 30, 50, 70])  # (few rows, with one and several row tiles, and many)
@pytest.mark.parametrize("bad", range(4))
def test_weights_beside_sequences_of_bad_offsets(new, bad):
    x = ref.make(11, 4, 2, 64, 16, [300, 290, 280], [new] * 3)
    scale = float(np.float32(8.0 ** -1))
    lse = np.float64(np.float32(ref.attend(x, 1, 0, scale)[1]))
    o = x.offsets
    offsets, spoilt = [
        ([0, o[2] + 1, o[2], o[3]], 1),      # the first sequence's rows reach into the second's
        ([0, o[1], o[2], o[3] + 9], 2),
        ([-4, o[1], o[2], o[3]], 0),
        ([0, o[1], 2 ** 31 - 1, o[3]], None),  # neither the second nor the third
    ][bad]
    x.offsets = np.array(offsets, np.int32)
    x.new = [0 if b == spoilt or (spoilt is None and b > 0) else int(x.offsets[b + 1]) - int(x.offsets[b]) for b in range(3)]
    got = run_weights(x, 1, 0, 1.0, None, lse, with_in=False, max_q=new)
    status(gdpa.GDPA_ERR_INVALID_ARG)
    want, tol = hist.weights(x, lse, True, 0, scale, 1.0, None)
    at = ~np.isnan(want)
    assert (np.abs(got - want)[at] <= tol[at]).all() and (got[~at] == SENTINEL).all()


@pytest.mark.parametrize("rows", [1, 70])
def test_weights_behind_many_sequences_without_rows(rows):
    """Millions of sequences that bring nothing, in front of one that does."""
    B, D, P = 1 << 22, 128, 16
    x = ref.make(5, 1, 1, D, P, [P], [rows])
    lse = np.float64(np.float32(ref.attend(x, 0, 0, float(np.float32(D ** -0.5)))[1]))
    want, tol = hist.weights(x, lse, False, 0, float(np.float32(D ** -0.5)), 1.0, None)
    page = int(x.table[0, 0])
    x.lens, x.new = [P] * B, [0] * (B - 1) + [rows]
    x.offsets = np.zeros(B + 1, np.int32)
    x.offsets[-1] = rows
    x.table = np.full((B, 1), page, np.int32)
    got = run_weights(x, 0, 0, 1.0, None, lse, with_in=False, max_q=rows)
    status()
    at = ~np.isnan(want)
    assert (np.abs(got - want)[at] <= tol[at]).all() and (got[~at] == SENTINEL).all()
