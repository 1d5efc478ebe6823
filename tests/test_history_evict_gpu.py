"""Evictions of few and many heads whose tokens lie on more CTAs, or are more, than other tests have."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from jagged_attention_recommender_gb300 import gdpa
from tests import history_ref as hist
from tests.test_history_gpu import NAMES, cu, evict_batch, same, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P", [64, 1024])
def test_a_history_on_a_wide_cluster_captured_as_its_first_call(P):
    """(64 and 1024: another size of shared memory each.)"""
    n, budget = 33000 if P == 64 else 90000, 700
    x, w = evict_batch(P, 1, 64, P, [n], budget)
    table = hist.spare_table(x, budget)
    codes = [cu(a) for a in (x.k_codes, x.v_codes, x.k_sf, x.v_sf)]
    cache, weights = gdpa.KvCache(*codes), cu(w)
    kept = torch.full((1, 1, budget), -1, dtype=torch.int32, device="cuda")
    new_lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens, old, new = cu(np.array([n], np.int32)), cu(x.table), cu(table)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gdpa.gdpa_cache_evict(cache, weights, lens, old, 1, old.shape[1], budget, 3, 50, new, new.shape[1], kept, new_lens)
    assert new_lens.item() == 0
    for _ in range(2):
        graph.replay()
        status()
        got = [t.cpu().numpy() for t in codes + [weights, kept, new_lens]]
        for name, a, b in zip(NAMES, got, hist.evict(x, w, budget, 3, 50, table)):
            same(a, b, name)
