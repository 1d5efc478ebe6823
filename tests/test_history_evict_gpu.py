"""Evictions of few and many heads whose tokens lie on more CTAs, or are more, than other tests have."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from jagged_attention_recommender_gb300 import gdpa
from tests import history_ref as hist
from tests.test_history_gpu import NAMES, check_evict, cu, evict_batch, same, status

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


def wide(x, tokens):
    """The batch with a table for so many tokens a sequence, as a server allocates one."""
    more = max(0, -(-tokens // x.P) - x.table.shape[1])
    x.table = np.concatenate([x.table, np.full((len(x.lens), more), -7, np.int32)], 1)
    return x


# A CTA holds up to 40 960 tokens' keys in shared memory; what is larger, by the table's width, is read anew for every
# digit.  (On 152 SMs: 80 heads take one CTA of 1024 threads each, 320 one of 256, one or two clusters of 16.)
@pytest.mark.parametrize("H,lens,tokens,budget", [
    (1, [45003, 300, 0, 2000, 41000, 64, 17, 1] * 10, 45056, 333),
    (2, [3000, 1, 700, 129, 0, 260, 33, 34] * 5, 50000, 64),
    (2, [300, 1, 500, 129, 0, 260, 33, 34] * 20, 41000, 40),
    (1, [660001], 660001, 1500),
    (1, [700, 200000], 700000, 900),
    (1, [5], 700000, 3),
])
@pytest.mark.parametrize("kind", ["random", "ties"])
def test_evict_of_tables_wider_than_shared_memory(H, lens, tokens, budget, kind):
    x, w = evict_batch(budget, H, 64, 16 if max(lens) < 41000 else 1024, lens, budget)
    rng = np.random.default_rng(7)
    if kind == "ties":
        w = rng.choice(np.array([0.0, 0.5, 0.5000001, 2.0, np.nan], np.float32), w.shape)
    check_evict(wide(x, tokens), w, budget, 2, budget // 4)
