"""How the operators for long histories are called: captured and replayed, on streams of their own, in place, at the ends
of their ranges."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from jagged_attention_recommender_gb300 import gdpa
from tests import cache_ref as ref
from tests import history_ref as hist
from tests.test_history_gpu import (NAMES, SENTINEL, check_evict, check_weights, cu, cu_bf16, evict_batch, rope_bound,
                                    run_weights, same, status)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,H,new", [(130, 1, [3, 1]), (300, 1, [1, 2]), (129, 1, [40, 1]), (258, 2, [1, 7])])
def test_weights_of_more_heads_than_columns(Hq, H, new):
    """A group of heads that does not fit the 128 columns of a chunk."""
    check_weights(ref.make(Hq, Hq, H, 64, 32, [150, 300], new), 1, 0)


@pytest.mark.parametrize("G", [3, 5, 7, 100])
@pytest.mark.parametrize("window", [0, 50])
def test_weights_of_chunks_that_do_not_fill_their_columns(G, window):
    check_weights(ref.make(G, 2 * G, 2, 128, 64, [400, 129, 700], [150, 60, 33]), 1, window)


@pytest.mark.parametrize("window", [1, 100, 256, 300, 5000])
@pytest.mark.parametrize("new", [1, 30, 200])
@pytest.mark.parametrize("in_place,decay", [(True, 1.0), (True, 0.5), (False, 1.0)])
def test_weights_through_windows(window, new, in_place, decay):
    """Keys in front of the window keep, or fade; in place without fading they are not touched."""
    x = ref.make(window, 4, 2, 64, 16, [1300, 40, 257], [new, min(new, 40), new])
    check_weights(x, 1, window, decay=decay, in_place=in_place)


@pytest.mark.parametrize("new,hint", [(3, 1), (40, 1), (200, 3), (200, 40), (1, 500), (60, 30)])
def test_weights_whatever_the_hint(new, hint):
    """max_q picks the kernel; sequences with more or fewer rows are computed all the same."""
    x = ref.make(new, 8, 2, 128, 32, [333, 500, 64], [new, 1, 2])
    check_weights(x, 1, 0, max_q=hint)


def test_weights_far_in_a_large_cache():
    """Pages whose codes lie more than 2^32 bytes from the first."""
    D, P, pages = 128, 1024, 36000
    codes = torch.empty((pages, 1, P, D), dtype=torch.uint8, device="cuda")
    sf = torch.full((pages, 1, P // 16), 120, dtype=torch.uint8, device="cuda")
    w = torch.zeros((pages, 1, P), dtype=torch.float32, device="cuda")
    x = ref.make(1, 4, 1, D, P, [1500], [1], jitter=0)
    for rows in (1, 70):
        y = ref.make(1, 4, 1, D, P, [1500], [rows], jitter=0)
        far = np.array([[pages - 1, pages - 3]], np.int32)
        for i in range(2):
            codes[int(far[0, i])].copy_(cu(y.k_codes[y.table[0, i]]))
        sf[far[0].tolist()] = 120
        y.k_sf[:] = 120
        cache = gdpa.KvCache(codes, codes, sf, sf)
        scale = float(np.float32(D ** -0.5))
        lse = np.float64(np.float32(ref.attend(y, True, 0, scale)[1]))
        gdpa.gdpa_cache_weights(cache, cu_bf16(y.q), 4 * D, cu(lse.astype(np.float32)), cu(y.offsets), cu(np.array([1500], np.int32)),
                                cu(far), rows, 1, 4, 2, rows, True, 0, scale, 1.0, None, w)
        status()
        want, tol = hist.weights(y, lse, True, 0, scale, 1.0, None)
        t = np.arange(1500)
        got = w.cpu().numpy()[far[0, t // P], 0, t % P]
        at = y.table[0, t // P], 0, t % P
        assert (np.abs(got - want[at]) <= tol[at]).all()
    # ... and an eviction from and to such pages
    kept = torch.full((1, 1, 300), -1, dtype=torch.int32, device="cuda")
    lens = torch.empty(1, dtype=torch.int32, device="cuda")
    v = codes.clone()
    cache = gdpa.KvCache(codes, v, sf, sf.clone())
    gdpa.gdpa_cache_evict(cache, w, cu(np.array([1500], np.int32)), cu(far), 1, 2, 300, 2, 9, cu(np.array([[pages - 2]], np.int32)), 1,
                          kept, lens)
    status()
    at = kept.cpu().numpy()[0, 0]
    old = np.where((np.arange(1500) < 2) | (np.arange(1500) >= 1491), np.inf, got)
    assert np.array_equal(at, np.sort(np.argsort(-old, kind="stable")[:300])) and lens.item() == 300
    src = codes[far[0].tolist()].reshape(-1, D)[torch.from_numpy(at).cuda().long()]
    assert torch.equal(codes[pages - 2, 0, :300], src)


def test_streams_and_graphs():
    """Each operator on a stream of its own, captured as its first call there would be, and replayed as lengths, tables and
    positions change."""
    side = torch.cuda.Stream()
    x, w0 = evict_batch(21, 2, 64, 16, [300, 200], 64)
    q = ref.make(22, 8, 2, 64, 16, [300, 200], [2, 1])
    f, m = hist.frequencies(64)
    rows = ref.bf16(np.random.default_rng(0).standard_normal((9, 3, 64)))
    offsets, first = np.array([0, 4, 9], np.int32), np.array([7, 100], np.int32)
    d_off, d_first = cu(offsets), cu(first)
    dx, dy = cu_bf16(rows), torch.zeros((9, 3, 64), dtype=torch.bfloat16, device="cuda")
    codes = [cu(a) for a in (x.k_codes, x.v_codes, x.k_sf, x.v_sf)]
    cache = gdpa.KvCache(*codes)
    table, lens = cu(x.table), cu(np.array(x.lens, np.int32))
    scale = float(np.float32(8.0 ** -1))
    x.q, x.offsets, x.new, x.Hq = q.q, q.offsets, q.new, 8
    lse = np.float64(np.float32(ref.attend(x, True, 0, scale)[1]))
    d_q, d_lse, d_qoff = cu_bf16(x.q), cu(lse.astype(np.float32)), cu(x.offsets)
    before, w = cu(w0), torch.full(w0.shape, SENTINEL, dtype=torch.float32, device="cuda")
    new_table = hist.spare_table(x, 64)
    d_new = cu(new_table)
    kept = torch.full((2, 2, 64), -1, dtype=torch.int32, device="cuda")
    new_lens = torch.zeros(2, dtype=torch.int32, device="cuda")

    def step():
        gdpa.gdpa_rope(dx, 192, d_off, d_first, 9, 2, 3, 64, f, 0, 1.0, 0, dy, 192)
        gdpa.gdpa_cache_weights(cache, d_q, 8 * 64, d_lse, d_qoff, lens, table, 3, 2, 8, x.table.shape[1], 2, True, 0, scale, 1.0, before, w)
        gdpa.gdpa_cache_evict(cache, w, lens, table, 2, x.table.shape[1], 64, 1, 8, d_new, d_new.shape[1], kept, new_lens)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    for turn in range(3):
        if turn == 2:  # shorter sequences, other positions
            x.lens = [250, 180]
            lens.copy_(cu(np.array(x.lens, np.int32)))
            first = np.array([1000, 3], np.int32)
            d_first.copy_(cu(first))
            lse = np.float64(np.float32(ref.attend(x, True, 0, scale)[1]))
            d_lse.copy_(cu(lse.astype(np.float32)))
        for t, a in zip(codes, (x.k_codes, x.v_codes, x.k_sf, x.v_sf)):
            t.copy_(cu(a))
        w.fill_(SENTINEL)
        dy.zero_()
        kept.fill_(-1)
        torch.cuda.synchronize()
        if turn == 0:
            with torch.cuda.stream(side):
                step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        status()
        want = hist.rope(rows, offsets, first, f, False)
        assert (np.abs(dy.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + rope_bound(rows, 64, f, 0, 1.0, 0) * 1.01).all()
        want, tol = hist.weights(x, lse, True, 0, scale, 1.0, np.float64(w0))
        got = w.cpu().numpy()
        old = {int(x.table[b, i]) for b in range(2) for i in range(-(-x.lens[b] // 16))}
        at = ~np.isnan(want)
        assert (np.abs(got - want)[at] <= tol[at]).all() and old == {int(p) for p in np.nonzero(at)[0]}
        mine = np.where(at, got, np.float32(SENTINEL)).astype(np.float32)
        for name, a, b in zip(NAMES, [t.cpu().numpy() for t in codes] + [got, kept.cpu().numpy(), new_lens.cpu().numpy()],
                              hist.evict(x, mine, 64, 1, 8, new_table)):
            same(a, b, name)


def test_two_calls_at_once():
    """Calls on two streams, over different pages of one cache, do not disturb each other."""
    x = ref.make(31, 8, 2, 128, 32, [900, 700, 800, 600], [40, 1, 40, 1])
    scale = float(np.float32(128 ** -0.5))
    lse = np.float64(np.float32(ref.attend(x, True, 0, scale)[1]))
    want, tol = hist.weights(x, lse, True, 0, scale, 1.0, None)
    cache = gdpa.KvCache(*(cu(a) for a in (x.k_codes, x.v_codes, x.k_sf, x.v_sf)))
    w = torch.full(x.k_codes.shape[:3], SENTINEL, dtype=torch.float32, device="cuda")
    q, d_lse = cu_bf16(x.q), cu(lse.astype(np.float32))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    parts = []
    for i in range(2):
        r0 = int(x.offsets[2 * i])
        parts.append((q[r0:r0 + 41], d_lse[r0:r0 + 41], cu(np.array([0, 40, 41], np.int32)), cu(np.array(x.lens[2 * i:2 * i + 2], np.int32)),
                      cu(x.table[2 * i:2 * i + 2])))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (qq, ll, off, lens, table) in zip(streams, parts):
            for hint in (40, 4):
                gdpa.gdpa_cache_weights(cache, qq, 8 * 128, ll, off, lens, table, 41, 2, 8, x.table.shape[1], hint, True, 0, scale, 1.0,
                                        None, w, stream=s)
    torch.cuda.synchronize()
    status()
    got = w.cpu().numpy()
    at = ~np.isnan(want)
    assert (np.abs(got - want)[at] <= tol[at]).all() and (got[~at] == SENTINEL).all()


def test_evict_of_many_sequences_and_heads():
    lens = [int(n) for n in np.random.default_rng(3).integers(0, 200, 90)]
    x, w = evict_batch(41, 4, 64, 16, lens, 50)
    check_evict(x, w, 50, 1, 6)


def test_rope_of_wide_rows():
    """More heads than a block takes, and rows more than 2^31 bytes from the first."""
    T, H, D = 6, 600, 128
    stride = 1 << 28
    x = torch.empty((T - 1) * stride + H * D, dtype=torch.bfloat16, device="cuda")
    rows = ref.bf16(np.random.default_rng(1).standard_normal((T, H, D)))
    view = x.as_strided((T, H, D), (stride, D, 1))
    view.copy_(cu_bf16(rows))
    y = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
    f, _ = hist.frequencies(128)
    gdpa.gdpa_rope(view, stride, cu(np.array([0, 2, 6], np.int32)), None, T, 2, H, D, f, 1, 1.0, 0, y, H * D)
    gdpa.gdpa_rope(view, stride, cu(np.array([0, 2, 6], np.int32)), None, T, 2, H, D, f, 1, 1.0, 0, view, stride)  # in place
    status()
    want = hist.rope(rows, [0, 2, 6], None, f, True)
    for got in (y, view):
        assert (np.abs(got.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + rope_bound(rows, 128, f, 0, 1.0, 1) * 1.01).all()


@pytest.mark.parametrize("rows", [1, 70])
@pytest.mark.parametrize("window", [0, 100])
def test_weights_at_the_largest_length(rows, window):
    """2^31 - 16 keys: all but the last page are one page again and again, whose weights are undefined; the last page's
    are right."""
    D, P = 128, 16
    n = 2 ** 31 - 16
    x = ref.make(5, 1, 1, D, P, [P], [rows], jitter=0)
    x.k_sf[:] = 120
    width = -(-n // P)
    table = torch.full((1, width), 1, dtype=torch.int32, device="cuda")
    table[0, -1] = 0
    codes = torch.zeros((2, 1, P, D), dtype=torch.uint8, device="cuda")
    codes[0] = cu(x.k_codes[x.table[0, 0]])
    sf = torch.full((2, 1, P // 16), 120, dtype=torch.uint8, device="cuda")
    held = n - (width - 1) * P  # tokens of the last page
    q = ref.bf16(np.random.default_rng(1).standard_normal((rows, 1, D)))
    lse = np.float32(np.random.default_rng(2).uniform(0, 2, (rows, 1)))
    w_in = torch.full((2, 1, P), 0.5, dtype=torch.float32, device="cuda")
    w = torch.full((2, 1, P), SENTINEL, dtype=torch.float32, device="cuda")
    scale = float(np.float32(D ** -0.5))
    gdpa.gdpa_cache_weights(gdpa.KvCache(codes, codes, sf, sf), cu_bf16(q), D, cu(lse), cu(np.array([0, rows], np.int32)),
                            cu(np.array([n], np.int32)), table, rows, 1, 1, width, rows, True, window, scale, 1.0, w_in, w)
    status()
    k = ref.e4m3_values(x.k_codes[x.table[0, 0], 0, :held]) * 2.0 ** -7
    pos, j = n - rows + np.arange(rows)[:, None], (width - 1) * P + np.arange(held)
    s = scale * q[:, 0] @ k.T
    p = np.where((j <= pos) & ((j > pos - window) if window else True), np.exp(s - np.float64(lse)), 0)
    want = p.sum(0) + np.where(j < n - rows, 0.5, 0)
    got = w[0, 0].double().cpu().numpy()
    # (a score is off by (D + 8) 2^-23 of sum |q k| / sqrt(D), at most 16 here, its exponential by as much: 2^-12)
    assert (np.abs(got[:held] - want) <= 2.0 ** -12 * want + 1e-30).all() and (got[held:] == SENTINEL).all()


def test_evict_at_the_largest_length():
    """2^31 - 16 tokens, on one page again and again but for the last: what stays is found there and among the first."""
    P, n = 16, 2 ** 31 - 16
    width = -(-n // P)
    table = torch.full((1, width), 1, dtype=torch.int32, device="cuda")
    table[0, -1] = 0
    codes = torch.from_numpy(np.random.default_rng(0).integers(0, 0x7E, (46, 1, P, 64)).astype(np.uint8)).cuda()
    sf = torch.full((46, 1, P // 16), 120, dtype=torch.uint8, device="cuda")
    w = torch.zeros((46, 1, P), dtype=torch.float32, device="cuda")
    held = n - (width - 1) * P
    w[0, 0, :held] = cu(np.float32(np.random.default_rng(1).uniform(-1, 1, held)))
    kept = torch.full((1, 1, 700), -1, dtype=torch.int32, device="cuda")
    lens = torch.empty(1, dtype=torch.int32, device="cuda")
    gdpa.gdpa_cache_evict(gdpa.KvCache(codes, codes.clone(), sf, sf.clone()), w, cu(np.array([n], np.int32)), table, 1, width, 700,
                          0, 5, cu(np.arange(2, 46, dtype=np.int32)[None]), 44, kept, lens)
    status()
    last = w[0, 0, :held].cpu().numpy()
    stays = np.flatnonzero((last > 0) | (np.arange(held) >= held - 5))
    want = np.concatenate([np.arange(700 - len(stays)), (width - 1) * P + stays])
    assert lens.item() == 700 and np.array_equal(kept.cpu().numpy()[0, 0], want)
    first = torch.arange(700 - len(stays), device="cuda") % P
    src = torch.cat([codes[1, 0, first], codes[0, 0, torch.from_numpy(stays).cuda()]])
    assert torch.equal(codes[2:, 0].reshape(-1, 64)[:700], src)


def test_evict_of_many_heads_at_the_largest_length():
    """As many heads as take one CTA each: what stays is the last page's alone."""
    P, H, n = 16, 80, 2 ** 31 - 16
    width = n // P
    table = torch.full((1, width), 1, dtype=torch.int32, device="cuda")
    table[0, -1] = 0
    codes = torch.from_numpy(np.random.default_rng(0).integers(0, 0x7E, (3, H, P, 64)).astype(np.uint8)).cuda()
    sf = torch.full((3, H, P // 16), 120, dtype=torch.uint8, device="cuda")
    w = torch.full((3, H, P), -1.0, dtype=torch.float32, device="cuda")
    w[0] = 1.0
    kept = torch.full((1, H, P), -1, dtype=torch.int32, device="cuda")
    lens = torch.empty(1, dtype=torch.int32, device="cuda")
    gdpa.gdpa_cache_evict(gdpa.KvCache(codes, codes.clone(), sf, sf.clone()), w, cu(np.array([n], np.int32)), table, 1, width, P, 0, 0,
                          cu(np.array([[2]], np.int32)), 1, kept, lens)
    status()
    assert lens.item() == P and (kept.cpu().numpy()[0] == n - P + np.arange(P)).all()
    assert torch.equal(codes[2], codes[0]) and torch.equal(w[2], w[0])
