"""The operators for long histories against their 64-bit forms: rotary positions, the weight that stored keys receive,
eviction."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from jagged_attention_recommender_gb300 import gdpa
from tests import cache_ref as ref
from tests import history_ref as hist

pytestmark = pytest.mark.gpu


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def cu_bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


def status(want=gdpa.GDPA_OK):
    assert gdpa.gdpa_device_status() == want


# ---------------------------------------------------------------- rotary positions

def rope_bound(x, r, inv_freq, pos_max, magnitude, interleaved):
    """Half a step of bf16, and of the pair's length: the angle's 2^-26 turns (and 2^-32 of the fraction), sine and cosine
    to 2^-22, their product with the magnitude, and the four roundings of the pair, 2^-24 each: 2^-20 has room."""
    pair = np.zeros(x.shape)
    if r:
        a, b = (np.s_[..., 0:r:2], np.s_[..., 1:r:2]) if interleaved else (np.s_[..., :r // 2], np.s_[..., r // 2:r])
        pair[a] = pair[b] = np.hypot(x[a], x[b])
    return 2.0 ** -20 * abs(magnitude) * pair


def run_rope(x, offsets, first, D, inv_freq, style, magnitude, inverse, fused=0, y_fused=0, in_place=False, stream=None):
    T, H = x.shape[:2]
    wide = torch.full((T, H + fused, D), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :H] = cu_bf16(x)
    y = wide if in_place else torch.full((T, H + y_fused, D), -3.0, dtype=torch.bfloat16, device="cuda")
    gdpa.gdpa_rope(wide[:, :H], wide.stride(0), cu(offsets), None if first is None else cu(first), T, len(offsets) - 1, H, D,
                   inv_freq, style, magnitude, inverse, y[:, :H], y.stride(0), stream=stream)
    return y.double().cpu().numpy(), H


@pytest.mark.parametrize("D,rot,H", [(64, 64, 1), (64, 16, 5), (128, 128, 8), (128, 64, 3), (128, 16, 41), (64, 0, 2), (128, 112, 4)])
@pytest.mark.parametrize("style", [gdpa.GDPA_ROPE_HALF, gdpa.GDPA_ROPE_INTERLEAVED])
@pytest.mark.parametrize("inverse", [0, 1])
def test_rope_matches_the_formula(D, rot, H, style, inverse):
    rng = np.random.default_rng(D + rot + H + style)
    rows = [0, 1, 17, 0, 0, 64, 3, 33, 1, 0]
    offsets = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    T = int(offsets[-1]) + 5  # rows of padding
    x = ref.bf16(rng.standard_normal((T, H, D)))
    first = np.array([5, 2 ** 31 - 2, 0, 1, 2, 130000, 7, 1 << 20, -9, 3], np.int32)
    f, m = hist.frequencies(rot, scaling=3, factor=8.0, trained=4096) if rot else (None, 1.25)
    for fused, y_fused, in_place in ((0, 0, False), (3, 0, False), (0, 2, False), (1, 1, True)):
        got, _ = run_rope(x, offsets, first, D, f, style, m, inverse, fused, y_fused, in_place)
        status()
        want = hist.rope(x, offsets, first, f, style == gdpa.GDPA_ROPE_INTERLEAVED, float(np.float32(m)), bool(inverse))
        n = int(offsets[-1])
        tol = 2.0 ** -8 * np.abs(want[:n]) + rope_bound(x[:n], rot, f, 0, m, style) * (1 + 2.0 ** -8) + 1e-38
        assert (np.abs(got[:n, :H] - want[:n]) <= tol).all()
        assert (got[:n, :H, rot:] == x[:n, :, rot:]).all()
        kept = x[n:] if in_place else np.full_like(x[n:], -3.0)
        assert (got[n:, :H] == kept).all()
        assert (got[:, H:] == (7.0 if in_place else -3.0)).all()


@pytest.mark.parametrize("T,B", [(1, 1), (2, 70), (4100, 3), (333, 333)])
def test_rope_row_and_sequence_counts(T, B):
    rng = np.random.default_rng(T + B)
    cuts = np.sort(rng.integers(0, T + 1, B - 1)) if T != B else np.arange(1, B)
    offsets = np.concatenate([[0], cuts, [T]]).astype(np.int32)
    x = ref.bf16(rng.standard_normal((T, 2, 64)))
    f, _ = hist.frequencies(64)
    got, _ = run_rope(x, offsets, None, 64, f, 0, 1.0, 0)
    status()
    want = hist.rope(x, offsets, None, f, False)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + rope_bound(x, 64, f, 0, 1.0, 0) * 1.01).all()


def test_rope_gradient_is_the_transpose_and_the_differences():
    """<dy, rope(x)> = <inverse(dy), x>, and the gradient of sum(dy rope(x)) by differences along coordinates."""
    rng = np.random.default_rng(4)
    offsets = np.array([0, 40, 41, 100], np.int32)
    f, m = hist.frequencies(64, scaling=3, factor=4.0, trained=2048)
    x, dy = ref.bf16(rng.standard_normal((100, 3, 128))), ref.bf16(rng.standard_normal((100, 3, 128)))
    first = np.array([9, 0, 4000], np.int32)
    y, _ = run_rope(x, offsets, first, 128, f, 0, m, 0)
    dx, _ = run_rope(dy, offsets, first, 128, f, 0, m, 1)
    status()
    # each side is a sum of rounded products: 2^-8 of the sum of their magnitudes at most
    assert abs((dy * y).sum() - (dx * x).sum()) <= 2.0 ** -8 * ((np.abs(dy * y)).sum() + np.abs(dx * x).sum())
    h = 0.5
    for t, head, d in [(0, 0, 0), (39, 1, 33), (40, 2, 63), (77, 0, 31), (99, 2, 127)]:
        up, down = x.copy(), x.copy()
        up[t, head, d] += h
        down[t, head, d] -= h
        g = lambda z: (dy * hist.rope(z, offsets, first, f, False, float(np.float32(m)))).sum()
        want = (g(up) - g(down)) / (2 * h)
        pair = np.abs(dy[t, head]).max() * 2 * m  # (linear: the difference is exact but for 64-bit rounding)
        assert abs(dx[t, head, d] - want) <= 2.0 ** -8 * abs(want) + 2.0 ** -19 * pair


def test_rope_offsets_out_of_range_are_flagged_and_skipped():
    x = ref.bf16(np.random.default_rng(0).standard_normal((20, 1, 64)))
    f, _ = hist.frequencies(64)
    for offsets, skipped in (([0, 8, 21], np.s_[8:20]), ([-1, 8, 20], np.s_[0:8])):
        got, _ = run_rope(x, np.array(offsets, np.int32), None, 64, f, 0, 1.0, 0)
        status(gdpa.GDPA_ERR_INVALID_ARG)
        assert (got[skipped] == -3.0).all() and (got != -3.0).any()
    got, _ = run_rope(x, np.array([0, 20], np.int32), None, 64, f, 0, 1.0, 0)
    status()


# ---------------------------------------------------------------- weights of stored keys

SENTINEL = -12345.0


def run_weights(x, causal, window, decay, w_in, lse, q=None, in_place=False, max_q=None, stride=0, with_in=True):
    cache = gdpa.KvCache(*(cu(a) for a in (x.k_codes, x.v_codes, x.k_sf, x.v_sf)))
    q = cu_bf16(x.q if q is None else q)
    if stride:
        wide = torch.full((q.shape[0], x.Hq + stride, x.D), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :x.Hq] = q
        q = wide[:, :x.Hq]
    w = torch.full(x.k_codes.shape[:3], SENTINEL, dtype=torch.float32, device="cuda")
    before = cu(w_in.astype(np.float32)) if with_in else None
    if in_place:
        w = before
    gdpa.gdpa_cache_weights(cache, q, q.stride(0), cu(lse.astype(np.float32)), cu(x.offsets), cu(np.array(x.lens, np.int32)),
                            cu(x.table), q.shape[0], len(x.lens), x.Hq, x.table.shape[1], max_q or max(max(x.new), 1), causal,
                            window, x.D ** -0.5, decay, before, w)
    return w.double().cpu().numpy()


def check_weights(x, causal, window, decay=1.0, seed=0, in_place=False, with_in=True, lse=None, **kw):
    rng = np.random.default_rng(seed)
    scale = float(np.float32(x.D ** -0.5))
    w_in = np.float64(np.float32(rng.exponential(0.2, x.k_codes.shape[:3])))
    if lse is None:
        lse = np.float64(np.float32(ref.attend(x, causal, window, scale)[1]))
    got = run_weights(x, causal, window, decay, w_in, lse, in_place=in_place, with_in=with_in, **kw)
    status()
    want, tol = hist.weights(x, lse, causal, window, scale, decay, w_in if with_in else None)
    at = ~np.isnan(want)
    assert np.isfinite(got[at]).all()
    err = np.abs(got - want)[at]
    assert (err <= tol[at]).all(), "off by %.3e, %.3g times the bound" % (err.max(), (err / tol[at]).max())
    untouched = w_in if in_place else np.full_like(got, SENTINEL)
    assert (got[~at] == untouched[~at]).all()
    return got


CASES = [
    # Hq, H, D, P, lens, new
    (1, 1, 64, 16, [1], [1]),
    (8, 2, 64, 16, [201], [1]),
    (8, 8, 128, 32, [0, 1, 15, 16, 17, 300], [1, 1, 1, 1, 1, 1]),
    (16, 2, 128, 64, [63, 64, 65, 129, 700], [1, 2, 0, 3, 1]),
    (7, 1, 128, 16, [33, 500], [5, 1]),
    (14, 2, 64, 128, [5, 260, 90], [9, 3, 2]),         # more rows than tokens
    (12, 4, 128, 32, [150, 40, 600], [20, 40, 7]),
    (8, 8, 64, 64, [100, 333], [32, 32]),
    (32, 4, 128, 64, [300, 70], [40, 70]),
    (8, 1, 128, 1024, [1100, 2060], [130, 33]),
    (4, 4, 64, 16, [777, 90, 401], [200, 90, 129]),
    (64, 1, 64, 32, [130, 520], [70, 1]),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("causal,window", [(1, 0), (0, 0), (1, 1), (1, 37)])
def test_weights_match_the_formula(case, causal, window):
    Hq, H, D, P, lens, new = CASES[case]
    x = ref.make(case, Hq, H, D, P, lens, new)
    check_weights(x, causal, window, decay=[1.0, 0.75][case % 2], in_place=bool(case % 3 == 0), stride=case % 4)


@pytest.mark.parametrize("D,P", [(64, 16), (128, 32)])
@pytest.mark.parametrize("hint", [1, 20, 40, 200])
def test_weights_of_many_sequences(D, P, hint):
    """More sequences than a warp has lanes, most of them shorter than a tile, whichever kernel the hint picks."""
    rng = np.random.default_rng(D)
    B = 150
    lens = [int(n) for n in rng.choice([0, 1, 20, 127, 128, 129, 200, 300, 700], B)]
    x = ref.make(14, 4, 4, D, P, lens, [int(n) for n in rng.choice([0, 1, 1, 2], B)])
    check_weights(x, 1, 0, max_q=hint)


@pytest.mark.parametrize("new", [[1, 1], [9, 1], [64, 80]])
def test_weights_without_earlier_ones(new):
    x = ref.make(5, 8, 2, 64, 32, [90, 400], new)
    check_weights(x, 1, 0, with_in=False)


@pytest.mark.parametrize("new", [1, 6, 100])
def test_weights_of_a_call_sum_to_the_rows(new):
    """Every row that sees a key gives 1 in all: with weights_in NULL the sum over a head's keys is its rows' number."""
    x = ref.make(6, 6, 2, 128, 32, [411, 128], [new, new])
    got = check_weights(x, 1, 0, with_in=False)
    for b in range(2):
        t = np.arange(x.lens[b])
        s = got[x.table[b, t // 32], :, t % 32].sum(0)
        # (a score is off by (D + 8) 2^-23 of sum |q k| / sqrt(D), at most 16 here: 2^-12)
        assert np.abs(s - 3 * new).max() <= 3 * new * 2.0 ** -12


@pytest.mark.parametrize("new", [1, 3, 60, 200])
def test_weights_of_empty_rows_and_infinite_statistics(new):
    """A row of logsumexp -inf gives nothing, one of +inf 0; NaN reaches exactly the keys that the row sees."""
    x = ref.make(7, 4, 2, 64, 16, [120, 75], [new, new])
    scale = float(np.float32(8.0 ** -1))
    lse = np.float64(np.float32(ref.attend(x, 1, 0, scale)[1]))
    lse[0, 0], lse[x.offsets[1], 1] = -np.inf, np.inf
    check_weights(x, 1, 0, lse=lse)
    lse[x.offsets[1] + new - 1, 2] = np.nan
    w = run_weights(x, 1, 0, 1.0, np.zeros(x.k_codes.shape[:3]), lse)
    status()
    t = np.arange(75)
    assert np.isnan(w[x.table[1, t // 16], 1, t % 16]).all() and np.isfinite(w[x.table[1, t // 16], 0, t % 16]).all()
    t = np.arange(120)
    assert np.isfinite(w[x.table[0, t // 16], :, t % 16]).all()


@pytest.mark.parametrize("new", [1, 5, 90])
def test_weights_of_nan_keys_stay_theirs(new):
    x = ref.make(8, 4, 2, 128, 32, [200, 130], [new, new])
    scale = float(np.float32(128 ** -0.5))
    lse = np.float64(np.float32(ref.attend(x, 1, 0, scale)[1]))
    want, tol = hist.weights(x, lse, True, 0, scale, 1.0, None)
    bad = (x.table[0, 30 // 32], 1, 30 % 32)
    x.k_codes[bad][5] = 0xFF
    got = run_weights(x, 1, 0, 1.0, None, lse, with_in=False)
    status()
    assert np.isnan(got[bad])
    got[bad] = want[bad]
    at = ~np.isnan(want)
    assert (np.abs(got - want)[at] <= tol[at]).all()


@pytest.mark.parametrize("new", [1, 50])
def test_weights_far_scales(new):
    """Blocks of K whose scales are far apart, and queries whose elements are."""
    x = ref.make(9, 4, 2, 128, 32, [180, 333], [new, new], jitter=9)
    x.q = ref.bf16(x.q * np.exp2(np.random.default_rng(2).integers(-12, 2, x.q.shape)))
    check_weights(x, 1, 0)


def test_weights_bits_do_not_depend_on_the_run():
    x = ref.make(10, 8, 2, 64, 64, [900, 64, 321], [30, 2, 100])
    scale = float(np.float32(8.0 ** -1))
    lse = np.float64(np.float32(ref.attend(x, 1, 0, scale)[1]))
    w_in = np.random.default_rng(1).random(x.k_codes.shape[:3])
    first = run_weights(x, 1, 0, 1.0, w_in, lse)
    for _ in range(3):
        assert (run_weights(x, 1, 0, 1.0, w_in, lse) == first).all()


def test_weights_bad_pages_offsets_and_lengths():
    """What is out of range is flagged; the other sequences' weights are right and nothing else is written."""
    for new in ([1, 1, 1], [40, 40, 40]):
        x = ref.make(11, 4, 2, 64, 16, [100, 90, 80], new)
        scale = float(np.float32(8.0 ** -1))
        lse = np.float64(np.float32(ref.attend(x, 1, 0, scale)[1]))
        want, tol = hist.weights(x, lse, True, 0, scale, 1.0, None)
        good = x.table.copy()
        for entry in (-1, x.k_codes.shape[0], 2 ** 31 - 1, -2 ** 31):
            x.table = good.copy()
            x.table[1, 2] = entry
            got = run_weights(x, 1, 0, 1.0, None, lse, with_in=False)
            status(gdpa.GDPA_ERR_INVALID_ARG)
            there = ~np.isnan(want)
            there[good[1, 2]] = False
            assert (np.abs(got - want)[there] <= tol[there]).all()
            assert (got[~there] == SENTINEL).all()
        x.table = good
        lens = list(x.lens)
        for bad in (-1, 16 * x.table.shape[1] + 1, 2 ** 31 - 1):
            x.lens = [100, bad, 80]
            got = run_weights(x, 1, 0, 1.0, None, lse, with_in=False)
            status(gdpa.GDPA_ERR_INVALID_ARG)
            t = np.arange(90)
            there = ~np.isnan(want)
            there[good[1, t // 16], :, t % 16] = False
            assert (np.abs(got - want)[there] <= tol[there]).all() and (got[~there] == SENTINEL).all()
        x.lens = lens
        offsets = x.offsets.copy()
        for bad in ([0, offsets[2] + 1, offsets[2], offsets[3]], [0, offsets[1], offsets[2], offsets[3] + 9], [-4, offsets[1], offsets[2], offsets[3]]):
            x.offsets = np.array(bad, np.int32)
            x.offsets, keep = np.array(bad, np.int32), offsets
            got = run_weights(x, 1, 0, 1.0, None, lse, with_in=False, max_q=max(new))
            status(gdpa.GDPA_ERR_INVALID_ARG)
            x.offsets = keep


# ---------------------------------------------------------------- eviction

def run_evict(x, w, budget, sink, recent, table):
    codes = [cu(a) for a in (x.k_codes, x.v_codes, x.k_sf, x.v_sf)]
    cache = gdpa.KvCache(*codes)
    weights = cu(w)
    B = len(x.lens)
    kept = torch.full((B, x.H, budget), -1, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    gdpa.gdpa_cache_evict(cache, weights, cu(np.array(x.lens, np.int32)), cu(x.table), B, x.table.shape[1], budget, sink, recent,
                          cu(table), table.shape[1], kept, lens)
    k, v, k_sf, v_sf = (c.cpu().numpy() for c in codes)
    return k, v, k_sf, v_sf, weights.cpu().numpy(), kept.cpu().numpy(), lens.cpu().numpy()


NAMES = ("k", "v", "k_sf", "v_sf", "weights", "kept", "lens")


def same(got, want, name):
    if got.dtype == np.float32:
        got, want = got.view(np.uint32), want.view(np.uint32)
    if name in "kv":  # every NaN is one
        nan = (want & 0x7F) == 0x7F
        assert (((got & 0x7F) == 0x7F) == nan).all()
        got, want = np.where(nan, 0, got), np.where(nan, 0, want)
        # (a rounded value of zero may have either sign)
        got, want = np.where(got == 0x80, 0, got), np.where(want == 0x80, 0, want)
    assert np.array_equal(got, want), name


def check_evict(x, w, budget, sink, recent):
    table = hist.spare_table(x, budget)
    got = run_evict(x, w, budget, sink, recent, table)
    status()
    for name, a, b in zip(NAMES, got, hist.evict(x, w, budget, sink, recent, table)):
        same(a, b, name)
    return got


def evict_batch(seed, H, D, P, lens, budget, jitter=3):
    x = ref.make(seed, H, H, D, P, lens, [0] * len(lens), spare=hist.pages_for(lens, P, budget) + 2, jitter=jitter)
    rng = np.random.default_rng(seed + 50)
    w = rng.lognormal(0, 2, x.k_codes.shape[:3]).astype(np.float32)
    w[rng.random(w.shape) < 0.1] = 0
    return x, w


@pytest.mark.parametrize("H,D,P,lens,budget,sink,recent", [
    (1, 64, 16, [1], 1, 0, 0),
    (1, 64, 16, [2], 1, 0, 0),
    (2, 64, 16, [150], 100, 4, 16),
    (3, 128, 32, [0, 1, 15, 16, 17, 64, 200], 16, 1, 2),
    (8, 128, 64, [500, 64, 65, 1000], 65, 0, 65),          # nothing but the last ones
    (2, 128, 16, [400, 33], 40, 40, 0),                    # nothing but the first ones
    (2, 64, 128, [700, 300, 20], 257, 3, 30),
    (1, 128, 1024, [3000, 1025], 1500, 5, 7),
    (2, 64, 32, [5000], 17, 0, 1),
    (5, 64, 32, [90, 91, 92], 1000, 10, 10),               # all stay
    (2, 64, 64, [20001, 300], 1200, 2, 40),                # several CTAs a head
    (1, 64, 1024, [400003], 333, 5, 1),                    # more keys than their shared memory holds
])
def test_evict_matches_the_definition(H, D, P, lens, budget, sink, recent):
    x, w = evict_batch(budget, H, D, P, lens, budget)
    check_evict(x, w, budget, sink, recent)


@pytest.mark.parametrize("kind", ["equal", "zeros", "signs", "infinite", "nan", "some_nan", "near", "tiny"])
@pytest.mark.parametrize("budget", [1, 31, 200])
def test_evict_of_odd_weights(kind, budget):
    """Ties go to the lower place; zeros of both signs are equal; NaN is less than any number."""
    lens = [300, 210, 31]
    x, w = evict_batch(3, 2, 64, 32, lens, budget)
    rng = np.random.default_rng(1)
    if kind == "equal":
        w[:] = 0.25
    elif kind == "zeros":
        w[:] = np.where(rng.random(w.shape) < 0.5, 0.0, -0.0)
    elif kind == "signs":
        w = rng.standard_normal(w.shape).astype(np.float32)
    elif kind == "infinite":
        w = rng.choice([np.inf, -np.inf, 1.0, np.finfo(np.float32).max, np.finfo(np.float32).min], w.shape).astype(np.float32)
    elif kind == "nan":
        w[:] = np.nan
    elif kind == "some_nan":
        w = np.where(rng.random(w.shape) < 0.9, np.nan, np.where(rng.random(w.shape) < 0.5, -np.inf, 1.0)).astype(np.float32)
    elif kind == "near":  # differ in the last bits alone
        w = (np.float32(1.0).view(np.uint32) + rng.integers(0, 5, w.shape).astype(np.uint32)).view(np.float32)
    else:
        w = rng.integers(0, 4, w.shape).astype(np.uint32).view(np.float32)  # subnormal numbers
    check_evict(x, w, budget, 0, min(budget - 1, 3))


@pytest.mark.parametrize("jitter", [0, 1, 9, 60])
def test_evict_of_far_scales(jitter):
    """Codes are rounded to the largest scale of their new block, to nothing where it is far above."""
    x, w = evict_batch(jitter, 2, 128, 32, [400, 222], 100, jitter)
    x.k_sf = np.where(x.k_sf == 255, 255, np.random.default_rng(0).integers(120 - jitter, 121 + jitter, x.k_sf.shape)).astype(np.uint8)
    x.k_codes = np.random.default_rng(1).integers(0, 256, x.k_codes.shape).astype(np.uint8)  # every code, NaN too
    check_evict(x, w, 100, 2, 5)


def test_evict_shared_old_pages():
    """Sequences that share pages of a prompt are cut independently: old pages are only read."""
    x, w = evict_batch(6, 2, 64, 16, [100, 100], 30)
    x.table[1, :3] = x.table[0, :3]
    check_evict(x, w, 30, 1, 4)


def test_evict_bad_pages_and_lengths():
    x, w = evict_batch(7, 2, 64, 16, [100, 90, 80], 40)
    table = hist.spare_table(x, 40)
    good = hist.evict(x, w, 40, 2, 3, table)
    clean = x.table.copy()
    for entry in (-1, x.k_codes.shape[0], 2 ** 31 - 1):
        x.table = clean.copy()
        x.table[1, 2] = entry
        got = run_evict(x, w, 40, 2, 3, table)
        status(gdpa.GDPA_ERR_INVALID_ARG)
        for b in (0, 2):
            assert np.array_equal(got[5][b], good[5][b])
            for i in range(3):
                assert np.array_equal(got[0][table[b, i]], good[0][table[b, i]])
        # the tokens on that page go before all others
        assert not ((got[5][1] >= 32) & (got[5][1] < 48)).any() and got[6].tolist() == [40, 40, 40]
    x.table = clean
    bad = table.copy()
    bad[1, 1] = x.k_codes.shape[0]
    got = run_evict(x, w, 40, 2, 3, bad)
    status(gdpa.GDPA_ERR_INVALID_ARG)
    assert np.array_equal(got[5], good[5])
    assert np.array_equal(got[0][table[1, 0]], good[0][table[1, 0]]) and np.array_equal(got[0][table[1, 1]], x.k_codes[table[1, 1]])
    for n in (-1, 16 * x.table.shape[1] + 1, 2 ** 31 - 1):
        y = ref.Batch(**{**x.__dict__, "lens": [100, n, 80]})
        got = run_evict(y, w, 40, 2, 3, table)
        status(gdpa.GDPA_ERR_INVALID_ARG)
        assert got[6].tolist() == [40, 0, 40] and (got[5][1] == -1).all()
        assert np.array_equal(got[0][table[1]], x.k_codes[table[1]])


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("Hq,H,D,new", [(8, 2, 64, 1), (4, 4, 128, 3)])
def test_a_history_is_served_and_cut(Hq, H, D, new):
    """A prompt, decoding steps and cuts as a program does them: rotate by the true positions, append to a cache without
    rotation, attend, accumulate the weights, cut when it is long, go on in the new pages.  Each step is checked against
    the 64-bit forms on the state that the library left."""
    P, B, budget, rot = 16, 2, 64, D
    f, m = gdpa.gdpa_rope_freqs(rot, scaling=gdpa.GDPA_ROPE_SCALE_RAMP, factor=4.0, trained=256)
    rng = np.random.default_rng(D)
    num = 40
    codes = [torch.full((num, H, P, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    codes += [torch.full((num, H, P // 16), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = gdpa.KvCache(*codes)
    w = torch.full((num, H, P), float("nan"), dtype=torch.float32, device="cuda")
    free, held = list(range(num)), [[], []]
    lens, pos = [0, 0], [0, 0]
    scale = float(np.float32(D ** -0.5))
    cuts = 0
    for step in range(16):
        rows = [70, 33] if step == 0 else [new, new]
        for b in range(B):
            lens[b] += rows[b]
            while len(held[b]) * P < lens[b]:
                held[b].append(free.pop())
        width = max(len(p) for p in held)
        table = np.full((B, width), -1, np.int32)
        for b in range(B):
            table[b, :len(held[b])] = held[b]
        offsets = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        T = int(offsets[-1])
        fused = cu_bf16(rng.standard_normal((T, Hq + 2 * H, D)))
        d_off, d_lens, d_table, d_pos = cu(offsets), cu(np.array(lens, np.int32)), cu(table), cu(np.array(pos, np.int32))
        raw = fused.double().cpu().numpy()
        gdpa.gdpa_rope(fused[:, :Hq + H], fused.stride(0), d_off, d_pos, T, B, Hq + H, D, f, gdpa.GDPA_ROPE_HALF, m, False,
                       fused[:, :Hq + H], fused.stride(0))
        q, k, v = fused[:, :Hq], fused[:, Hq:Hq + H], fused[:, Hq + H:]
        gdpa.gdpa_cache_append(cache, None, 0, k, k.stride(0), v, v.stride(0), d_off, d_lens, d_table, T, B, Hq, width, None)
        out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((T, Hq), dtype=torch.float32, device="cuda")
        ws = torch.empty(gdpa.gdpa_cache_workspace_size(cache, Hq, max(rows)), dtype=torch.uint8, device="cuda")
        gdpa.gdpa_cache_fwd(cache, q, q.stride(0), d_off, d_lens, d_table, T, B, Hq, width, max(rows), True, 0, scale, out, lse, ws)
        before = w.double().cpu().numpy()
        gdpa.gdpa_cache_weights(cache, q, q.stride(0), lse, d_off, d_lens, d_table, T, B, Hq, width, max(rows), True, 0, scale,
                                0.875, w, w)
        status()
        # the rotation, the attention and the weights of this step
        want = hist.rope(raw[:, :Hq + H], offsets, pos, f, False, m)
        turned = fused.double().cpu().numpy()
        assert (np.abs(turned[:, :Hq + H] - want) <= 2.0 ** -8 * np.abs(want)
                + 1.01 * rope_bound(raw[:, :Hq + H], rot, f, 0, m, 0)).all()
        host = [c.cpu().numpy() for c in codes]
        x = ref.Batch(Hq, H, D, P, list(lens), rows, *host, table, offsets, turned[:, :Hq], turned[:, Hq:Hq + H], raw[:, Hq + H:])
        ro = ref.attend(x, True, 0, scale)
        tol, tol_lse = ref.attend_bounds(x, *ro)
        assert (np.abs(out.double().cpu().numpy() - ro[0]) <= tol).all()
        got_lse = lse.double().cpu().numpy()
        assert (np.abs(got_lse - ro[1]) <= tol_lse).all()
        want_w, tol_w = hist.weights(x, got_lse, True, 0, scale, 0.875, before)
        at = ~np.isnan(want_w)
        assert (np.abs(w.double().cpu().numpy() - want_w)[at] <= tol_w[at]).all()
        pos = [p + r for p, r in zip(pos, rows)]
        if max(lens) > budget + 4:
            cuts += 1
            to = [[free.pop() for _ in range(-(-min(n, budget) // P))] for n in lens]
            new_table = np.full((B, budget // P), -1, np.int32)
            for b in range(B):
                new_table[b, :len(to[b])] = to[b]
            kept = torch.full((B, H, budget), -1, dtype=torch.int32, device="cuda")
            new_lens = torch.empty(B, dtype=torch.int32, device="cuda")
            old_w = w.cpu().numpy()
            gdpa.gdpa_cache_evict(cache, w, d_lens, d_table, B, width, budget, 2, 8, cu(new_table), budget // P, kept, new_lens)
            status()
            want = hist.evict(x, old_w, budget, 2, 8, new_table)
            got = [c.cpu().numpy() for c in codes] + [w.cpu().numpy(), kept.cpu().numpy(), new_lens.cpu().numpy()]
            for name, a, b in zip(NAMES, got, want):
                same(a, b, name)
            for b in range(B):
                free += held[b]
            held, lens = to, new_lens.cpu().tolist()
    assert cuts >= 2


@pytest.mark.parametrize("new", [65, 112, 113])
@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("causal,window", [(1, 0), (0, 0), (1, 50)])
def test_weights_between_few_rows_and_many(new, P, causal, window):
    """Heads of 64 with more rows than the least kernels hold, on both sides of the rule for many."""
    x = ref.make(15, 2, 2, 64, P, [511, 130, new], [new, 66, new])
    check_weights(x, causal, window)
