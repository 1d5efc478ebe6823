"""Calls of the paged cache that programs may make and that the other GPU tests leave out: offsets, windows, pages and
values at the ends of what the documentation allows."""
from __future__ import annotations

import dataclasses
import math
import os
import subprocess
import sys

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


@pytest.mark.parametrize("D", [64, 128])
def test_the_plain_form_may_take_longer_than_a_wait_may(D):
    """Every segment has a block of V far below the others and takes the plain form (about 50 ms a segment here), in
    front of another segment of the same run: with a wait limit of 5 ms the roles that wait for it must not give up.
    In a process of its own, for the limit."""
    code = """
import sys; sys.path.insert(0, %r)
import math
import dataclasses
import math
import os
import subprocess
import sys

import numpy as np
from tests import cache_ref as ref
from tests.test_cache_gpu import Dev, gdpa, host
B, new, n, D = 160, 40, 2000, %d
x = ref.make(72, 4, 1, D, 64, [n], [new], jitter=1)
x.v_sf[x.table[0, 5], :, 1] = 60
ro = ref.attend(x, True, 0, float(np.float32(1 / math.sqrt(D))))
tol, tl = ref.attend_bounds(x, *ro)
# the same sequence many times over (its pages are only read)
x.table, x.lens, x.new = np.repeat(x.table, B, 0), [n] * B, [new] * B
x.offsets = (np.arange(B + 1) * new).astype(np.int32)
x.q, x.k, x.v = (np.tile(a, (B, 1, 1)) for a in (x.q, x.k, x.v))
d = Dev(x)
d.fwd()
status = gdpa.gdpa_device_status()
assert status == gdpa.GDPA_OK, status
got, lse = host(d.out).reshape(B, new, 4, D), host(d.lse).reshape(B, new, 4)
assert (np.abs(got - ro[0]) <= tol).all() and (np.abs(lse - ro[1]) <= tl).all()
print("fine")
""" % (os.path.dirname(os.path.dirname(os.path.abspath(__file__))), D)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, GDPA_WAIT_TIMEOUT_MS="5"))
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stderr[-2000:]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,heads", [(2, (4, 1)), (3, (8, 1)), (12, (4, 1)), (30, (1, 1)), (70, (2, 1)), (130, (2, 1))])
@pytest.mark.parametrize("sf,rest", [(254, 120), (254, 100), (247, 70), (254, 60), (247, 40)])
def test_a_huge_value_that_only_the_first_row_s_window_holds(D, new, heads, sf, rest):
    """The last key of its block that any row sees, far above all others: it decides the first row and leaves no trace
    in the next ones."""
    window = 100
    for keys in (497, 2593):
        x = ref.make(71, *heads, D, 32, [keys], [new], jitter=1)
        at = keys - new - window + 1
        x.v_sf[x.v_sf != 255] = rest
        page, slot = x.table[0, at // 32], at % 32
        x.v_sf[page, :, slot // 16] = sf
        block = x.v_codes[page, :, slot // 16 * 16:slot // 16 * 16 + 16]
        block[:, :slot % 16 + 1] = block[:, :slot % 16 + 1] & 0x87 | 1  # from 2^-9 to 2^-6: finite in the result
        block[:, slot % 16 + 1:] = 0
        d = Dev(x)
        d.fwd(window=window)
        check_fwd(x, d, True, window)


def attend_kept(x, causal, window, scale):
    """ref.attend over the keys whose page the cache has."""
    pages = x.k_codes.shape[0]
    bad = (x.table < 0) | (x.table >= pages)
    y = dataclasses.replace(x, table=np.where(bad, 0, x.table))
    G = x.Hq // x.H
    out, lse, big = np.zeros((x.T, x.Hq, x.D)), np.full((x.T, x.Hq), -np.inf), np.zeros((x.T, x.Hq))
    mag = np.zeros_like(out)
    for b, (n, new) in enumerate(zip(x.lens, x.new)):
        k, v = ref.gather(y, b, x.k_codes, x.k_sf), ref.gather(y, b, x.v_codes, x.v_sf)
        there = ~bad[b, np.arange(n) // x.P]
        for i in range(new):
            j0, j1 = ref.seen(n, new, i, causal, window)
            j = np.arange(j0, max(j0, j1))
            j = j[there[j]]
            if not len(j):
                continue
            r = x.offsets[b] + i
            for h in range(x.H):
                qq, kk, vv = x.q[r, h * G:(h + 1) * G], k[j, h], v[j, h]
                s = scale * (qq @ kk.T)
                m = s.max(-1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(-1, keepdims=True)
                at = np.s_[r, h * G:(h + 1) * G]
                out[at], mag[at], lse[at] = p @ vv / l, p @ np.abs(vv) / l, (np.log(l) + m)[:, 0]
                big[at] = (abs(scale) * (np.abs(qq) @ np.abs(kk).T)).max(-1)
    return out, lse, mag, big


def check_kept(x, d, causal, window, skipped=()):
    """The rows of all sequences but the skipped ones, which keep what the outputs held."""
    ro = attend_kept(x, causal, window, float(np.float32(1 / math.sqrt(x.D))))
    tol, tl = ref.attend_bounds(x, *ro)
    got, lse = host(d.out), host(d.lse)
    rows = np.zeros(d.T, bool)
    for b in range(len(x.lens)):
        if b not in skipped:
            rows[x.offsets[b]:x.offsets[b + 1]] = True
    assert (got[~rows] == 7).all() and (lse[~rows] == 7).all()
    rows = rows[:x.T]
    bad = ~(np.abs(got[:x.T] - ro[0]) <= tol)[rows]
    assert not bad.any(), (np.argwhere(bad)[:5], got[:x.T][rows][bad][:5], ro[0][rows][bad][:5])
    none = np.isneginf(ro[1])[rows]
    np.testing.assert_array_equal(np.isneginf(lse[:x.T][rows]), none)
    assert (none | (np.abs(np.where(none, 0, lse[:x.T][rows]) - np.where(none, 0, ro[1][rows])) <= tl[rows])).all()


ROWS = [(1, (1, 1)), (3, (8, 1)), (6, (4, 1)), (12, (4, 1)), (65, (2, 1)), (70, (4, 1))]  # every tile and kernel


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,heads", ROWS)
@pytest.mark.parametrize("keys", [300, 2603])
@pytest.mark.parametrize("P,causal,window", [(16, True, 0), (32, True, 77), (128, False, 0)])
def test_keys_on_a_page_out_of_range_are_not_seen(D, new, heads, keys, P, causal, window):
    """Bad entries first, in the middle, last, several and all of them; with and without a block of V so far below the
    others that many rows take the plain form."""
    for low in (False, True):
        x = ref.make(70, *heads, D, P, [keys, 55], [new, 2], jitter=1)
        if low:
            x.v_sf[x.table[0, 130 // P], :, 130 % P // 16] = 60
        n = -(-keys // P)
        spans = [ref.seen(keys, new, i, causal, window) for i in (0, new - 1)]
        for bad in ([0], [n // 2], [n - 1], [0, 1, n - 2], list(range(n))):
            y = dataclasses.replace(x, table=x.table.copy())
            y.table[0, bad] = [[-1, -2 ** 31, x.k_codes.shape[0], 2 ** 31 - 1][i % 4] for i in range(len(bad))]
            d = Dev(y, pad=1)
            d.fwd(causal, window)
            read = any(j0 < (b + 1) * P and b * P < j1 for b in bad for j0, j1 in spans)
            assert gdpa.gdpa_device_status() == (gdpa.GDPA_ERR_INVALID_ARG if read else gdpa.GDPA_OK), bad
            check_kept(y, d, causal, window)


@pytest.mark.parametrize("new,heads", ROWS)
@pytest.mark.parametrize("spoil", ["long", "negative", "offsets"])
def test_other_sequences_are_right_beside_a_spoilt_one(new, heads, spoil):
    x = ref.make(73, *heads, 64, 32, [90, 2203, 41], [new, 1, new])
    d = Dev(x, pad=2)
    if spoil == "offsets":  # of the last sequence: past the rows there are
        d.offsets[3] = d.T + 1
    else:
        d.lens[1] = x.table.shape[1] * 32 + 1 if spoil == "long" else -5
    d.fwd()
    assert gdpa.gdpa_device_status() == gdpa.GDPA_ERR_INVALID_ARG
    check_kept(x, d, True, 0, skipped=[2 if spoil == "offsets" else 1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,heads", ROWS)
def test_a_cache_without_pages(D, new, heads):
    """Nothing is stored and nothing can be: rows see nothing, and lengths above zero are reported."""
    for lens, status in (([0, 0], gdpa.GDPA_OK), ([new + 40, 0], gdpa.GDPA_ERR_INVALID_ARG)):
        x = ref.make(74, *heads, D, 32, [0, 0], [new, 1], spare=0)
        x.lens, x.table = lens, np.full((2, 5), -1, np.int32)
        d = Dev(x, inv_freq(D), pad=1)
        assert d.k_codes.numel() == 0
        d.fwd()
        assert gdpa.gdpa_device_status() == status
        assert (host(d.out)[:x.T] == 0).all() and np.isneginf(host(d.lse)[:x.T]).all()
        assert (host(d.out)[x.T:] == 7).all() and (host(d.lse)[x.T:] == 7).all()
    x.lens = [new, 1]  # an append keeps nothing, and rotates the queries
    d = Dev(x, inv_freq(D))
    d.append()
    assert gdpa.gdpa_device_status() == gdpa.GDPA_ERR_INVALID_ARG
    q = np.concatenate([ref.rotate(x.q[:new], np.arange(new), inv_freq(D), False), x.q[new:]])
    slack = 2.0 ** -21 * np.sqrt(2) * np.linalg.norm(x.q, axis=-1, keepdims=True)
    assert (np.abs(host(d.q_out) - q) <= 2.0 ** -8 * np.abs(q) + slack).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(300, 1), (1000, 2), (600, 600), (1023, 341)])
@pytest.mark.parametrize("new", [1, 3])
def test_many_heads(D, heads, new):
    """Groups of more heads than a tile has rows, and more key heads than a CTA has tiles."""
    x = ref.make(75, *heads, D, 16, [70, new], [new, new], jitter=1)
    d = Dev(x)
    d.fwd()
    check_fwd(x, d, True, 0)
    d.append()  # (unrotated: so many blocks hold some whose scale a rotation's rounding decides)
    check_append(x, d, None, False)


@pytest.mark.parametrize("D", [64, 128])
def test_calls_for_many_and_few_rows_at_once(D):
    """Four streams with a workspace each, two of them with the kernel for many rows."""
    xs = [ref.make(90 + i, 8, 2, D, 64, [3000, 100 * i + 99, 700], [n, 30, 99]) for i, n in enumerate((90, 1, 140, 6))]
    ds = [Dev(x) for x in xs]
    hints = (140, 1, 140, 6)
    spaces = [torch.empty(gdpa.gdpa_cache_workspace_size(d.cache, 8, n), dtype=torch.uint8, device="cuda")
              for d, n in zip(ds, hints)]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, w, s, n in zip(ds, spaces, streams, hints):
            d.fwd(workspace=w, stream=s, max_q=n)
    torch.cuda.synchronize()
    for x, d in zip(xs, ds):
        check_fwd(x, d, True, 0)
