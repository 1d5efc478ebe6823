"""The paged cache on the GPU against its plain 64-bit forms (tests/cache_ref.py).

Every page and block that belongs to no stored token holds NaN codes and NaN
scales in these tests, so a read of one shows in the result."""
from __future__ import annotations

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

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()
    yield


def inv_freq(rot, base=10000.0):
    return base ** (-np.arange(0, rot, 2) / rot) if rot else None


class Dev:
    """A batch on the device."""

    def __init__(self, x: ref.Batch, freq=None, interleaved=False, fused=False, pad=0):
        self.x = x
        cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.k_codes, self.v_codes, self.k_sf, self.v_sf = cu(x.k_codes), cu(x.v_codes), cu(x.k_sf), cu(x.v_sf)
        self.cache = gdpa.KvCache(self.k_codes, self.v_codes, self.k_sf, self.v_sf, freq,
                                  gdpa.GDPA_ROPE_INTERLEAVED if interleaved else gdpa.GDPA_ROPE_HALF)
        self.table, self.offsets = cu(x.table), cu(x.offsets)
        self.lens = cu(np.array(x.lens, np.int32))
        rows = [np.concatenate([a, np.full((pad,) + a.shape[1:], np.nan)]) for a in (x.q, x.k, x.v)]
        rows = [torch.from_numpy(a).to(torch.bfloat16) for a in rows]
        if fused:  # heads of q, k and v side by side in one row, and 8 elements between the rows
            n = x.Hq + 2 * x.H
            buf = torch.full((x.T + pad, n * x.D + 8), float("nan"), dtype=torch.bfloat16)
            buf[:, :n * x.D] = torch.cat(rows, 1).reshape(x.T + pad, -1)
            buf = buf.cuda()
            cut = [0, x.Hq, x.Hq + x.H, n]
            self.q, self.k, self.v = (buf[:, cut[i] * x.D:cut[i + 1] * x.D].unflatten(1, (-1, x.D)) for i in range(3))
        else:
            self.q, self.k, self.v = (a.cuda() for a in rows)
        self.T = x.T + pad
        self.q_out = torch.full((self.T, x.Hq, x.D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.out = torch.full((self.T, x.Hq, x.D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.T, x.Hq), 7.0, dtype=torch.float32, device="cuda")

    def append(self, with_q=True, q_out=None, stream=None):
        x = self.x
        out = self.q_out if q_out is None else q_out
        gdpa.gdpa_cache_append(self.cache, self.q if with_q else None, self.q.stride(0), self.k, self.k.stride(0),
                               self.v, self.v.stride(0), self.offsets, self.lens, self.table, self.T, len(x.lens), x.Hq,
                               x.table.shape[1], out if with_q else None, stream=stream)

    def fwd(self, causal=True, window=0, scale=None, max_q=None, q=None, lse=True, workspace=None, stream=None):
        x = self.x
        max_q = max(1, max(x.new)) if max_q is None else max_q
        q = self.q if q is None else q
        if workspace is None:
            workspace = torch.full((gdpa.gdpa_cache_workspace_size(self.cache, x.Hq, max_q),), 0xFF, dtype=torch.uint8,
                                   device="cuda")
        gdpa.gdpa_cache_fwd(self.cache, q, q.stride(0), self.offsets, self.lens, self.table, self.T, len(x.lens), x.Hq,
                            x.table.shape[1], max_q, causal, window, 1 / math.sqrt(x.D) if scale is None else scale,
                            self.out, self.lse if lse else None, workspace, stream=stream)
        return workspace


def host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def check_append(x, d, freq, interleaved, with_q=True):
    """q, codes and scales.  A rotated value is off by at most 2^-21 (|x| + |y|): 2^-23.3 of it from the angle
    (rounded to 24 bits of half a turn, 2^-25 pi), two units of sine and cosine, three roundings.  Stored values
    then are off by half a step: 2^-8 (bf16), 2^-4 or half of 2^-9 scales (e4m3).  What is not rotated is exact."""
    q, k, v = ref.append(x, freq, interleaved)
    assert gdpa.gdpa_device_status() == gdpa.GDPA_OK
    if with_q:
        slack = 2.0 ** -21 * np.sqrt(2) * np.linalg.norm(x.q, axis=-1, keepdims=True) if freq is not None else 0
        got = host(d.q_out)[:x.T]
        assert (np.abs(got - q) <= 2.0 ** -8 * np.abs(q) + slack).all()
        assert (host(d.q_out)[x.T:] == 7).all()
    for name, (codes, sf, val, near), raw in (("k", k, x.k), ("v", v, x.v)):
        got, got_sf = host(getattr(d, name + "_codes")), host(getattr(d, name + "_sf"))
        rotated = name == "k" and freq is not None
        assert not rotated or near > 1e-5  # the draw decides no exponent by a rounding
        np.testing.assert_array_equal(got_sf, sf)
        new = np.isfinite(val)
        if rotated:
            unit = np.ldexp(1.0, sf.astype(np.int64) - 127).repeat(ref.BLOCK, -1)[..., None]
            unit = np.where(new, unit, 0)
            y = np.where(new, val, 0)
            err = np.abs(np.where(new, ref.e4m3_values(got), 0) * unit - y)
            big = np.abs(raw).max(initial=0) * 2
            assert (err <= 2.0 ** -4 * np.abs(y) + 2.0 ** -10 * unit + 2.0 ** -21 * big).all()
            same = ~new
        else:
            same = np.ones_like(new)
        np.testing.assert_array_equal(got[same], codes[same])


HEADS = [(1, 1), (8, 8), (8, 2), (14, 2), (32, 4)]
APPEND = [
    # (lens after, new): first tokens, ends and starts inside blocks and pages, sequences without new tokens
    ([1], [1]),
    ([16], [16]),
    ([17, 33, 5], [1, 17, 5]),
    ([40, 0, 70, 16], [3, 0, 70, 0]),
    ([100 + i for i in range(37)], [1] * 37),
    ([131, 64, 200], [131, 31, 130]),
    ([300, 15, 1], [300, 15, 1]),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", range(len(APPEND)))
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(D, case, interleaved):
    lens, new = APPEND[case]
    Hq, H = HEADS[case % len(HEADS)]
    P = [16, 32, 64, 128][case % 4]
    rot = [D, D // 2, 16, 0][(case + interleaved) % 4]
    held = [n - m for n, m in zip(lens, new)]
    x = ref.make(case, Hq, H, D, P, lens, new, held)
    f = inv_freq(rot)
    d = Dev(x, f, interleaved, fused=case % 2 == 1, pad=case % 3)
    d.append()
    check_append(x, d, f, interleaved)
    d.append()  # the same tokens again: the same contents (a block's scale only grows)
    check_append(x, d, f, interleaved)


def test_append_without_queries_and_in_place():
    f = inv_freq(64)
    x = ref.make(3, 8, 2, 64, 32, [50, 20], [30, 1], [20, 19])
    d = Dev(x, f)
    d.append(with_q=False)
    check_append(x, d, f, False, with_q=False)
    assert (host(d.q_out) == 7).all()
    d.append(q_out=d.q)
    d.q_out = d.q
    check_append(x, d, f, False)


def test_append_grows_scales_and_keeps_what_is_not_finite():
    D, P = 128, 32
    x = ref.make(5, 4, 2, D, P, [21, 32, 9], [4, 10, 9], [17, 22, 0])
    x.k *= 16                       # larger than what the blocks hold: earlier codes are rounded again
    x.v[4:14] *= 2.0 ** 60          # by so much that they become zero
    x.v[14:] = 0                    # an all-zero block
    x.k[14, 0, :] = 0
    x.k[15, 1, 5], x.k[16, 1, 6], x.v[2, 0, 7], x.v[3, 1, 8] = np.inf, np.nan, -np.inf, np.nan
    d = Dev(x, None)
    d.append()
    check_append(x, d, None, False)
    codes = host(d.v_codes)
    assert (codes[x.table[0, 0], 0, 19, 7] & 0x7F) == 0x7F and (codes[x.table[0, 0], 1, 20, 8] & 0x7F) == 0x7F
    assert (host(d.v_sf)[x.table[2, 0], :, 0] == 0).all() and (codes[x.table[2, 0], :, :9] == 0).all()


@pytest.mark.parametrize("top", [3.3e38, 1e-39, 448.0, 449.0, 1.75 * 2.0 ** -100])
def test_append_extreme_magnitudes(top):
    x = ref.make(6, 1, 1, 64, 16, [16], [16], [0])
    x.k[:] = ref.bf16(np.clip(x.k, -3, 3) / 3 * top)
    x.v[:] = ref.bf16(x.v / np.abs(x.v).max() * top)
    d = Dev(x, None)
    d.append()
    check_append(x, d, None, False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_far_positions(interleaved):
    """Angles near the last position that fits (2^31), and attention through a window there."""
    P, D = 1024, 64
    end = (1 << 31) - 5 * P - 3
    n = 45  # from the start of a block: nothing in front of them is stored
    x = ref.make(7, 2, 1, D, P, [3 * P], [n], [0], spare=0)
    x.table = np.full((1, (1 << 31) // P - 1), -1, np.int32)
    last = (end - 1) // P
    x.table[0, last - 1:last + 1] = [2, 1]
    x.lens = [end]
    f = inv_freq(D)
    d = Dev(x, f, interleaved)
    d.append()
    check_append(x, d, f, interleaved)
    x.k_codes, x.k_sf, x.v_codes, x.v_sf = host(d.k_codes), host(d.k_sf), host(d.v_codes), host(d.v_sf)
    d.fwd(window=17, q=d.q_out)
    assert gdpa.gdpa_device_status() == gdpa.GDPA_OK
    # the same rows as a sequence of its own: the window never reaches behind the new tokens for rows 16 on
    y = ref.Batch(x.Hq, x.H, D, P, [last * P + P - (last - 1) * P], [n], x.k_codes, x.v_codes, x.k_sf, x.v_sf,
                  np.array([[2, 1]], np.int32), x.offsets, x.q, x.k, x.v)
    y.lens = [end - (last - 1) * P]
    q = host(d.q_out)
    out, lse, mag, big = ref.attend(y, True, 17, 1 / math.sqrt(D), q=q)
    tol, tl = ref.attend_bounds(y, out, lse, mag, big)
    assert (np.abs(host(d.out) - out) <= tol)[16:].all()
    assert (np.abs(host(d.lse) - lse) <= tl)[16:].all()


def test_cache_beyond_32_bits():
    """Codes more than 2^31 and 2^32 bytes into the cache."""
    H, P, D = 8, 128, 128
    pages = (1 << 32) // (H * P * D) + 2
    codes = [torch.zeros((pages, H, P, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    sf = [torch.zeros((pages, H, P // 16), dtype=torch.uint8, device="cuda") for _ in range(2)]
    x = ref.make(8, 8, H, D, P, [2 * P], [2 * P], [0], spare=0)
    d = Dev(x, None)
    d.cache = gdpa.KvCache(codes[0], codes[1], sf[0], sf[1])
    big = torch.tensor([[pages - 1, pages // 2]], dtype=torch.int32, device="cuda")
    width = x.table.shape[1]
    d.table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    d.table[:, :2] = big
    d.append()
    d.fwd()
    assert gdpa.gdpa_device_status() == gdpa.GDPA_OK
    _, k, v = ref.append(x, None, False)
    for c, s, want in ((codes[0], sf[0], k), (codes[1], sf[1], v)):
        at = x.table[0, :2].astype(np.int64)
        np.testing.assert_array_equal(host(c[big[0].long()]), want[0][at])
        np.testing.assert_array_equal(host(s[big[0].long()]), want[1][at])
    x.k_codes, x.k_sf, x.v_codes, x.v_sf = k[0], k[1], v[0], v[1]
    check_fwd(x, d, True, 0)


def test_append_skips_what_is_out_of_range():
    f = inv_freq(64)
    for spoil in ("page", "negative", "len", "short", "offsets", "decreasing"):
        x = ref.make(9, 4, 2, 64, 16, [40, 50, 20], [3, 20, 2], [37, 30, 18])
        d = Dev(x, f)
        before = host(d.k_codes).copy()
        if spoil == "page":
            d.table[1] = x.k_codes.shape[0]
        elif spoil == "negative":
            d.table[1] = -1
        elif spoil == "len":
            d.lens[1] = x.table.shape[1] * 16 + 1
        elif spoil == "short":
            d.lens[1] = 19
        elif spoil == "offsets":
            d.offsets[3] = x.T + 9
        else:
            d.offsets[1:] = torch.tensor([23, 3, 25], dtype=torch.int32)
        d.append()
        assert gdpa.gdpa_device_status() == gdpa.GDPA_ERR_INVALID_ARG, spoil
        assert gdpa.gdpa_device_status() == gdpa.GDPA_OK
        if spoil in ("page", "negative", "len", "short"):
            own = x.table[1, :4]
            np.testing.assert_array_equal(host(d.k_codes)[own], before[own])
            _, _, (want, _, _, _) = ref.append(x, f, False)  # the other sequences are stored
            for b, n in ((0, 3), (2, 2)):
                np.testing.assert_array_equal(host(d.v_codes)[x.table[b, :n]], want[x.table[b, :n]])


# ------------------------------------------------------------------ attention

def check_fwd(x, d, causal, window, scale=None, q=None, lse=True):
    assert gdpa.gdpa_device_status() == gdpa.GDPA_OK
    scale = float(np.float32(1 / math.sqrt(x.D) if scale is None else scale))
    ro = ref.attend(x, causal, window, scale, q=q)
    tol, tl = ref.attend_bounds(x, *ro)
    got, got_lse = host(d.out), host(d.lse)
    bad = ~(np.abs(got[:x.T] - ro[0]) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[:x.T][bad][:5], ro[0][bad][:5], bad.sum())
    assert (got[x.T:] == 7).all()
    if lse:
        none = np.isneginf(ro[1])
        np.testing.assert_array_equal(np.isneginf(got_lse[:x.T]), none)
        bad = ~none & ~(np.abs(np.where(none, 0, got_lse[:x.T]) - np.where(none, 0, ro[1])) <= tl)
        assert not bad.any(), (np.argwhere(bad)[:5], got_lse[:x.T][bad][:5], ro[1][bad][:5])
        assert (got_lse[x.T:] == 7).all()
    else:
        assert (got_lse == 7).all()


ATTEND = [
    # (lens, new, causal, window)
    ([1], [1], True, 0),
    ([0], [1], True, 0),
    ([17, 0, 1, 16, 15, 33], [1] * 6, True, 0),
    ([200, 0, 511, 64, 1000], [1] * 5, True, 0),
    ([90, 33, 400], [1, 1, 1], True, 32),
    ([300, 40, 7], [5, 3, 7], True, 0),
    ([300, 40, 7], [5, 3, 7], False, 0),
    ([2, 3], [5, 6], True, 0),             # more rows than tokens: the first rows see nothing
    ([130, 0, 600], [70, 2, 100], True, 0),
    ([130, 0, 600], [70, 2, 100], False, 0),
    ([257, 700], [200, 130], True, 19),
    ([3000], [1], True, 0),
    ([1500, 12], [33, 0], True, 100),
    ([64] * 40, [1] * 40, True, 1),
    # more segments than CTAs: runs of whole short ones, and of cut longer ones
    ([(37 * i) % 300 for i in range(160)], [1] * 160, True, 0),
    ([(97 * i) % 900 for i in range(160)], [1 + i % 2 for i in range(160)], True, 0),
    ([2500, 40, 2100], [3, 1, 2], True, 0),
    ([2100, 3000], [70, 33], True, 0),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_fwd(D, heads, case):
    lens, new, causal, window = ATTEND[case]
    Hq, H = heads
    P = [16, 64, 32, 128, 1024][(case + Hq) % 5]
    x = ref.make(100 + case, Hq, H, D, P, lens, new)
    d = Dev(x, fused=case % 2 == 0, pad=case % 3)
    d.fwd(causal, window)
    check_fwd(x, d, causal, window)


@pytest.mark.parametrize("heads", [(3, 1), (20, 2), (16, 1), (48, 1), (40, 1)])
@pytest.mark.parametrize("new", [1, 2, 9])
def test_fwd_odd_groups(heads, new):
    x = ref.make(11, *heads, 128, 32, [100, 333, 31], [new] * 3)
    d = Dev(x)
    d.fwd()
    check_fwd(x, d, True, 0)


def test_fwd_does_not_depend_on_the_hint():
    x = ref.make(12, 8, 2, 64, 16, [500, 90, 33], [70, 1, 33])
    for max_q in (1, 3, 40, 70, 5000):
        d = Dev(x)
        d.fwd(max_q=max_q, lse=False)
        check_fwd(x, d, True, 0, lse=False)


@pytest.mark.parametrize("scale", [0.0, -0.5, 3.0, 1e-3])
def test_fwd_scales(scale):
    x = ref.make(13, 8, 2, 128, 64, [700, 31], [2, 2], jitter=1)
    d = Dev(x)
    d.fwd(scale=scale)
    check_fwd(x, d, True, 0, scale=scale)


def test_fwd_wide_ranges():
    """Large scores (one key takes all), queries and scales far from 1, a value block far above the others."""
    x = ref.make(14, 8, 2, 64, 16, [400, 300], [1, 3])
    x.q = ref.bf16(x.q * 30)
    d = Dev(x)
    d.fwd()
    check_fwd(x, d, True, 0)
    x = ref.make(15, 8, 2, 64, 16, [400, 300], [1, 3], jitter=0)
    x.q = ref.bf16(x.q * 2.0 ** -90)
    x.k_sf[x.k_sf != 255] += 90
    x.v_sf[x.table[0, 3], :, 0] += 40
    x.v_sf[x.table[1, 2], :, 0] = 0
    d = Dev(x)
    d.fwd()
    check_fwd(x, d, True, 0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["grows", "drops", "jumps", "zeros", "steps"])
def test_fwd_many_rows_wide_value_scales(D, kind):
    """Value blocks whose scales lie far apart, in the order of the keys, for many rows at once."""
    n, new = 500, 70
    x = ref.make(24, 4, 1, D, 16, [n], [new], jitter=0)
    sf = np.full(-(-n // 16), 120)
    j = np.arange(len(sf))
    sf = {"grows": 60 + 3 * j, "drops": 180 - 3 * j, "jumps": 120 + 25 * (j % 4 == 1), "zeros": 120 - 120 * (j % 3 == 0),
          "steps": 120 + 7 * (j // 4 % 2) - 8 * (j % 2)}[kind]
    x.v_sf[x.table[0, :len(sf)], 0, 0] = sf
    if kind == "zeros":
        for b in j[j % 3 == 0]:
            x.v_codes[x.table[0, b], 0] = np.where(x.v_codes[x.table[0, b], 0] == 127, 127, 0x80 * (b % 2))
    for window in (0, 33):
        d = Dev(x)
        d.fwd(window=window)
        check_fwd(x, d, True, window)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["grows", "drops", "jumps", "zeros", "steps"])
@pytest.mark.parametrize("new,keys", [(1, 500), (1, 2600), (2, 700), (3, 500), (4, 2600)])
def test_fwd_few_rows_wide_value_scales(D, kind, new, keys):
    """The same for one token and for a few, in one CTA and cut into parts."""
    x = ref.make(25, 16, 2, D, 32, [keys, 33], [new, 1], jitter=0)
    j = np.arange(-(-keys // 16))
    sf = {"grows": 60 + j % 100, "drops": 220 - j % 200, "jumps": 120 + 25 * (j % 4 == 1), "zeros": 120 * (j % 3 != 0),
          "steps": 120 + 7 * (j // 4 % 2) - 8 * (j % 2)}[kind]
    x.v_sf[x.table[0, :-(-keys // 32)].repeat(2)[:len(j)], :, j % 2] = sf[:, None]
    for window in (0, 33):
        d = Dev(x)
        d.fwd(window=window)
        check_fwd(x, d, True, window)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [7, 8, 9, 16, 17, 24, 25, 32, 33, 48, 49, 64, 96, 97])
@pytest.mark.parametrize("keys,causal", [(300, True), (900, False), (2600, True)])
def test_fwd_row_counts(D, rows, keys, causal):
    """Both sides of every number of rows at which another kernel or tile takes over, few keys and many."""
    x = ref.make(26 + rows, 2, 2, D, 32, [keys, rows // 2, rows + 40], [rows, rows // 3, rows - 1])
    d = Dev(x, pad=1)
    d.fwd(causal)
    check_fwd(x, d, causal, 0)


@pytest.mark.parametrize("new,window,heads", [(6, 0, (4, 1)), (20, 0, (8, 2)), (150, 0, (4, 2)), (5, 9, (2, 2)),
                                              (150, 9, (8, 1))])
def test_fwd_hidden_keys_never_count(new, window, heads):
    """NaN and infinite-scale keys and values inside the sequence: rows that do not see them are as if they were not
    there; rows that see a NaN key are NaN, rows that see a NaN value have NaN in its coordinate."""
    n = 300
    x = ref.make(16, *heads, 64, 32, [n], [new])
    at = n - new // 2  # a key of the middle new token
    page, slot = x.table[0, at // 32], at % 32
    clean = x.v_codes.copy(), x.k_codes.copy()
    x.v_codes[page, :, slot, 5] = 0x7F
    if new > 10:
        at2 = n - 2
        x.k_codes[x.table[0, at2 // 32], :, at2 % 32, 3] = 0xFF
    d = Dev(x)
    d.fwd(window=window)
    got = host(d.out)
    x.v_codes, x.k_codes = clean
    out, lse, mag, big = ref.attend(x, True, window, 1 / math.sqrt(64))
    tol, _ = ref.attend_bounds(x, out, lse, mag, big)
    for i in range(new):
        j0, j1 = ref.seen(n, new, i, True, window)
        if new > 10 and j0 <= n - 2 < j1:
            assert np.isnan(got[i]).all()
        elif j0 <= at < j1:
            assert np.isnan(got[i, :, 5]).all()
            ok = np.abs(got[i] - out[i]) <= tol[i]
            assert np.delete(ok, 5, -1).all()
        else:
            assert (np.abs(got[i] - out[i]) <= tol[i]).all(), i


def test_fwd_skips_pages_out_of_range():
    x = ref.make(17, 8, 2, 64, 16, [100, 90], [1, 2])
    d = Dev(x)
    d.table[0, 2] = 10 ** 6
    d.fwd()
    assert gdpa.gdpa_device_status() == gdpa.GDPA_ERR_INVALID_ARG
    assert torch.isfinite(d.out).all()
    d = Dev(x)
    d.lens[0] = x.table.shape[1] * 16 + 1
    d.fwd()
    assert gdpa.gdpa_device_status() == gdpa.GDPA_ERR_INVALID_ARG
    d = Dev(x)
    d.offsets[2] = 50
    d.fwd()
    assert gdpa.gdpa_device_status() == gdpa.GDPA_ERR_INVALID_ARG


def test_fwd_small_workspace_is_refused():
    x = ref.make(18, 8, 2, 64, 16, [100], [1])
    d = Dev(x)
    n = gdpa.gdpa_cache_workspace_size(d.cache, 8, 1)
    with pytest.raises(gdpa.GdpaError) as e:
        d.fwd(workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.code == gdpa.GDPA_ERR_NO_MEMORY


def test_same_inputs_same_bits():
    x = ref.make(19, 16, 2, 128, 64, [5000, 3, 900], [1, 1, 1])
    first = None
    for _ in range(4):
        d = Dev(x)
        d.fwd()
        got = d.out.clone(), d.lse.clone()
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, got))
        first = got


def test_a_run_of_both():
    """Prompts in two pieces, then single tokens: as a serving program calls them."""
    Hq, H, D, P = 8, 2, 64, 32
    f = inv_freq(D)
    rng = np.random.default_rng(20)
    total = [150, 40, 77]
    x = ref.make(20, Hq, H, D, P, total, [0, 0, 0], [0, 0, 0])
    steps = [[100, 0, 33], [30, 20, 40]] + [[1, 1, 1]] * 4 + [[1, 0, 0]] * 16 + [[0, 15, 0]]
    have = np.zeros(3, np.int64)
    d = Dev(x, f)
    for new in steps:
        have += new
        x.lens, x.new = [int(n) for n in have], list(new)
        x.offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        x.q, x.k, x.v = (ref.bf16(rng.standard_normal((x.T, h, D))) for h in (Hq, H, H))
        now = Dev(x, f)
        now.cache, now.k_codes, now.v_codes, now.k_sf, now.v_sf = d.cache, d.k_codes, d.v_codes, d.k_sf, d.v_sf
        now.append()
        check_append(x, now, f, False)
        x.k_codes, x.k_sf, x.v_codes, x.v_sf = host(d.k_codes), host(d.k_sf), host(d.v_codes), host(d.v_sf)
        now.fwd(q=now.q_out)
        check_fwd(x, now, True, 0, q=host(now.q_out))


def test_agrees_with_the_causal_forward():
    """The same attention through gdpa_fwd_sliding on the cache's values (exact in bf16)."""
    H, D, P, n = 4, 128, 64, 900
    x = ref.make(21, H, H, D, P, [n], [n], jitter=1)
    d = Dev(x)
    d.fwd()
    k, v = (torch.from_numpy(ref.gather(x, 0, c, s)).to(torch.bfloat16).cuda() for c, s in
            ((x.k_codes, x.k_sf), (x.v_codes, x.v_sf)))
    out = torch.empty_like(d.out)
    lse = torch.empty_like(d.lse)
    off = np.array([0, n], np.int32)
    dev = torch.from_numpy(off).cuda()
    gdpa.gdpa_fwd_sliding(d.q, k, v, off, off, dev, dev, 1, H, D, 0, n, 1 / math.sqrt(D), out, lse)
    ro = ref.attend(x, True, 0, 1 / math.sqrt(D))
    tol, tl = ref.attend_bounds(x, *ro)
    # the other side rounds its weights to bf16: 2^-8 where this one has 2^-11
    assert (np.abs(host(d.out) - host(out)) <= 2 * tol + 2.0 ** -8 * ro[2] * 1.01).all()
    assert (np.abs(host(d.lse) - host(lse)) <= 4 * tl).all()


# ------------------------------------------------------------------ streams and graphs

def test_graph_replays_read_lengths_anew():
    """A captured decoding step: append and attention, replayed with grown lengths and new tokens, in a batch padded
    to a fixed number of rows."""
    Hq, H, D, P, B = 8, 2, 64, 16, 4
    f = inv_freq(D)
    x = ref.make(22, Hq, H, D, P, [41, 64, 17, 30], [1, 1, 1, 0], [40, 63, 16, 30])
    for b in range(B):  # room for what comes
        x.table[b, -(-x.lens[b] // P):] = -7
    num = x.k_codes.shape[0]
    extra = np.arange(num, num + 2 * B, dtype=np.int32).reshape(B, 2)
    grow = lambda a, v: np.concatenate([a, np.full((2 * B,) + a.shape[1:], v, np.uint8)])
    x.k_codes, x.v_codes, x.k_sf, x.v_sf = grow(x.k_codes, 127), grow(x.v_codes, 127), grow(x.k_sf, 255), grow(x.v_sf, 255)
    table = np.full((B, x.table.shape[1] + 2), -7, np.int32)
    for b in range(B):
        n = -(-x.lens[b] // P)
        table[b, :n] = x.table[b, :n]
        table[b, n:n + 2] = extra[b]
    x.table = table
    d = Dev(x, f, pad=3)
    ws = torch.empty(gdpa.gdpa_cache_workspace_size(d.cache, Hq, 1), dtype=torch.uint8, device="cuda")
    state = [t.clone() for t in (d.k_codes, d.v_codes, d.k_sf, d.v_sf)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            d.append()
            d.fwd(q=d.q_out, workspace=ws, max_q=1)
    for t, was in zip((d.k_codes, d.v_codes, d.k_sf, d.v_sf), state):
        assert torch.equal(t, was)  # capture ran nothing
    rng = np.random.default_rng(23)
    torch.cuda.current_stream().wait_stream(s)
    for step in range(6):
        new = [[1, 1, 1, 0], [1, 1, 1, 1], [0, 1, 1, 1], [2, 1, 0, 1], [1, 0, 1, 0], [1, 1, 1, 1]][step]
        if step:
            x.lens = [a + b for a, b in zip(x.lens, new)]
        x.new = new
        x.offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        rows = [ref.bf16(rng.standard_normal((x.T, h, D))) for h in (Hq, H, H)]
        x.q, x.k, x.v = rows
        for t, a in zip((d.q, d.k, d.v), rows):
            t.fill_(float("nan"))
            t[:x.T] = torch.from_numpy(a).to(torch.bfloat16).cuda()
        d.lens.copy_(torch.tensor(x.lens, dtype=torch.int32))
        d.offsets.copy_(torch.from_numpy(x.offsets))
        d.q_out.fill_(7), d.out.fill_(7), d.lse.fill_(7)
        g.replay()
        check_append(x, d, f, False)
        x.k_codes, x.k_sf, x.v_codes, x.v_sf = host(d.k_codes), host(d.k_sf), host(d.v_codes), host(d.v_sf)
        check_fwd(x, d, True, 0, q=host(d.q_out)[:x.T])


def test_two_streams_with_a_workspace_each():
    xs = [ref.make(30 + i, 16, 2, 128, 64, [3000, 100 * i + 1], [1, 1]) for i in range(2)]
    ds = [Dev(x) for x in xs]
    ws = [torch.empty(gdpa.gdpa_cache_workspace_size(d.cache, 16, 1), dtype=torch.uint8, device="cuda") for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, w, s in zip(ds, ws, streams):
            d.fwd(workspace=w, stream=s)
    torch.cuda.synchronize()
    for x, d in zip(xs, ds):
        check_fwd(x, d, True, 0)


def test_the_first_call_of_a_process_may_be_captured():
    """Nothing but the capture has run: modules, kernels and their settings are loaded inside it."""
    code = """
import sys; sys.path.insert(0, %r)
import torch
from tests import cache_ref as ref
from tests.test_cache_gpu import Dev, check_append, check_fwd, host, inv_freq, gdpa
for new in ([1, 1], [3, 2], [90, 20]):
    f = inv_freq(64)
    x = ref.make(40, 8, 2, 64, 16, [300, 41], new, [300 - new[0], 41 - new[1]])
    d = Dev(x, f)
    ws = torch.empty(gdpa.gdpa_cache_workspace_size(d.cache, 8, max(new)), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.append()
        d.fwd(q=d.q_out, workspace=ws)
    for _ in range(2):
        g.replay()
    check_append(x, d, f, False)
    x.k_codes, x.k_sf, x.v_codes, x.v_sf = host(d.k_codes), host(d.k_sf), host(d.v_codes), host(d.v_sf)
    check_fwd(x, d, True, 0, q=host(d.q_out))
print("fine")
""" % os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stderr[-2000:]


# ------------------------------------------------------------------ calls that programs make and the tests above do not

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 5, 40])
def test_two_sequences_share_a_prefix(D, new):
    """The same page numbers twice in the table: both read them, neither writes."""
    x = ref.make(41, 8, 2, D, 16, [new + 300, new + 200], [new, new])
    x.table[1, :10] = x.table[0, :10]
    d = Dev(x)
    d.fwd()
    check_fwd(x, d, True, 0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,heads", [(2, (8, 2)), (6, (4, 1)), (24, (2, 1)), (90, (4, 2)), (130, (2, 2))])
def test_same_inputs_same_bits_with_more_rows(D, new, heads):
    x = ref.make(42, *heads, D, 64, [4000, 500, new], [new, new // 2, new])
    d = Dev(x)
    d.fwd()
    first = d.out.clone(), d.lse.clone()
    for _ in range(3):
        d.out.fill_(7), d.lse.fill_(7)
        d.fwd()
        assert torch.equal(first[0], d.out) and torch.equal(first[1], d.lse)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,heads", [(2, (4, 1)), (3, (8, 1)), (12, (4, 1)), (30, (1, 1)), (130, (2, 1))])
@pytest.mark.parametrize("sf", [230, 254])
def test_fwd_a_huge_value_hidden_from_all_but_the_last_row(D, new, heads, sf):
    """The last token alone in its block, of a scale far above the others: it decides the last row and leaves no trace
    in the others."""
    for keys in (497, 2593):
        x = ref.make(43, *heads, D, 32, [keys], [new], jitter=1)
        block = (keys - 1) // 16
        x.v_sf[x.table[0, block // 2], :, block % 2] = sf
        codes = x.v_codes[x.table[0, block // 2], :, (keys - 1) % 32]
        x.v_codes[x.table[0, block // 2], :, (keys - 1) % 32] = codes & 0x87  # below 2^-5: finite in the result
        d = Dev(x)
        d.fwd()
        check_fwd(x, d, True, 0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,heads", [(1, (4, 1)), (3, (8, 1)), (12, (4, 1)), (40, (2, 1)), (130, (2, 1))])
@pytest.mark.parametrize("sf", [3, 246])
def test_fwd_largest_and_smallest_values(D, new, heads, sf):
    """Values up to 448 2^119 (a sum of two is not finite in fp32) and from 2^-133 on."""
    for keys in (497, 2593):
        x = ref.make(48, *heads, D, 32, [keys], [new], jitter=1)
        x.v_sf[x.v_sf != 255] = sf
        d = Dev(x)
        d.fwd()
        check_fwd(x, d, True, 0)
        x.v_sf[x.table[0, 3], :, 0] = 200 - sf // 2  # blocks far apart as well: many rows take the plain form
        d = Dev(x)
        d.fwd()
        check_fwd(x, d, True, 0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,heads", [(3, (2, 1)), (3, (5, 1)), (6, (4, 1)), (28, (1, 1)), (48, (1, 1)), (140, (1, 1))])
def test_fwd_a_nan_value_stays_with_the_rows_that_see_it(D, new, heads):
    for keys in (299, 2603):
        x = ref.make(44, *heads, D, 32, [keys], [new])
        at = keys - max(1, new // 2)
        page, slot = x.table[0, at // 32], at % 32
        was = x.v_codes[page, :, slot, 9].copy()
        x.v_codes[page, :, slot, 9] = 0x7F
        d = Dev(x)
        d.fwd()
        x.v_codes[page, :, slot, 9] = was
        got = host(d.out)
        ro = ref.attend(x, True, 0, 1 / math.sqrt(D))
        tol, _ = ref.attend_bounds(x, *ro)
        for i in range(new):
            sees = at < ref.seen(keys, new, i, True, 0)[1]
            ok = np.abs(got[i] - ro[0][i]) <= tol[i]
            assert np.delete(ok, 9, -1).all(), (keys, i)
            assert np.isnan(got[i, :, 9]).all() if sees else ok[:, 9].all(), (keys, i)


def test_two_graphs_take_turns_with_one_workspace():
    xs = [ref.make(45 + i, 16, 2, 128, 64, [3000 + 500 * i, 70], [n, 1]) for i, n in enumerate((1, 12))]
    ds = [Dev(x) for x in xs]
    size = max(gdpa.gdpa_cache_workspace_size(d.cache, 16, 12) for d in ds)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    graphs = []
    for d in ds:
        d.fwd(workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            d.fwd(workspace=ws)
        graphs.append(g)
    for d in ds:
        d.out.fill_(7), d.lse.fill_(7)
    for _ in range(5):
        for g in graphs:
            g.replay()
    for x, d in zip(xs, ds):
        check_fwd(x, d, True, 0)


def test_a_slice_of_a_wider_table_is_refused():
    x = ref.make(49, 8, 2, 64, 16, [100, 50], [1, 1])
    d = Dev(x)
    d.table = torch.nn.functional.pad(d.table, (0, 3))[:, :d.table.shape[1]]
    with pytest.raises(ValueError, match="contiguous"):
        d.fwd()
    with pytest.raises(ValueError, match="contiguous"):
        d.append()
