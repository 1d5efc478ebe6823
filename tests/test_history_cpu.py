"""The argument checks of the operators for long histories (all before any CUDA call), the scaled frequencies, and the
tests' own 64-bit forms against brute force."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from jagged_attention_recommender_gb300 import build as gbuild
from jagged_attention_recommender_gb300 import gdpa
from tests import cache_ref as ref
from tests import history_ref as hist
from tests.test_cache_cpu import A, BAD_DESC, INV, UNS, Desc


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()
    yield


def rope(**kw):
    a = dict(x=A, x_stride=256, offsets=A, first=A, T=4, B=2, H=2, D=128, inv_freq=np.ones(64), rope_style=0, magnitude=1.0,
             inverse=0, y=2 * A, y_stride=256)
    a.update(kw)
    gdpa.gdpa_rope(stream=0, **a)


def weights(cache=None, **kw):
    a = dict(q=A, q_stride=1024, lse=A, offsets=A, kv_lens=A, page_table=A, T=4, B=2, Hq=8, max_pages=3, max_q=1, causal=1,
             window_tokens=0, scale=1.0, decay=1.0, weights_in=A, weights=A)
    a.update(kw)
    gdpa.gdpa_cache_weights(cache or Desc(), stream=0, **a)


def evict(cache=None, **kw):
    a = dict(weights=A, kv_lens=A, page_table=A, B=2, max_pages=3, budget=100, sink=2, recent=8, new_table=A, new_max_pages=2,
             kept=A, new_lens=2 * A)
    a.update(kw)
    gdpa.gdpa_cache_evict(cache or Desc(), stream=0, **a)


def refused(call, code, *args, **kw):
    with pytest.raises(gdpa.GdpaError) as e:
        call(*args, **kw)
    assert e.value.code == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INV), (dict(B=-1), INV), (dict(H=0), INV), (dict(D=96, inv_freq=np.ones(48)), UNS), (dict(D=256), UNS),
    (dict(inv_freq=np.ones(65)), INV), (dict(inv_freq=np.ones(4)), UNS), (dict(inv_freq=np.full(64, np.inf)), INV),
    (dict(inv_freq=np.full(64, np.nan)), INV), (dict(rope_style=2), INV), (dict(rope_style=-1), INV), (dict(inverse=2), INV),
    (dict(magnitude=float("nan")), INV), (dict(magnitude=float("inf")), INV), (dict(x=None), INV), (dict(y=None), INV),
    (dict(x=A + 8), INV), (dict(y=A + 2), INV), (dict(x_stride=255), INV), (dict(x_stride=260), UNS), (dict(y_stride=248), INV),
    (dict(y_stride=257), UNS), (dict(offsets=None), INV), (dict(offsets=A + 2), INV), (dict(first=A + 1), INV),
    (dict(H=1 << 14, x_stride=1 << 22, y_stride=1 << 22), UNS), (dict(T=2 ** 31 - 256), UNS), (dict(B=2 ** 31 - 4097), UNS),
    (dict(y=A, y_stride=512), INV),                                # in place with another stride
    (dict(y=A + 16), INV), (dict(y=A - 16), INV), (dict(y=A + 512), INV), (dict(y=A + 3 * 512), INV),
    (dict(x_stride=512, y_stride=512, y=A + 510 * 2 - 12), INV),   # the next row's heads
])
def test_rope_refusals(kw, code):
    refused(rope, code, **kw)


def test_rope_of_nothing():
    rope(T=0, x=None, y=None, offsets=None)
    rope(B=0, x=None, y=None, offsets=None)
    refused(rope, INV, T=0, inverse=5)


@pytest.mark.parametrize("kw,code", BAD_DESC)
def test_cache_descriptors_are_refused(kw, code):
    refused(weights, code, Desc(**kw))
    refused(evict, code, Desc(**kw))


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INV), (dict(B=-1), INV), (dict(max_pages=-1), INV), (dict(max_pages=0), INV), (dict(Hq=0), INV), (dict(Hq=3), INV),
    (dict(max_q=0), INV), (dict(causal=2), INV), (dict(window_tokens=-1), INV), (dict(causal=0, window_tokens=5), INV),
    (dict(scale=float("nan")), INV), (dict(decay=float("nan")), INV), (dict(decay=-0.5), INV), (dict(decay=float("inf")), INV),
    (dict(q=None), INV), (dict(q=A + 8), INV), (dict(q_stride=1023), INV), (dict(q_stride=1028), UNS), (dict(lse=None), INV),
    (dict(lse=A + 2), INV), (dict(offsets=None), INV), (dict(kv_lens=None), INV), (dict(page_table=None), INV),
    (dict(weights=None), INV), (dict(weights=A + 4), INV), (dict(weights_in=A + 8), INV), (dict(weights_in=A + 64), INV),
    (dict(T=2 ** 31 - 256), UNS), (dict(B=2 ** 31 - 4097), UNS), (dict(max_pages=1 << 26), UNS), (dict(Hq=1 << 14), UNS),
    (dict(T=2 ** 30), UNS),                                        # query rows of a key head: T Hq / H
])
def test_weights_refusals(kw, code):
    refused(weights, code, **kw)


def test_weights_of_nothing():
    weights(T=0, q=None, lse=None, weights=None, weights_in=None, offsets=None)
    weights(B=0, q=None, lse=None, weights=None, weights_in=None, offsets=None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INV), (dict(max_pages=-1), INV), (dict(max_pages=0), INV), (dict(budget=0), INV), (dict(budget=-1), INV),
    (dict(sink=-1), INV), (dict(recent=-1), INV), (dict(sink=60, recent=41), INV), (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), INV),
    (dict(new_max_pages=-1), INV), (dict(new_max_pages=1), INV), (dict(budget=2 ** 31 - 1, new_max_pages=2), INV),
    (dict(weights=None), INV), (dict(weights=A + 8), INV), (dict(kv_lens=None), INV), (dict(page_table=None), INV),
    (dict(new_table=None), INV), (dict(kept=None), INV), (dict(new_lens=None), INV), (dict(new_lens=A), INV),
    (dict(new_lens=A + 4), INV), (dict(new_lens=A - 4), INV), (dict(B=2 ** 31 - 4097), UNS), (dict(max_pages=1 << 26), UNS),
])
def test_evict_refusals(kw, code):
    refused(evict, code, **kw)


def test_evict_of_nothing():
    evict(B=0, weights=None, kv_lens=None, kept=None)


# ---------------------------------------------------------------- frequencies

@pytest.mark.parametrize("rot", [16, 32, 64, 128])
@pytest.mark.parametrize("scaling", range(4))
@pytest.mark.parametrize("factor,trained,base", [(1.0, 2048, 10000.0), (8.0, 4096, 10000.0), (40.0, 100, 500000.0), (2.5, 10 ** 7, 100.0)])
def test_frequencies(rot, scaling, factor, trained, base):
    f, m = gdpa.gdpa_rope_freqs(rot, base, scaling, factor, trained)
    want, wm = hist.frequencies(rot, base, scaling, factor, trained)
    assert f.shape == (rot // 2,) and np.allclose(f, want, rtol=1e-13, atol=0) and abs(m - wm) <= 2.0 ** -23 * wm
    plain = base ** (-np.arange(0, rot, 2) / rot)
    assert (f <= plain * (1 + 1e-12)).all() and (f >= plain / factor * (1 - 1e-12)).all()  # positions are only stretched
    if scaling == gdpa.GDPA_ROPE_SCALE_BASE:
        assert f[0] == 1 and abs(f[-1] * factor / plain[-1] - 1) < 1e-12
    if scaling == gdpa.GDPA_ROPE_SCALE_RAMP:
        turns = trained * plain / (2 * np.pi)
        # (the ramp's ends are whole pairs: one pair of room on either side)
        step = base ** (2 / rot)
        assert np.allclose(f[turns >= 32 * step], plain[turns >= 32 * step]) or hist_ramp_is_short(rot, base, trained)
        assert np.allclose(f[turns <= 1 / step], plain[turns <= 1 / step] / factor) or hist_ramp_is_short(rot, base, trained)


def hist_ramp_is_short(rot, base, trained):
    """The ramp is cut off at the first or the last pair."""
    at = lambda turns: rot * np.log(trained / (2 * np.pi * turns)) / (2 * np.log(base))
    return at(32.0) < 0 or at(1.0) > rot // 2 - 1


@pytest.mark.parametrize("kw,code", [
    (dict(rot_dim=0), INV), (dict(rot_dim=-16), INV), (dict(rot_dim=24), UNS), (dict(rot_dim=144), UNS), (dict(base=1.0), INV),
    (dict(base=float("nan")), INV), (dict(base=float("inf")), INV), (dict(scaling=4), INV), (dict(scaling=-1), INV),
    (dict(scaling=1, factor=0.5), INV), (dict(scaling=1, factor=float("nan")), INV), (dict(scaling=3, factor=2.0), INV),
    (dict(scaling=3, factor=2.0, trained=100, fast=1.0, slow=1.0), INV), (dict(scaling=3, factor=2.0, trained=100, slow=0.0), INV),
    (dict(scaling=3, factor=2.0, trained=100, slow=-1.0), INV), (dict(scaling=3, factor=2.0, trained=100, fast=float("inf")), INV),
])
def test_frequency_refusals(kw, code):
    a = dict(rot_dim=64)
    a.update(kw)
    refused(gdpa.gdpa_rope_freqs, code, **a)


# ---------------------------------------------------------------- the 64-bit forms themselves

def test_the_rotation_form_turns_pairs():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((7, 2, 32))
    f = hist.frequencies(16)[0]
    for inter in (False, True):
        y = hist.rope(x, [0, 3, 7], [5, -2], f, inter, 1.5)
        for t, pos in enumerate([5, 6, 7, -2, -1, 0, 1]):
            for i in range(8):
                a, b = (2 * i, 2 * i + 1) if inter else (i, i + 8)
                z = (x[t, :, a] + 1j * x[t, :, b]) * np.exp(1j * pos * f[i]) * 1.5
                assert np.allclose(y[t, :, a], z.real) and np.allclose(y[t, :, b], z.imag)
        assert (y[..., 16:] == x[..., 16:]).all()
        assert np.allclose(hist.rope(y, [0, 3, 7], [5, -2], f, inter, 1 / 1.5, inverse=True), x)


def test_the_weights_form_against_a_padded_softmax():
    """Without earlier weights and with the attention's own logsumexp: the column sums of the softmax maps."""
    x = ref.make(1, 4, 2, 64, 16, [37, 20], [5, 3])
    lse = ref.attend(x, True, 9, 0.125)[1]
    w, _ = hist.weights(x, lse, True, 9, 0.125, 1.0, None)
    for b in range(2):
        k = torch.from_numpy(ref.gather(x, b, x.k_codes, x.k_sf))
        n, new = x.lens[b], x.new[b]
        q = torch.from_numpy(x.q[x.offsets[b]:x.offsets[b + 1]]).unflatten(1, (2, 2))
        s = torch.einsum("ihgd,jhd->hgij", q, k) * 0.125
        pos, j = n - new + torch.arange(new)[:, None], torch.arange(n)
        p = torch.softmax(s.masked_fill((j > pos) | (j <= pos - 9), -torch.inf), -1).sum((1, 2))
        t = np.arange(n)
        assert np.allclose(w[x.table[b, t // 16], :, t % 16], p.T.numpy(), atol=1e-12)


def test_the_evict_form_keeps_what_a_sort_keeps():
    x = ref.make(2, 2, 2, 64, 16, [100, 9], [0, 0], spare=8)
    w = np.random.default_rng(0).random(x.k_codes.shape[:3]).astype(np.float32)
    table = hist.spare_table(x, 40)
    k, v, k_sf, v_sf, w2, kept, lens = hist.evict(x, w, 40, 3, 5, table)
    assert lens.tolist() == [40, 9]
    y = ref.Batch(**{**x.__dict__, "lens": [40, 9], "table": table, "k_codes": k, "k_sf": k_sf})
    for b in range(2):
        t = np.arange(x.lens[b])
        old = w[x.table[b, t // 16], :, t % 16]
        for h in range(2):
            at = kept[b, h, :lens[b]]
            assert (np.diff(at) > 0).all() and set(range(min(3, lens[b]))) <= set(at)
            out = np.setdiff1d(t, at)
            if len(out):
                free = np.setdiff1d(at, np.r_[0:3, x.lens[b] - 5:x.lens[b]])
                assert old[out, h].max() <= old[free, h].min()
            # the kept values are the old ones but for codes that a larger scale cuts: half its last step
            new, was = ref.gather(y, b, k, k_sf)[:, h], ref.gather(x, b, x.k_codes, x.k_sf)[at, h]
            step = np.ldexp(2.0 ** -9, k_sf[table[b, np.arange(lens[b]) // 16], h, np.arange(lens[b]) % 16 // 16].astype(int) - 127)
            assert (np.abs(new - was) <= 2.0 ** -4 * np.abs(was) + step[:, None] / 2).all()
