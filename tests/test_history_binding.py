"""What the Python binding of the operators for long histories refuses: tensors that the library would misread.  On
the CPU, as tests/test_cache_binding.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from jagged_attention_recommender_gb300 import gdpa
from tests.test_cache_binding import B, D, H, HQ, PAGES, T, WIDTH, bf, cache, i32, rows, wrong


class Calls:
    """Stands for the library."""

    def __init__(self):
        self.n = 0

    def _count(self, *a):
        self.n += 1
        return gdpa.GDPA_OK

    gdpa_cache_weights = gdpa_cache_evict = gdpa_rope = _count


@pytest.fixture()
def calls(monkeypatch):
    c = Calls()
    gdpa._device()  # (loads what the binding knows of torch)
    monkeypatch.setattr(gdpa, "_device", lambda: -1)
    monkeypatch.setattr(gdpa, "lib", lambda: c)
    monkeypatch.setattr(gdpa, "_check", lambda code, where: None)
    return c


def f32(*s):
    return torch.zeros(s, dtype=torch.float32)


def weights(**kw):
    a = dict(q=bf(T, HQ, D), lse=f32(T, HQ), offsets=i32(B + 1), kv_lens=i32(B), page_table=i32(B, WIDTH), T=T, B=B, Hq=HQ,
             max_pages=WIDTH, max_q=1, causal=1, window_tokens=0, scale=1.0, decay=1.0, weights_in=f32(PAGES, H, 32),
             weights=f32(PAGES, H, 32))
    a.update(kw)
    if "q_stride" not in a:
        a["q_stride"] = a["q"].stride(0)
    gdpa.gdpa_cache_weights(a.pop("cache", None) or cache(), stream=0, **a)


def evict(**kw):
    a = dict(weights=f32(PAGES, H, 32), kv_lens=i32(B), page_table=i32(B, WIDTH), B=B, max_pages=WIDTH, budget=40, sink=1, recent=2,
             new_table=i32(B, 2), new_max_pages=2, kept=i32(B, H, 40), new_lens=i32(B))
    a.update(kw)
    gdpa.gdpa_cache_evict(a.pop("cache", None) or cache(), stream=0, **a)


def rope(**kw):
    a = dict(x=bf(T, HQ, D), offsets=i32(B + 1), first=i32(B), T=T, B=B, H=HQ, D=D, inv_freq=np.ones(D // 2), rope_style=0,
             magnitude=1.0, inverse=0, y=bf(T, HQ, D))
    a.update(kw)
    for n in "xy":
        if n + "_stride" not in a:
            a[n + "_stride"] = a[n].stride(0)
    gdpa.gdpa_rope(stream=0, **a)


def test_layouts_that_the_library_reads(calls):
    for t, stride in rows(HQ):
        weights(q=t, q_stride=stride)
        rope(x=t, x_stride=stride)
        rope(y=t, y_stride=stride)
    weights(weights_in=None)
    weights(weights=f32(PAGES * H * 32 + 5), lse=f32(T + 1, HQ))
    evict(kept=i32(B * H * 40), page_table=i32(B * WIDTH), new_lens=i32(B + 3))
    rope(first=None, inv_freq=None)
    rope(inv_freq=[1.0] * 16)
    weights(T=0, lse=f32(0), offsets=i32(0), kv_lens=i32(0), page_table=i32(0))
    evict(B=0, kv_lens=i32(0), page_table=i32(0), new_table=i32(0), kept=i32(0), new_lens=i32(0))
    assert calls.n == 3 * len(list(rows(HQ))) + 7


@pytest.mark.parametrize("i", range(13))
def test_layouts_that_it_would_misread(calls, i):
    t, stride = list(wrong(HQ))[i]
    for call, name in ((weights, "q"), (rope, "x"), (rope, "y")):
        with pytest.raises(ValueError, match="rows of"):
            call(**{name: t, name + "_stride": stride})
    assert calls.n == 0


@pytest.mark.parametrize("call,kw", [
    (weights, dict(lse=f32(T, HQ - 1))), (weights, dict(offsets=i32(B))), (weights, dict(kv_lens=i32(B - 1))),
    (weights, dict(page_table=i32(B - 1, WIDTH))), (weights, dict(page_table=i32(B, WIDTH + 1))),
    (weights, dict(weights=f32(PAGES, H, 31))), (weights, dict(weights_in=f32(PAGES - 1, H, 32))),
    (weights, dict(weights=f32(PAGES, 32, H).transpose(1, 2))),
    (evict, dict(weights=f32(PAGES, H, 16))), (evict, dict(kv_lens=i32(B - 1))), (evict, dict(page_table=i32(B, WIDTH + 1))),
    (evict, dict(new_table=i32(B, 3))), (evict, dict(new_table=i32(1, 2))), (evict, dict(kept=i32(B, H, 39))),
    (evict, dict(kept=i32(B, 40, H).transpose(1, 2))), (evict, dict(new_lens=i32(B - 1))),
    (rope, dict(offsets=i32(B))), (rope, dict(first=i32(B - 1))), (rope, dict(offsets=i32(2 * B + 2)[::2])),
])
def test_tensors_that_are_too_small_or_not_contiguous(calls, call, kw):
    with pytest.raises(ValueError):
        call(**kw)
    assert calls.n == 0


@pytest.mark.parametrize("call,kw", [
    (weights, dict(q=f32(T, HQ, D))), (weights, dict(lse=bf(T, HQ))), (weights, dict(weights=bf(PAGES, H, 32))),
    (weights, dict(weights_in=torch.zeros(PAGES, H, 32, dtype=torch.float64))), (weights, dict(kv_lens=i32(B).long())),
    (evict, dict(kept=i32(B, H, 40).long())), (evict, dict(weights=bf(PAGES, H, 32))), (evict, dict(new_lens=f32(B))),
    (rope, dict(x=f32(T, HQ, D))), (rope, dict(y=bf(T, HQ, D).half())), (rope, dict(first=i32(B).long())),
])
def test_other_types(calls, call, kw):
    with pytest.raises(TypeError):
        call(**kw)
    assert calls.n == 0


def test_tensors_and_caches_on_another_device(calls, monkeypatch):
    c = cache()
    monkeypatch.setattr(gdpa, "_device", lambda: 1)
    for call in (lambda: weights(cache=c), lambda: evict(cache=c), rope):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
    assert calls.n == 0
