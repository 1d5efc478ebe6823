"""What the paged cache's Python binding refuses: tensors that the library would misread.  On the CPU: it is told
that host memory is the current device, and the C calls are replaced by one that only counts."""
from __future__ import annotations

import pytest
import torch

from jagged_attention_recommender_gb300 import gdpa

H, HQ, D, T, B, PAGES, WIDTH = 2, 8, 64, 6, 3, 5, 4


class Calls:
    """Stands for the library."""

    def __init__(self):
        self.append = self.fwd = 0

    def gdpa_cache_append(self, *a):
        self.append += 1
        return gdpa.GDPA_OK

    def gdpa_cache_fwd(self, *a):
        self.fwd += 1
        return gdpa.GDPA_OK


@pytest.fixture()
def calls(monkeypatch):
    c = Calls()
    gdpa._device()  # (loads what the binding knows of torch)
    monkeypatch.setattr(gdpa, "_device", lambda: -1)
    monkeypatch.setattr(gdpa, "lib", lambda: c)
    monkeypatch.setattr(gdpa, "_check", lambda code, where: None)
    return c


def cache():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    return gdpa.KvCache(u8(PAGES, H, 32, D), u8(PAGES, H, 32, D), u8(PAGES, H, 2), u8(PAGES, H, 2))


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def append(**kw):
    a = dict(q=bf(T, HQ, D), k=bf(T, H, D), v=bf(T, H, D), offsets=i32(B + 1), kv_lens=i32(B), page_table=i32(B, WIDTH),
             T=T, B=B, Hq=HQ, max_pages=WIDTH, q_out=bf(T, HQ, D))
    a.update(kw)
    for n in "qkv":
        if n + "_stride" not in a:
            a[n + "_stride"] = a[n].stride(0)
    gdpa.gdpa_cache_append(a.pop("cache", None) or cache(), stream=0, **a)


def fwd(**kw):
    a = dict(q=bf(T, HQ, D), offsets=i32(B + 1), kv_lens=i32(B), page_table=i32(B, WIDTH), T=T, B=B, Hq=HQ,
             max_pages=WIDTH, max_q=1, causal=1, window_tokens=0, scale=1.0, out=bf(T, HQ, D), lse=torch.zeros(T, HQ),
             workspace=torch.zeros(64, dtype=torch.uint8))
    a.update(kw)
    if "q_stride" not in a:
        a["q_stride"] = a["q"].stride(0)
    gdpa.gdpa_cache_fwd(a.pop("cache", None) or cache(), stream=0, **a)


def rows(heads):
    """Layouts of T rows of heads of D, with the stride of a row, that the library reads right."""
    n = heads * D
    fused = bf(T, HQ + 2 * H, D)
    yield bf(T, heads, D), n
    yield bf(T + 3, heads, D), n                      # rows to spare
    yield bf(T, n), n                                 # not cut into heads
    yield bf(T * n), n                                # nor into rows
    yield bf(T * heads, D), n
    yield fused[:, 1:1 + heads], (HQ + 2 * H) * D     # some heads of a fused projection
    yield fused.flatten(1)[:, D:D + n], (HQ + 2 * H) * D
    yield bf(T, n + 8)[:, :n].unflatten(1, (heads, D)), n + 8
    yield bf(T, 1, heads, D), n
    yield bf(T, heads, 1, D), n
    yield bf(T // 2, 2, heads, D), n                  # samples of two rows


def test_layouts_that_the_library_reads(calls):
    for t, stride in rows(HQ):
        append(q=t, q_stride=stride)
        fwd(q=t, q_stride=stride)
    for t, stride in rows(H):
        append(k=t, k_stride=stride)
        append(v=t, v_stride=stride)
    append(q=None, q_stride=0)
    one = bf(1, H, 3 * D)[:, :, :D]                   # one head of one row has no layout to get wrong
    append(k=bf(1, H, D), v=bf(1, H, D), q=bf(1, HQ, D), T=1, k_stride=H * D)
    with pytest.raises(ValueError):
        append(k=one, v=bf(1, H, D), q=bf(1, HQ, D), T=1, k_stride=H * D)
    append(T=0, k=bf(0, H, D), v=bf(0, H, D), q=bf(0, HQ, D))
    assert calls.append and calls.fwd


def wrong(heads):
    """Layouts that it would misread."""
    n = heads * D
    yield bf(T, heads, 3 * D)[:, :, :D], heads * 3 * D            # heads further apart than D
    yield bf(T, heads, 3 * D)[:, :, D:2 * D], heads * 3 * D
    yield bf(T, heads, 2 * D)[:, :, ::2], heads * 2 * D           # coordinates that are not adjacent
    yield bf(T, D, heads).transpose(1, 2), n                      # coordinates outermost in a row
    yield bf(heads, T, D).transpose(0, 1), n                      # rows inside heads
    yield bf(heads, T, D), T * D
    yield bf(T // 2, heads, 2, D), n * 2                          # samples of two rows, heads outermost
    yield bf(T, heads, D), n + 8                                  # another stride than its own
    yield bf(2 * T, heads, D)[::2], n
    yield bf(T - 1, heads, D), n                                  # too few rows
    yield bf(T * n - 1), n
    yield bf(T, heads // 2, D), n
    yield bf(T, heads, D // 2), n


@pytest.mark.parametrize("i", range(13))
def test_layouts_that_it_would_misread(calls, i):
    t, stride = list(wrong(HQ))[i]
    for call in (append, fwd):
        with pytest.raises(ValueError, match="rows of"):
            call(q=t, q_stride=stride)
    t, stride = list(wrong(H))[i]
    for name in "kv":
        with pytest.raises(ValueError, match="rows of"):
            append(**{name: t, name + "_stride": stride})
    assert calls.append == calls.fwd == 0


def test_tensors_that_are_too_small_for_the_call(calls):
    short = dict(offsets=i32(B), kv_lens=i32(B - 1), page_table=i32(B - 1, WIDTH))
    for name, t in short.items():
        for call in (append, fwd):
            with pytest.raises(ValueError, match="elements or more"):
                call(**{name: t})
    with pytest.raises(ValueError, match="elements or more"):
        append(q_out=bf(T, HQ - 1, D))
    for kw in (dict(out=bf(T - 1, HQ, D)), dict(lse=torch.zeros(T, HQ - 1)), dict(workspace_bytes=65)):
        with pytest.raises(ValueError, match="elements or more"):
            fwd(**kw)
    for call in (append, fwd):  # rows wider or narrower than max_pages: another sequence's pages would be read
        for width in (WIDTH - 1, WIDTH + 2):
            with pytest.raises(ValueError, match="entries a row|elements or more"):
                call(page_table=i32(2 * B, width))
    assert calls.append == calls.fwd == 0


def test_tensors_with_room_to_spare(calls):
    more = dict(offsets=i32(B + 9), kv_lens=i32(B + 8), page_table=i32(B + 8, WIDTH))
    append(q_out=bf(T + 2, HQ, D), **more)
    append(page_table=i32(B * WIDTH))
    append(q=None, q_stride=0, q_out=bf(0))
    fwd(out=bf(T + 2, HQ, D), lse=torch.zeros(T + 2, HQ), **more)
    fwd(lse=None, workspace_bytes=60)
    fwd(page_table=i32(1, WIDTH + 3), B=1)  # one sequence: its row may be wider
    for kw in (dict(T=0), dict(B=0)):  # nothing to do
        append(offsets=i32(0), kv_lens=i32(0), page_table=i32(0), q_out=bf(0), **kw)
        fwd(offsets=i32(0), kv_lens=i32(0), page_table=i32(0), out=bf(0), lse=torch.zeros(0), **kw)
    assert calls.append == 5 and calls.fwd == 5


def test_a_cache_on_another_device_than_the_current_one(calls, monkeypatch):
    """Codes of one device must not be read by a launch on another, whatever the other tensors are."""
    c = cache()
    bare = dict(q=1 << 20, k=1 << 20, v=1 << 20, offsets=1 << 20, kv_lens=1 << 20, page_table=1 << 20, q_stride=HQ * D)
    monkeypatch.setattr(gdpa, "_device", lambda: 1)
    with pytest.raises(ValueError, match="current CUDA device"):
        append(cache=c, q_out=1 << 20, k_stride=H * D, v_stride=H * D, **bare)
    del bare["k"], bare["v"]
    with pytest.raises(ValueError, match="current CUDA device"):
        fwd(cache=c, out=1 << 20, lse=None, workspace=1 << 20, workspace_bytes=64, **bare)
    assert calls.append == calls.fwd == 0
