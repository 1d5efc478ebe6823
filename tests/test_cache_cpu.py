"""The paged cache's argument checks (all before any CUDA call), and the tests' own 64-bit forms."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

from jagged_attention_recommender_gb300 import build as gbuild
from jagged_attention_recommender_gb300 import gdpa
from tests import cache_ref as ref

A = 1 << 20  # an aligned address that no refused call may touch
INV = gdpa.GDPA_ERR_INVALID_ARG
UNS = gdpa.GDPA_ERR_UNSUPPORTED
MEM = gdpa.GDPA_ERR_NO_MEMORY


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()
    yield


class Desc:
    """A descriptor over bare addresses."""

    def __init__(self, **kw):
        self.freq = np.ones(64)
        d = dict(k_codes=A, v_codes=A, k_sf=A, v_sf=A, num_pages=4, page_tokens=64, H=2, D=128,
                 inv_freq=self.freq.ctypes.data, rot_dim=128, rope_style=0)
        if "freq" in kw:
            self.freq[:] = kw.pop("freq")
        d.update(kw)
        self.desc = gdpa._CacheDesc(**d)
        self.addr = ctypes.addressof(self.desc)


class Null:
    addr = None


def append(cache, **kw):
    a = dict(q=A, q_stride=1024, k=A, k_stride=256, v=A, v_stride=256, offsets=A, kv_lens=A, page_table=A, T=4, B=2,
             Hq=8, max_pages=3, q_out=A)
    a.update(kw)
    gdpa.gdpa_cache_append(cache, stream=0, **a)


def fwd(cache, **kw):
    a = dict(q=A, q_stride=1024, offsets=A, kv_lens=A, page_table=A, T=4, B=2, Hq=8, max_pages=3, max_q=1, causal=1,
             window_tokens=0, scale=1.0, out=A, lse=None, workspace=A, workspace_bytes=1 << 40)
    a.update(kw)
    gdpa.gdpa_cache_fwd(cache, stream=0, **a)


BAD_DESC = [
    (dict(D=96), UNS), (dict(D=256), UNS), (dict(page_tokens=8), UNS), (dict(page_tokens=48), UNS),
    (dict(page_tokens=2048), UNS), (dict(page_tokens=0), INV), (dict(page_tokens=-64), INV), (dict(H=0), INV),
    (dict(H=-1), INV), (dict(H=1 << 14), UNS), (dict(num_pages=-1), INV), (dict(k_codes=None), INV),
    (dict(v_codes=A + 8), INV), (dict(k_sf=None), INV), (dict(k_sf=A + 2), INV), (dict(v_sf=A + 1), INV), (dict(v_sf=None), INV), (dict(rot_dim=-16), INV),
    (dict(rot_dim=144), INV), (dict(rot_dim=24), UNS), (dict(inv_freq=None), INV), (dict(rope_style=2), INV),
    (dict(freq=math.nan), INV), (dict(freq=math.inf), INV),
]


@pytest.mark.parametrize("kw,code", BAD_DESC)
def test_bad_descriptors_are_refused(kw, code):
    for call in (append, fwd, lambda c: gdpa.gdpa_cache_workspace_size(c, 8, 1)):
        with pytest.raises(gdpa.GdpaError) as e:
            call(Desc(**kw))
        assert e.value.code == code
    for call in (append, fwd, lambda c: gdpa.gdpa_cache_workspace_size(c, 8, 1)):
        with pytest.raises(gdpa.GdpaError) as e:
            call(Null())
        assert e.value.code == INV


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INV), (dict(B=-1), INV), (dict(max_pages=-1), INV), (dict(max_pages=0), INV), (dict(T=1 << 31), UNS),
    (dict(max_pages=1 << 25), UNS), (dict(Hq=0), INV), (dict(Hq=1 << 14), UNS), (dict(k=None), INV),
    (dict(v=None), INV), (dict(k=A + 2), INV), (dict(v=A + 8), INV), (dict(q=A + 8), INV), (dict(q_out=None), INV),
    (dict(q_out=A + 4), INV), (dict(k_stride=255), INV), (dict(v_stride=248), INV), (dict(q_stride=1016), INV),
    (dict(k_stride=260), UNS), (dict(q_stride=1025), UNS), (dict(offsets=None), INV), (dict(kv_lens=None), INV),
    (dict(page_table=None), INV)])
def test_append_refuses(kw, code):
    with pytest.raises(gdpa.GdpaError) as e:
        append(Desc(), **kw)
    assert e.value.code == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INV), (dict(B=-1), INV), (dict(max_pages=0), INV), (dict(T=1 << 31), UNS), (dict(T=1 << 29), UNS),
    (dict(max_pages=1 << 25), UNS), (dict(Hq=0), INV), (dict(Hq=7), INV), (dict(Hq=1 << 14), UNS), (dict(max_q=0), INV),
    (dict(causal=2), INV), (dict(causal=-1), INV), (dict(window_tokens=-1), INV),
    (dict(causal=0, window_tokens=5), INV), (dict(scale=math.nan), INV), (dict(scale=math.inf), INV),
    (dict(q=None), INV), (dict(q=A + 8), INV), (dict(q_stride=1016), INV), (dict(q_stride=1028), UNS),
    (dict(out=None), INV), (dict(out=A + 8), INV), (dict(lse=A + 2), INV), (dict(offsets=None), INV),
    (dict(kv_lens=None), INV), (dict(page_table=None), INV), (dict(workspace=None), INV),
    (dict(workspace=A + 8), INV)])
def test_fwd_refuses(kw, code):
    with pytest.raises(gdpa.GdpaError) as e:
        fwd(Desc(), **kw)
    assert e.value.code == code


def test_empty_calls_do_nothing():
    append(Desc(), T=0)
    append(Desc(), B=0)
    append(Desc(num_pages=0, k_codes=None, v_codes=None, k_sf=None, v_sf=None), T=0)
    fwd(Desc(), T=0, workspace_bytes=0)
    fwd(Desc(), B=0, workspace_bytes=0)


@pytest.mark.parametrize("Hq,max_q", [(0, 1), (7, 1), (8, 0), (8, -1)])
def test_workspace_size_refuses(Hq, max_q):
    with pytest.raises(gdpa.GdpaError) as e:
        gdpa.gdpa_cache_workspace_size(Desc(), Hq, max_q)
    assert e.value.code == INV
    assert gdpa.lib().gdpa_cache_workspace_size(Desc().addr, 8, 1, None) == INV


def test_the_binding_refuses_tensors_of_another_kind():
    f = torch.zeros(8, 128)
    with pytest.raises(TypeError):
        append(Desc(), k=f)
    with pytest.raises(ValueError):  # host memory
        append(Desc(), k=f.to(torch.bfloat16))
    with pytest.raises(TypeError):
        fwd(Desc(), offsets=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        fwd(Desc(), lse=f.double())
    codes, sf = torch.zeros(2, 1, 16, 64, dtype=torch.uint8), torch.zeros(2, 1, 1, dtype=torch.uint8)
    with pytest.raises(ValueError):  # host memory
        gdpa.KvCache(codes, codes, sf, sf)
    with pytest.raises(ValueError):  # another shape
        gdpa.KvCache(codes, codes, sf, sf[:1])
    with pytest.raises(ValueError):  # not contiguous
        gdpa.KvCache(codes.transpose(1, 2), codes, sf, sf)


def test_reference_codes_are_torch_s():
    x = np.concatenate([np.linspace(-448, 448, 4001), np.ldexp(1.0, np.arange(-14, 9)), ref.e4m3_values(np.arange(127)),
                        (ref._TABLE[1:] + ref._TABLE[:-1]) / 2, -(ref._TABLE[1:] + ref._TABLE[:-1]) / 2])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = ref.e4m3_codes(x.astype(np.float32))
    assert np.array_equal(got, want)
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3_values(np.arange(256)), v, equal_nan=True)


def test_reference_exponent():
    for e in (-127, -60, -3, 0, 5, 100):
        assert ref.block_exponent(448 * 2.0 ** e) == e
        assert ref.block_exponent(449 * 2.0 ** e) == e + 1
        assert ref.block_exponent(225 * 2.0 ** e) == e
    assert ref.block_exponent(0.0) == -127
    assert ref.block_exponent(1e-45) == -127
