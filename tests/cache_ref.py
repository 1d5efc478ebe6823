"""Plain 64-bit forms of the paged cache's two operators (numpy, sequence by sequence), and random batches for them."""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

BLOCK = 16
NAN_CODE = 0x7F


def e4m3_values(codes) -> np.ndarray:
    """float64 values of e4m3 codes."""
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    ex, m = (c >> 3) & 15, c & 7
    v = np.where(ex > 0, np.ldexp(1.0 + m / 8.0, ex - 7), np.ldexp(m / 8.0, -6))
    v = np.where((c & 0x7F) == NAN_CODE, np.nan, v)
    return np.where(c & 0x80, -v, v)


_TABLE = e4m3_values(np.arange(0x7F))  # the magnitudes, increasing


def e4m3_codes(x) -> np.ndarray:
    """Nearest e4m3 codes, ties to even; what is not finite becomes NaN.  |x| <= 448 is expected."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.clip(np.searchsorted(_TABLE, a), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    up, down = _TABLE[hi] - a, a - _TABLE[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    c = np.where(a >= _TABLE[0x7E], 0x7E, c) | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isfinite(x), c, NAN_CODE).astype(np.uint8)


def block_exponent(amax: float) -> int:
    """The smallest integer e >= -127 with amax <= 448 2^e."""
    if amax == 0:
        return -127
    e = int(np.ceil(np.log2(amax / 448.0)))
    while amax <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return max(e, -127)


def rotate(x, pos, inv_freq, interleaved) -> np.ndarray:
    """x [n, H, D] float64 at positions pos [n]."""
    y = np.array(x, dtype=np.float64)
    if inv_freq is None:
        return y
    r = 2 * len(inv_freq)
    a, b = (np.s_[..., 0:r:2], np.s_[..., 1:r:2]) if interleaved else (np.s_[..., :r // 2], np.s_[..., r // 2:r])
    ang = (np.asarray(pos, dtype=np.float64)[:, None] * inv_freq)[:, None]
    c, s = np.cos(ang), np.sin(ang)
    y[a], y[b] = x[a] * c - x[b] * s, x[b] * c + x[a] * s
    return y


@dataclasses.dataclass
class Batch:
    """Host arrays of one batch: the cache, its table and the new tokens (float64 values of bf16 numbers)."""
    Hq: int
    H: int
    D: int
    P: int
    lens: list
    new: list
    k_codes: np.ndarray
    v_codes: np.ndarray
    k_sf: np.ndarray
    v_sf: np.ndarray
    table: np.ndarray
    offsets: np.ndarray
    q: np.ndarray
    k: np.ndarray
    v: np.ndarray

    @property
    def T(self):
        return int(self.offsets[-1])


def bf16(x) -> np.ndarray:
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).double().numpy()


def make(seed, Hq, H, D, P, lens, new, held=None, spare=2, jitter=3, spread=1.0) -> Batch:
    """Random values in the first held[b] tokens of each sequence (default: all lens[b]); NaN codes and NaN scales
    everywhere else, so that whatever reads there shows."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    held = list(lens) if held is None else held
    pages = [-(-n // P) for n in lens]
    num = sum(pages) + spare
    shape = (num, H, P, D)
    order = rng.permutation(num).astype(np.int32)
    width = max(1, max(pages, default=1)) + 1
    table = np.full((B, width), -7, np.int32)
    codes = [np.full(shape, NAN_CODE, np.uint8) for _ in range(2)]
    sf = [np.full((num, H, P // BLOCK), 255, np.uint8) for _ in range(2)]
    at = 0
    for b in range(B):
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += pages[b]
        for c, f in zip(codes, sf):
            for i in range(pages[b]):
                n = min(P, held[b] - i * P)
                if n <= 0:
                    break
                pg = table[b, i]
                c[pg, :, :n] = e4m3_codes(np.clip(rng.standard_normal((H, n, D)) * 100, -448, 448))
                f[pg, :, :-(-n // BLOCK)] = rng.integers(120 - jitter, 121 + jitter, (H, -(-n // BLOCK)))
    offsets = np.zeros(B + 1, np.int32)
    offsets[1:] = np.cumsum(new)
    T = int(offsets[-1])
    q, k, v = (bf16(rng.standard_normal((T, h, D)) * spread) for h in (Hq, H, H))
    return Batch(Hq, H, D, P, list(lens), list(new), codes[0], codes[1], sf[0], sf[1], table, offsets, q, k, v)


def append(x: Batch, inv_freq, interleaved):
    """Rotated q, and for k and v: codes, scales (after the append), the new tokens' values before their rounding
    (float64 [pages, H, P, D], NaN elsewhere) and how near the largest rotated value of a block is to a border of its
    exponent."""
    q = np.array(x.q)
    rot = 0 if inv_freq is None else 2 * len(inv_freq)
    res = []
    for which, codes, sf in (("k", x.k_codes.copy(), x.k_sf.copy()), ("v", x.v_codes.copy(), x.v_sf.copy())):
        val = np.full(codes.shape, np.nan)
        near = np.inf
        for b, (n, new) in enumerate(zip(x.lens, x.new)):
            rows = np.s_[x.offsets[b]:x.offsets[b + 1]]
            pos = np.arange(n - new, n)
            if which == "k":
                q[rows] = rotate(x.q[rows], pos, inv_freq, interleaved)
                y = rotate(x.k[rows], pos, inv_freq, interleaved)
            else:
                y = x.v[rows]
            for j in range((n - new) // BLOCK, -(-n // BLOCK)) if new else ():
                t0, t1 = max(j * BLOCK, n - new), min((j + 1) * BLOCK, n)
                page, s0 = x.table[b, t0 // x.P], j * BLOCK % x.P
                held = t0 - j * BLOCK
                for h in range(x.H):
                    z = y[t0 - (n - new):t1 - (n - new), h]
                    amax = np.abs(np.where(np.isfinite(z), z, 0)).max()
                    e = block_exponent(amax)
                    turned = np.abs(np.where(np.isfinite(z), z, 0))[:, :rot].max(initial=0)
                    if turned > 0:  # the other coordinates are exact: they decide the same exponent on both sides
                        near = min(near, abs(turned / (448 * 2.0 ** e) - 1), abs(turned / (224 * 2.0 ** e) - 1))
                    if held:
                        e0 = int(sf[page, h, s0 // BLOCK]) - 127
                        if e > e0:
                            old = codes[page, h, s0:s0 + held]
                            codes[page, h, s0:s0 + held] = e4m3_codes(e4m3_values(old) * 2.0 ** (e0 - e))
                        e = max(e, e0)
                    sf[page, h, s0 // BLOCK] = e + 127
                    at = np.s_[page, h, s0 + held:s0 + held + len(z)]
                    codes[at] = e4m3_codes(z * 2.0 ** -e)
                    val[at] = z
        res.append((codes, sf, val, near))
    return q, res[0], res[1]


def gather(x: Batch, b, codes, sf):
    """float64 [len, H, D] of sequence b."""
    n = x.lens[b]
    t = np.arange(n)
    page, slot = x.table[b, t // x.P], t % x.P
    return e4m3_values(codes[page, :, slot]) * np.ldexp(1.0, sf[page, :, slot // BLOCK].astype(np.int64) - 127)[..., None]


def seen(n, new, i, causal, window):
    pos = n - new + i
    return (max(0, pos - window + 1) if window else 0), (max(0, min(n, pos + 1)) if causal else n)


def attend(x: Batch, causal, window, scale, q=None):
    """out [T, Hq, D], lse [T, Hq], sum p |v| / sum p [T, Hq, D] and the largest scale sum |q k| [T, Hq]."""
    q = x.q if q is None else q
    G = x.Hq // x.H
    out = np.zeros((x.T, x.Hq, x.D))
    mag = np.zeros_like(out)
    lse = np.full((x.T, x.Hq), -np.inf)
    big = np.zeros((x.T, x.Hq))
    for b in range(len(x.lens)):
        if not x.new[b]:
            continue
        k, v = gather(x, b, x.k_codes, x.k_sf), gather(x, b, x.v_codes, x.v_sf)
        for i in range(x.new[b]):
            j0, j1 = seen(x.lens[b], x.new[b], i, causal, window)
            if j1 <= j0:
                continue
            r = x.offsets[b] + i
            for h in range(x.H):
                qq = q[r, h * G:(h + 1) * G]
                kk, vv = k[j0:j1, h], v[j0:j1, h]
                s = scale * (qq @ kk.T)
                m = s.max(-1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(-1, keepdims=True)
                out[r, h * G:(h + 1) * G] = p @ vv / l
                mag[r, h * G:(h + 1) * G] = p @ np.abs(vv) / l
                lse[r, h * G:(h + 1) * G] = (np.log(l) + m)[:, 0]
                big[r, h * G:(h + 1) * G] = (abs(scale) * (np.abs(qq) @ np.abs(kk).T)).max(-1)
    return out, lse, mag, big


def attend_bounds(x: Batch, out, lse, mag, big):
    """How far a result may be off.  A score is a sum of D products in fp32, in any order and grouping: off by at
    most d = (D + 8) 2^-23 times the sum of their magnitudes (2^-23, not 2^-24: the tensor core may cut where others
    round); exp2 adds 2^-21 (its own 2^-22 and its argument's rounding for the few units it spans here).  A weight is
    then off by a factor 1 +- d, and its rounding to fp16 adds 2^-11: both move a weighted mean by at most their size
    times sum p |v| / sum p (twice for d: numerator and sum).  The result is rounded to bf16: 2^-8 of it."""
    w = 2.0 ** -11
    d = (x.D + 8) * 2.0 ** -23 * big + 2.0 ** -21
    tol = 2.0 ** -8 * np.abs(out) + (w + 2 * d[..., None]) * mag * 1.01 + 1e-38
    return tol, np.where(np.isfinite(lse), d + 2.0 ** -22 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0))), 0)
