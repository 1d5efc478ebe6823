"""Plain 64-bit forms of the operators for long histories (numpy, sequence by sequence): rotary positions of jagged
rows, the attention weight that stored keys receive, and the cache's eviction by it."""
from __future__ import annotations

import numpy as np

from tests import cache_ref as ref

BLOCK = ref.BLOCK


def frequencies(rot, base=10000.0, scaling=0, factor=1.0, trained=0, fast=32.0, slow=1.0):
    """(radians per position of each pair, magnitude)."""
    if scaling == 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-np.arange(0, rot, 2) / rot)
    if scaling == 1:
        return f / factor, 1.0
    if scaling != 3:
        return f, 1.0
    # the (real) index of the pair that turns so often over the trained context
    index = lambda turns: rot * np.log(trained / (2 * np.pi * turns)) / (2 * np.log(base))
    lo, hi = max(np.floor(index(fast)), 0), min(np.ceil(index(slow)), rot - 1)
    ramp = np.array([min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(rot // 2)])
    return f / factor * ramp + f * (1 - ramp), 0.1 * np.log(factor) + 1


def rope(x, offsets, first, inv_freq, interleaved, magnitude=1.0, inverse=False):
    """x [T, H, D] float64; rows behind the last sequence come back as NaN."""
    y = np.full(x.shape, np.nan)
    r = 0 if inv_freq is None else 2 * len(inv_freq)
    for b in range(len(offsets) - 1):
        rows = np.s_[offsets[b]:offsets[b + 1]]
        pos = np.arange(offsets[b + 1] - offsets[b], dtype=np.float64) + (0 if first is None else int(first[b]))
        y[rows] = ref.rotate(x[rows], pos, None if not r else np.asarray(inv_freq) * (-1 if inverse else 1), interleaved)
        y[rows][..., :r] *= magnitude
    return y


def weights(x: ref.Batch, lse, causal, window, scale, decay, w_in, q=None):
    """Weights [num_pages, H, P] (NaN where nothing is written) and how far each may be off.

    A score is off by d (tests/cache_ref.py: attend_bounds) and by what the rounding of a query to fp16 adds (2^-25 of
    the row's largest element, each); the argument of exp2 is a difference of two products, each rounded, and 2^x itself
    is off by 2^-22: (3 + |s| + |lse|) 2^-23 log2(e) and 2^-22, twice for room.  A sum of N positive terms is off
    by N 2^-24 of itself, an earlier weight by 2^-23."""
    q = x.q if q is None else q
    G = x.Hq // x.H
    out = np.full(x.k_codes.shape[:3], np.nan)
    tol = np.zeros_like(out)
    for b, (n, new) in enumerate(zip(x.lens, x.new)):
        if not new or not n:
            continue
        k = ref.gather(x, b, x.k_codes, x.k_sf)
        t = np.arange(n)
        page, slot = x.table[b, t // x.P], t % x.P
        w, e = np.zeros((n, x.H)), np.zeros((n, x.H))
        if w_in is not None:
            old = max(0, n - new)
            w[:old] = np.float64(np.float32(decay)) * w_in[page[:old], :, slot[:old]]
            e[:old] = 2.0 ** -23 * np.abs(w[:old])
        for i in range(new):
            j0, j1 = ref.seen(n, new, i, causal, window)
            r = x.offsets[b] + i
            for hq in range(x.Hq if j1 > j0 else 0):
                if lse[r, hq] == -np.inf:
                    continue
                kk, qq = k[j0:j1, hq // G], q[r, hq]
                s = scale * (kk @ qq)
                with np.errstate(over="ignore", invalid="ignore"):
                    p = np.exp(s - lse[r, hq])
                    d = (x.D + 8) * 2.0 ** -23 * abs(scale) * (np.abs(kk) @ np.abs(qq))
                    d = d + 2.0 ** -25 * np.abs(qq).max() * abs(scale) * np.abs(kk).sum(-1)
                    d = d + 2 * (2.0 ** -22 + 1.5 * 2.0 ** -23 * (3 + np.abs(s) + abs(lse[r, hq])))
                    w[j0:j1, hq // G] += p
                    e[j0:j1, hq // G] += p * np.expm1(np.minimum(d, 50))
        out[page, :, slot] = w
        tol[page, :, slot] = e + (new * G + 2) * 2.0 ** -23 * np.abs(w) + 1e-37
    return out, tol


def evict(x: ref.Batch, w, budget, sink, recent, new_table):
    """Codes and scales of K and V, weights, kept [B, H, budget] (-1 behind the kept ones) and new lengths."""
    k, v, k_sf, v_sf, w_out = (a.copy() for a in (x.k_codes, x.v_codes, x.k_sf, x.v_sf, w))
    B = len(x.lens)
    kept = np.full((B, x.H, budget), -1, np.int32)
    lens = np.array([min(n, budget) for n in x.lens], np.int32)
    for b, n in enumerate(x.lens):
        t = np.arange(n)
        page, slot = x.table[b, t // x.P], t % x.P
        for h in range(x.H if n else 0):
            always = (t < sink) | (t >= n - recent)
            old = w[page, h, slot].astype(np.float64)
            # the always kept first, then by weight (NaN last), equal ones in their order
            order = sorted(range(n), key=lambda j: (not always[j], bool(np.isnan(old[j])), 0.0 if np.isnan(old[j]) else -old[j], j))
            at = np.sort(np.array(order[:lens[b]], np.int64))
            kept[b, h, :lens[b]] = at
            i = np.arange(lens[b])
            to, ts = new_table[b, i // x.P], i % x.P
            w_out[to, h, ts] = w[page[at], h, slot[at]]
            for codes, sf, c0, f0 in ((k, k_sf, x.k_codes, x.k_sf), (v, v_sf, x.v_codes, x.v_sf)):
                for i0 in range(0, lens[b], BLOCK):
                    src = at[i0:i0 + BLOCK]
                    e = f0[page[src], h, slot[src] // BLOCK].astype(np.int64)
                    sf[to[i0], h, ts[i0] // BLOCK] = e.max()
                    for m, j in enumerate(src):
                        c = c0[page[j], h, slot[j]]
                        if e[m] < e.max():
                            c = ref.e4m3_codes(ref.e4m3_values(c) * 2.0 ** float(e[m] - e.max()))
                        codes[to[i0 + m], h, ts[i0 + m]] = c
    return k, v, k_sf, v_sf, w_out, kept, lens


def spare_table(x: ref.Batch, budget, seed=3):
    """A table of pages that no sequence uses, wide enough for `budget` tokens (x needs enough spare ones)."""
    need = [-(-min(n, budget) // x.P) for n in x.lens]
    used = {int(x.table[b, i]) for b, n in enumerate(x.lens) for i in range(-(-n // x.P))}
    free = np.random.default_rng(seed).permutation([p for p in range(x.k_codes.shape[0]) if p not in used])
    width = max(1, max(need, default=0), -(-min(budget, x.table.shape[1] * x.P) // x.P))
    table = np.full((len(x.lens), width), -5, np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = free[at:at + m]
        at += m
    return table


def pages_for(lens, P, budget):
    return sum(-(-min(n, budget) // P) for n in lens)
