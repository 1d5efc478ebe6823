"""Operators for long histories: rotary positions of jagged rows (and their gradient), the attention weight that each
key of the paged cache has received, and the cache's eviction by it.

The cache holds keys and values as e4m3 codes, one power-of-two scale for each block of 16 tokens and head.  ``own``
false computes the operators in plain torch operations in 32 bits (angles in 64); ``own`` true calls this repository's
library.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16  # tokens of a scale block


def _rope(name, **kw):
    c = dict(op="rope", name=name, lo=1, hi=1, first=0, heads_of=0, interleaved=False, scaled=1.0, inverse=False)
    c.update(kw)
    return c


def _weights(name, **kw):
    c = dict(op="weights", name=name, window=0, causal=True, decay=1.0)
    c.update(kw)
    return c


def _evict(name, **kw):
    c = dict(op="evict", name=name)
    c.update(kw)
    return c


def listed():
    """Rope: lo, hi: rows of a sequence; first: the largest first position; heads_of: heads of the fused row that the
    rotated ones lie in (0: rows of their own); scaled: the context's extension.  Cache: lo, hi: tokens of a sequence;
    new_lo, new_hi: rows of a sequence; page: tokens of a page."""
    return [
        # one decoding step of four sequences whose caches were cut (positions are no lengths): launch latency
        _rope("rope_few", B=4, H=10, D=64, rot=64, first=900),
        # queries and keys of a training batch, side by side in the fused projection's rows
        _rope("rope_train", B=128, H=8, D=128, rot=128, lo=100, hi=4096, heads_of=12),
        # the gradient on its way back into the fused projection's rows
        _rope("rope_grad", B=128, H=8, D=128, rot=128, lo=100, hi=4096, heads_of=12, inverse=True),
        # pieces of far longer contexts than were trained on: scaled frequencies, half of each head, interleaved pairs
        _rope("rope_pieces", B=48, H=9, D=64, rot=32, lo=1, hi=1501, first=120000, interleaved=True, scaled=8.0),
        # one token of one short sequence: launch latency
        _weights("weights_one", B=1, Hq=8, Hkv=2, D=64, page=16, lo=201, hi=201, new_lo=1, new_hi=1),
        # one decoding step of a batch of ragged histories
        _weights("weights_step", B=64, Hq=32, Hkv=8, D=128, page=64, lo=100, hi=8192, new_lo=1, new_hi=1),
        # one token of two very long histories, older weight fading
        _weights("weights_long", B=2, Hq=16, Hkv=2, D=128, page=128, lo=130001, hi=131071, new_lo=1, new_hi=1,
                 decay=0.96875),
        # 32 candidate rows a sample against its stored history, every row sees all of it
        _weights("weights_candidates", B=128, Hq=8, Hkv=8, D=64, page=64, lo=100, hi=6000, new_lo=32, new_hi=32,
                 causal=False),
        # pieces of prompts behind what the cache already holds
        _weights("weights_prompts", B=4, Hq=32, Hkv=8, D=128, page=64, lo=2100, hi=8192, new_lo=300, new_hi=1024),
        # one short sequence is cut: launch latency
        _evict("evict_one", B=1, Hkv=2, D=64, page=16, lo=150, hi=150, budget=100, sink=4, recent=16),
        # a batch of ragged histories is cut to 2048 tokens each
        _evict("evict_step", B=64, Hkv=8, D=128, page=64, lo=1500, hi=8192, budget=2048, sink=4, recent=256),
        # two very long histories are cut to an eighth
        _evict("evict_long", B=2, Hkv=2, D=128, page=128, lo=130001, hi=131071, budget=16384, sink=16, recent=2049),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    D = rng.choice([64, 128])
    op = rng.choice(["rope", "weights", "evict"])
    if op == "rope":
        H = rng.choice([1, 2, 5, 8, 12, 40])
        B = _log(rng, 1, 300)
        # at most the rows of the largest listed batch, in elements
        most = max(1, min(8192, 128 * 2098 * 8 * 128 // (H * D) // B))
        hi = 1 if rng.random() < 0.3 else _log(rng, 1, most)
        return _rope("", op=op, B=B, H=H, D=D, rot=rng.choice([16, D // 2, D]), lo=rng.choice([0, 1, hi]), hi=hi,
                     first=rng.choice([0, _log(rng, 1, 1 << 20)]), heads_of=rng.choice([0, H + rng.choice([1, 4])]),
                     interleaved=rng.random() < 0.5, scaled=rng.choice([1.0, 4.0, 32.0]), inverse=rng.random() < 0.4)
    Hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, D=D, Hkv=Hkv, page=rng.choice([16, 32, 64, 128]), B=_log(rng, 1, 300))
    most = max(64, min(131072, 64 * 8192 * 8 * 128 // (Hkv * D) // c["B"]))  # codes of the largest listed step
    c["hi"] = _log(rng, 2, most)
    if op == "evict":
        c["lo"] = rng.choice([0, 1, c["hi"] // 2, c["hi"]])
        c["budget"] = _log(rng, 1, c["hi"] + 10)
        c["sink"] = rng.choice([0, min(4, c["budget"] // 2)])
        c["recent"] = rng.randrange(c["budget"] - c["sink"] + 1) if rng.random() < 0.3 else c["budget"] // 8
        return c
    c["lo"] = rng.choice([0, 1, c["hi"] // 8, c["hi"]])
    c["Hq"] = Hkv * rng.choice([1, 2, 4, 7, 8])
    kind = rng.random()
    rows = 1 if kind < 0.5 else 40 if kind < 0.8 else 1024
    # fewer products than the listed pieces of prompts
    rows = max(1, min(rows, 4 * 512 * 4096 * 32 * 128 // (c["B"] * c["hi"] * c["Hq"] * D)))
    c["new_hi"] = _log(rng, 1, rows)
    c["new_lo"] = rng.choice([1, c["new_hi"]])
    c["causal"] = rng.random() < 0.8
    c["window"] = rng.choice([0, 0, _log(rng, 1, 4096)]) if c["causal"] else 0
    c["decay"] = rng.choice([1.0, 0.5, 0.99])
    return c


def _spread(n, lo, hi, a):
    """n lengths spread evenly over lo..hi, in no order (multiples of an irrational number, less whole parts)."""
    return [lo + int((hi - lo + 1) * (((i + 1) * a) % 1.0)) for i in range(n)]


def _lengths(c):
    """Tokens in the cache and rows of each sequence (rope: rows and first positions): by the case alone."""
    if c["op"] == "rope":
        return _spread(c["B"], c["lo"], c["hi"], 0.6180339887498949), _spread(c["B"], 0, c["first"], 0.7548776662466927)
    lens = _spread(c["B"], c["lo"], c["hi"], 0.6180339887498949)
    if c["op"] == "evict":
        return lens, [min(n, c["budget"]) for n in lens]
    return lens, _spread(c["B"], c["new_lo"], c["new_hi"], 0.7548776662466927)


def _frequencies(c):
    """Radians a position of each pair, and the magnitude: the interpolation by wave length of scaled contexts
    (trained on 4096 positions, base 10000)."""
    rot, s = c["rot"], c["scaled"]
    f = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if s == 1.0:
        return f, 1.0
    # a pair that turns 32 times or more over the trained context stays, one that turns once or less is stretched
    dim = rot * np.log(4096 / (2 * math.pi * np.array([32.0, 1.0]))) / (2 * math.log(10000.0))
    lo, hi = max(math.floor(dim[0]), 0), min(math.ceil(dim[1]), rot - 1)
    ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
    return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1


def _offsets(rows):
    offsets = np.zeros(len(rows) + 1, np.int32)
    offsets[1:] = np.cumsum(rows)
    return offsets


def prepare(case, seed):
    if case["op"] == "rope":
        return _prepare_rope(case, seed)
    dev = torch.device("cuda")
    B, Hkv, D, P = case["B"], case["Hkv"], case["D"], case["page"]
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, new = _lengths(case)
    pages = [-(-n // P) for n in lens]
    fresh = [-(-n // P) for n in new] if case["op"] == "evict" else []  # pages that take what is kept
    num_pages = sum(pages) + sum(fresh) + 3
    # every sequence's pages lie anywhere; entries behind its last page are -1
    order = torch.randperm(num_pages, device=dev, generator=g).to(torch.int32)

    def tables(counts, skip):
        width = max(1, max(counts))
        n = torch.tensor(counts, device=dev)
        at = torch.arange(width, device=dev)[None] < n[:, None]
        begin = torch.cumsum(n, 0) - n + skip
        index = (begin[:, None] + torch.arange(width, device=dev)[None]).clamp(max=num_pages - 1)
        return torch.where(at, order[index], torch.full_like(order[:1], -1)).contiguous(), width

    table, max_pages = tables(pages, 0)
    s = dict(case=case, B=B, Hkv=Hkv, D=D, P=P, max_pages=max_pages, max_len=max(lens), table=table,
             lens=torch.tensor(lens, dtype=torch.int32, device=dev))

    # The cache's contents: values of about N(0, 1), whose largest in a block is about 3.5 = 448 / 2^7; blocks a
    # factor of two larger and smaller among them.
    shape = (num_pages, Hkv, P, D)

    def codes():
        x = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
        for p in range(0, num_pages, 4096):
            n = min(4096, num_pages - p)
            x[p:p + n] = torch.randn((n,) + shape[1:], device=dev, generator=g).mul_(100).clamp_(-448, 448)
        return x.view(torch.uint8)

    def scales():
        return torch.randint(119, 122, shape[:2] + (P // BLOCK,), device=dev, generator=g).to(torch.uint8)

    s.update(k_codes=codes(), v_codes=codes(), k_sf=scales(), v_sf=scales())
    # accumulated weight: a few keys took most of it, a tenth of them none that fp32 holds
    w = torch.randn((num_pages, Hkv, P), device=dev, generator=g).mul_(2).exp_().mul_(2.0 ** -10)
    w = torch.where(torch.rand(w.shape, device=dev, generator=g) < 0.1, torch.zeros((), device=dev), w)
    if case["op"] == "evict":
        s["weights"] = w
        s["new_table"], s["new_max_pages"] = tables(fresh, sum(pages))
        s["kept"] = torch.full((B, Hkv, case["budget"]), -1, dtype=torch.int32, device=dev)
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device=dev)
        s["result"] = {"k": s["k_codes"].view(torch.float8_e4m3fn), "v": s["v_codes"].view(torch.float8_e4m3fn),
                       "k_scale": s["k_sf"].view(torch.float8_e8m0fnu), "v_scale": s["v_sf"].view(torch.float8_e8m0fnu),
                       "weights": w, "kept": s["kept"], "lens": s["new_lens"]}
    else:
        offsets = _offsets(new)
        T, Hq = int(offsets[-1]), case["Hq"]
        s.update(T=T, Hq=Hq, max_new=max(new), offsets=torch.from_numpy(offsets).to(dev), before=w, scale=1.0 / math.sqrt(D))
        s["weights"] = torch.zeros_like(w)
        s["q"] = torch.randn((T, Hq, D), device=dev, generator=g).to(torch.bfloat16)
        # the attention's own logsumexp of each row
        score, _ = _scores(s)
        lse = torch.logsumexp(score, -1)
        row = torch.arange(T, device=dev)
        b = torch.searchsorted(s["offsets"].long()[1:], row, right=True)
        s["lse"] = lse.permute(0, 2, 1, 3).reshape(B, s["max_new"], Hq)[b, row - s["offsets"].long()[b]].contiguous()
        del score
    if own:  # the descriptor that a program keeps beside the cache
        from jagged_attention_recommender_gb300 import gdpa
        s["cache"] = gdpa.KvCache(s["k_codes"], s["v_codes"], s["k_sf"], s["v_sf"])
    return s


def _prepare_rope(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rows, first = _lengths(case)
    offsets = _offsets(rows)
    T, H, D = int(offsets[-1]), case["H"], case["D"]

    def fused(fill):
        x = torch.empty((T, max(H, case["heads_of"]), D), dtype=torch.bfloat16, device=dev)
        if fill:
            for t in range(0, T, 65536):
                n = min(65536, T - t)
                x[t:t + n] = torch.randn((n,) + x.shape[1:], device=dev, generator=g)
        return x[:, :H]

    own_rows = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev)
    if case["inverse"]:
        for t in range(0, T, 65536):
            n = min(65536, T - t)
            own_rows[t:t + n] = torch.randn((n, H, D), device=dev, generator=g)
    x, y = (own_rows, fused(False)) if case["inverse"] else (fused(True), own_rows)
    f, magnitude = _frequencies(case)
    return dict(case=case, T=T, x=x, y=y, inv_freq=f, d_inv_freq=torch.from_numpy(f).to(dev), magnitude=magnitude,
                offsets=torch.from_numpy(offsets).to(dev), first=torch.tensor(first, dtype=torch.int32, device=dev))


def run(s):
    return {"rope": _run_rope, "weights": _run_weights, "evict": _run_evict}[s["case"]["op"]](s)


def _run_rope(s):
    c, x, y = s["case"], s["x"], s["y"]
    if own:
        from jagged_attention_recommender_gb300 import gdpa
        style = gdpa.GDPA_ROPE_INTERLEAVED if c["interleaved"] else gdpa.GDPA_ROPE_HALF
        gdpa.gdpa_rope(x, x.stride(0), s["offsets"], s["first"], s["T"], c["B"], c["H"], c["D"], s["inv_freq"], style,
                       s["magnitude"], c["inverse"], y, y.stride(0))
        return y
    offsets = s["offsets"].long()
    row = torch.arange(s["T"], device=x.device)
    b = torch.searchsorted(offsets[1:], row, right=True)
    pos = s["first"].long()[b] + row - offsets[b]
    angle = pos.double()[:, None, None] * s["d_inv_freq"]  # far positions: angles in 64 bits
    cos, sin = (angle.cos() * s["magnitude"]).float(), (angle.sin() * s["magnitude"]).float()
    if c["inverse"]:
        sin = -sin
    z, rot = x.float(), c["rot"]
    if c["interleaved"]:
        u, v = z[..., 0:rot:2], z[..., 1:rot:2]
        t = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
    else:
        u, v = z[..., :rot // 2], z[..., rot // 2:rot]
        t = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
    y[..., :rot] = t
    y[..., rot:] = x[..., rot:]
    return y


def _scores(s):
    """Scores [B, Hkv, rows G, tokens] in 32 bits, -inf where a row does not see a key, and whether a key is stored."""
    c = s["case"]
    B, Hkv, D, P, M = s["B"], s["Hkv"], s["D"], s["P"], s["max_new"]
    G = s["Hq"] // Hkv
    offsets, lens = s["offsets"].long(), s["lens"].long()
    n = offsets[1:] - offsets[:-1]
    N = s["max_pages"] * P
    i = torch.arange(M, device=n.device)
    j = torch.arange(N, device=n.device)
    pos = (lens - n)[:, None] + i  # [B, M]
    stored = j < lens[:, None]
    seen = stored[:, None] & (i < n[:, None])[:, :, None]
    if c["causal"]:
        seen = seen & (j <= pos[:, :, None])
    if c["window"]:
        seen = seen & (j > pos[:, :, None] - c["window"])
    rows = (offsets[:-1, None] + i).clamp(max=s["T"] - 1)
    q = s["q"][rows].float().reshape(B, M, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * G, D)
    pages = s["table"].long().clamp(min=0)
    k = s["k_codes"].view(torch.float8_e4m3fn)[pages].float()  # [B, pages, Hkv, P, D]
    k = k * torch.exp2(s["k_sf"][pages].float() - 127).repeat_interleave(BLOCK, -1)[..., None]
    k = k.permute(0, 2, 1, 3, 4).reshape(B, Hkv, N, D)
    score = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).reshape(B, Hkv, M, G, N)
    return score.masked_fill_(~seen[:, None, :, None], float("-inf")), stored


def _run_weights(s):
    c = s["case"]
    if own:
        from jagged_attention_recommender_gb300 import gdpa
        gdpa.gdpa_cache_weights(s["cache"], s["q"], s["q"].stride(0), s["lse"], s["offsets"], s["lens"], s["table"], s["T"],
                                s["B"], s["Hq"], s["max_pages"], s["max_new"], c["causal"], c["window"], s["scale"],
                                c["decay"], s["before"], s["weights"])
        return s["weights"]
    score, stored = _scores(s)
    B, Hkv, P, M = s["B"], s["Hkv"], s["P"], s["max_new"]
    offsets, lens = s["offsets"].long(), s["lens"].long()
    rows = (offsets[:-1, None] + torch.arange(M, device=lens.device)).clamp(max=s["T"] - 1)
    lse = s["lse"][rows].reshape(B, M, Hkv, -1).permute(0, 2, 1, 3)[..., None]
    # a row that sees no key has a logsumexp of -inf, and no score to go with it
    lse = torch.where(torch.isfinite(lse), lse, torch.zeros((), device=lse.device))
    w = score.sub_(lse).exp_().sum((2, 3))  # [B, Hkv, tokens]
    pages = s["table"].long()
    old = s["before"][pages.clamp(min=0)].permute(0, 2, 1, 3).reshape(w.shape)
    earlier = torch.arange(w.shape[-1], device=w.device) < (lens - (offsets[1:] - offsets[:-1]))[:, None]
    w = w + torch.where(earlier[:, None], old * c["decay"], torch.zeros((), device=w.device))
    b, j = stored.nonzero(as_tuple=True)
    s["weights"][pages[b, j // P], :, j % P] = w[b, :, j]
    return s["weights"]


def _run_evict(s):
    c = s["case"]
    if own:
        from jagged_attention_recommender_gb300 import gdpa
        gdpa.gdpa_cache_evict(s["cache"], s["weights"], s["lens"], s["table"], s["B"], s["max_pages"], c["budget"],
                              c["sink"], c["recent"], s["new_table"], s["new_max_pages"], s["kept"], s["new_lens"])
        return s["result"]
    B, Hkv, P, N = s["B"], s["Hkv"], s["P"], s["max_pages"] * s["P"]
    lens, pages = s["lens"].long()[:, None, None], s["table"].long()
    new_lens = lens.clamp(max=c["budget"])
    j = torch.arange(N, device=lens.device)
    # what is always kept comes first, then the largest weights, equal ones by their place; what is not stored is last
    w = s["weights"][pages.clamp(min=0)].permute(0, 2, 1, 3).reshape(B, Hkv, N)
    w = torch.where((j < c["sink"]) | (j >= lens - c["recent"]), torch.full((), float("inf"), device=w.device), w)
    w = torch.where(j < lens, w, torch.full((), float("-inf"), device=w.device))
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, j.expand_as(order))
    b, h, src = (rank < new_lens).nonzero(as_tuple=True)  # in the order of sequences, heads and tokens
    count = new_lens[:, 0, 0]
    begin = (torch.cumsum(count, 0) - count)[b] * Hkv + h * count[b]
    i = torch.arange(len(src), device=src.device) - begin
    s["kept"][b, h, i] = src.int()
    s["new_lens"].copy_(count)
    page, to = pages[b, src // P], s["new_table"].long()[b, i // P]
    s["weights"][to, h, i % P] = s["weights"][page, h, src % P]
    # a block of 16 kept tokens takes the largest of their scales
    block = (torch.cumsum((count + BLOCK - 1) // BLOCK, 0) - (count + BLOCK - 1) // BLOCK)[b] * Hkv
    block = block + h * ((count[b] + BLOCK - 1) // BLOCK) + i // BLOCK
    for codes, sf in ((s["k_codes"], s["k_sf"]), (s["v_codes"], s["v_sf"])):
        was = sf[page, h, src % P // BLOCK].int()
        top = torch.zeros(int(block.shape[0]) + 1, dtype=torch.int32, device=was.device)
        top = top.scatter_reduce_(0, block, was, "amax")[block]
        x = codes[page, h, src % P].view(torch.float8_e4m3fn).float() * torch.exp2((was - top).float())[:, None]
        codes[to, h, i % P] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        sf[to, h, i % P // BLOCK] = top.to(torch.uint8)
    return s["result"]


def _seen(c, length, n, i):
    """First and one past the last key that query i of n sees in a sequence of `length` tokens."""
    pos = length - n + i
    end = min(length, pos + 1) if c["causal"] else length
    return max(0, pos - c["window"] + 1) if c["window"] else 0, max(0, end)


def work(case):
    lens, new = _lengths(case)
    if case["op"] == "rope":
        elements = sum(lens) * case["H"] * case["D"]
        return {"bytes": 4 * elements + 8 * case["B"], "flops": 3 * sum(lens) * case["H"] * case["rot"]}
    Hkv, D = case["Hkv"], case["D"]
    table = 4 * sum(-(-n // case["page"]) for n in lens)
    if case["op"] == "evict":
        # all weights in; what is kept in and out, its weights and places out
        kept, blocks = sum(new), sum(-(-n // BLOCK) for n in new)
        return {"bytes": Hkv * (4 * sum(lens) + kept * (4 * D + 8) + 4 * blocks) + table, "flops": Hkv * sum(lens)}
    keys = pairs = 0
    for m, n in zip(lens, new):
        spans = [_seen(case, m, n, i) for i in range(n)]
        pairs += sum(max(0, e - a) for a, e in spans)
        spans = [x for x in spans if x[1] > x[0]]
        keys += max((e for _, e in spans), default=0) - min((a for a, _ in spans), default=0)
    earlier = sum(max(0, m - n) for m, n in zip(lens, new))
    return {"bytes": keys * Hkv * D + keys * Hkv // BLOCK + 4 * Hkv * (earlier + sum(lens))
            + sum(new) * case["Hq"] * (2 * D + 4) + table, "flops": 2 * pairs * case["Hq"] * D}


def exact(case, seed):
    """The same from the definition, sequence by sequence in 64 bits; codes and scales as values, codes unrounded."""
    s = prepare(case, seed)
    lens, new = _lengths(case)
    if case["op"] == "rope":
        x = s["x"].double()
        r, k = case["rot"], 0
        first, second = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
        for n, p in zip(lens, new):
            pos = np.arange(p, p + n, dtype=np.float64)
            turn = np.exp((-1j if case["inverse"] else 1j) * pos[:, None] * s["inv_freq"]) * s["magnitude"]
            z = torch.complex(x[k:k + n, :, first], x[k:k + n, :, second])
            z = z * torch.from_numpy(turn).to(x.device)[:, None]
            x[k:k + n, :, first], x[k:k + n, :, second] = z.real, z.imag
            k += n
        return x
    P, Hkv = s["P"], s["Hkv"]
    table = s["table"].cpu().numpy()
    dev = s["lens"].device
    if case["op"] == "evict":
        res = {"k": s["k_codes"].view(torch.float8_e4m3fn).double(), "v": s["v_codes"].view(torch.float8_e4m3fn).double(),
               "k_scale": torch.pow(2.0, s["k_sf"].double() - 127), "v_scale": torch.pow(2.0, s["v_sf"].double() - 127),
               "weights": s["weights"].double(), "kept": None, "lens": None}
        to = s["new_table"].cpu().numpy()
        for b in range(s["B"]):
            if not lens[b]:
                continue
            n, t = new[b], torch.arange(lens[b], device=dev)
            page, slot = torch.from_numpy(table[b].astype(np.int64)).to(dev)[t // P], t % P
            w = s["weights"][page, :, slot].double()  # [tokens, heads]
            w[:case["sink"]] = float("inf")
            w[max(0, lens[b] - case["recent"]):] = float("inf")
            at = torch.argsort(-w, dim=0, stable=True)[:n].sort(0).values  # [kept, heads]
            h = torch.arange(Hkv, device=dev).expand_as(at)
            i = torch.arange(n, device=dev)
            new_page = torch.from_numpy(to[b].astype(np.int64)).to(dev)[i // P][:, None].expand_as(at)
            new_slot = (i % P)[:, None].expand_as(at)
            res["weights"][new_page, h, new_slot] = s["weights"][page[at], h, slot[at]].double()
            for name in ("k", "v"):
                code, unit = res[name], res[name + "_scale"]
                u = unit[page[at], h, slot[at] // BLOCK]
                full = torch.zeros((-(-n // BLOCK) * BLOCK, Hkv), dtype=torch.float64, device=dev)
                full[:n] = u
                top = full.reshape(-1, BLOCK, Hkv).amax(1).repeat_interleave(BLOCK, 0)[:n]
                code[new_page, h, new_slot] = code[page[at], h, slot[at]] * (u / top)[..., None]
                unit[new_page, h, new_slot // BLOCK] = top
        return res
    if work(case)["flops"] > 2e12:
        return None
    out = torch.zeros(s["weights"].shape, dtype=torch.float64, device=dev)
    G, k0 = s["Hq"] // Hkv, 0
    for b in range(s["B"]):
        rows = slice(k0, k0 + new[b])
        k0 += new[b]
        if not lens[b]:
            continue
        t = torch.arange(lens[b], device=dev)
        page, slot = torch.from_numpy(table[b].astype(np.int64)).to(dev)[t // P], t % P
        k = s["k_codes"][page, :, slot].view(torch.float8_e4m3fn).double()  # [tokens, heads, D]
        k = k * torch.pow(2.0, s["k_sf"][page, :, slot // BLOCK].double() - 127)[..., None]
        spans = torch.tensor([_seen(case, lens[b], new[b], i) for i in range(new[b])], device=dev)
        hidden = (t < spans[:, :1]) | (t >= spans[:, 1:])
        w = s["before"][page, :, slot].double() * case["decay"]
        w[max(0, lens[b] - new[b]):] = 0
        for h in range(Hkv):
            x = torch.einsum("igd,jd->gij", s["q"][rows, h * G:(h + 1) * G].double(), k[:, h]) * (1.0 / math.sqrt(s["D"]))
            p = torch.exp(x - s["lse"][rows, h * G:(h + 1) * G].double().T[..., None])
            w[:, h] += torch.where(hidden, torch.zeros((), dtype=p.dtype, device=dev), p).sum((0, 1))
        out[page, :, slot] = w
    return out
