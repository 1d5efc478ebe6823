"""The paged key/value cache's operators: appending new tokens with their
position rotation, and attention over the cache.

The cache holds keys and values as e4m3 codes, one power-of-two scale for each
block of 16 tokens and head.  ``own`` false computes the operators in plain
torch operations in 32 bits; ``own`` true calls this repository's library.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16        # tokens of a scale block
E4M3_MAX = 448.0  # the largest e4m3 value


def _append(name, **kw):
    c = dict(op="append", name=name, strided=False, interleaved=False)
    c.update(kw)
    return c


def _attend(name, **kw):
    c = dict(op="attend", name=name, window=0, causal=True)
    c.update(kw)
    return c


def listed():
    """lo, hi: tokens of a sequence in the cache (after the append); new_lo,
    new_hi: new tokens of a sequence; page: tokens of a page; rot: rotated
    coordinates of a head."""
    return [
        # one decoding step of four short sequences: launch latency
        _append("append_few", B=4, Hq=8, Hkv=2, D=64, page=16, lo=1, hi=90, new_lo=1, new_hi=1, rot=64),
        # one decoding step of a full batch, from the fused projection's rows
        _append("append_step", B=256, Hq=32, Hkv=8, D=128, page=64, lo=1, hi=4095, new_lo=1, new_hi=1, rot=128,
                strided=True),
        # pieces of prompts that begin and end inside scale blocks, half of each head rotated, interleaved pairs
        _append("append_pieces", B=48, Hq=8, Hkv=8, D=64, page=32, lo=301, hi=2500, new_lo=1, new_hi=300, rot=32,
                strided=True, interleaved=True),
        # whole prompts of hundreds to thousands of tokens into an empty cache
        _append("append_prompts", B=32, Hq=32, Hkv=8, D=128, page=64, lo=100, hi=4096, new_lo=4096, new_hi=4096,
                rot=128),
        # one token of one short sequence: launch latency
        _attend("attend_one", B=1, Hq=8, Hkv=2, D=64, page=16, lo=201, hi=201, new_lo=1, new_hi=1),
        # one decoding step of a batch of ragged histories
        _attend("attend_step", B=64, Hq=32, Hkv=8, D=128, page=64, lo=100, hi=8192, new_lo=1, new_hi=1),
        # one token of two very long histories: the key axis has to be split
        _attend("attend_long", B=2, Hq=16, Hkv=2, D=128, page=128, lo=130001, hi=131071, new_lo=1, new_hi=1),
        # many short and empty histories, as many key heads as query heads
        _attend("attend_many", B=512, Hq=8, Hkv=8, D=64, page=16, lo=0, hi=1023, new_lo=1, new_hi=1),
        # five drafted tokens a sequence are checked at once
        _attend("attend_verify", B=48, Hq=32, Hkv=4, D=128, page=32, lo=500, hi=6001, new_lo=5, new_hi=5),
        # a sliding window over long histories
        _attend("attend_window", B=96, Hq=16, Hkv=4, D=128, page=64, lo=900, hi=16384, new_lo=1, new_hi=2, window=1024),
        # 32 candidate rows a sample against its stored history, every row sees all of it
        _attend("attend_candidates", B=128, Hq=8, Hkv=8, D=64, page=64, lo=100, hi=6000, new_lo=32, new_hi=32,
                causal=False),
        # pieces of prompts behind what the cache already holds
        _attend("attend_prompts", B=4, Hq=32, Hkv=8, D=128, page=64, lo=2100, hi=8192, new_lo=300, new_hi=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=rng.choice(["append", "attend"]), D=D, Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 4, 7, 8]),
             page=rng.choice([16, 32, 64, 128]))
    if c["op"] == "append":
        c["B"] = _log(rng, 1, 300)
        # at most 2^16 new tokens of 32 query heads and 8 key heads of 128
        most = max(1, min(4096, 65536 * 48 * 128 // ((c["Hq"] + 2 * Hkv) * D) // c["B"]))
        c["new_lo"] = 1
        c["new_hi"] = 1 if rng.random() < 0.4 else _log(rng, 1, most)
        c["lo"] = c["new_hi"] + rng.randrange(40)
        c["hi"] = c["lo"] + _log(rng, 1, 4000)
        c["rot"] = rng.choice([0, D // 2, D])
        c["strided"] = rng.random() < 0.5
        c["interleaved"] = rng.random() < 0.5
        return c
    c["B"] = _log(rng, 1, 300)
    most = max(64, min(131072, 64 * 8192 * 8 * 128 // (Hkv * D) // c["B"]))  # codes of the largest listed step
    c["hi"] = _log(rng, 2, most)
    c["lo"] = rng.choice([0, 1, c["hi"] // 8, c["hi"]])
    kind = rng.random()
    rows = 1 if kind < 0.5 else 40 if kind < 0.8 else 1024
    # fewer products than the listed pieces of prompts
    rows = max(1, min(rows, 4 * 512 * 4096 * 32 * 128 // (c["B"] * c["hi"] * c["Hq"] * D)))
    c["new_hi"] = _log(rng, 1, rows)
    c["new_lo"] = rng.choice([1, c["new_hi"]])
    c["causal"] = rng.random() < 0.8
    c["window"] = rng.choice([0, 0, _log(rng, 1, 4096)]) if c["causal"] else 0
    return c


def _spread(n, lo, hi, a):
    """n lengths spread evenly over lo..hi, in no order (multiples of an irrational number, less whole parts)."""
    return [lo + int((hi - lo + 1) * (((i + 1) * a) % 1.0)) for i in range(n)]


def _lengths(c):
    """Tokens in the cache and new tokens of each sequence: by the case alone."""
    lens = _spread(c["B"], c["lo"], c["hi"], 0.6180339887498949)
    new = _spread(c["B"], c["new_lo"], c["new_hi"], 0.7548776662466927)
    if c["op"] == "append":
        new = [min(n, m) for n, m in zip(new, lens)]
    return lens, new


def _inv_freq(rot):
    return 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot) if rot else None


def prepare(case, seed):
    dev = torch.device("cuda")
    B, Hq, Hkv, D, P = case["B"], case["Hq"], case["Hkv"], case["D"], case["page"]
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, new = _lengths(case)
    max_pages = max(1, -(-max(lens) // P))
    pages = [-(-n // P) for n in lens]
    num_pages = sum(pages) + 3
    # every sequence's pages lie anywhere; entries behind its last page are -1
    order = torch.randperm(num_pages, device=dev, generator=g).to(torch.int32)
    n_pages = torch.tensor(pages, device=dev)
    at = torch.arange(max_pages, device=dev)[None] < n_pages[:, None]
    first = torch.cumsum(n_pages, 0) - n_pages
    index = (first[:, None] + torch.arange(max_pages, device=dev)[None]).clamp(max=num_pages - 1)
    table = torch.where(at, order[index], torch.full_like(order[:1], -1)).contiguous()
    offsets = np.zeros(B + 1, np.int32)
    offsets[1:] = np.cumsum(new)
    T = int(offsets[-1])
    s = dict(case=case, B=B, Hq=Hq, Hkv=Hkv, D=D, P=P, T=T, max_pages=max_pages, max_len=max(lens), max_new=max(new),
             table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev),
             offsets=torch.from_numpy(offsets).to(dev))

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
    if case["op"] == "append":
        fused = torch.randn((T, Hq + 2 * Hkv, D), device=dev, generator=g).to(torch.bfloat16)
        parts = torch.split(fused, [Hq, Hkv, Hkv], dim=1)
        s["q"], s["k"], s["v"] = parts if case["strided"] else [x.contiguous() for x in parts]
        s["inv_freq"] = _inv_freq(case["rot"])
        s["d_inv_freq"] = None if s["inv_freq"] is None else torch.from_numpy(s["inv_freq"]).to(dev)
        s["q_out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
        # the scale blocks that take new tokens: (sequence, block)
        touched = [(b, j) for b in range(B) if new[b] for j in range((lens[b] - new[b]) // BLOCK, -(-lens[b] // BLOCK))]
        s["touched"] = torch.tensor(touched, dtype=torch.int64, device=dev)
        s["result"] = {"q": s["q_out"], **_values(s)}
    else:
        s["q"] = torch.randn((T, Hq, D), device=dev, generator=g).to(torch.bfloat16)
        s["out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty((T, Hq), dtype=torch.float32, device=dev)
        s["scale"] = 1.0 / math.sqrt(D)
    if own:  # the descriptor and the workspace that a program keeps beside the cache
        from jagged_attention_recommender_gb300 import gdpa
        style = gdpa.GDPA_ROPE_INTERLEAVED if case.get("interleaved") else gdpa.GDPA_ROPE_HALF
        s["cache"] = gdpa.KvCache(s["k_codes"], s["v_codes"], s["k_sf"], s["v_sf"], s.get("inv_freq"), style)
        if case["op"] == "attend":
            n = gdpa.gdpa_cache_workspace_size(s["cache"], Hq, s["max_new"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=dev)
    return s


def _values(s):
    """The cache's own buffers as the values their codes and scales stand for (types of 8 bits)."""
    return {"k": s["k_codes"].view(torch.float8_e4m3fn), "v": s["v_codes"].view(torch.float8_e4m3fn),
            "k_scale": s["k_sf"].view(torch.float8_e8m0fnu), "v_scale": s["v_sf"].view(torch.float8_e8m0fnu)}


def run(s):
    if s["case"]["op"] == "append":
        return _run_append(s)
    return _run_attend(s)


def _run_append(s):
    if own:
        from jagged_attention_recommender_gb300 import gdpa
        q, k, v = s["q"], s["k"], s["v"]
        gdpa.gdpa_cache_append(s["cache"], q, q.stride(0), k, k.stride(0), v, v.stride(0), s["offsets"], s["lens"],
                               s["table"], s["T"], s["B"], s["Hq"], s["max_pages"], s["q_out"])
        return s["result"]
    offsets, lens = s["offsets"].long(), s["lens"].long()
    start = lens - (offsets[1:] - offsets[:-1])
    row = torch.arange(s["T"], device=lens.device)
    b = torch.searchsorted(offsets[1:], row, right=True)
    pos = start[b] + row - offsets[b]
    q, k = _rotate(s, s["q"].float(), pos), _rotate(s, s["k"].float(), pos)
    s["q_out"].copy_(q)
    _store(s, k, s["k_codes"], s["k_sf"], start)
    _store(s, s["v"].float(), s["v_codes"], s["v_sf"], start)
    return s["result"]


def _rotate(s, x, pos):
    if s["inv_freq"] is None:
        return x
    angle = pos.double()[:, None, None] * s["d_inv_freq"]  # far positions: angles in 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    rot = s["case"]["rot"]
    if s["case"]["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _store(s, x, codes, sf, start):
    """New rows x [T, Hkv, D] into the touched blocks: a block's scale only grows, its earlier codes follow it."""
    b, j = s["touched"][:, 0], s["touched"][:, 1]
    pos = j[:, None] * BLOCK + torch.arange(BLOCK, device=x.device)  # [n, 16]
    new = (pos >= start[b][:, None]) & (pos < s["lens"].long()[b][:, None])
    old = pos < start[b][:, None]
    row = (s["offsets"].long()[b][:, None] + pos - start[b][:, None]).clamp(0, s["T"] - 1)
    val = torch.where(new[:, :, None, None], x[row], torch.zeros((), device=x.device))  # [n, 16, Hkv, D]
    m, ex = torch.frexp(val.abs().amax((1, 3)))
    e = torch.where(m > 0, ex - 9 + (m > E4M3_MAX / 512).int(), -127).clamp(min=-127)  # [n, Hkv]
    page = s["table"].long()[b, j * BLOCK // s["P"]]
    first = j * BLOCK % s["P"]
    h = torch.arange(s["Hkv"], device=x.device)
    at_sf = (page[:, None], h[None], (first // BLOCK)[:, None])
    before = sf[at_sf].int() - 127
    e = torch.where(old.any(1)[:, None], torch.maximum(e, before), e)
    slot = first[:, None] + torch.arange(BLOCK, device=x.device)
    at = (page[:, None, None], h[None, None], slot[:, :, None])  # [n, 16, Hkv]
    cur = codes[at]
    kept = cur.view(torch.float8_e4m3fn).float() * torch.exp2((before - e).float())[:, None, :, None]
    val = torch.where(old[:, :, None, None], kept, val * torch.exp2(-e.float())[:, None, :, None])
    val = val.to(torch.float8_e4m3fn).view(torch.uint8)
    codes[at] = torch.where((new | old)[:, :, None, None], val, cur)
    sf[at_sf] = (e + 127).to(torch.uint8)


def _run_attend(s):
    c = s["case"]
    if own:
        from jagged_attention_recommender_gb300 import gdpa
        gdpa.gdpa_cache_fwd(s["cache"], s["q"], s["q"].stride(0), s["offsets"], s["lens"], s["table"], s["T"], s["B"],
                            s["Hq"], s["max_pages"], s["max_new"], c["causal"], c["window"], s["scale"], s["out"],
                            s["lse"], s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    B, Hkv, D, P, M = s["B"], s["Hkv"], s["D"], s["P"], s["max_new"]
    G = s["Hq"] // Hkv
    offsets, lens = s["offsets"].long(), s["lens"].long()
    n = offsets[1:] - offsets[:-1]
    N = s["max_pages"] * P
    i = torch.arange(M, device=n.device)
    j = torch.arange(N, device=n.device)
    pos = (lens - n)[:, None] + i  # [B, M]
    seen = (j < lens[:, None])[:, None].expand(B, M, N)
    if c["causal"]:
        seen = seen & (j <= pos[:, :, None])
    if c["window"]:
        seen = seen & (j > pos[:, :, None] - c["window"])
    rows = (offsets[:-1, None] + i).clamp(max=s["T"] - 1)
    q = s["q"][rows].float().reshape(B, M, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * G, D)
    pages = s["table"].long().clamp(min=0)

    def values(codes, sf):
        x = codes.view(torch.float8_e4m3fn)[pages].float()  # [B, pages, Hkv, P, D]
        f = torch.exp2(sf[pages].float() - 127).repeat_interleave(BLOCK, -1)
        return (x * f[..., None]).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N, D)

    score = torch.matmul(q, values(s["k_codes"], s["k_sf"]).transpose(-1, -2)).mul_(s["scale"])
    score = score.reshape(B, Hkv, M, G, N).masked_fill_(~seen[:, None, :, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros((), device=top.device))
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = values(s["v_codes"], s["v_sf"])
    # what lies behind a sequence's last token is no value of it
    v = torch.where((j < lens[:, None])[:, None, :, None], v, torch.zeros((), device=v.device))
    o = torch.matmul(p.reshape(B, Hkv, M * G, N), v).reshape(B, Hkv, M, G, D)
    o = o / torch.where(total > 0, total, torch.ones((), device=o.device))
    lse = (total.log() + top).squeeze(-1)
    row = torch.arange(s["T"], device=n.device)
    b = torch.searchsorted(offsets[1:], row, right=True)
    at = row - offsets[b]
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(B, M, s["Hq"], D)[b, at])
    s["lse"].copy_(lse.permute(0, 2, 1, 3).reshape(B, M, s["Hq"])[b, at])
    return {"out": s["out"], "lse": s["lse"]}


def _seen(c, length, n, i):
    """First and one past the last key that query i of n sees in a sequence of `length` tokens."""
    pos = length - n + i
    end = min(length, pos + 1) if c["causal"] else length
    return max(0, pos - c["window"] + 1) if c["window"] else 0, max(0, end)


def work(case):
    lens, new = _lengths(case)
    Hq, Hkv, D, T = case["Hq"], case["Hkv"], case["D"], sum(new)
    table = 4 * sum(-(-n // case["page"]) for n in lens)
    if case["op"] == "append":
        # q in and out, k and v in, their codes and the touched scales out
        blocks = sum(-(-m // BLOCK) - (m - n) // BLOCK for m, n in zip(lens, new) if n)
        return {"bytes": T * D * (4 * Hq + 6 * Hkv) + 2 * blocks * Hkv + table,
                "flops": 3 * T * case["rot"] * (Hq + Hkv) + 2 * T * D * 2 * Hkv}
    keys = pairs = 0
    for m, n in zip(lens, new):
        spans = [_seen(case, m, n, i) for i in range(n)]
        pairs += sum(max(0, e - a) for a, e in spans)
        spans = [x for x in spans if x[1] > x[0]]
        keys += max((e for _, e in spans), default=0) - min((a for a, _ in spans), default=0)
    return {"bytes": 2 * keys * Hkv * D + 2 * keys * Hkv // BLOCK + T * Hq * (4 * D + 4) + table,
            "flops": 4 * pairs * Hq * D}


def exact(case, seed):
    """The same from the definition, sequence by sequence in 64 bits; codes and scales as values, codes unrounded."""
    s = prepare(case, seed)
    lens, new = _lengths(case)
    P, G = s["P"], s["Hq"] // s["Hkv"]
    starts = np.concatenate([[0], np.cumsum(new)])
    table = s["table"].cpu().numpy()
    dev = s["q"].device
    if case["op"] == "append":
        res = {"q": torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)}
        f = _inv_freq(case["rot"])

        def turned(x, pos):
            x = x.double().clone()
            if f is None:
                return x
            r = case["rot"]
            first, second = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
            z = torch.complex(x[..., first], x[..., second])
            z = z * torch.from_numpy(np.exp(1j * pos[:, None] * f)).to(dev)[:, None]
            x[..., first], x[..., second] = z.real, z.imag
            return x

        for name in ("k", "v"):
            codes = s[name + "_codes"].view(torch.float8_e4m3fn).double()
            scale = torch.pow(2.0, s[name + "_sf"].double() - 127)
            for b in range(s["B"]):
                rows = slice(int(starts[b]), int(starts[b + 1]))
                at = lens[b] - new[b]
                pos = np.arange(at, lens[b], dtype=np.float64)
                x = turned(s["k"][rows], pos) if name == "k" else s["v"][rows].double()
                if name == "k":
                    res["q"][rows] = turned(s["q"][rows], pos)
                j0, j1 = at // BLOCK, -(-lens[b] // BLOCK)
                full = torch.zeros(((j1 - j0) * BLOCK,) + x.shape[1:], dtype=torch.float64, device=dev)
                full[at - j0 * BLOCK:lens[b] - j0 * BLOCK] = x
                full = full.reshape(j1 - j0, BLOCK, s["Hkv"], s["D"])
                page = torch.from_numpy(table[b, np.arange(j0, j1) * BLOCK // P].astype(np.int64)).to(dev)
                sub = torch.arange(j0, j1, device=dev) % (P // BLOCK)
                e = torch.ceil(torch.log2(full.abs().amax((1, 3)) / E4M3_MAX)).clamp(min=-127)  # [blocks, Hkv]
                unit = torch.pow(2.0, e)
                cur = codes.reshape(-1, s["Hkv"], P // BLOCK, BLOCK, s["D"])[page, :, sub].transpose(1, 2)
                held = torch.zeros(full.shape[:2], dtype=torch.bool, device=dev)
                held.view(-1)[:at - j0 * BLOCK] = True
                fresh = torch.zeros_like(held)
                fresh.view(-1)[at - j0 * BLOCK:lens[b] - j0 * BLOCK] = True
                was = scale[page, :, sub]
                unit = torch.where(held.any(1)[:, None], torch.maximum(unit, was), unit)
                kept = cur * (was / unit)[:, None, :, None]
                put = torch.where(held[..., None, None], kept, torch.where(fresh[..., None, None], full / unit[:, None, :, None], cur))
                codes.view(-1, s["Hkv"], P // BLOCK, BLOCK, s["D"])[page, :, sub] = put.transpose(1, 2)
                scale[page, :, sub] = unit
            res[name], res[name + "_scale"] = codes, scale
        return res
    w = work(case)
    if w["flops"] > 4e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.full(s["q"].shape[:2], float("-inf"), dtype=torch.float64, device=dev)
    for b in range(s["B"]):
        if not new[b] or not lens[b]:
            continue
        page = torch.from_numpy(table[b, :-(-lens[b] // P)].astype(np.int64)).to(dev)
        kv = []
        for name in ("k", "v"):
            x = s[name + "_codes"][page].view(torch.float8_e4m3fn).double()
            x = x.reshape(len(page), s["Hkv"], P // BLOCK, BLOCK, s["D"])
            x = x * torch.pow(2.0, s[name + "_sf"][page].double() - 127)[..., None, None]
            kv.append(x.reshape(len(page), s["Hkv"], P, s["D"]).transpose(0, 1).reshape(s["Hkv"], -1, s["D"])[:, :lens[b]])
        rows = slice(int(starts[b]), int(starts[b + 1]))
        spans = torch.tensor([_seen(case, lens[b], new[b], i) for i in range(new[b])], device=dev)
        at = torch.arange(lens[b], device=dev)
        hidden = (at < spans[:, :1]) | (at >= spans[:, 1:])
        q = s["q"][rows].double()
        for h in range(s["Hkv"]):
            heads = slice(h * G, (h + 1) * G)
            t = torch.einsum("igd,jd->gij", q[:, heads], kv[0][h]) * (1.0 / math.sqrt(s["D"]))
            t = t.masked_fill(hidden, float("-inf"))
            lse[rows, heads] = torch.logsumexp(t, -1).T
            t = torch.softmax(t, -1).nan_to_num(0.0)
            out[rows, heads] = torch.einsum("gij,jd->igd", t, kv[1][h])
    return {"out": out, "lse": lse}
