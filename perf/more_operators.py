"""Cases for drafted tokens and branching sequences on the 8-bit paged cache.

Four operators of a server that has several tokens checked at once, or several
continuations of one prompt:

  append   normalise each head of new queries and keys (root mean square, with
           a weight), rotate them by a given position, put keys and values
           into the paged e4m3 cache                     (q8_kv_append_norm)
  tree     attention of a tree of drafted tokens: each sees the cached tokens
           and the drafted ones that its mask names  (q8_attention_kv8_tree)
  compact  the drafted tokens that were kept go to the front of their slots,
           in every layer                                    (q8_kv_compact)
  fork     sequences become copies of others: full pages are shared and
           counted, open ones copied in every layer, pages that nobody holds
           freed and room for new tokens taken from them        (q8_kv_fork)

`run` makes one call of an operator: in elementary torch operations where `own`
is false, through this package where it is true.  Cache layout: keys uint8
[pages, kv_heads, page, dim], values uint8 [pages, kv_heads, dim, page] (tokens
innermost), both e4m3 codes; one exponent byte b per page and head, a code c
standing for e4m3(c) * 2^(b - 127).  Codes come back as float8_e4m3fn and
exponent bytes as float8_e8m0fnu views of the same buffers.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
E4M3_MAX = 448.0
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def _append(name, seqs, new, past, heads, kv_heads, dim, page, rot, interleaved, drafted, dtype, ragged):
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "past": past, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "rot": rot, "interleaved": interleaved, "drafted": drafted, "dtype": dtype,
            "ragged": ragged}


def _tree(name, seqs, new, past, heads, kv_heads, dim, page, window, dtype, ragged):
    return {"name": name, "op": "tree", "seqs": seqs, "new": new, "past": past, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "window": window, "dtype": dtype, "ragged": ragged}


def _compact(name, layers, seqs, new, past, kv_heads, dim, page, ragged):
    return {"name": name, "op": "compact", "layers": layers, "seqs": seqs, "new": new, "past": past,
            "kv_heads": kv_heads, "dim": dim, "page": page, "ragged": ragged}


def _fork(name, layers, seqs, outs, past, kv_heads, dim, page, room, ragged):
    return {"name": name, "op": "fork", "layers": layers, "seqs": seqs, "outs": outs, "past": past,
            "kv_heads": kv_heads, "dim": dim, "page": page, "room": room, "ragged": ragged}


def listed():
    return [
        # one chat user, a small tree of drafts: the call's latency is what counts
        _append("append drafts of one", 1, 12, 700, 32, 8, 128, 64, 128, False, True, "bf16", 1),
        # a decode step of a busy server
        _append("append decode batch", 128, 1, 4000, 32, 8, 128, 64, 128, False, False, "bf16", 3),
        # prompts of odd lengths continued after a cached prefix; half the head rotated, neighbours as pairs
        _append("append prompts", 6, 3001, 900, 32, 8, 128, 128, 64, True, False, "fp16", 5),
        # one user, a short conversation
        _tree("tree of one", 1, 12, 700, 32, 8, 128, 64, 0, "bf16", 1),
        # drafts of a busy server's users, sequences of all lengths
        _tree("tree batch", 32, 24, 4099, 32, 8, 128, 64, 0, "bf16", 7),
        # two users with very long documents and wide trees: the long axis has to be split
        _tree("tree long", 2, 70, 100001, 32, 8, 128, 128, 0, "bf16", 2),
        # small heads that are not shared, a sliding window
        _tree("tree window", 9, 33, 2777, 16, 16, 64, 32, 1024, "fp16", 11),
        # one user's kept path, in all layers
        _compact("compact of one", 12, 1, 12, 700, 8, 128, 64, 4),
        # a busy server's
        _compact("compact batch", 12, 64, 24, 300, 8, 128, 64, 9),
        # a step of one user's beams
        _fork("fork beams of one", 12, 4, 4, 350, 8, 128, 64, 1, 6),
        # many samples of one prompt
        _fork("fork samples", 12, 1, 16, 2900, 8, 128, 64, 16, 2),
        # a step of many users' beams
        _fork("fork beams batch", 12, 64, 64, 500, 8, 128, 64, 1, 8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "tree", "tree", "compact", "fork"])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8] if kv_heads <= 4 else [1, 2, 4])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([32, 64, 128])
    ragged = rng.randrange(1, 1 << 20)
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "append":
        seqs = _log(rng, 1, 128)
        most = 16384 * 48 * 128 // ((heads + 2 * kv_heads) * dim) // seqs
        new = rng.choice([1, _log(rng, 2, 64), _log(rng, 2, max(2, most))])
        past = _log(rng, 1, max(1, 400000 // seqs // kv_heads))
        c = _append("", seqs, new, past, heads, kv_heads, dim, page, rng.choice([dim, dim // 2, 0]), rng.random() < 0.5,
                    1 < new <= 128 and rng.random() < 0.7, rng.choice([dtype, dtype, "fp32"]), ragged)
    elif op == "tree":
        seqs = _log(rng, 1, 64)
        new = min(_log(rng, 1, 150), max(1, 100000 // (seqs * heads)))
        past = _log(rng, 1, min(100000, 150000000 // (kv_heads * dim) // seqs, 400000000 // (seqs * new * heads)))
        c = _tree("", seqs, new, past, heads, kv_heads, dim, page, rng.choice([0, 0, 0, 300, 1000]), dtype, ragged)
    elif op == "compact":
        seqs = _log(rng, 1, 64)
        new = _log(rng, 1, 150)
        layers = rng.randint(1, max(1, min(12, (12 * 64 * 24 * 8 * 128) // (seqs * new * kv_heads * dim))))
        past = _log(rng, 1, max(1, 20000 // seqs * 4 // kv_heads))
        c = _compact("", layers, seqs, new, past, kv_heads, dim, page, ragged)
    else:
        kv_heads, dim = min(kv_heads, 8), min(dim, 128)
        seqs = _log(rng, 1, 64)
        outs = rng.choice([seqs, _log(rng, 1, 64)])
        past = _log(rng, 1, max(1, 20000 // seqs * 4 // kv_heads))
        layers = rng.randint(1, max(1, min(12, (12 * 64 * 8 * 128 * 64) // (outs * kv_heads * dim * page))))
        c = _fork("", layers, seqs, outs, past, kv_heads, dim, page, rng.choice([0, 1, 1, 16, 100]), ragged)
    del c["name"]
    return c


def _lengths(case):
    """New tokens and cached tokens before them, of each sequence."""
    s, new, past = case["seqs"], case["new"], case["past"]
    if s == 1:
        return [new], [past]
    r = random.Random(case["ragged"])
    return [r.randint((new + 1) // 2, new) for _ in range(s)], [r.randint(past // 8, past) for _ in range(s)]


def _parents(case):
    """The drafted trees: of each new token the one that it continues, -1 where that is the last cached token."""
    r = random.Random(case["ragged"] + 1)
    return [[-1 if i == 0 or r.random() < 0.08 else max(0, i - 1 - int(r.expovariate(0.4))) for i in range(n)]
            for n in _lengths(case)[0]]


def _paths(case):
    """Of each sequence the drafted tokens that are kept: a token and those that it continues."""
    r = random.Random(case["ragged"] + 2)
    paths = []
    for up in _parents(case):
        at = r.randrange(len(up)) if case["seqs"] == 1 or r.random() < 0.9 else -1
        if case["seqs"] == 1:
            at = len(up) - 1
        path = []
        while at >= 0:
            path.append(at)
            at = up[at]
        paths.append(path[::-1])
    return paths


def _origins(case):
    """The lengths of the sequences that are there, and which of them each new one continues (-1: none)."""
    r = random.Random(case["ragged"] + 3)
    n, past = case["seqs"], case["past"]
    held = [r.randint((past + 1) // 2, past) if n > 1 else past for _ in range(n)]
    return held, [-1 if n > 8 and r.random() < 0.05 else r.randrange(n) for _ in range(case["outs"])]


# ------------------------------------------------------------------ inputs
def _exponent(amax):
    """The byte b of the smallest power of two 2^(b - 127) with amax <= 448 * 2^(b - 127); 0 for small amax."""
    bits = amax.contiguous().view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(0, 254)


def _two_to(e):
    """2^e for whole e from -250 to 250, exactly."""
    half = e // 2
    rest = e - half
    return ((half + 127) << 23).int().view(torch.float32) * ((rest + 127) << 23).int().view(torch.float32)


def _cache(gen, dev, layers, pages, hk, page, d):
    """Pages of `layers` layers, all of them filled: keys and values of layer i at [i]."""
    # channels of keys differ in size, some by a lot; values are even; tokens of a page are alike, those of pages not
    channel = 1.0 + 7.0 * (torch.rand(hk, 1, d, generator=gen, device=dev) < 0.03)
    k = torch.empty(layers, pages, hk, page, d, dtype=torch.float8_e4m3fn, device=dev)
    v = torch.empty(layers, pages, hk, d, page, dtype=torch.float8_e4m3fn, device=dev)
    ke = torch.empty(layers, pages, hk, dtype=torch.uint8, device=dev)
    ve = torch.empty_like(ke)
    for i in range(layers):
        size = 1.0 + 2.0 * torch.rand(pages, hk, 1, 1, generator=gen, device=dev)
        x = torch.randn(pages, hk, page, d, generator=gen, device=dev) * channel * size
        e = _exponent(x.abs().amax((2, 3)))
        k[i] = (x * _two_to(127 - e)[:, :, None, None]).to(torch.float8_e4m3fn)
        ke[i] = e.byte()
        x = torch.randn(pages, hk, d, page, generator=gen, device=dev) * size
        e = _exponent(x.abs().amax((2, 3)))
        v[i] = (x * _two_to(127 - e)[:, :, None, None]).to(torch.float8_e4m3fn)
        ve[i] = e.byte()
    return {"k": k, "v": v, "ke": ke.view(torch.float8_e8m0fnu), "ve": ve.view(torch.float8_e8m0fnu), "channel": channel}


def _prepare_batch(case, gen, dev, layers):
    new, past = _lengths(case)
    page = case["page"]
    total = [a + b for a, b in zip(new, past)]
    need = [-(-t // page) for t in total]
    pages = sum(need) + 3
    s = _cache(gen, dev, layers, pages, case["kv_heads"], page, case["dim"])
    order = torch.randperm(pages, generator=gen, device=dev).int()
    table = torch.full((len(need), max(need)), -1, dtype=torch.int32, device=dev)
    start, at = [0], 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
        start.append(start[-1] + new[i])
    s.update({"op": case["op"], "table": table, "start": torch.tensor(start, dtype=torch.int32, device=dev),
              "len": torch.tensor(total, dtype=torch.int32, device=dev), "max_new": max(new), "max_len": max(total),
              "tokens": start[-1], "page": page})
    return s


def _prepare_tree(case, s, dev):
    """Masks of the new tokens in words of 64 and their positions, which count the tokens that they continue."""
    (new, past), words = _lengths(case), -(-case["new"] // 64)
    rows, pos = [], []
    for up, p in zip(_parents(case), past):
        sees = []
        for i, u in enumerate(up):
            sees.append((sees[u] if u >= 0 else 0) | 1 << i)
            rows.append([sees[i] >> 64 * w & (1 << 64) - 1 for w in range(words)])
            pos.append(p + bin(sees[i]).count("1") - 1)
    rows = [[w - (1 << 64) if w >> 63 else w for w in r] for r in rows]
    s["mask"] = torch.tensor(rows, dtype=torch.int64, device=dev)
    s["pos"] = torch.tensor(pos, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    if case["op"] == "fork":
        page, room, d = case["page"], case["room"], case["dim"]
        held, origin = _origins(case)
        need = [-(-t // page) for t in held]
        width = max(-(-(t + room) // page) for t in held) + 2
        pages = sum(need) + case["outs"] * (-(-room // page) + 1) + 5
        s = _cache(gen, dev, case["layers"], pages, case["kv_heads"], page, d)
        order = torch.randperm(pages, generator=gen, device=dev).int()
        table = torch.full((len(need), width), -1, dtype=torch.int32, device=dev)
        refs = torch.zeros(pages, dtype=torch.int32, device=dev)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        refs[order[:at].long()] = 1
        s.update({"op": "fork", "table": table, "len": torch.tensor(held, dtype=torch.int32, device=dev), "refs": refs,
                  "parent": torch.tensor(origin, dtype=torch.int32, device=dev), "room": room, "page": page})
        s["caches"] = list(zip(s["k"].unbind(), s["ke"].unbind(), s["v"].unbind(), s["ve"].unbind()))
        return s
    s = _prepare_batch(case, gen, dev, case.get("layers", 1))
    t, hk, d = s["tokens"], case["kv_heads"], case["dim"]
    s["caches"] = list(zip(s["k"].unbind(), s["ke"].unbind(), s["v"].unbind(), s["ve"].unbind()))
    if case["op"] == "compact":
        paths = _paths(case)
        width = max(1, max(len(p) for p in paths))
        s["keep"] = torch.tensor([p + [-1] * (width - len(p)) for p in paths], dtype=torch.int32, device=dev)
        s["kept"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=dev)
        return s
    h, dt = case["heads"], DTYPES[case["dtype"]]
    if case["op"] == "tree":
        _prepare_tree(case, s, dev)
        s["q"] = (torch.randn(t, h, d, generator=gen, device=dev) * 1.5).to(dt)
        s["window"] = case["window"]
        return s
    # what the fused projection of a layer gives: a token's queries, keys and values beside each other
    qkv = torch.randn(t, h + 2 * hk, d, generator=gen, device=dev)
    qkv *= torch.exp(torch.randn(t, h + 2 * hk, 1, generator=gen, device=dev))
    qkv = qkv.to(dt)
    s["q"], s["new_k"], s["new_v"] = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
    s["wq"] = (1.0 + 0.3 * torch.randn(d, generator=gen, device=dev)).to(dt)
    s["wk"] = (1.0 + 0.3 * torch.randn(d, generator=gen, device=dev)).to(dt)
    s["cos"] = s["sin"] = s["pos"] = None
    if case["rot"]:
        f = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
        angle = torch.arange(s["max_len"], device=dev, dtype=torch.float64)[:, None] * f
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    if case["drafted"]:
        _prepare_tree(case, s, dev)
    s["interleaved"] = case["interleaved"]
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["op"]
    if own:
        from w8a8_quantized_linear_channel_amd import ops as q8

        if op == "fork":
            f = q8.q8_kv_fork(state["caches"], state["table"], state["len"], state["refs"], state["parent"],
                              room=state["room"])
            return _with_cache(state, {"table": f.block_table, "len": f.kv_len, "refs": f.refs, "missing": f.missing})
        batch = q8.KvBatch(state["start"], state["len"], state["table"], state["max_new"], state["max_len"])
        if op == "compact":
            length = q8.q8_kv_compact(state["caches"], batch, state["keep"], state["kept"])
            return _with_cache(state, {"len": length})
        cache = q8.KvCache(*state["caches"][0])
        if op == "tree":
            return q8.q8_attention_kv8_tree(state["q"], cache, batch, state["mask"], positions=state["pos"],
                                            window=state["window"])
        q = q8.q8_kv_append_norm(state["new_k"], state["new_v"], cache, batch, q=state["q"], q_weight=state["wq"],
                                 k_weight=state["wk"], eps=EPS, cos=state["cos"], sin=state["sin"],
                                 interleaved=state["interleaved"], positions=state["pos"])
        return _with_cache(state, {"q": q})
    if op == "fork":
        return _plain_fork(state)
    if op == "compact":
        return _plain_compact(state)
    return _plain_append(state) if op == "append" else _plain_tree(state)


def _with_cache(state, more):
    names = ("k", "k_exp", "v", "v_exp")
    more.update({"%s%d" % (n, i): t for i, c in enumerate(state["caches"]) for n, t in zip(names, c)})
    return more


def _normed(x, weight):
    """x over the root of its features' mean square, times the weight, in 32 bits; the mean in 64."""
    r = (x.double().square().mean(-1, keepdim=True) + EPS).rsqrt().float()
    return x.float() * r * weight.float()


def _rotated(x, pos, s):
    """x [tokens, heads, dim] in 32 bits, its first 2 r features rotated by cos, sin [positions, r]."""
    if s["cos"] is None:
        return x
    c, z = s["cos"][pos][:, None], s["sin"][pos][:, None]
    r = c.shape[2]
    if s["interleaved"]:
        a, b = x[:, :, 0:2 * r:2], x[:, :, 1:2 * r:2]
        y = torch.stack((a * c - b * z, b * c + a * z), 3).flatten(2)
    else:
        a, b = x[:, :, :r], x[:, :, r:2 * r]
        y = torch.cat((a * c - b * z, b * c + a * z), 2)
    return torch.cat((y, x[:, :, 2 * r:]), 2)


def _put(codes, exps, at, rows, fresh, old, tokens_last):
    """rows [layers, pages, heads, page, dim] in 32 bits into the pages `at` where `fresh` [pages, page]; the older
    tokens `old` of a page at its new scale; codes [layers, all pages, ...], exps [layers, all pages, heads]."""
    is_new, is_old = fresh[:, None, :, None], old[:, None, :, None]
    rows = torch.where(is_new, rows, 0.0)
    had = exps.view(torch.uint8)[:, at].int()
    want = _exponent(rows.abs().amax((3, 4)))
    e = torch.where(old.any(1)[:, None], torch.maximum(had, want), want)
    e = torch.where(fresh.any(1)[:, None], e, had)
    before = codes[:, at].float()
    if tokens_last:
        before = before.transpose(3, 4)
    kept = torch.where(is_old, before * _two_to(had - e)[..., None, None], before)
    got = torch.where(is_new, rows * _two_to(127 - e)[..., None, None], kept).to(torch.float8_e4m3fn)
    codes.view(torch.uint8)[:, at] = (got.transpose(3, 4) if tokens_last else got).view(torch.uint8)
    exps.view(torch.uint8)[:, at] = e.byte()


def _pages_of(s, low, high, most):
    """The pages that slots low .. high - 1 of each sequence fall in, as many for each as `most` slots may need (the
    last one repeated): page numbers [pages], their slots [pages, page], and sequence [pages]."""
    page = s["page"]
    reach = (most + page - 2) // page + 1
    first, last = low // page, (high - 1).clamp(min=0) // page
    logical = torch.minimum(first[:, None] + torch.arange(reach, device=low.device), torch.maximum(first, last)[:, None])
    logical = logical.clamp(max=s["table"].shape[1] - 1)
    at = s["table"].gather(1, logical).long().flatten()
    place = (logical[:, :, None] * page + torch.arange(page, device=low.device)).flatten(0, 1)
    return at, place, torch.arange(len(low), device=low.device).repeat_interleave(reach)


def _plain_append(s):
    t = s["tokens"]
    start, total = s["start"].long(), s["len"].long()
    past = total - (start[1:] - start[:-1])
    token = torch.arange(t, device=start.device)
    seq = torch.searchsorted(start[1:], token, right=True)
    pos = past[seq] + token - start[seq] if s["pos"] is None else s["pos"].long()
    q = _rotated(_normed(s["q"], s["wq"]), pos, s).to(s["q"].dtype)
    at, place, of = _pages_of(s, past, total, s["max_new"])
    low, high = past[of][:, None], total[of][:, None]
    old, fresh = place < low, (place >= low) & (place < high)
    source = (start[:-1][of][:, None] + place - low).clamp(0, t - 1)
    k = _rotated(_normed(s["new_k"], s["wk"]), pos, s)
    _put(s["k"], s["ke"], at, k[source].transpose(1, 2)[None], fresh, old, False)
    _put(s["v"], s["ve"], at, s["new_v"].float()[source].transpose(1, 2)[None], fresh, old, True)
    return _with_cache(s, {"q": q})


def _plain_compact(s):
    page, width = s["page"], s["keep"].shape[1]
    total, keep, kept = s["len"].long(), s["keep"].long(), s["kept"].long()
    past = total - (s["start"][1:] - s["start"][:-1]).long()
    i = torch.arange(width, device=past.device)
    moved = (i < kept[:, None]) & (keep != i)
    stay = ((i < kept[:, None]) & (keep == i)).sum(1)                 # those at the front that are in place
    at, place, of = _pages_of(s, past, past + kept, width)
    which = place - past[of][:, None]
    inside = which.clamp(0, width - 1)
    fresh = (which >= 0) & (which < width) & moved[of].gather(1, inside)
    old = which < stay[of][:, None]
    slot = (past[of][:, None] + keep[of].gather(1, inside)).clamp(min=0)
    src = s["table"][of].gather(1, (slot // page).clamp(max=s["table"].shape[1] - 1)).long().clamp(min=0)
    off = slot % page
    head = torch.arange(s["k"].shape[2], device=past.device)
    size = lambda e: _two_to(e.view(torch.uint8)[:, src].int() - 127).unsqueeze(-1)  # noqa: E731  [layers, pages, page, heads, 1]
    layer = torch.arange(s["k"].shape[0], device=past.device)[:, None, None, None]
    where = (layer, src[None, :, :, None], head[None, None, None])
    k = s["k"].view(torch.uint8)[where + (off[None, :, :, None],)].view(torch.float8_e4m3fn).float() * size(s["ke"])
    v = s["v"].view(torch.uint8).transpose(3, 4)[where + (off[None, :, :, None],)].view(torch.float8_e4m3fn).float() * size(s["ve"])
    _put(s["k"], s["ke"], at, k.transpose(2, 3), fresh, old, False)
    _put(s["v"], s["ve"], at, v.transpose(2, 3), fresh, old, True)
    return _with_cache(s, {"len": (past + kept).int()})


def _plain_fork(s):
    page, table, refs, parent = s["page"], s["table"].long(), s["refs"].long(), s["parent"].long()
    (n, width), pages, outs = table.shape, len(refs), len(parent)
    dev = table.device
    there = (parent >= 0) & (parent < n)
    p = parent.clamp(0, n - 1)
    length = torch.where(there, s["len"].long()[p].clamp(0, width * page), 0)
    full = length // page
    need = torch.where(there, ((length + s["room"] + page - 1) // page).clamp(max=width), 0)
    j = torch.arange(width, device=dev)
    entry = table[p]
    known = (entry >= 0) & (entry < pages)
    held = entry.clamp(0, pages - 1)
    first = there & ~((parent[:, None] == parent) & torch.ones(outs, outs, dtype=torch.bool, device=dev).tril(-1)).any(1)
    shared = (j < full[:, None]) & known
    own_page = (j >= full[:, None]) & (j < need[:, None]) & first[:, None] & known & (refs[held] == 1)
    fresh = (j >= full[:, None]) & (j < need[:, None]) & ~own_page
    copied = fresh & (j == full[:, None]) & (length % page > 0)[:, None] & known

    def count(of, which):
        return torch.zeros(pages + 1, dtype=torch.long, device=dev).scatter_add_(
            0, torch.where(which, of, pages).flatten(), which.flatten().long())[:pages]

    after = refs - count(table.clamp(0, pages - 1), (table >= 0) & (table < pages)) + count(held, shared | own_page)
    free = after + count(held, copied) == 0
    by_rank = torch.full((pages + 1,), -1, dtype=torch.long, device=dev)
    by_rank.scatter_(0, torch.where(free, free.long().cumsum(0) - 1, pages), torch.arange(pages, device=dev))
    by_rank = torch.where(torch.arange(pages + 1, device=dev) < free.sum(), by_rank, -1)
    taken = by_rank[(fresh.flatten().long().cumsum(0) - 1).clamp(0, pages).view(outs, width)]
    out = torch.where(fresh, taken, torch.where(shared | own_page, held, -1))
    got = fresh & (taken >= 0)
    after = after + count(taken.clamp(min=0), got)
    open_page = full.clamp(max=width - 1)[:, None]
    lost = (fresh & ~got & (j == full[:, None])).any(1) & (length % page > 0)
    # rows without a copy repeat one that has one
    does = (copied & got).any(1)
    row = torch.where(does, torch.arange(outs, device=dev), does.long().argmax())
    src, dst = held.gather(1, open_page)[row, 0], out.gather(1, open_page)[row, 0]
    dst = torch.where(does.any(), dst, src)
    s["k"].view(torch.uint8)[:, dst] = s["k"].view(torch.uint8)[:, src]
    s["v"].view(torch.uint8)[:, dst] = s["v"].view(torch.uint8)[:, src]
    s["ke"].view(torch.uint8)[:, dst] = s["ke"].view(torch.uint8)[:, src]
    s["ve"].view(torch.uint8)[:, dst] = s["ve"].view(torch.uint8)[:, src]
    return _with_cache(s, {"table": out.int(), "len": torch.where(lost, full * page, length).int(), "refs": after.int(),
                           "missing": (fresh & ~got).sum().int().view(1)})


def _plain_tree(s):
    q, page = s["q"], s["page"]
    t, h, d = q.shape
    start, total = s["start"].long(), s["len"].long()
    cache_k, cache_v, ke, ve = s["k"][0], s["v"][0], s["ke"][0], s["ve"][0]
    n, hk, wide = len(total), cache_k.shape[1], s["max_new"]
    past = total - (start[1:] - start[:-1])
    at = s["table"].long().clamp(min=0)
    length = at.shape[1] * page
    k = cache_k[at].float() * ke[at].float()[:, :, :, None, None]               # [seqs, pages, heads, page, dim]
    k = k.transpose(1, 2).reshape(n, hk, length, d)
    v = cache_v[at].float() * ve[at].float()[:, :, :, None, None]               # [seqs, pages, heads, dim, page]
    v = v.permute(0, 2, 1, 4, 3).reshape(n, hk, length, d)
    rows = (start[:-1, None] + torch.arange(wide, device=q.device)).clamp(max=t - 1)
    x = q[rows].float().view(n, wide, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, d)
    p = (x @ k.transpose(2, 3)).view(n, hk, h // hk, wide, length)
    p *= 1.0 / math.sqrt(d)
    key = torch.arange(length, device=q.device)
    which = key - past[:, None]                                                  # of the new tokens
    bit = which.clamp(0, 64 * s["mask"].shape[1] - 1)[:, None].expand(n, wide, length)
    drafted = (s["mask"][rows].gather(2, bit // 64) >> bit % 64) & 1 == 1
    drafted = drafted & (which >= 0)[:, None] & (key < total[:, None])[:, None]
    cached = (which < 0)[:, None].expand(n, wide, length)
    if s["window"]:
        cached = cached & (key > s["pos"].long()[rows][:, :, None] - s["window"])
    seen = (drafted | cached)[:, None, None]
    p = p.masked_fill_(~seen, -math.inf)
    top = p.amax(4, keepdim=True).clamp(min=-3e38)
    p = p.sub_(top).exp_()
    p = p / p.sum(4, keepdim=True).clamp(min=1e-30)
    y = (p.view(n, hk, -1, length) @ v).view(n, hk, h // hk, wide, d).permute(0, 3, 1, 2, 4)
    token = torch.arange(t, device=q.device)
    seq = torch.searchsorted(start[1:], token, right=True)
    return y[seq, token - start[seq]].reshape(t, h, d).to(q.dtype)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    hk, d, page, op = case["kv_heads"], case["dim"], case["page"], case["op"]
    if op == "fork":
        held, origin = _origins(case)
        copies = sum(p >= 0 and p in origin[:i] and held[p] % page > 0 for i, p in enumerate(origin))
        width = max(-(-(t + case["room"]) // page) for t in held) + 2
        pages = sum(-(-t // page) for t in held) + case["outs"] * (-(-case["room"] // page) + 1) + 5
        moved = copies * case["layers"] * 2 * (2 * hk * page * d + 2 * hk)
        return {"bytes": moved + 4 * (width + 1) * (len(held) + len(origin)) + 8 * pages + 4 * len(origin), "flops": 0}
    new, past = _lengths(case)
    t = sum(new)
    if op == "compact":
        paths, moved, pages = _paths(case), 0, 0
        for path, p in zip(paths, past):
            slots = [i for i, u in enumerate(path) if u != i]
            moved += len(slots)
            pages += len({(p + i) // page for i in slots} | {(p + path[i]) // page for i in slots})
        return {"bytes": case["layers"] * (4 * moved * hk * d + 2 * hk * pages) + 4 * sum(map(len, paths)) + 16 * len(new),
                "flops": case["layers"] * 2 * moved * hk * d}
    h, es = case["heads"], BYTES[case["dtype"]]
    if op == "append":
        pages = sum((p + n - 1) // page - p // page + 1 for n, p in zip(new, past))
        moved = t * (2 * hk + 2 * h) * d * es + 2 * t * hk * d + 2 * pages * hk + t * case["rot"] * 4
        return {"bytes": moved + 2 * d * es + (4 * t if case["drafted"] else 0),
                "flops": 3 * t * (h + hk) * case["rot"] + 5 * t * (h + hk) * d + 3 * t * 2 * hk * d}
    pairs = keys = 0
    for up, p in zip(_parents(case), past):
        deep = []
        for u in up:
            deep.append(deep[u] + 1 if u >= 0 else 0)
        lows = [max(0, p + x - case["window"] + 1) if case["window"] else 0 for x in deep]
        pairs += sum(max(0, p - low) + x + 1 for low, x in zip(lows, deep))
        keys += len(up) + max(0, p - min(lows))
    words = -(-case["new"] // 64)
    return {"bytes": 2 * t * h * d * es + 2 * keys * hk * d + 2 * hk * keys // page + 8 * t * words, "flops": 4 * pairs * h * d}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _exp2(e):
    """2^e in 64 bits for whole e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3_nearest(x):
    """x (64 bits) to the nearest e4m3 value, ties to the even one, 448 at most."""
    size = x.abs().clamp(max=E4M3_MAX)
    _, e = torch.frexp(size)                             # size = f * 2^e, f in [0.5, 1)
    ulp = _exp2((e - 4).clamp(min=-9))
    return torch.copysign(torch.round(size / ulp) * ulp, x)


def _byte_of(largest):
    """As in the definition, of one number: the least b >= 0 with largest <= 448 * 2^(b - 127)."""
    b = 0 if largest <= 0.0 else max(0, math.ceil(math.log2(largest / E4M3_MAX)) + 127)
    while largest > E4M3_MAX * 2.0 ** (b - 127):
        b += 1
    while b > 0 and largest <= E4M3_MAX * 2.0 ** (b - 128):
        b -= 1
    return b


def _power(e, dev):
    return torch.tensor([2.0 ** u for u in e], dtype=torch.float64, device=dev)[:, None, None]


def _exact_put(codes, exps, at, lo, hi, rows):
    """rows [heads, hi - lo, dim] (64 bits) into slots lo .. hi - 1 of page `at`; codes [pages, heads, page, dim] (64
    bits) and exps (lists of bytes) are changed."""
    want = [_byte_of(u) for u in rows.abs().amax((1, 2)).tolist()]
    held = exps[at]
    if lo > 0:
        want = [max(u, w) for u, w in zip(held, want)]
        codes[at, :, :lo] = _e4m3_nearest(codes[at, :, :lo] * _power([u - w for u, w in zip(held, want)], rows.device))
    codes[at, :, lo:hi] = _e4m3_nearest(rows * _power([127 - w for w in want], rows.device))
    exps[at] = want


def _exact_outputs(state, codes, exps, more):
    dev = state["table"].device
    for i in range(len(state["caches"])):
        for n in ("k", "v"):
            more["%s%d" % (n, i)] = codes[n][i] if n == "k" else codes[n][i].transpose(2, 3)
            more["%s_exp%d" % (n, i)] = _exp2(torch.tensor(exps[n][i], device=dev) - 127)
    return more


def exact(case, seed):
    s = prepare(case, seed)
    page, d, dev = case["page"], case["dim"], s["table"].device
    table = s["table"].tolist()
    if case["op"] != "tree":
        codes = {"k": [k.double() for k in s["k"]], "v": [v.double().transpose(2, 3) for v in s["v"]]}
        exps = {n: [e.view(torch.uint8).tolist() for e in s[n + "e"]] for n in ("k", "v")}
    if case["op"] == "fork":
        lens, refs, width = s["len"].tolist(), s["refs"].tolist(), len(table[0])
        before, out, length, wanted, copies = list(refs), [], [], [], []
        for row in table:
            for u in row:
                if u >= 0:
                    refs[u] -= 1
        seen = set()
        for i, p in enumerate(s["parent"].tolist()):
            row, have = [-1] * width, 0
            if p >= 0:
                have = lens[p]
                for x in range(min(width, -(-(have + case["room"]) // page))):
                    old = table[p][x]
                    if x < have // page or (p not in seen and old >= 0 and before[old] == 1):
                        row[x] = old
                        refs[old] += 1
                    else:
                        wanted.append((i, x, old if x == have // page and have % page else -1))
                seen.add(p)
            out.append(row)
            length.append(have)
        held = {old for _, _, old in wanted if old >= 0}
        free = iter([u for u in range(len(refs)) if refs[u] == 0 and u not in held])
        missing = 0
        for i, x, old in wanted:
            u = next(free, -1)
            out[i][x] = u
            if u < 0:
                missing += 1
                length[i] = min(length[i], x * page)
                continue
            refs[u] += 1
            if old >= 0:
                copies.append((old, u))
        for old, u in copies:
            for n in ("k", "v"):
                for c, e in zip(codes[n], exps[n]):
                    c[u] = c[old]
                    e[u] = list(e[old])
        whole = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        return _exact_outputs(s, codes, exps, {"table": whole(out), "len": whole(length), "refs": whole(refs),
                                               "missing": whole([missing])})
    new, past = _lengths(case)
    start = s["start"].tolist()
    if case["op"] == "compact":
        for n in ("k", "v"):
            for c, e in zip(codes[n], exps[n]):
                for i, (path, p) in enumerate(zip(_paths(case), past)):
                    slots = [x for x, u in enumerate(path) if u != x]
                    if not slots:
                        continue
                    from_page = [table[i][(p + path[x]) // page] for x in slots]
                    value = c[from_page, :, [(p + path[x]) % page for x in slots]]          # [moved, heads, dim]
                    value = value * _exp2(torch.tensor([e[u] for u in from_page], device=dev) - 127)[:, :, None]
                    a = p + slots[0]
                    while a < p + len(path):
                        b = min(p + len(path), (a // page + 1) * page)
                        rows = value[a - p - slots[0]:b - p - slots[0]].transpose(0, 1)
                        _exact_put(c, e, table[i][a // page], a % page, (b - 1) % page + 1, rows)
                        a = b
        return _exact_outputs(s, codes, exps, {"len": torch.tensor([p + len(u) for p, u in zip(past, _paths(case))],
                                                                   dtype=torch.int32, device=dev)})
    q = s["q"].double()
    if case["op"] == "append":
        k, v = s["new_k"].double(), s["new_v"].double()
        q = q / torch.sqrt((q * q).sum(2, keepdim=True) / d + EPS) * s["wq"].double()
        k = k / torch.sqrt((k * k).sum(2, keepdim=True) / d + EPS) * s["wk"].double()
        pos = torch.cat([torch.arange(p, p + n) for n, p in zip(new, past)]).to(dev)
        if case["drafted"]:
            pos = s["pos"].long()
        if case["rot"]:
            r = case["rot"] // 2
            turn = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None]
            here = [slice(0, 2 * r, 2), slice(1, 2 * r, 2)] if case["interleaved"] else [slice(0, r), slice(r, 2 * r)]
            for x in (q, k):
                z = torch.complex(x[:, :, here[0]], x[:, :, here[1]]) * turn
                x[:, :, here[0]], x[:, :, here[1]] = z.real, z.imag
        for i, (n, p) in enumerate(zip(new, past)):
            a = p
            while a < p + n:
                b = min(p + n, (a // page + 1) * page)
                for name, x in (("k", k), ("v", v)):
                    rows = x[start[i] + a - p:start[i] + b - p].transpose(0, 1)
                    _exact_put(codes[name][0], exps[name][0], table[i][a // page], a % page, (b - 1) % page + 1, rows)
                a = b
        return _exact_outputs(s, codes, exps, {"q": q})
    h, hk = case["heads"], case["kv_heads"]
    y = torch.zeros_like(q)
    for i, (up, n, p) in enumerate(zip(_parents(case), new, past)):
        at = [u for u in table[i] if u >= 0]
        sees = torch.zeros(n, n, dtype=torch.bool)
        for a, u in enumerate(up):
            if u >= 0:
                sees[a] = sees[u]
            sees[a, a] = True
        depth = sees.sum(1) - 1
        hide = torch.cat((torch.zeros(n, p, dtype=torch.bool), ~sees), 1)
        if case["window"]:
            hide[:, :p] = torch.arange(p) <= (p + depth - case["window"])[:, None]
        hide = hide.to(dev).repeat_interleave(h // hk, 0)
        for g in range(hk):
            k = (s["k"][0][at, g].double() * s["ke"][0][at, g].double()[:, None, None]).reshape(-1, d)[:n + p]
            v = (s["v"][0][at, g].double() * s["ve"][0][at, g].double()[:, None, None]).transpose(1, 2).reshape(-1, d)[:n + p]
            rows = q[start[i]:start[i + 1], g * (h // hk):(g + 1) * (h // hk)].reshape(-1, d)
            score = (rows @ k.t().contiguous() / math.sqrt(d)).masked_fill(hide, -math.inf)
            y[start[i]:start[i + 1], g * (h // hk):(g + 1) * (h // hk)] = (torch.softmax(score, 1) @ v).view(n, h // hk, d)
    return y
