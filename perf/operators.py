"""Cases for the block-scaled FP8 product and the 8-bit paged key/value cache.

Three operators of a decoder layer served in 8 bits:

  append     rotate new keys (and queries) by their position and put keys and
             values into a paged e4m3 cache whose scale is one power of two per
             page and head                                  (q8_kv_append)
  attention  softmax attention of new queries over that cache, from one token
             to a whole prompt                              (q8_attention_kv8)
  linear     Y = X W^T in e4m3 with one scale per token and 128 features for X
             and one per 128 x 128 block for W              (q8_linear_fp8_block)

`run` makes one call of an operator: in elementary torch operations in 32 bits
where `own` is false, through this package where it is true.  Cache layout:
keys uint8 [pages, kv_heads, page, dim], values uint8 [pages, kv_heads, dim,
page] (tokens innermost), both e4m3 codes; one exponent byte b per page and
head, a code c standing for e4m3(c) * 2^(b - 127).  Codes come back as
float8_e4m3fn and exponent bytes as float8_e8m0fnu views of the same buffers.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = 128      # features (and weight rows) that share a scale
E4M3_MAX = 448.0


# ------------------------------------------------------------------ the cases
def _append(name, seqs, new, past, heads, kv_heads, dim, page, rot, interleaved, dtype, ragged):
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "past": past, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "rot": rot, "interleaved": interleaved, "dtype": dtype, "ragged": ragged}


def _attention(name, seqs, new, past, heads, kv_heads, dim, page, causal, window, dtype, ragged):
    return {"name": name, "op": "attention", "seqs": seqs, "new": new, "past": past, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "causal": causal, "window": window, "dtype": dtype,
            "ragged": ragged}


def _linear(name, m, n, k, bias, x_dtype, y_dtype):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "bias": bias, "x_dtype": x_dtype, "y_dtype": y_dtype}


def listed():
    return [
        # one chat user, one token: the call's latency is what counts
        _append("append one token", 1, 1, 700, 32, 8, 128, 64, 128, False, "bf16", 0),
        # a decode step of a busy server, sequences of all lengths
        _append("append decode batch", 128, 1, 4000, 32, 8, 128, 64, 128, False, "bf16", 3),
        # prompts of odd lengths continued after a cached prefix; half the head rotated, neighbours as pairs
        _append("append prompts", 6, 3001, 900, 32, 8, 128, 128, 64, True, "fp16", 5),
        # one user, a short conversation
        _attention("attention one token", 1, 1, 512, 32, 8, 128, 64, True, 0, "bf16", 0),
        # a decode step of a busy server
        _attention("attention decode batch", 64, 1, 4099, 32, 8, 128, 64, True, 0, "bf16", 7),
        # two users with very long documents: the long axis has to be split
        _attention("attention long", 2, 1, 120001, 32, 8, 128, 128, True, 0, "bf16", 0),
        # prompt chunks after cached prefixes, small heads, no shared heads, a sliding window
        _attention("attention chunks", 5, 333, 2777, 16, 16, 64, 32, True, 1024, "fp16", 11),
        # one long prompt, nothing cached before
        _attention("attention prompt", 1, 8192, 0, 32, 8, 128, 64, True, 0, "bf16", 0),
        # a projection for one token
        _linear("linear one token", 1, 4096, 4096, False, "bf16", "bf16"),
        # the wide feed-forward product for a few users
        _linear("linear 16 tokens", 16, 14336, 4096, False, "bf16", "bf16"),
        # odd everything: rows and columns that fill no tile, features that end inside a block
        _linear("linear odd", 333, 1000, 2064, True, "fp16", "fp16"),
        # the narrow feed-forward product of a prompt
        _linear("linear prompt", 4096, 4096, 14336, False, "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "linear"])
    if op == "linear":
        k = rng.choice([80 * _log(rng, 4, 179), 640 * _log(rng, 1, 22)])     # ending inside a block, or with one
        n = _log(rng, 64, 14336)
        m = min(_log(rng, 1, 4096), max(1, (1 << 37) // (n * k)))
        x_dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        c = _linear("", m, n, k, rng.random() < 0.5, x_dtype, "bf16" if x_dtype == "fp32" else x_dtype)
    else:
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8] if kv_heads <= 4 else [1, 2, 4])
        dim = rng.choice([64, 128, 128, 256])
        page = rng.choice([32, 64, 128])
        ragged = rng.randrange(1, 1 << 20)
        seqs = _log(rng, 1, 128)
        if op == "append":
            new = rng.choice([1, _log(rng, 2, max(2, 16384 // seqs))])
            past = _log(rng, 1, max(1, 400000 // seqs // kv_heads))
            rot = rng.choice([dim, dim // 2, 0])
            c = _append("", seqs, new, past, heads, kv_heads, dim, page, rot, rng.random() < 0.5,
                        rng.choice(["bf16", "fp16", "fp32"]), ragged)
        else:
            if rng.random() < 0.5:
                new = rng.choice([1, 1, rng.randrange(2, 9)])
                past = _log(rng, 1, min(131072, 240000000 // (kv_heads * dim) // seqs))
            else:
                seqs = rng.randrange(1, 9)
                new = _log(rng, 16, 4096 // seqs)
                past = _log(rng, 1, 8192 // seqs)
            c = _attention("", seqs, new, past, heads, kv_heads, dim, page, rng.random() < 0.8,
                           rng.choice([0, 0, 256, 1000]), rng.choice(["bf16", "fp16"]), ragged)
    del c["name"]
    return c


def _lengths(case):
    """New tokens and cached tokens before them, of each sequence."""
    s, new, past = case["seqs"], case["new"], case["past"]
    if not case["ragged"]:
        return [new] * s, [past] * s
    r = random.Random(case["ragged"])
    return [r.randint((new + 1) // 2, new) for _ in range(s)], [r.randint(past // 8, past) for _ in range(s)]


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


def _prepare_cache(case, gen, dev):
    new, past = _lengths(case)
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    total = [a + b for a, b in zip(new, past)]
    need = [-(-t // page) for t in total]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=dev).int()
    width = max(need)
    table = torch.full((len(need), width), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    # channels of keys differ in size, some by a lot; values are even
    channel = 1.0 + 7.0 * (torch.rand(hk, 1, d, generator=gen, device=dev) < 0.03)
    kf = torch.randn(pages, hk, page, d, generator=gen, device=dev) * channel
    ke = _exponent(kf.abs().amax((2, 3)))
    kq = (kf * _two_to(127 - ke)[:, :, None, None]).to(torch.float8_e4m3fn)
    del kf
    vf = torch.randn(pages, hk, d, page, generator=gen, device=dev)
    ve = _exponent(vf.abs().amax((2, 3)))
    vq = (vf * _two_to(127 - ve)[:, :, None, None]).to(torch.float8_e4m3fn)
    del vf
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    return {
        "op": case["op"], "k": kq, "v": vq, "ke": ke.byte().view(torch.float8_e8m0fnu),
        "ve": ve.byte().view(torch.float8_e8m0fnu), "table": table, "channel": channel,
        "start": torch.tensor(start, dtype=torch.int32, device=dev),
        "len": torch.tensor(total, dtype=torch.int32, device=dev),
        "max_new": max(new), "max_len": max(total), "tokens": start[-1], "page": page,
    }


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        x = torch.randn(m, k, generator=gen, device=dev)
        x *= 1.0 + 19.0 * (torch.rand(m, k, generator=gen, device=dev) < 0.001)
        w = torch.randn(n, k, generator=gen, device=dev) * 0.02
        rows, cols = -(-n // BLOCK), -(-k // BLOCK)
        padded = torch.zeros(rows * BLOCK, cols * BLOCK, device=dev)
        padded[:n, :k] = w
        amax = padded.view(rows, BLOCK, cols, BLOCK).abs().amax((1, 3))
        scale = (amax / E4M3_MAX).clamp(min=1e-8)
        wq = w / scale.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
        wq = wq.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        bias = torch.randn(n, generator=gen, device=dev) * 0.1 if case["bias"] else None
        return {"op": "linear", "x": x.to(DTYPES[case["x_dtype"]]), "wq": wq, "scale": scale, "bias": bias,
                "y_dtype": DTYPES[case["y_dtype"]]}
    s = _prepare_cache(case, gen, dev)
    t, h, hk, d = s["tokens"], case["heads"], case["kv_heads"], case["dim"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "append":
        # what the fused projection of a layer gives: a token's queries, keys and values beside each other
        qkv = torch.randn(t, h + 2 * hk, d, generator=gen, device=dev)
        qkv[:, h:h + hk] *= s["channel"].view(1, hk, d)
        qkv[:, h:h + hk] *= 1.0 + 3.0 * (torch.rand(t, hk, 1, generator=gen, device=dev) < 0.01)
        qkv = qkv.to(dt)
        s["q"], s["new_k"], s["new_v"] = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        s["cos"] = s["sin"] = None
        if case["rot"]:
            f = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
            angle = torch.arange(s["max_len"], device=dev, dtype=torch.float64)[:, None] * f
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["interleaved"] = case["interleaved"]
    else:
        s["q"] = (torch.randn(t, h, d, generator=gen, device=dev) * 1.5).to(dt)
        s["causal"], s["window"] = case["causal"], case["window"]
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        from w8a8_quantized_linear_channel_amd import ops as q8

        if state["op"] == "linear":
            return q8.q8_linear_fp8_block(state["x"], state["wq"], state["scale"], bias=state["bias"],
                                          out_dtype=state["y_dtype"])
        cache = q8.KvCache(state["k"], state["ke"], state["v"], state["ve"])
        batch = q8.KvBatch(state["start"], state["len"], state["table"], state["max_new"], state["max_len"])
        if state["op"] == "append":
            q = q8.q8_kv_append(state["new_k"], state["new_v"], cache, batch, q=state["q"], cos=state["cos"],
                                sin=state["sin"], interleaved=state["interleaved"])
            return {"k": state["k"], "k_exp": state["ke"], "v": state["v"], "v_exp": state["ve"], "q": q}
        return q8.q8_attention_kv8(state["q"], cache, batch, causal=state["causal"], window=state["window"])
    if state["op"] == "linear":
        return _plain_linear(state)
    return _plain_append(state) if state["op"] == "append" else _plain_attention(state)


def _plain_linear(s):
    x, (n, k) = s["x"].float(), s["wq"].shape
    m, cols = x.shape[0], s["scale"].shape[1]
    x = torch.nn.functional.pad(x, (0, cols * BLOCK - k)).view(m, cols, BLOCK)
    xs = (x.abs().amax(2, keepdim=True) / E4M3_MAX).clamp(min=1e-8)
    x = ((x / xs).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).float() * xs).view(m, cols * BLOCK)[:, :k]
    w = s["wq"].view(torch.float8_e4m3fn).float()
    w = w * s["scale"].repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    y = x @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["y_dtype"])


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


def _plain_append(s):
    page, t = s["page"], s["tokens"]
    start, total = s["start"].long(), s["len"].long()
    new = start[1:] - start[:-1]
    past = total - new
    token = torch.arange(t, device=start.device)
    seq = torch.searchsorted(start[1:], token, right=True)
    pos = past[seq] + token - start[seq]
    q = _rotated(s["q"].float(), pos, s).to(s["q"].dtype)
    # the pages that new tokens fall in, as many for each sequence as the longest may need (the last repeated)
    reach = (s["max_new"] + page - 2) // page + 1
    first, last = past // page, (total - 1).clamp(min=0) // page
    logical = torch.minimum(first[:, None] + torch.arange(reach, device=start.device), last[:, None])
    at = s["table"].gather(1, logical).long().flatten()
    place = (logical[:, :, None] * page + torch.arange(page, device=start.device)).flatten(0, 1)
    low, high = past.repeat_interleave(reach)[:, None], total.repeat_interleave(reach)[:, None]
    old, fresh = place < low, (place >= low) & (place < high)
    source = (start[:-1].repeat_interleave(reach)[:, None] + place - low).clamp(0, t - 1)

    def put(codes, exps, rows, tokens_last):
        rows = rows[source].transpose(1, 2)                              # [pages, heads, page, dim]
        is_new, is_old = fresh[:, None, :, None], old[:, None, :, None]
        rows = torch.where(is_new, rows, 0.0)
        had = exps.view(torch.uint8)[at].int()
        want = _exponent(rows.abs().amax((2, 3)))
        e = torch.where(old.any(1)[:, None], torch.maximum(had, want), want)
        e = torch.where(fresh.any(1)[:, None], e, had)
        before = codes[at].float()
        if tokens_last:
            before = before.transpose(2, 3)
        kept = torch.where(is_old, before * _two_to(had - e)[:, :, None, None], before)
        got = torch.where(is_new, rows * _two_to(127 - e)[:, :, None, None], kept).to(torch.float8_e4m3fn)
        codes.view(torch.uint8)[at] = (got.transpose(2, 3) if tokens_last else got).view(torch.uint8)
        exps.view(torch.uint8)[at] = e.byte()

    put(s["k"], s["ke"], _rotated(s["new_k"].float(), pos, s), False)
    put(s["v"], s["ve"], s["new_v"].float(), True)
    return {"k": s["k"], "k_exp": s["ke"], "v": s["v"], "v_exp": s["ve"], "q": q}


def _plain_attention(s):
    q, page = s["q"], s["page"]
    t, h, d = q.shape
    start, total = s["start"].long(), s["len"].long()
    n, hk, wide = len(total), s["k"].shape[1], s["max_new"]
    new = start[1:] - start[:-1]
    at = s["table"].long().clamp(min=0)
    length = at.shape[1] * page
    k = s["k"][at].float() * s["ke"][at].float()[:, :, :, None, None]           # [seqs, pages, heads, page, dim]
    k = k.transpose(1, 2).reshape(n, hk, length, d)
    v = s["v"][at].float() * s["ve"][at].float()[:, :, :, None, None]           # [seqs, pages, heads, dim, page]
    v = v.permute(0, 2, 1, 4, 3).reshape(n, hk, length, d)
    step = torch.arange(wide, device=q.device)
    rows = (start[:-1, None] + step).clamp(max=t - 1)
    x = q[rows].float().view(n, wide, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, d)
    p = (x @ k.transpose(2, 3)).view(n, hk, h // hk, wide, length)
    p *= 1.0 / math.sqrt(d)
    key = torch.arange(length, device=q.device)
    pos = (total - new)[:, None] + step                                         # of each query
    seen = (key < total[:, None, None]).expand(n, wide, length)
    if s["causal"]:
        seen = seen & (key <= pos[:, :, None])
    if s["window"]:
        seen = seen & (key > pos[:, :, None] - s["window"])
    seen = seen[:, None, None]
    p = p.masked_fill_(~seen, -math.inf)
    top = p.amax(4, keepdim=True).clamp(min=-3e38)
    p = p.sub_(top).exp_()
    p = p / p.sum(4, keepdim=True).clamp(min=1e-30)
    y = (p.view(n, hk, -1, length) @ v).view(n, hk, h // hk, wide, d).permute(0, 3, 1, 2, 4)
    token = torch.arange(t, device=q.device)
    seq = torch.searchsorted(start[1:], token, right=True)
    return y[seq, token - start[seq]].reshape(t, h, d).to(q.dtype)


# ------------------------------------------------------------------ what a pass cannot do without
def _pairs(case):
    """Query-key pairs (of one head) that the mask leaves, and keys that any query of their sequence sees."""
    pairs = keys = 0
    for n, p in zip(*_lengths(case)):
        total, w = n + p, case["window"]
        lows = [max(0, p + i - w + 1) if w else 0 for i in range(n)]
        highs = [p + i + 1 if case["causal"] else total for i in range(n)]
        pairs += sum(b - a for a, b in zip(lows, highs))
        keys += highs[-1] - lows[0]
    return pairs, keys


def work(case):
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        blocks = -(-n // BLOCK) * -(-k // BLOCK)
        moved = m * k * BYTES[case["x_dtype"]] + n * k + 4 * blocks + m * n * BYTES[case["y_dtype"]]
        return {"bytes": moved + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    new, past = _lengths(case)
    t, h, hk, d, es = sum(new), case["heads"], case["kv_heads"], case["dim"], BYTES[case["dtype"]]
    if case["op"] == "append":
        pages = sum((p + n - 1) // case["page"] - p // case["page"] + 1 for n, p in zip(new, past))
        moved = t * (2 * hk + 2 * h) * d * es + 2 * t * hk * d + 2 * pages * hk + t * case["rot"] * 4
        return {"bytes": moved, "flops": 3 * t * (h + hk) * case["rot"] + 3 * t * 2 * hk * d}
    pairs, keys = _pairs(case)
    return {"bytes": 2 * t * h * d * es + 2 * keys * hk * d + 2 * hk * keys // case["page"], "flops": 4 * pairs * h * d}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _e4m3_nearest(x):
    """x (64 bits) to the nearest e4m3 value, ties to the even one, 448 at most."""
    size = x.abs().clamp(max=E4M3_MAX)
    _, e = torch.frexp(size)                             # size = f * 2^e, f in [0.5, 1)
    ulp = torch.ldexp(torch.ones_like(size), (e - 4).clamp(min=-9))
    return torch.copysign(torch.round(size / ulp) * ulp, x)


def _byte_of(largest):
    """As in the definition, of one number: the least b >= 0 with largest <= 448 * 2^(b - 127)."""
    b = 0 if largest <= 0.0 else max(0, math.ceil(math.log2(largest / E4M3_MAX)) + 127)
    while largest > E4M3_MAX * 2.0 ** (b - 127):
        b += 1
    while b > 0 and largest <= E4M3_MAX * 2.0 ** (b - 128):
        b -= 1
    return b


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        x, k = s["x"].double(), case["k"]
        y = torch.zeros(case["m"], case["n"], dtype=torch.float64, device=x.device)
        codes = s["wq"].view(torch.float8_e4m3fn).double()
        for j, a in enumerate(range(0, k, BLOCK)):
            part = x[:, a:a + BLOCK]
            scale = (part.abs().amax(1, keepdim=True) / E4M3_MAX).clamp(min=1e-8)
            across = s["scale"][:, j].double().repeat_interleave(BLOCK)[:case["n"]]
            y += scale * (_e4m3_nearest(part / scale) @ codes[:, a:a + BLOCK].t().contiguous()) * across
        return y if s["bias"] is None else y + s["bias"].double()
    new, past = _lengths(case)
    start, page, d = s["start"].tolist(), s["page"], case["dim"]
    table = s["table"].tolist()
    if case["op"] == "append":
        q, k, v = s["q"].double(), s["new_k"].double(), s["new_v"].double()
        pos = torch.cat([torch.arange(p, p + n) for n, p in zip(new, past)]).to(q.device)
        if case["rot"]:
            r = case["rot"] // 2
            turn = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None]
            here = [slice(0, 2 * r, 2), slice(1, 2 * r, 2)] if case["interleaved"] else [slice(0, r), slice(r, 2 * r)]
            for x in (q, k):
                z = torch.complex(x[:, :, here[0]], x[:, :, here[1]]) * turn
                x[:, :, here[0]], x[:, :, here[1]] = z.real, z.imag
        out = {"k": s["k"].double(), "v": s["v"].double().transpose(2, 3)}
        exps = {"k": s["ke"].view(torch.uint8).tolist(), "v": s["ve"].view(torch.uint8).tolist()}
        for i, (n, p) in enumerate(zip(new, past)):
            for j in range(p // page, (p + n - 1) // page + 1):
                a, b, at = max(p, j * page), min(p + n, (j + 1) * page), table[i][j]
                for name, x in (("k", k), ("v", v)):
                    rows = x[start[i] + a - p:start[i] + b - p].transpose(0, 1)
                    tops = rows.abs().amax((1, 2)).tolist()
                    want = [_byte_of(u) for u in tops]
                    held = exps[name][at]
                    if a > j * page:
                        want = [max(u, w) for u, w in zip(held, want)]
                    to = torch.tensor([2.0 ** (127 - w) for w in want], dtype=torch.float64, device=x.device)
                    drop = torch.tensor([2.0 ** (u - w) for u, w in zip(held, want)], dtype=torch.float64, device=x.device)
                    old = out[name][at, :, :a - j * page]
                    out[name][at, :, :a - j * page] = _e4m3_nearest(old * drop[:, None, None])
                    out[name][at, :, a - j * page:b - j * page] = _e4m3_nearest(rows * to[:, None, None])
                    exps[name][at] = want
        value = {n: torch.tensor(e, dtype=torch.float64, device=q.device).sub(127).exp2() for n, e in exps.items()}
        return {"k": out["k"], "k_exp": value["k"], "v": out["v"].transpose(2, 3), "v_exp": value["v"], "q": q}
    q = s["q"].double()
    h, hk = case["heads"], case["kv_heads"]
    y = torch.zeros_like(q)
    for i, (n, p) in enumerate(zip(new, past)):
        at = [u for u in table[i] if u >= 0]
        total = n + p
        key = torch.arange(total, device=q.device)
        for g in range(hk):
            k = (s["k"][at, g].double() * s["ke"][at, g].double()[:, None, None]).reshape(-1, d)[:total]
            v = (s["v"][at, g].double() * s["ve"][at, g].double()[:, None, None]).transpose(1, 2).reshape(-1, d)[:total]
            for u in range(g * (h // hk), (g + 1) * (h // hk)):
                for a in range(0, n, 2048):
                    b = min(n, a + 2048)
                    score = q[start[i] + a:start[i] + b, u] @ k.t().contiguous() / math.sqrt(d)
                    at_q = torch.arange(p + a, p + b, device=q.device)[:, None]
                    hide = key > at_q if case["causal"] else torch.zeros_like(score, dtype=torch.bool)
                    if case["window"]:
                        hide = hide | (key <= at_q - case["window"])
                    score[hide] = -math.inf
                    y[start[i] + a:start[i] + b, u] = torch.softmax(score, 1) @ v
    return y
