"""Plain CPU forms of the paged 8-bit cache, the attention over it and the
block-scaled FP8 product, from their definitions, for the tests: rotation in
binary32 as it is defined, everything else in 64 bits."""
import math

import numpy as np
import torch

E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def e4m3_codes(x):
    """Codes of the e4m3 values nearest to x (float64), ties to even, 448 at most."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    _, e = np.frexp(a)
    ulp = np.ldexp(1.0, np.maximum(e - 4, -9))
    a = np.rint(a / ulp) * ulp
    pos = E4M3[:127]                                     # 0 .. 448, ascending
    return (np.searchsorted(pos, a) + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def exponent(amax):
    b = 0
    while amax > 448.0 * 2.0 ** (b - 127):
        b += 1
    return b


def rotate(x, pos, cos, sin, interleaved):
    """x float32 [tokens, heads, dim]; every product and sum rounded to binary32."""
    if cos is None:
        return x
    y = x.copy()
    r = cos.shape[1]
    c, s = cos[pos][:, None], sin[pos][:, None]
    ia, ib = (slice(0, 2 * r, 2), slice(1, 2 * r, 2)) if interleaved else (slice(0, r), slice(r, 2 * r))
    a, b = x[:, :, ia], x[:, :, ib]
    y[:, :, ia] = a * c - b * s
    y[:, :, ib] = b * c + a * s
    return y


def append(cache, table, q_start, kv_len, k, v, cos=None, sin=None, interleaved=False):
    """cache: dict of numpy uint8 arrays k, ke, v, ve, changed in place; k, v float32
    [tokens, heads, dim]."""
    page = cache["k"].shape[2]
    P, H = cache["ke"].shape
    for s in range(len(kv_len)):
        n = q_start[s + 1] - q_start[s]
        past = kv_len[s] - n
        pos = np.arange(past, kv_len[s])
        rows = np.arange(q_start[s], q_start[s + 1])
        keep = (pos >= 0) & (pos < table.shape[1] * page)
        pos, rows = pos[keep], rows[keep]
        if len(pos) == 0:
            continue
        kr = rotate(k[rows], np.minimum(pos, len(cos) - 1) if cos is not None else pos, cos, sin, interleaved)
        for lp in range(pos[0] // page, pos[-1] // page + 1):
            at = table[s, lp]
            if not 0 <= at < P:
                continue
            here = pos // page == lp
            off, lo = pos[here] % page, max(past, 0) - lp * page
            for name, x in (("k", kr), ("v", v[rows])):
                codes = cache[name][at]                  # [heads, page, dim] or [heads, dim, page]
                for h in range(H):
                    new = x[here, h].astype(np.float64)
                    want, had = exponent(np.abs(new).max()), int(cache[name + "e"][at, h])
                    b = want if lo <= 0 else max(want, had)
                    view = codes[h] if name == "k" else codes[h].T
                    if lo > 0 and b != had:
                        view[:lo] = e4m3_codes(E4M3[view[:lo]] * 2.0 ** (had - b))
                    view[off] = e4m3_codes(new * 2.0 ** (127 - b))
                    cache[name + "e"][at, h] = b


def gathered(cache, table_row, total, name):
    """Float64 [heads, total, dim] of one sequence."""
    page = cache["k"].shape[2]
    at = table_row[:-(-total // page)]
    x = E4M3[cache[name][at]] * 2.0 ** (cache[name + "e"][at].astype(np.float64) - 127)[:, :, None, None]
    if name == "v":
        x = x.transpose(0, 1, 3, 2)
    return x.transpose(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :total]


def attention(cache, table, q_start, kv_len, q, scale=None, causal=True, window=0):
    """q float64 [tokens, heads, dim].  Returns out, lse and, per output, the
    weighted mean of |v| and the largest scale * sum |q k| over the keys seen
    (for error bounds)."""
    T, Hq, D = q.shape
    Hk = cache["ke"].shape[1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    av, aqk = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for s in range(len(kv_len)):
        n, total = q_start[s + 1] - q_start[s], kv_len[s]
        if n == 0 or total == 0:
            continue
        lo_key = max(0, total - n - window + 1) if window else 0
        row = table[s].copy()
        row[:lo_key // cache["k"].shape[2]] = 0          # pages no query sees
        k, v = gathered(cache, row, total, "k"), gathered(cache, row, total, "v")
        k, v = k[:, lo_key:], v[:, lo_key:]
        for i in range(n):
            p = total - n + i
            j = np.arange(lo_key, total)
            seen = np.ones(len(j), bool)
            if causal:
                seen &= j <= p
            if window:
                seen &= j > p - window
            if not seen.any():
                continue
            t = q_start[s] + i
            for h in range(Hq):
                kk, vv = k[h // (Hq // Hk)][seen], v[h // (Hq // Hk)][seen]
                sc = kk @ q[t, h] * scale
                m = sc.max()
                w = np.exp(sc - m)
                lse[t, h] = m + math.log(w.sum())
                w /= w.sum()
                out[t, h], av[t, h] = w @ vv, w @ np.abs(vv)
                aqk[t, h] = (np.abs(kk) @ np.abs(q[t, h])).max() * abs(scale)
    return out, lse, av, aqk


def block_quantize_act(x):
    """x float32 [M, K] -> codes [M, K], scale float32 [ceil(K/128), M]."""
    M, K = x.shape
    G = -(-K // 128)
    codes, scale = np.zeros((M, K), np.uint8), np.zeros((G, M), np.float32)
    for j in range(G):
        part = x[:, 128 * j:128 * j + 128]
        s = np.maximum(np.abs(part).max(1) / np.float32(448), np.float32(1e-8)).astype(np.float32)
        scale[j] = s
        codes[:, 128 * j:128 * j + 128] = e4m3_codes((part / s[:, None]).astype(np.float32))
    return codes, scale


def block_quantize_weight(w):
    N, K = w.shape
    codes, scale = np.zeros((N, K), np.uint8), np.zeros((-(-N // 128), -(-K // 128)), np.float32)
    for i in range(scale.shape[0]):
        for j in range(scale.shape[1]):
            part = w[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            s = np.maximum(np.float32(np.abs(part).max()) / np.float32(448), np.float32(1e-8))
            scale[i, j] = s
            codes[128 * i:128 * i + 128, 128 * j:128 * j + 128] = e4m3_codes((part / s).astype(np.float32))
    return codes, scale


def block_product(xq, xs, wq, ws, bias=None):
    """Exact product in 64 bits, and the same of the absolute values."""
    M, K = xq.shape
    N = wq.shape[0]
    y, a = np.zeros((M, N)), np.zeros((M, N))
    for j in range(xs.shape[0]):
        x, w = E4M3[xq[:, 128 * j:128 * j + 128]], E4M3[wq[:, 128 * j:128 * j + 128]]
        s = xs[j].astype(np.float64)[:, None] * np.repeat(ws[:, j].astype(np.float64), 128)[:N][None]
        y += s * (x @ w.T)
        a += s * (np.abs(x) @ np.abs(w).T)
    return (y if bias is None else y + bias), a
