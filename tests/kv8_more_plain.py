"""Plain CPU forms of the normalising append, the attention of drafted trees, the
compaction of kept drafts and the forks of paged sequences, from their
definitions, for the tests: norms and attention in 64 bits, codes exactly."""
import math

import numpy as np

import kv8_plain as P


def normalised(x, weight, eps):
    """x float32 [tokens, heads, dim]; r in 64 bits, rounded to binary32 as both products are."""
    if weight is None:
        return x
    m = np.square(x.astype(np.float64)).mean(2, keepdims=True)
    r = (1.0 / np.sqrt(m + float(np.float32(eps)))).astype(np.float32)
    return (x * r) * weight.astype(np.float32)


def rotated(x, pos, cos, sin, interleaved):
    if cos is None:
        return x
    return P.rotate(x, np.clip(pos, 0, len(cos) - 1), cos, sin, interleaved)


def slots(q_start, kv_len):
    """Slot of every token that belongs to a sequence."""
    return np.concatenate([np.arange(b - n, b) for n, b in zip(np.diff(q_start), kv_len)] or [np.zeros(0, int)]).astype(int)


def tree_of(rng, n, root=0.1):
    """Parents of n drafted tokens (-1: the last cached one) and which of them each sees."""
    up = [-1 if i == 0 or rng.random() < root else max(0, i - 1 - int(rng.exponential(2.0))) for i in range(n)]
    sees = np.zeros((n, n), bool)
    for i, u in enumerate(up):
        if u >= 0:
            sees[i] = sees[u]
        sees[i, i] = True
    return up, sees


def words_of(sees, words):
    """Rows of truth values [tokens, up to 64 words] as uint64 [tokens, words]."""
    out = np.zeros((len(sees), words), np.uint64)
    for j in range(sees.shape[1]):
        out[:, j // 64] |= sees[:, j].astype(np.uint64) << np.uint64(j % 64)
    return out


def tree_seen(n, total, sees, pos, window):
    """[n, max(total, 0)]: the keys that each of n new tokens sees; sees [n, any], pos: their positions or None."""
    past, key = total - n, np.arange(max(total, 0))
    seen = np.zeros((n, len(key)), bool)
    for i in range(n):
        p = past + i if pos is None else min(max(int(pos[i]), past), past + n - 1)
        seen[i] = key < past
        if window:
            seen[i] &= key > p - window
        for j in np.flatnonzero(sees[i][:n]):
            if past + j >= 0:
                seen[i, past + j] = True
    return seen


def tree_attention(cache, table, q_start, kv_len, q, sees, pos=None, scale=None, window=0):
    """As kv8_plain.attention; sees: of each sequence a truth array [its new tokens, any]; pos [tokens]."""
    T, Hq, D = q.shape
    Hk = cache["ke"].shape[1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    av, aqk = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    page = cache["k"].shape[2]
    for s in range(len(kv_len)):
        first, n, total = q_start[s], q_start[s + 1] - q_start[s], kv_len[s]
        if n == 0 or total <= 0:
            continue
        seen = tree_seen(n, total, sees[s], None if pos is None else pos[first:first + n], window)
        row = table[s].copy()
        for j in range(-(-total // page)):               # pages that nobody sees need not exist
            if not seen[:, j * page:(j + 1) * page].any():
                row[j] = 0
        k, v = P.gathered(cache, row, total, "k"), P.gathered(cache, row, total, "v")
        for i in range(n):
            if not seen[i].any():
                continue
            for h in range(Hq):
                kk, vv = k[h // (Hq // Hk)][seen[i]], v[h // (Hq // Hk)][seen[i]]
                sc = kk @ q[first + i, h] * scale
                m = sc.max()
                w = np.exp(sc - m)
                lse[first + i, h] = m + math.log(w.sum())
                w /= w.sum()
                out[first + i, h], av[first + i, h] = w @ vv, w @ np.abs(vv)
                aqk[first + i, h] = (np.abs(kk) @ np.abs(q[first + i, h])).max() * abs(scale)
    return out, lse, av, aqk


def rescaled(codes, shift):
    """Codes whose values are taken times 2^shift; NaN codes as they are."""
    nan = (codes & 0x7F) == 0x7F
    value = np.where(nan, 0.0, P.E4M3[np.where(nan, 0, codes)])
    new = P.e4m3_codes(value * 2.0 ** np.asarray(shift, np.float64))
    new = np.where((new & 0x7F) == 0, (codes & 0x80) | (new & 0x7F), new)      # the sign of a zero stays
    return np.where(nan, codes, new).astype(np.uint8)


def path(keep, n):
    """As much of a list of kept tokens as is one."""
    out, last = [], -1
    for i, u in enumerate(keep):
        if u < i or u <= last or u >= n:
            break
        out.append(int(u))
        last = u
    return out


def compact(cache, table, q_start, kv_len, keep, n_keep):
    """cache: dict of numpy uint8 arrays, changed in place (one layer); returns the new lengths."""
    page = cache["k"].shape[2]
    pages, heads = cache["ke"].shape
    cap = table.shape[1] * page
    lens = []
    for s in range(len(kv_len)):
        n = max(0, q_start[s + 1] - q_start[s])
        past = max(kv_len[s], 0) - n
        kept = path(keep[s][:max(0, min(n_keep[s], keep.shape[1]))], n)
        lens.append(max(0, past + len(kept)))
        moves = [(past + i, past + u) for i, u in enumerate(kept) if i != u]
        there = lambda slot: 0 <= slot < cap and 0 <= table[s, slot // page] < pages  # noqa: E731
        # per target page, the slots from the first on that some kept token goes to
        for lp in sorted({t // page for t, _ in moves if 0 <= t < cap}):
            mine = [(t, f) for t, f in moves if t // page == lp and t >= 0]
            at = table[s, lp]
            if not 0 <= at < pages:
                continue
            low = mine[0][0] % page
            mine = [(t, f) for t, f in mine if there(f)]
            if not mine:
                continue
            for name in ("k", "v"):
                exps = cache[name + "e"]
                view = cache[name] if name == "k" else cache[name].transpose(0, 1, 3, 2)
                for h in range(heads):
                    had = int(exps[at, h])
                    rows = [(t % page, view[table[s, f // page], h, f % page].copy(), int(exps[table[s, f // page], h]))
                            for t, f in mine]
                    want = 0
                    for _, c, b in rows:
                        for m in np.abs(P.E4M3[c[(c & 0x7F) != 0x7F]]):
                            w = 0
                            while m > 448.0 * 2.0 ** (w - b):
                                w += 1
                            want = max(want, w)
                    b = want if low == 0 else max(want, had)
                    if low > 0 and b != had:
                        view[at, h, :low] = rescaled(view[at, h, :low], had - b)
                    for t, c, u in rows:
                        view[at, h, t] = rescaled(c, u - b)
                    exps[at, h] = b
    return np.array(lens, np.int32)


def fork(caches, table, kv_len, refs, parent, room):
    """caches: list of dicts, changed in place; returns table, lengths, counts and the number missing."""
    page = caches[0]["k"].shape[2]
    pages = len(refs)
    S, width = table.shape
    known = lambda e: 0 <= e < pages  # noqa: E731
    count = refs.astype(np.int64).copy()
    for e in table.flatten():
        if known(e):
            count[e] -= 1
    out, lens, wanted, heirs = np.full((len(parent), width), -1, np.int32), [], [], set()
    for s, p in enumerate(parent):
        if not 0 <= p < S:
            lens.append(0)
            continue
        L = min(max(int(kv_len[p]), 0), width * page)
        for j in range(min(width, -(-(L + room) // page))):
            e = table[p, j]
            if j < L // page or (p not in heirs and known(e) and refs[e] == 1):
                if known(e):
                    out[s, j] = e
                    count[e] += 1
            else:
                wanted.append((s, j, int(e) if j == L // page and L % page and known(e) else -1))
        heirs.add(p)
        lens.append(L)
    held = {e for _, _, e in wanted if e >= 0}
    free = iter([x for x in range(pages) if count[x] == 0 and x not in held])
    missing, copies = 0, []
    for s, j, e in wanted:
        x = next(free, None)
        if x is None:
            missing += 1
            L = lens[s]
            if j == L // page and L % page:
                lens[s] = L // page * page
            continue
        out[s, j] = x
        count[x] += 1
        if e >= 0:
            copies.append((e, x))
    for c in caches:
        before = {n: a.copy() for n, a in c.items()}
        for e, x in copies:
            for n in c:
                c[n][x] = before[n][e]
    return out, np.array(lens, np.int32), count.astype(np.int32), missing
