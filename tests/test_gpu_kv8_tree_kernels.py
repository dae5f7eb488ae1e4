"""q8_attention_kv8_tree in each of its kernels, which the calls' bounds choose (kv8_tree_cases.py)."""
import numpy as np
import pytest
import torch

import kv8_more_plain as M
import kv8_plain as P
from kv8_tree_cases import KERNELS
from test_gpu_kv8 import BF, DEV, HF, batch_of, bounds, device, random_cache, table_of
from test_gpu_kv8_drafts import any_mask, run_tree, up
from w8a8_quantized_linear_channel_amd import ops as q8

pytestmark = pytest.mark.gpu


def even_values(rng, pages, heads, page, dim):
    """A cache whose value features are alike in all tokens, on exponent bytes up to 3 apart, and those features."""
    cache = random_cache(rng, pages, heads, page, dim)
    cache["ve"] = rng.integers(124, 128, (pages, heads)).astype(np.uint8)
    mantissa, power, sign = rng.integers(0, 8, dim), rng.integers(-2, 3, dim), rng.integers(0, 2, dim)
    # e4m3: 7 + exponent in bits 3 to 6; a page at byte b holds 2^(127 - b) as much
    raised = power[None, None] + 127 - cache["ve"][:, :, None].astype(int)
    codes = sign * 128 + (7 + raised) * 8 + mantissa
    cache["v"] = np.repeat(codes.astype(np.uint8)[..., None], page, 3)
    return cache, (1 - 2 * sign) * (1 + mantissa / 8) * 2.0 ** power


@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("name", KERNELS)
def test_mean_of_even_values_is_the_value(name, dt):
    """sum(w c) / sum(w) is c whatever w is rounded to, if both sums have the rounded w (f16; a bf16 output hides
    2^-11).  In binary32 the upper sum is off by a rounding a key, 1200 2^-24 of itself, the lower one by fewer,
    together under 2^-12.  c has 4 significant bits, 1.875 2^e at most, and half a step of f16 is 2^-11 2^e: a border
    over 2^-12 of c away.  So the output is c itself."""
    _, _, seqs, heads, kv_heads, dim, page, max_q, max_kv, window = KERNELS[name]
    rng = np.random.default_rng(dim + max_q)
    news, lens = ([20, 33, 5] + [1] * seqs)[:seqs], ([20, 1200, 433] + [37] * seqs)[:seqs]
    news, lens = [min(n, max_q) for n in news], [min(n, max_kv) for n in lens]
    lens[0] = news[0]
    table, pages = table_of(rng, lens, page)
    cache, want = even_values(rng, pages, kv_heads, page, dim)
    start, batch = batch_of(news, lens, table, max_q, max_kv)
    T = int(start[-1])
    want = torch.from_numpy(want).to(dt)
    for kind, size in (("self", 1.0), ("any", 1.0), ("tree", 6.0)):
        sees = [np.eye(n, dtype=bool) if kind == "self" else any_mask(rng, n, kind) for n in news]
        seen = np.concatenate([M.tree_seen(n, t, s, None, window).any(1) for n, t, s in zip(news, lens, sees)])
        q = torch.from_numpy((rng.standard_normal((T, heads, dim)) * size).astype(np.float32)).to(dt)
        mask = up(np.concatenate([M.words_of(s, 1) for s in sees]).view(np.int64))
        out = q8.q8_attention_kv8_tree(q.to(DEV), device(cache), batch, mask, window=window).cpu()
        off = (out[seen] != want).any(2)
        assert off.sum().item() == 0, (kind, off.numel(), (out[seen].float() / want.float() - 1).abs().max())
        assert (out[~seen] == 0).all()


def sizes(name, new, length):
    """New tokens and lengths of a call that is to see several shares of the keys: the first two sequences', the others
    small; whole heads of rows that end inside a wave's."""
    _, split, seqs, _, _, _, _, max_q, max_kv, window = KERNELS[name]
    if window > 1000:
        new, length = min(new, 5), window + 900            # (few rows: each costs 64-bit passes over 20000 keys)
    elif not split:
        length = min(length, 700)
    news, lens = ([new, 3, 1] + [1] * seqs)[:seqs], ([length, 90, 40] + [37] * seqs)[:seqs]
    return [min(n, max_q) for n in news], [min(n, max_kv) for n in lens]


@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("name", KERNELS)
def test_kernels_against_64_bits(name, dt):
    """Trees and masks of any kind, a last block that ends inside a wave's rows, more rows than a block, windows."""
    _, _, _, heads, kv_heads, dim, page, max_q, max_kv, window = KERNELS[name]
    rng = np.random.default_rng(dim + max_kv % 997)
    kw = dict(window=window, max_q=max_q, max_kv=max_kv)
    run_tree(rng, *sizes(name, 50, 4000), heads, kv_heads, dim, page, dt, **kw)
    run_tree(rng, *sizes(name, 9, 1100), heads, kv_heads, dim, page, dt, kind="any", strided=True, **kw)
    if window < 1000:
        # past the bound on new tokens: blocks one after the other, the first among them before the sequence's start
        run_tree(rng, *sizes(name, 9, 5), heads, kv_heads, dim, page, dt, kind="chain", deep=False, **kw)
        news, lens = sizes(name, 9, 2300)
        run_tree(rng, [70] + news[1:], [max(lens[0], 71)] + lens[1:], heads, kv_heads, dim, page, dt, kind="any", words=1, **kw)


@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("name", [n for n in KERNELS if KERNELS[n][9] < 1000])
def test_kernels_values_of_very_different_size(name, dt):
    """Value pages up to 2^60 apart (f16: 2^33), scores that spread far: each row against 64 bits with a bound of its own.

    As check_range of test_gpu_kv8_range.py has it: a key's term is off by its score and the sum's (ds), by the
    exponents inside the exponential's argument (2^-15), by f16's 2^-11 and by binary32 sums (2^-22 a key), of the
    weighted mean of |v|; what f16 cannot hold is 2^-24 of the row's largest weight for each key and code.  An f16
    output's divisor has the rounded weights of some pages, another 2^-11 of the output.  Then the output's rounding."""
    _, _, _, heads, kv_heads, dim, page, max_q, max_kv, window = KERNELS[name]
    rng = np.random.default_rng(dim + page)
    news, lens = sizes(name, 20, 2600)
    table, pages = table_of(rng, lens, page)
    cache = random_cache(rng, pages, kv_heads, page, dim)
    cache["ve"] = rng.choice([97, 112, 120, 127, 130, 157] if dt == BF else [97, 112, 118, 124, 130], (pages, kv_heads)).astype(np.uint8)
    start, batch = batch_of(news, lens, table, max_q, max_kv)
    half, floor = (2.0 ** -8, 2.0 ** -133) if dt == BF else (2.0 ** -11, 2.0 ** -24)
    for size in (1.0, 30.0):
        sees = [any_mask(rng, n, "any") for n in news]
        q = torch.from_numpy((rng.standard_normal((int(start[-1]), heads, dim)) * size).astype(np.float32)).to(dt)
        mask = up(np.concatenate([M.words_of(a, 1) for a in sees]).view(np.int64))
        out, lse = q8.q8_attention_kv8_tree(q.to(DEV), device(cache), batch, mask, window=window, lse=True)
        got, gl, x = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().numpy()
        for s, (n, total) in enumerate(zip(news, lens)):
            seen = M.tree_seen(n, total, sees[s], None, window)
            k = P.gathered(cache, table[s], total, "k")
            codes = P.gathered({**cache, "ve": np.full_like(cache["ve"], 127)}, table[s], total, "v")
            b = cache["ve"][table[s][:-(-total // page)]].astype(np.float64).T.repeat(page, 1)[:, :total] - 127
            for i in range(0, n, 3):
                for h in range(0, heads, 3):
                    g = h // (heads // kv_heads)
                    if not seen[i].any():
                        assert (got[start[s] + i, h] == 0).all()
                        continue
                    kk, c, e = k[g][seen[i]], codes[g][seen[i]], b[g][seen[i]]
                    sc = kk @ x[start[s] + i, h] / np.sqrt(dim)
                    w = np.exp(sc - sc.max())
                    want_l = sc.max() + np.log(w.sum())
                    w = w / w.sum() * 2.0 ** e
                    want, mean = w @ c, w @ np.abs(c)
                    ds = (dim + 16) * 2.0 ** -23 * (np.abs(kk) @ np.abs(x[start[s] + i, h])).max() / np.sqrt(dim) + 2.0 ** -21
                    rel = 2 * ds + 2.0 ** -15 + 2.0 ** -11 + total * 2.0 ** -22
                    tol = rel * mean + 2.0 ** -24 * w.max() * np.abs(c).sum(0) + (half + 2.0 ** -11 * (dt == HF)) * np.abs(want) + floor
                    err = np.abs(got[start[s] + i, h] - want)
                    assert (err <= tol).all(), (size, s, i, h, (err / tol).max())
                    assert abs(gl[start[s] + i, h] - want_l) <= ds + total * 2.0 ** -23 + 2.0 ** -21 * abs(want_l), (size, s, i, h)


@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("name", [n for n in KERNELS if KERNELS[n][9] < 1000])
def test_kernels_keep_nan_codes_to_the_rows_that_see_them(name, dt):
    """A NaN among the values makes its feature NaN in the rows that see its key and changes no other bit; one among the
    keys makes those rows NaN, and leaves the others where 64 bits have them."""
    _, _, _, heads, kv_heads, dim, page, max_q, max_kv, window = KERNELS[name]
    rng = np.random.default_rng(dim + page + 1)
    news, lens = sizes(name, 30, 2600)
    table, pages = table_of(rng, lens, page)
    cache = random_cache(rng, pages, kv_heads, page, dim)
    start, batch = batch_of(news, lens, table, max_q, max_kv)
    n, total, group = news[0], lens[0], heads // kv_heads
    sees = [any_mask(rng, m, "any") for m in news]
    mask = up(np.concatenate([M.words_of(a, 1) for a in sees]).view(np.int64))
    seen = M.tree_seen(n, total, sees[0], None, window)
    q = torch.from_numpy(rng.standard_normal((int(start[-1]), heads, dim)).astype(np.float32)).to(dt)
    call = lambda c: q8.q8_attention_kv8_tree(q.to(DEV), device(c), batch, mask, window=window, lse=True)  # noqa: E731
    clean, clean_lse = call(cache)
    want, wl, av, aqk = M.tree_attention(cache, table, start, lens, q.double().numpy(), sees, None, None, window)
    tol, ltol = bounds(av, aqk, wl, want, dim, max(lens), dt)
    for at in sorted({max(total - n - 30, 0), total - n, total - n // 2, total - 1}):
        rows = torch.from_numpy(np.flatnonzero(seen[:, at])).to(DEV)
        c = {**cache, "v": cache["v"].copy()}
        c["v"][table[0, at // page], 0, [3, dim - 1], at % page] = [0x7F, 0xFF]
        out, lse = call(c)
        bad = clean.clone()
        for f in (3, dim - 1):
            bad[rows, :group, f] = float("nan")
        assert torch.equal(out.isnan(), bad.isnan()), at
        assert torch.equal(out.nan_to_num(), bad.nan_to_num()) and torch.equal(lse, clean_lse), at
        c = {**cache, "k": cache["k"].copy()}
        c["k"][table[0, at // page], 0, at % page, dim - 2] = 0x7F
        out, lse = call(c)
        hit = torch.zeros(out.shape[:2], dtype=torch.bool, device=DEV)
        hit[rows, :group] = True
        assert out[hit].isnan().all() and lse[hit].isnan().all(), at
        free = ~hit.cpu().numpy()
        assert (np.abs(out.double().cpu().numpy() - want) <= tol)[free].all(), at
        ok = free & np.isfinite(wl)
        assert (np.abs(lse.double().cpu().numpy() - np.where(ok, wl, 0)) <= ltol)[ok].all(), at
