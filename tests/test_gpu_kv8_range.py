"""q8_attention_kv8 where pages differ in size by far: what a row's mask hides
has no say in it, and what it sees is held relative to its own largest term."""
import numpy as np
import pytest
import torch

import kv8_plain as P
from test_gpu_kv8 import BF, DEV, HF, batch_of, device, random_cache, table_of
from w8a8_quantized_linear_channel_amd import ops as q8

pytestmark = pytest.mark.gpu


def check_range(rng, news, lens, Hq, Hk, D, page, dt, cache, table, qscale, causal=True, window=0, **bounds):
    """Against 64 bits with a bound of each row's own.

    The weight of a key's codes is p 2^(b - 127), p its share of the softmax.
    It is off by its score and the sum's: D exact products in binary32, at most
    D + 16 roundings of 2^-23 of the largest sum of magnitudes, and 2^-21 of the
    hardware's exponentials (twice: numerator and sum); by the exponents inside
    the exponential's argument, rounded at up to 2^9 (2^-15 of a weight); by f16's
    2^-11; and by the binary32 sums, 2^-22 a key.  That scales the weighted mean
    of |v|.  What f16 cannot hold is at most 2^-24 of the row's largest weight,
    for each key and code: 2^-24 W sum |c|.  Then the output's rounding
    (subnormals included)."""
    start, batch = batch_of(news, lens, table, **bounds)
    T = int(start[-1])
    q = torch.from_numpy((rng.standard_normal((T, Hq, D)) * qscale).astype(np.float32)).to(dt)
    out, lse = q8.q8_attention_kv8(q.to(DEV), device(cache), batch, causal=causal, window=window, lse=True)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(got).all()
    half, floor = (2.0 ** -8, 2.0 ** -133) if dt == BF else (2.0 ** -11, 2.0 ** -24)
    x = q.double().numpy()
    for s, (n, total) in enumerate(zip(news, lens)):
        k = P.gathered(cache, table[s], total, "k")
        codes = P.gathered({**cache, "ve": np.full_like(cache["ve"], 127)}, table[s], total, "v")
        b = cache["ve"][table[s][:-(-total // page)]].astype(np.float64).T.repeat(page, 1)[:, :total] - 127
        j = np.arange(total)
        for i in range(n):
            p = total - n + i
            seen = (j <= p if causal else j >= 0) & (j > p - window if window else j >= 0)
            for h in range(Hq):
                g = h // (Hq // Hk)
                kk, c, e = k[g][seen], codes[g][seen], b[g][seen]
                sc = kk @ x[start[s] + i, h] / np.sqrt(D)
                w = np.exp(sc - sc.max())
                want_l = sc.max() + np.log(w.sum())
                w = w / w.sum() * 2.0 ** e
                want, mean = w @ c, w @ np.abs(c)
                ds = (D + 16) * 2.0 ** -23 * (np.abs(kk) @ np.abs(x[start[s] + i, h])).max() / np.sqrt(D) + 2.0 ** -21
                rel = 2 * ds + 2.0 ** -15 + 2.0 ** -11 + total * 2.0 ** -22
                tol = rel * mean + 2.0 ** -24 * w.max() * np.abs(c).sum(0) + half * np.abs(want) + floor
                err = np.abs(got[start[s] + i, h] - want)
                assert (err <= tol).all(), (s, i, h, (err / tol).max())
                assert abs(gl[start[s] + i, h] - want_l) <= ds + total * 2.0 ** -23 + 2.0 ** -21 * abs(want_l)
    return out


def test_pages_hidden_by_the_mask_have_no_say():
    """Under the causal mask rows 0 to 31 see the first page only, whose values are 2^35 below the next's."""
    rng = np.random.default_rng(0)
    table, pages = table_of(rng, [256], 32)
    cache = random_cache(rng, pages, 1, 32, 64)
    cache["ve"][table[0]] = np.array([105, 140] * 4)[:, None]
    cache["ke"][:] = 118
    for dt, base in ((BF, 0), (HF, 14)):
        cache["ve"][table[0]] = np.array([105 + base, 140 - base // 2] * 4)[:, None]
        check_range(rng, [256], [256], 2, 1, 64, 32, dt, cache, table, 1.0)
        check_range(rng, [30], [256], 2, 1, 64, 32, dt, cache, table, 1.0)
        check_range(rng, [30], [256], 2, 1, 64, 32, dt, cache, table, 1.0, window=45)
        check_range(rng, [200], [256], 2, 1, 64, 32, dt, cache, table, 1.0, window=45)


def test_later_pages_do_not_change_a_bit():
    """The first rows of a prompt, with and without far larger values behind them."""
    rng = np.random.default_rng(1)
    table, pages = table_of(rng, [300], 64)
    cache = random_cache(rng, pages, 2, 64, 128)
    start, batch = batch_of([300], [300], table)
    q = torch.from_numpy(rng.standard_normal((300, 8, 128)).astype(np.float32)).to(BF).to(DEV)
    one = q8.q8_attention_kv8(q, device(cache), batch)
    cache["ve"][table[0, 2:]] = 200
    two = q8.q8_attention_kv8(q, device(cache), batch)
    assert torch.equal(one[:128], two[:128]) and not torch.equal(one[128:], two[128:])


@pytest.mark.parametrize("D,page,Hq,Hk", [(64, 32, 2, 1), (128, 64, 4, 2), (256, 128, 3, 1)])
@pytest.mark.parametrize("new,length", [([1, 1], [700, 90]), ([9, 30], [600, 64]), ([300], [700]), ([1], [5000])])
def test_weight_on_small_pages(D, page, Hq, Hk, new, length):
    """Value pages up to 2^60 apart and scores that spread over some 2^100: the largest term of a row
    may lie on any page, and its largest weight on another."""
    rng = np.random.default_rng(D + len(new) + length[0])
    table, pages = table_of(rng, length, page)
    cache = random_cache(rng, pages, Hk, page, D)
    cache["ve"] = rng.choice([97, 112, 120, 127, 130, 157], (pages, Hk)).astype(np.uint8)
    check_range(rng, new, length, Hq, Hk, D, page, BF, cache, table, 50.0)
    check_range(rng, new, length, Hq, Hk, D, page, BF, cache, table, 1.0, causal=False)
    check_range(rng, new, length, Hq, Hk, D, page, BF, cache, table, 8.0, window=150)


def test_values_of_zero_pages_and_extreme_exponents():
    rng = np.random.default_rng(3)
    for new in (1, 100):
        table, pages = table_of(rng, [400], 32)
        cache = random_cache(rng, pages, 1, 32, 64)
        cache["ve"][:] = rng.choice([0, 1, 60, 127, 220], (pages, 1))
        cache["v"][table[0, 1:4]] = 0
        cache["ve"][table[0, 1:4]] = 0
        check_range(rng, [new], [400], 2, 1, 64, 32, BF, cache, table, 30.0)


def test_reference_does_not_drift():
    """Every fifth page far below the others: most steps move the rows' references, which must stay where the
    largest term is over hundreds of them.  (The bound on the lengths keeps the keys in one share.)"""
    rng = np.random.default_rng(9)
    for new, D in ((100, 64), (100, 128), (4, 128)):
        table, pages = table_of(rng, [6000], 32)
        cache = random_cache(rng, pages, 1, 32, D)
        cache["ve"][table[0, ::5]] = 96
        check_range(rng, [new], [6000], 2, 1, D, 32, BF, cache, table, 20.0, max_kv=100)
