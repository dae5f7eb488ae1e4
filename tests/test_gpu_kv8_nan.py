"""NaN codes in the cache: they reach the rows that see them, and no others."""
import numpy as np
import pytest
import torch

from test_gpu_kv8 import BF, DEV, HF, batch_of, device, random_cache, table_of
from w8a8_quantized_linear_channel_amd import ops as q8

pytestmark = pytest.mark.gpu

# new tokens and lengths, heads, features, page, window: few rows in one and in several blocks of 16, many rows,
# keys split over workgroups, a window whose lower edge crosses a block
SHAPES = [([1, 5], [70, 90], 2, 1, 64, 32, 0), ([30, 1], [300, 33], 4, 1, 128, 64, 0), ([30], [300], 2, 1, 256, 32, 50),
          ([130], [130], 4, 2, 64, 32, 0), ([300], [500], 4, 1, 128, 64, 0), ([200], [400], 2, 1, 256, 64, 70),
          ([40], [9000], 8, 2, 128, 64, 0), ([3], [20000], 8, 2, 64, 128, 3000), ([150], [3000], 4, 1, 64, 64, 1000),
          ([70], [40], 2, 1, 64, 32, 0)]


def places(rng, news, lens, window):
    """Positions of one sequence that some of its rows see and some do not, that all do, or none."""
    n, total = news[0], lens[0]
    past = total - n
    at = {total - 1, max(total - 2, 0), max(past + 1, 0), max(past - 1, 0), max(past - window + 2, 0) if window else 0}
    return sorted(at | {int(rng.integers(max(past, 0), total))})


@pytest.mark.parametrize("news,lens,Hq,Hk,D,page,window", SHAPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dt", [BF, HF])
def test_nan_value_codes(news, lens, Hq, Hk, D, page, window, causal, dt):
    rng = np.random.default_rng(sum(lens) + D)
    table, pages = table_of(rng, lens, page)
    cache = random_cache(rng, pages, Hk, page, D)
    start, batch = batch_of(news, lens, table)
    q = torch.from_numpy(rng.standard_normal((int(start[-1]), Hq, D)).astype(np.float32)).to(dt).to(DEV)
    call = lambda c: q8.q8_attention_kv8(q, device(c), batch, causal=causal, window=window, lse=True)  # noqa: E731
    clean, clean_lse = call(cache)
    features = [3, D - 1]
    head = Hk - 1
    mine = slice(head * (Hq // Hk), (head + 1) * (Hq // Hk))
    n, total = news[0], lens[0]
    for at in places(rng, news, lens, window):
        c = {**cache, "v": cache["v"].copy()}
        c["v"][table[0, at // page], head, features, at % page] = [0x7F, 0xFF]
        out, lse = call(c)
        pos = total - n + np.arange(n)
        seen = np.full(n, at < total)
        if causal:
            seen &= at <= pos
        if window:
            seen &= at > pos - window
        want = clean.clone()
        rows = torch.from_numpy(np.flatnonzero(seen)).to(DEV)
        for f in features:
            sub = want[:, mine, f]
            sub[rows] = float("nan")
        assert torch.equal(torch.isnan(out), torch.isnan(want)), at
        assert torch.equal(out.nan_to_num(), want.nan_to_num()), at
        assert torch.equal(lse, clean_lse)


@pytest.mark.parametrize("news,lens,Hq,Hk,D,page,window", SHAPES)
def test_nan_scores(news, lens, Hq, Hk, D, page, window):
    """A key or a query with a NaN: outputs and log-sum-exp of the rows that see it are NaN, not 'no key'."""
    rng = np.random.default_rng(sum(lens) + D + 1)
    table, pages = table_of(rng, lens, page)
    cache = random_cache(rng, pages, Hk, page, D)
    start, batch = batch_of(news, lens, table)
    q = torch.from_numpy(rng.standard_normal((int(start[-1]), Hq, D)).astype(np.float32)).to(BF).to(DEV)
    clean, clean_lse = q8.q8_attention_kv8(q, device(cache), batch, window=window, lse=True)
    assert torch.equal(torch.isneginf(clean_lse), (clean == 0).all(2))
    n, total = news[0], lens[0]
    at = total - 1 if n == 1 else total - max(1, min(n, total) // 2)
    c = {**cache, "k": cache["k"].copy()}
    c["k"][table[0, at // page], 0, at % page, D - 2] = 0x7F
    out, lse = q8.q8_attention_kv8(q, device(c), batch, window=window, lse=True)
    pos = total - n + np.arange(n)
    rows = np.flatnonzero((at <= pos) & ((at > pos - window) if window else True))
    bad = torch.zeros(clean_lse.shape, dtype=torch.bool)
    bad[torch.from_numpy(rows), :Hq // Hk] = True
    bad = bad.to(DEV)
    assert len(rows) and out[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], clean_lse[~bad])
    x = q.clone()
    x[-1, Hq - 1, 0] = float("nan")
    out, lse = q8.q8_attention_kv8(x, device(cache), batch, window=window, lse=True)
    assert out[-1, Hq - 1].isnan().all() and lse[-1, Hq - 1].isnan()
    out[-1, Hq - 1], lse[-1, Hq - 1] = clean[-1, Hq - 1], clean_lse[-1, Hq - 1]
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
