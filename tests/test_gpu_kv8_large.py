"""Calls over the cache whose grids come near what one launch takes."""
import numpy as np
import pytest
import torch

from test_gpu_kv8 import BF, DEV, batch_of, device, random_cache, table_of
from w8a8_quantized_linear_channel_amd import ops as q8

pytestmark = pytest.mark.gpu


def test_one_prompt_among_thousands_of_sequences():
    """4095 sequences of one new token and a prompt of 16384: the blocks of the longest for every sequence
    are 2^32 threads.  Cut differently, each part is what it is alone, to within both roundings."""
    rng = np.random.default_rng(0)
    S, n, Hq, Hk, D, page = 4096, 16384, 32, 8, 64, 64
    news, lens = [n] + [1] * (S - 1), [n] + rng.integers(1, 64, S - 1).tolist()
    table, pages = table_of(rng, lens, page)
    start, batch = batch_of(news, lens, table)
    gen = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randn(int(start[-1]), Hq + 2 * Hk, D, generator=gen, device=DEV).to(BF)
    cache = q8.q8_kv_cache(pages, Hk, D, page=page, device=DEV)
    parts = [slice(0, 1), slice(1, S)]
    alone = [c.clone() for c in cache]
    q = q8.q8_kv_append(x[:, Hq:Hq + Hk], x[:, Hq + Hk:], cache, batch, q=x[:, :Hq])
    assert torch.equal(q, x[:, :Hq])
    y = q8.q8_attention_kv8(q, cache, batch)
    for p in parts:
        t = slice(int(start[p.start]), int(start[p.stop]))
        st, b = batch_of(news[p], lens[p], table[p])
        c = q8.KvCache(*alone)
        q8.q8_kv_append(x[t, Hq:Hq + Hk], x[t, Hq + Hk:], c, b)
        z = q8.q8_attention_kv8(x[t, :Hq], cache, b)
        # weights off by 2^-11 and the sums by far less, of values below 6; bf16 outputs
        assert ((y[t].float() - z.float()).abs() <= 2 * (6 * 2.0 ** -11 + 2.0 ** -8 * z.float().abs())).all()
    for a, b in zip(alone, cache):
        assert torch.equal(a, b)


def test_most_sequences_and_heads():
    """32768 sequences of 1024 heads: the append is two launches, the attention takes its grid's other axes.
    A few sequences have tokens, at both ends of each launch."""
    rng = np.random.default_rng(1)
    S, H, D, page = 32768, 1024, 64, 32
    have = {0: (2, 5), 16383: (1, 1), 16384: (2, 30), 32767: (3, 3)}
    news, lens, table = [0] * S, [0] * S, np.full((S, 1), -1, np.int32)
    for i, (s, (n, total)) in enumerate(have.items()):
        news[s], lens[s], table[s] = n, total, (i + 1) % 4
    start, batch = batch_of(news, lens, table)
    base = random_cache(rng, 4, H, page, D)
    x = torch.from_numpy(rng.standard_normal((int(start[-1]), 3 * H, D)).astype(np.float32)).to(BF)
    cache, xd = device(base), x.to(DEV)
    q = q8.q8_kv_append(xd[:, H:2 * H], xd[:, 2 * H:], cache, batch, q=xd[:, :H])
    assert torch.equal(q, xd[:, :H])
    y, lse = q8.q8_attention_kv8(q, cache, batch, lse=True)
    some = list(have)
    few_start, few = batch_of([news[s] for s in some], [lens[s] for s in some], table[some])
    alone = device(base)
    q8.q8_kv_append(xd[:, H:2 * H], xd[:, 2 * H:], alone, few)
    for a, b in zip(alone, cache):
        assert torch.equal(a, b)
    z, z_lse = q8.q8_attention_kv8(q, alone, few, lse=True)
    assert torch.equal(y, z) and torch.equal(lse, z_lse)
