"""q8_attention_kv8_tree in each of its kernels, which the calls' bounds choose (kv8_tree_cases.py)."""
import numpy as np
import pytest
import torch

import kv8_more_plain as M
from kv8_tree_cases import KERNELS
from test_gpu_kv8 import BF, DEV, HF, batch_of, device, random_cache, table_of
from test_gpu_kv8_drafts import any_mask, up
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
