"""Caches of several layers in one allocation: side by side they are taken, over one another refused."""
import numpy as np
import pytest
import torch

import kv8_more_plain as M
from test_gpu_kv8 import DEV, batch_of, device, random_cache, table_of
from test_gpu_kv8_drafts import interpreted, up
from test_gpu_kv8_pages import same
from w8a8_quantized_linear_channel_amd import _lib
from w8a8_quantized_linear_channel_amd import ops as q8

pytestmark = pytest.mark.gpu


def test_layers_side_by_side_and_over_one_another():
    rng = np.random.default_rng(0)
    news, lens = [9, 5], [70, 40]
    table, pages = table_of(rng, lens, 32)
    caches = [random_cache(rng, pages, 3, 32, 64) for _ in range(4)]
    whole = [torch.stack(t) for t in zip(*(device(c) for c in caches))]         # [layers, ...] of each array
    parts = lambda a: [q8.KvCache(*c) for c in zip(*(t.unbind() for t in a))]  # noqa: E731
    got = parts(whole)
    start, batch = batch_of(news, lens, table)
    keep, kept = np.array([[1, 4, 8], [0, 3, -1]], np.int32), np.array([3, 2], np.int32)
    out = q8.q8_kv_compact(got, batch, up(keep), up(kept))
    want = [M.compact(c, table, start, lens, keep, kept) for c in caches]
    assert np.array_equal(out.cpu().numpy(), want[0])
    same(got, caches)
    refs = np.zeros(pages, np.int32)
    refs[table[table >= 0]] = 1
    fork = lambda c: q8.q8_kv_fork(c, batch.block_table, batch.kv_len, up(refs), up(np.array([0, 0], np.int32)), room=1)  # noqa: E731
    assert isinstance(fork(got), q8.KvFork)
    was = [t.clone() for t in whole]
    for name in q8.KvCache._fields:
        a = getattr(got[1], name)
        one = torch.empty((pages + 1, *a.shape[1:]), dtype=a.dtype, device=DEV)             # a page apart
        for x, y in ((a, got[0]), (one[1:], got[0]._replace(**{name: one[:-1]}))):
            bad = [y, got[1]._replace(**{name: x}), got[2]] if x is not a else [got[0]._replace(**{name: a}), *got[1:]]
            for call in (lambda: q8.q8_kv_compact(bad, batch, up(keep), up(kept)), lambda: fork(bad)):
                for way in (lambda f: f(), interpreted):
                    with pytest.raises(_lib.Q8Error):
                        way(call)
    assert all(torch.equal(a, b) for a, b in zip(whole, was))
