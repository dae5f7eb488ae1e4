"""Token arrays of one head, whose heads' stride says nothing."""
import numpy as np
import pytest
import torch

from test_gpu_kv8 import BF, DEV, batch_of, device, random_cache, table_of
from w8a8_quantized_linear_channel_amd import ops as q8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 40])
def test_one_head_as_a_transposed_view(T):
    rng = np.random.default_rng(T)
    table, pages = table_of(rng, [T + 9], 64)
    base = random_cache(rng, pages, 1, 64, 128)
    _, batch = batch_of([T], [T + 9], table)
    x = torch.randn(3, T, 128, device=DEV).to(BF)
    got = []
    for dense in (True, False):
        q, k, v = (x[i:i + 1].transpose(0, 1) for i in range(3))           # [T, 1, 128], heads T * 128 apart
        assert T == 1 or k.stride() == (128, T * 128, 1)
        if dense:
            q, k, v = (t.contiguous().view(T, 128)[:, None] for t in (q, k, v))
        cache = device(base)
        r = q8.q8_kv_append(k, v, cache, batch, q=q)
        y, lse = q8.q8_attention_kv8(q, cache, batch, lse=True)
        got.append([r, y, lse, q8.q8_attention_kv8(q, cache, batch), *cache])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        q8.q8_attention_kv8(torch.randn(T, 128, 2, device=DEV).to(BF)[:, :, :1].transpose(1, 2), cache, batch)
