"""The kernels that calls of serving size reach, each at a size that reaches it (the comments name the
rule), against 64 bits on sampled rows or all."""
import numpy as np
import pytest
import torch

import kv8_plain as P
from test_gpu_fp8_block import BF, DEV, HF, check, inputs
from test_gpu_kv8 import random_cache, run_attention, table_of
from test_gpu_kv8_range import check_range
from w8a8_quantized_linear_channel_amd import ops as q8

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- block-scaled product
# 3700 x 3336: 15 x 14 tiles of 256 (192 and more take them); 1100 x 2100: 18 x 33 tiles of 64 (over 512)
# and 5 x 9 of 256, so tiles of 128.  Rows, columns and features end inside a tile.
@pytest.mark.parametrize("M,N", [(3700, 3336), (1100, 2100)])
@pytest.mark.parametrize("K", [16, 128, 144, 256, 272, 400, 1040])
@pytest.mark.parametrize("dt", [BF, HF])
def test_large_tiles(M, N, K, dt):
    x, w, bias = inputs(M + K, M, N, K, dt)
    wq, ws = q8.q8_quantize_weight_block(w.to(DEV))
    xq, xs = q8.q8_quantize_act_block(x.to(DEV))
    y = q8.q8_gemm_fp8_block(xq, xs, wq, ws, bias=torch.from_numpy(bias).to(DEV), out_dtype=dt)
    assert torch.equal(y, q8.q8_linear_fp8_block(x.to(DEV), wq, ws, bias=torch.from_numpy(bias).to(DEV)))
    rng = np.random.default_rng(M + K)
    edges = [0, 15, 16, 127, 128, 255, 256, M - M % 256 - 1, M - M % 256, M - M % 128, M - 1]
    rows = sorted(set(edges) | set(rng.integers(0, M, 30).tolist()))
    rq, rs = P.block_quantize_act(x.float().numpy()[rows])
    check(y[rows], rq, rs, wq.cpu().numpy(), ws.cpu().numpy(), bias, dt)


def test_large_tiles_of_many_blocks():
    """Every buffer of the tiles' rings in turn, several times."""
    for M, N, K in ((3600, 3400, 2064), (1100, 2100, 4112)):
        x, w, _ = inputs(K, M, N, K, BF)
        wq, ws = q8.q8_quantize_weight_block(w.to(DEV))
        y = q8.q8_linear_fp8_block(x.to(DEV), wq, ws)
        rows = [0, 100, 255, 256, 1000, M - 1]
        rq, rs = P.block_quantize_act(x.float().numpy()[rows])
        check(y[rows], rq, rs, wq.cpu().numpy(), ws.cpu().numpy(), None, BF)


@pytest.mark.parametrize("M,N", [(3700, 3336), (1100, 2100)])
@pytest.mark.parametrize("K", [128, 144, 400])
def test_large_tiles_keep_nan_codes_in_their_row_and_column(M, N, K):
    x, w, _ = inputs(5, M, N, K, BF)
    wq, ws = q8.q8_quantize_weight_block(w.to(DEV))
    xq, xs = q8.q8_quantize_act_block(x.to(DEV))
    clean = q8.q8_gemm_fp8_block(xq, xs, wq, ws)
    nan_w, nan_x = [1, 700, N - 1], [0, 300, M - 1]
    wq[nan_w] = 0x7F
    xq[nan_x] = 0xFF
    y = q8.q8_gemm_fp8_block(xq, xs, wq, ws)
    assert y[:, nan_w].isnan().all() and y[nan_x].isnan().all()
    y[:, nan_w] = clean[:, nan_w]
    y[nan_x] = clean[nan_x]
    assert torch.equal(y, clean)


# ---------------------------------------------------------------- attention of few rows
# more than 256 workgroups (sequences x kv heads x splits): 4 waves each, at every head size
@pytest.mark.parametrize("D,page,dt", [(64, 32, BF), (64, 128, HF), (128, 64, BF), (128, 32, HF), (256, 64, BF)])
def test_many_sequences_of_one_token(D, page, dt):
    rng = np.random.default_rng(D + page)
    lens = rng.integers(1, 700, 70).tolist()
    lens[:4] = [700, 1, 64, 65]
    run_attention(rng, [1] * 70, lens, 16, 8, D, page, dt)


@pytest.mark.parametrize("D,page,dt", [(64, 64, HF), (128, 128, BF)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 70)])
def test_many_sequences_of_a_few_tokens(D, page, dt, causal, window):
    rng = np.random.default_rng(D + window)
    news = rng.integers(0, 4, 40).tolist()
    news[0] = 3
    lens = [n + int(a) for n, a in zip(news, rng.integers(0, 400, 40))]
    run_attention(rng, news, lens, 16, 8, D, page, dt, causal=causal, window=window, strided=True)


@pytest.mark.parametrize("D", [64, 128])
def test_long_sequences_of_one_token(D):
    """20 splits of 2 sequences and 8 kv heads: 320 workgroups, then the join."""
    rng = np.random.default_rng(D)
    run_attention(rng, [1, 1], [20000, 13001], 16, 8, D, 128, BF)


# ---------------------------------------------------------------- attention of many rows
def test_64_features_on_8_waves():
    """32 sequences x 8 kv heads, 160 rows each: blocks of 256 rows fill the chip."""
    rng = np.random.default_rng(1)
    news = rng.integers(33, 41, 32).tolist()
    news[5] = 40
    lens = [n + int(a) for n, a in zip(news, rng.integers(0, 200, 32))]
    run_attention(rng, news, lens, 32, 8, 64, 64, BF)


@pytest.mark.parametrize("D,page,dt", [(64, 64, BF), (128, 32, HF), (256, 64, BF), (256, 128, HF)])
@pytest.mark.parametrize("new,length,Hq,Hk,window", [([200], [5000], 2, 1, 0), ([300], [3000], 4, 1, 0),
                                                     ([150, 90], [2500, 1200], 4, 2, 500)])
def test_many_rows_with_split_keys(D, page, dt, new, length, Hq, Hk, window):
    """Up to 27 splits of the tile kernels, and rows of a window to which a whole split is hidden."""
    rng = np.random.default_rng(D + len(new) + page)
    run_attention(rng, new, length, Hq, Hk, D, page, dt, window=window)


@pytest.mark.parametrize("D,page,dt", [(64, 64, BF), (128, 32, BF), (128, 64, HF), (256, 128, BF)])
def test_many_rows_on_more_than_8192_keys_of_one_share(D, page, dt):
    """A bound on the lengths that is too small keeps the keys whole: pages and exponents are held for 8192
    keys at a time.  Value exponents differ before and after, and grow."""
    rng = np.random.default_rng(D)
    lens = [9100]
    table, pages = table_of(rng, lens, page)
    cache = random_cache(rng, pages, 1, page, D)
    run_attention(rng, [100], lens, 2, 1, D, page, dt, cache=cache, table=table, max_kv=100, garbage=False)
    spread = (96, 118, 150) if dt == BF else (112, 120, 131)
    exps = np.full(len(table[0]), spread[1])
    exps[::5] = spread[0]
    exps[8192 // page:] = spread[2]
    cache["ve"][table[0, :len(exps)]] = exps[:, None]
    check_range(rng, [100], lens, 2, 1, D, page, dt, cache, table, 1.0, max_kv=100)
    check_range(rng, [100], lens, 2, 1, D, page, dt, cache, table, 20.0, max_kv=100)
