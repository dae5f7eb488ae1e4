"""The paged 8-bit cache: q8_kv_append against its definition bit for bit, and
q8_attention_kv8 against softmax attention in 64 bits over the same codes."""
import math

import numpy as np
import pytest
import torch

import kv8_plain as P
from w8a8_quantized_linear_channel_amd import _lib
from w8a8_quantized_linear_channel_amd import ops as q8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def host(cache):
    return {n: t.cpu().numpy().copy() for n, t in zip(("k", "ke", "v", "ve"), cache)}


def device(cache):
    return q8.KvCache(*(torch.from_numpy(cache[n]).to(DEV) for n in ("k", "ke", "v", "ve")))


def batch_of(news, lens, table, max_q=None, max_kv=None):
    start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    t = lambda a: torch.tensor(np.asarray(a, np.int32), device=DEV)  # noqa: E731
    return start, q8.KvBatch(t(start), t(lens), t(table), max(news) if max_q is None else max_q,
                             max(lens) if max_kv is None else max_kv)


def table_of(rng, lens, page, spare=2):
    """Pages in random order, -1 past each sequence's last, and the page count."""
    need = [-(-n // page) for n in lens]
    order = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(max(need), 1)), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


def random_cache(rng, pages, heads, page, dim, spread=2):
    """Codes of N(0, 1)-like values (no NaN codes) and exponents around 120."""
    codes = lambda *shape: P.e4m3_codes(rng.standard_normal(shape) * 60)  # noqa: E731
    exps = lambda: rng.integers(120 - spread, 121 + spread, (pages, heads)).astype(np.uint8)  # noqa: E731
    return {"k": codes(pages, heads, page, dim), "ke": exps(), "v": codes(pages, heads, dim, page), "ve": exps()}


def tables_of_angles(positions, rot):
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(positions)[:, None] * f
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


# ---------------------------------------------------------------- append
def run_append(rng, news, lens, Hq, Hk, D, page, dt, rot=None, interleaved=False, spike=True, positions=None):
    table, pages = table_of(rng, [max(n, 1) for n in lens], page)
    cache = random_cache(rng, pages, Hk, page, D)
    start, batch = batch_of(news, lens, table)
    T = int(start[-1])
    x = rng.standard_normal((T, Hq + 2 * Hk, D)).astype(np.float32)
    if spike and T:
        x[rng.random((T, Hq + 2 * Hk)) < 0.2] *= 9.0         # new maxima: older codes are re-expressed
    x = torch.from_numpy(x).to(dt)
    cos = sin = None
    if rot:
        cos, sin = tables_of_angles(positions or max(lens), rot)
    got = device(cache)
    xd = x.to(DEV)
    g = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
    q = q8.q8_kv_append(xd[:, Hq:Hq + Hk], xd[:, Hq + Hk:], got, batch, q=xd[:, :Hq], cos=g(cos), sin=g(sin),
                        interleaved=interleaved)
    xf = x.float().numpy()
    P.append(cache, table, start, lens, xf[:, Hq:Hq + Hk], xf[:, Hq + Hk:], cos, sin, interleaved)
    got = host(got)
    for name in ("ke", "ve", "k", "v"):
        bad = np.argwhere(got[name] != cache[name])
        assert len(bad) == 0, (name, len(bad), bad[:3])
    pos = np.concatenate([np.arange(b - n, b) for n, b in zip(news, lens)]) if T else np.zeros(0, int)
    lim = len(cos) - 1 if rot else 0
    want = torch.from_numpy(P.rotate(xf[:, :Hq], np.clip(pos, 0, lim) if rot else pos, cos, sin, interleaved)).to(dt)
    assert torch.equal(q.cpu(), want)


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt", [BF, HF, F32])
def test_append_shapes(page, D, dt):
    rng = np.random.default_rng(page + D)
    run_append(rng, [1, 3, page + 5, 0, 2 * page], [1, 40, 2 * page + 9, 7, 2 * page], 4, 2, D, page, dt, rot=D)


@pytest.mark.parametrize("rot,interleaved", [(None, False), (16, False), (32, True), (64, False), (128, True)])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (10, 2), (7, 1)])
def test_append_rotations_and_heads(rot, interleaved, Hq, Hk):
    rng = np.random.default_rng(Hq)
    run_append(rng, [1, 17, 1], [65, 150, 64], Hq, Hk, 128, 64, BF, rot=rot, interleaved=interleaved)


def test_append_step_by_step_is_the_state_update():
    """64 single tokens in turn: each step as the definition says, from the state the last one left."""
    rng = np.random.default_rng(5)
    table = np.array([[1]], np.int32)
    cache = random_cache(rng, 2, 2, 64, 64)
    got = device(cache)
    for p in range(64):
        x = torch.from_numpy((rng.standard_normal((1, 4, 64)) * (1 + p % 9)).astype(np.float32)).to(BF)
        start, batch = batch_of([1], [p + 1], table)
        xd = x.to(DEV)
        assert q8.q8_kv_append(xd[:, :2], xd[:, 2:], got, batch) is None
        P.append(cache, table, start, [p + 1], x[:, :2].float().numpy(), x[:, 2:].float().numpy())
    got = host(got)
    for name in cache:
        assert np.array_equal(got[name], cache[name]), name


def test_append_edges():
    rng = np.random.default_rng(9)
    # more new tokens than positions (the first fall away), positions past the angle table (its last row)
    run_append(rng, [9, 5], [4, 70], 2, 1, 64, 64, HF, rot=64, positions=50)
    # zeros and tiny values: exponent byte 0, and values far below e4m3's range of the page
    table, pages = table_of(rng, [40], 64)
    for scale in (0.0, 1e-30, 1e-38):
        cache = random_cache(rng, pages, 1, 64, 64)
        x = (rng.standard_normal((40, 2, 64)) * scale).astype(np.float32)
        got = device(cache)
        start, batch = batch_of([40], [40], table)
        xd = torch.from_numpy(x).to(DEV)
        q8.q8_kv_append(xd[:, :1], xd[:, 1:], got, batch)
        P.append(cache, table, start, [40], x[:, :1], x[:, 1:])
        got = host(got)
        for name in cache:
            assert np.array_equal(got[name], cache[name]), (scale, name)


def test_append_pages_outside_are_skipped_and_bounds_too_small_still_append():
    rng = np.random.default_rng(2)
    cache = random_cache(rng, 3, 1, 32, 64)
    table = np.array([[0, 99, 2], [-1, 1, -7]], np.int32)
    news, lens = [96, 50], [96, 60]
    start, _ = batch_of(news, lens, table)
    for max_q in (1, 96):
        got = device(cache)
        ref = {n: a.copy() for n, a in cache.items()}
        _, batch = batch_of(news, lens, table, max_q=max_q)
        x = torch.from_numpy(rng.standard_normal((146, 3, 64)).astype(np.float32)).to(BF)
        xd = x.to(DEV)
        q = q8.q8_kv_append(xd[:, 1:2], xd[:, 2:], got, batch, q=xd[:, :1])
        P.append(ref, table, start, lens, x[:, 1:2].float().numpy(), x[:, 2:].float().numpy())
        got = host(got)
        for name in ref:
            assert np.array_equal(got[name], ref[name]), (max_q, name)
        assert torch.equal(q.cpu(), x[:, :1])


def test_append_no_tokens_and_queries_in_place():
    cache = q8.q8_kv_cache(2, 1, 64, page=32, device=DEV)
    _, batch = batch_of([0], [0], [[0]])
    empty = torch.empty(0, 1, 64, dtype=BF, device=DEV)
    assert q8.q8_kv_append(empty, empty, cache, batch, q=empty).shape == (0, 1, 64)
    _, batch = batch_of([3], [3], [[0]])
    q = torch.randn(3, 2, 64, device=DEV).to(BF)
    k = torch.randn(3, 1, 64, device=DEV).to(BF)
    cos, sin = (torch.from_numpy(a).to(DEV) for a in tables_of_angles(3, 64))
    want = q8.q8_kv_append(k, k, cache, batch, q=q, cos=cos, sin=sin, interleaved=True)
    assert torch.equal(q8.q8_kv_append(k, k, cache, batch, q=q, cos=cos, sin=sin, interleaved=True, out=q), want)


# ---------------------------------------------------------------- attention
def bounds(av, aqk, lse, out, D, keys, dt):
    """Error bounds of the attention against 64 bits on the same codes.
    Scores: D exact products summed in binary32 in some order, each of at most
    D + 8 roundings (MFMA chain, key scale, softmax scale) within 2^-23 of the
    sum of magnitudes, then the subtraction of the maximum (|s| <= aqk) and the
    hardware exponential (2^-22 relative): ds = (D + 16) 2^-23 aqk + 2^-21.
    A weight is off by 2 ds (its own score and the sum's), its f16 rounding
    (2^-11 relative, 2^-25 of the largest weight below f16's normal range, which
    is at most `keys` 2^-25 of the weights' sum) and the binary32 sums over the
    keys (keys 2^-23).  All of it scales the weighted mean of |v|, or its
    maximum for the absolute part; then the output's own rounding."""
    ds = (D + 16) * 2.0 ** -23 * aqk + 2.0 ** -21
    rel = 2 * ds + 2.0 ** -11 + keys * 2.0 ** -22
    half = 2.0 ** -8 if dt == BF else 2.0 ** -11
    floor = 0.0 if dt == BF else 2.0 ** -24
    return rel[:, :, None] * (av + av.max(2, keepdims=True)) + half * np.abs(out) + floor, ds + keys * 2.0 ** -23 + 2.0 ** -21 * np.abs(np.where(np.isfinite(lse), lse, 0))


def run_attention(rng, news, lens, Hq, Hk, D, page, dt, causal=True, window=0, cache=None, table=None, scale=None,
                  max_q=None, max_kv=None, qscale=1.0, strided=False, garbage=True):
    if table is None:
        table, pages = table_of(rng, lens, page)
    if cache is None:
        cache = random_cache(rng, pages, Hk, page, D)
    if garbage:
        # NaN codes in every slot that no query sees
        for s, (n, total) in enumerate(zip(news, lens)):
            low = max(0, total - n - window + 1) if window else 0
            for lp in range(table.shape[1]):
                at = table[s, lp]
                if 0 <= at < len(cache["ke"]):
                    off = lp * page + np.arange(page)
                    hide = (off >= total) | (off < low)
                    cache["k"][at][:, hide] = 0x7f
                    cache["v"][at][:, :, hide] = 0xff
    start, batch = batch_of(news, lens, table, max_q, max_kv)
    T = int(start[-1])
    q = torch.from_numpy((rng.standard_normal((T, Hq + (2 if strided else 0), D)) * qscale).astype(np.float32)).to(dt)
    qd = q.to(DEV)[:, :Hq]
    out, lse = q8.q8_attention_kv8(qd, device(cache), batch, causal=causal, window=window, scale=scale, lse=True)
    want, wl, av, aqk = P.attention(cache, table, start, lens, q[:, :Hq].double().numpy(), scale, causal, window)
    tol, ltol = bounds(av, aqk, wl, want, D, max(lens) if lens else 0, dt)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= tol).all(), (err - tol).max()
    gl = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
    ok = np.isfinite(wl)
    assert (np.abs(gl - np.where(ok, wl, 0))[ok] <= ltol[ok]).all()
    return out


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt", [BF, HF])
def test_attention_single_tokens(page, D, dt):
    rng = np.random.default_rng(D + page)
    run_attention(rng, [1] * 9, [1, 31, 32, 33, 127, 128, 129, 500, 1000], 8, 2, D, page, dt)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (2, 2), (5, 1), (12, 4), (16, 1), (17, 1), (48, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_heads(Hq, Hk, causal):
    rng = np.random.default_rng(Hq)
    run_attention(rng, [1, 2, 3], [300, 77, 3], Hq, Hk, 64, 32, BF, causal=causal, strided=True)


@pytest.mark.parametrize("D,page,dt", [(64, 32, HF), (128, 64, BF), (256, 128, HF)])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,length", [([9, 1, 0, 5], [900, 1, 70, 1500]), ([30, 7, 29], [30, 2000, 333])])
def test_attention_few_rows(D, page, dt, window, causal, new, length):
    """Several blocks of 16 rows a sequence, a last one that is not full, sequences with fewer."""
    rng = np.random.default_rng(D + window + len(new))
    run_attention(rng, new, length, 6, 2, D, page, dt, causal=causal, window=window)


@pytest.mark.parametrize("D,page,dt", [(64, 32, HF), (128, 64, BF), (128, 128, HF), (256, 64, BF), (256, 32, HF),
                                       (64, 128, BF), (128, 32, BF)])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_prompts(D, page, dt, window, causal):
    rng = np.random.default_rng(D + window)
    run_attention(rng, [130, 1, 65, 0, 33], [130, 200, 300, 50, 34], 4, 2, D, page, dt, causal=causal, window=window)


@pytest.mark.parametrize("window", [1, 33, 700])
def test_attention_windows_of_long_sequences(window):
    rng = np.random.default_rng(window)
    run_attention(rng, [1, 4, 80], [2000, 1500, 900], 4, 1, 64, 32, BF, window=window)


def test_attention_rows_and_sequences_without_keys():
    rng = np.random.default_rng(1)
    table = np.array([[0, 1], [2, -1], [-1, -1], [-1, -1]], np.int32)
    cache = random_cache(rng, 3, 2, 32, 64)
    # more queries than keys (the first see nothing), a sequence of length 0, one of no tokens
    out = run_attention(rng, [70, 1, 3, 0], [40, 1, 0, 0], 4, 2, 64, 32, BF, cache=cache, table=table)
    assert (out[:30] == 0).all() and (out[71:] == 0).all()


def test_attention_long_keys_are_split_and_joined():
    rng = np.random.default_rng(3)
    out = run_attention(rng, [1, 2], [20011, 9000], 8, 2, 128, 128, BF)
    rng = np.random.default_rng(3)
    again = run_attention(rng, [1, 2], [20011, 9000], 8, 2, 128, 128, BF)
    assert torch.equal(out, again)                       # the same bits, run to run
    run_attention(np.random.default_rng(4), [40], [9000], 8, 2, 128, 64, HF)
    run_attention(np.random.default_rng(4), [5, 1], [5000, 12], 8, 2, 64, 32, HF, causal=False)


def test_attention_bounds_that_are_too_small():
    rng = np.random.default_rng(8)
    run_attention(rng, [70, 3], [600, 2000], 4, 2, 64, 64, BF, max_q=1, max_kv=1)
    run_attention(rng, [1, 1], [3000, 2000], 4, 2, 128, 64, BF, max_kv=100)


def test_attention_values_of_very_different_size():
    """Pages whose values differ by 2^40, pages of zeros, and weights on the small ones."""
    rng = np.random.default_rng(6)
    page, D = 32, 64
    lens = [512, 300]
    table, pages = table_of(rng, lens, page)
    cache = random_cache(rng, pages, 1, page, D)
    cache["ve"][:] = rng.choice([90, 100, 118, 130], (pages, 1))
    cache["v"][table[0, 3]] = 0
    cache["ve"][table[0, 3]] = 0
    run_attention(rng, [1, 40], lens, 2, 1, D, page, BF, cache=cache, table=table)
    cache["ke"][:] = rng.choice([100, 119, 121], (pages, 1))
    run_attention(rng, [1, 40], lens, 2, 1, D, page, HF, cache=cache, table=table, qscale=3.0)


def test_attention_sharp_and_flat_scores():
    rng = np.random.default_rng(12)
    run_attention(rng, [1, 70], [900, 500], 4, 2, 128, 64, BF, qscale=40.0)
    run_attention(rng, [1, 70], [900, 500], 4, 2, 128, 64, HF, qscale=1e-3)
    run_attention(rng, [1, 70], [900, 500], 4, 2, 128, 64, BF, scale=-0.05)
    run_attention(rng, [1, 70], [900, 500], 4, 2, 128, 64, BF, scale=0.0)


def test_offsets_past_32_bits():
    """A cache of over 2^32 bytes a tensor, used at its end."""
    page, D, Hk = 128, 128, 8
    pages = (1 << 32) // (page * D * Hk) + 40
    cache = q8.q8_kv_cache(pages, Hk, D, page=page, device=DEV)
    rng = np.random.default_rng(0)
    table = np.array([[pages - 1, pages - 7, 3]], np.int32)
    x = torch.from_numpy(rng.standard_normal((300, 4 + 2 * Hk, D)).astype(np.float32)).to(BF)
    start, batch = batch_of([300], [300], table)
    xd = x.to(DEV)
    q8.q8_kv_append(xd[:, 4:4 + Hk], xd[:, 4 + Hk:], cache, batch)
    small = {"k": np.zeros((3, Hk, page, D), np.uint8), "ke": np.zeros((3, Hk), np.uint8),
             "v": np.zeros((3, Hk, D, page), np.uint8), "ve": np.zeros((3, Hk), np.uint8)}
    t3 = np.array([[0, 1, 2]], np.int32)
    xf = x.float().numpy()
    P.append(small, t3, start, [300], xf[:, 4:4 + Hk], xf[:, 4 + Hk:])
    for name, big in zip(("k", "ke", "v", "ve"), cache):
        assert np.array_equal(big[table[0].tolist()].cpu().numpy(), small[name]), name
    qd = torch.from_numpy(rng.standard_normal((300, 8, D)).astype(np.float32)).to(BF)
    got = q8.q8_attention_kv8(qd.to(DEV), cache, batch).double().cpu().numpy()
    want, lse, av, aqk = P.attention(small, t3, start, [300], qd.double().numpy())
    tol, _ = bounds(av, aqk, lse, want, D, 300, BF)
    assert (np.abs(got - want) <= tol).all()


def test_other_stream_and_graph():
    """On a stream of its own, and replayed from a graph with changed inputs between the replays."""
    rng = np.random.default_rng(21)
    lens = [700, 90]
    table, pages = table_of(rng, [800, 800], 64)
    base = random_cache(rng, pages, 2, 64, 128)
    x = [torch.from_numpy(rng.standard_normal((2, 12, 128)).astype(np.float32)).to(BF).to(DEV) for _ in range(4)]
    cos, sin = (torch.from_numpy(a).to(DEV) for a in tables_of_angles(800, 128))

    def step(xin, cache, batch, out, ws):
        q = q8.q8_kv_append(xin[:, 8:10], xin[:, 10:], cache, batch, q=xin[:, :8], cos=cos, sin=sin, out=out[0])
        return q8.q8_attention_kv8(q, cache, batch, out=out[1], workspace=ws)

    ws = torch.empty(q8.q8_attention_workspace_bytes(2, 8, 2, 128, 2, 1, 800) + 16, dtype=torch.uint8, device=DEV)
    outs = lambda: (torch.empty(2, 8, 128, dtype=BF, device=DEV), torch.empty(2, 8, 128, dtype=BF, device=DEV))  # noqa: E731
    _, batch = batch_of([1, 1], lens, table, 1, 800)
    eager_cache, eager = device(base), []
    for xin in x:
        eager.append(step(xin, eager_cache, batch, outs(), ws).clone())
    side = torch.cuda.Stream()
    cache, xin, out = device(base), x[0].clone(), outs()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(xin, cache, batch, out, ws)
    side.synchronize()
    assert torch.equal(out[1], eager[0])
    cache2 = device(base)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(xin, cache2, batch, out, ws)
    for i, want in enumerate(eager):
        xin.copy_(x[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[1], want), i
        (torch.randn(256, 256, device=DEV) @ torch.randn(256, 256, device=DEV)).sum().item()


# ---------------------------------------------------------------- the binding
def test_compiled_and_interpreted_calls_agree():
    """The compiled half of the binding takes ordinary arguments and gives what the checked path gives."""
    fast = q8._fast()
    rng = np.random.default_rng(4)
    table, pages = table_of(rng, [300, 90], 64)
    base = random_cache(rng, pages, 2, 64, 128)
    _, batch = batch_of([2, 1], [300, 90], table)
    qkv = torch.from_numpy(rng.standard_normal((3, 12, 128)).astype(np.float32)).to(BF).to(DEV)
    cos, sin = (torch.from_numpy(a).to(DEV) for a in tables_of_angles(300, 128))
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    got = []
    for compiled in (True, False):
        cache = device(base)
        if compiled:
            r = fast.kv_append(k, v, cache, batch, q, cos, sin, False, None)
            assert isinstance(r, torch.Tensor)
            o = fast.attention_kv8(r, cache, batch, None, True, 0, None)
            assert isinstance(o, torch.Tensor)
        else:
            hold = q8._FAST
            q8._FAST = type("none", (), {n: staticmethod(lambda *a: NotImplemented)
                                         for n in ("kv_append", "attention_kv8", "linear_fp8_block")})
            try:
                r = q8.q8_kv_append(k, v, cache, batch, q=q, cos=cos, sin=sin)
                o = q8.q8_attention_kv8(r, cache, batch)
            finally:
                q8._FAST = hold
        got.append([r, o, *cache])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    # what the call refuses comes back as its status, what is not its kind of argument as NotImplemented
    assert fast.attention_kv8(q, device(base), batch, None, True, -1, None) == _lib.Q8_ERR_BAD_ARG
    assert fast.attention_kv8(q.cpu(), device(base), batch, None, True, 0, None) is NotImplemented
    assert fast.attention_kv8(q, device(base), batch, "x", True, 0, None) is NotImplemented
    assert fast.kv_append(k, v, device(base), batch, None, None, sin, False, None) is NotImplemented
    with pytest.raises(TypeError):
        fast.kv_append(k, v)


def test_binding_refusals():
    cache = q8.q8_kv_cache(4, 2, 64, page=32, device=DEV)
    _, batch = batch_of([2], [2], [[0, 1]])
    q = torch.zeros(2, 4, 64, dtype=BF, device=DEV)
    k = torch.zeros(2, 2, 64, dtype=BF, device=DEV)
    att = lambda **kw: q8.q8_attention_kv8(**{**dict(q=q, cache=cache, batch=batch), **kw})  # noqa: E731
    app = lambda **kw: q8.q8_kv_append(**{**dict(k=k, v=k, cache=cache, batch=batch), **kw})  # noqa: E731
    with pytest.raises(TypeError):
        att(q=q.float())
    with pytest.raises(TypeError):
        att(q=q.cpu())
    with pytest.raises(ValueError):
        att(q=q.transpose(0, 1))
    with pytest.raises(ValueError):
        att(q=q[:, :, :32])
    with pytest.raises(_lib.Q8Error):
        att(q=q[:, :3].contiguous())                     # 3 query heads over 2 kv heads
    with pytest.raises(_lib.Q8Error):
        att(window=-1)
    with pytest.raises(_lib.Q8Error):
        att(scale=float("nan"))
    with pytest.raises(TypeError):
        att(batch=batch._replace(kv_len=batch.kv_len.long()))
    with pytest.raises(ValueError):
        att(batch=batch._replace(q_start=batch.q_start[:1]))
    with pytest.raises(ValueError):
        att(cache=cache._replace(v=cache.k))
    with pytest.raises(ValueError):
        att(cache=cache._replace(v_exp=cache.v_exp[:2]))
    with pytest.raises(_lib.Q8Error):
        q8.q8_attention_kv8(q[:, :, :16].contiguous(), q8.q8_kv_cache(4, 2, 16, page=32, device=DEV), batch)
    with pytest.raises(_lib.Q8Error):
        att(cache=q8.q8_kv_cache(4, 2, 64, page=48, device=DEV))
    with pytest.raises(TypeError):
        app(v=k.half())
    with pytest.raises(ValueError):
        app(v=k[:1])
    with pytest.raises(ValueError):
        app(cos=torch.zeros(4, 16, device=DEV))
    with pytest.raises(ValueError):
        app(out=q)
    with pytest.raises(_lib.Q8Error):
        app(cos=torch.zeros(4, 4, device=DEV), sin=torch.zeros(4, 4, device=DEV))     # rot_dim 8
    with pytest.raises(_lib.Q8Error):
        app(cos=torch.zeros(4, 64, device=DEV), sin=torch.zeros(4, 64, device=DEV))   # rot_dim past dim
    long = batch_of([1, 1], [9000, 9000], [[0] * 300, [0] * 300])[1]
    with pytest.raises(_lib.Q8Error):
        att(batch=long, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
