"""q8_kv_append_norm against its definition bit for bit, and q8_attention_kv8_tree
against softmax attention in 64 bits over the same codes and masks."""
import numpy as np
import pytest
import torch

import kv8_more_plain as M
import kv8_plain as P
from test_gpu_kv8 import BF, DEV, F32, HF, batch_of, bounds, device, host, random_cache, table_of, tables_of_angles
from w8a8_quantized_linear_channel_amd import _lib
from w8a8_quantized_linear_channel_amd import ops as q8

pytestmark = pytest.mark.gpu


def up(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


# ---------------------------------------------------------------- append
def run_append(rng, news, lens, Hq, Hk, D, page, dt, rot=None, interleaved=False, positions=None, weights="both", wdt=None,
               eps=1e-6, size=1.0, max_q=None, angles=None):
    table, pages = table_of(rng, [max(n, 1) for n in lens], page)
    cache = random_cache(rng, pages, Hk, page, D)
    start, batch = batch_of(news, lens, table, max_q)
    T = int(start[-1])
    x = rng.standard_normal((T, Hq + 2 * Hk, D)) * np.exp(2 * rng.standard_normal((T, Hq + 2 * Hk, 1))) * size
    x = torch.from_numpy(x.astype(np.float32)).to(dt)
    weight = lambda on: torch.from_numpy((1 + 0.5 * rng.standard_normal(D)).astype(np.float32)).to(wdt or dt) if on else None  # noqa: E731
    wq, wk = weight(weights in ("both", "q")), weight(weights in ("both", "k"))
    cos, sin = tables_of_angles(angles or max(lens), rot) if rot else (None, None)
    pos = M.slots(start, lens)
    if positions is not None:
        pos = positions(pos).astype(np.int32)
    got, xd = device(cache), x.to(DEV)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    q = q8.q8_kv_append_norm(xd[:, Hq:Hq + Hk], xd[:, Hq + Hk:], got, batch, q=xd[:, :Hq], q_weight=dev(wq), k_weight=dev(wk),
                             eps=eps, cos=up(cos), sin=up(sin), interleaved=interleaved,
                             positions=None if positions is None else up(pos))
    xf, f = x.float().numpy(), lambda t: None if t is None else t.float().numpy()  # noqa: E731
    turn = lambda a: M.rotated(a, pos, cos, sin, interleaved)  # noqa: E731
    P.append(cache, table, start, lens, turn(M.normalised(xf[:, Hq:Hq + Hk], f(wk), eps)), xf[:, Hq + Hk:])
    got = host(got)
    for name in ("ke", "ve", "k", "v"):
        bad = np.argwhere(got[name] != cache[name])
        assert len(bad) == 0, (name, len(bad), bad[:3])
    want = torch.from_numpy(turn(M.normalised(xf[:, :Hq], f(wq), eps))).to(dt)
    assert torch.equal(q.cpu(), want)


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt", [BF, HF, F32])
def test_append_shapes(page, D, dt):
    rng = np.random.default_rng(page + D)
    run_append(rng, [1, 3, page + 5, 0, 2 * page], [1, 40, 2 * page + 9, 7, 2 * page], 4, 2, D, page, dt, rot=D)
    run_append(rng, [1, 1, 1], [1, page, page + 9], 4, 2, D, page, dt, rot=D // 2)


@pytest.mark.parametrize("rot,interleaved", [(None, False), (16, False), (32, True), (64, False), (112, False), (128, True), (128, False)])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (10, 2), (7, 1)])
def test_append_rotations_and_heads(rot, interleaved, Hq, Hk):
    rng = np.random.default_rng(Hq)
    run_append(rng, [1, 17, 1], [65, 150, 64], Hq, Hk, 128, 64, BF, rot=rot, interleaved=interleaved)
    run_append(rng, [1, 1], [65, 150], Hq, Hk, 128, 64, HF, rot=rot, interleaved=interleaved)


@pytest.mark.parametrize("weights", ["both", "q", "k", "none"])
@pytest.mark.parametrize("wdt", [F32, HF, BF])
def test_append_weights_and_positions(weights, wdt):
    rng = np.random.default_rng(5)
    # depths of a tree, positions that are not there (the table's first and last row stand in)
    for positions in (lambda p: p - p % 3, lambda p: p - 60, lambda p: p + 60, lambda p: p * 0 - 2 ** 31, lambda p: p * 0 + 2 ** 31 - 1):
        run_append(rng, [12, 1, 40], [70, 33, 45], 4, 2, 64, 32, BF, rot=64, positions=positions, weights=weights, wdt=wdt)
    run_append(rng, [1, 1], [70, 33], 4, 2, 256, 32, BF, rot=64, positions=lambda p: p - 5, weights=weights, wdt=wdt)


def test_append_sizes_of_values():
    rng = np.random.default_rng(6)
    # squares beyond binary32, rows far below eps, many tokens (heads share their angles), bounds too small
    run_append(rng, [9, 1], [40, 7], 4, 2, 128, 64, BF, rot=128, size=1e30)
    run_append(rng, [9, 1], [40, 7], 4, 2, 128, 64, F32, rot=128, size=1e-30)
    run_append(rng, [9, 1], [40, 7], 4, 2, 128, 64, HF, rot=128, size=1e-3, eps=0.1)
    run_append(rng, [700, 333], [900, 333], 10, 2, 64, 64, BF, rot=64)
    run_append(rng, [700, 333], [900, 333], 10, 2, 64, 64, HF, rot=32, interleaved=True)
    run_append(rng, [70, 1, 5], [90, 33, 5], 3, 1, 64, 32, BF, rot=64, max_q=1)
    # more new tokens than positions (the first fall away), positions past the angle table
    run_append(rng, [9, 5], [4, 70], 2, 1, 64, 64, HF, rot=64, angles=50)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_infinite_and_nan_queries(D):
    """A NaN makes its head NaN; beside an infinity (r = 0) the other features are 0; other heads are as they were."""
    rng = np.random.default_rng(D)
    x = torch.from_numpy(rng.standard_normal((9, 6, D)).astype(np.float32)).to(BF)
    x[0, 1, 3], x[2, 0, D - 1], x[4, 3, 5], x[8, 2, 0] = float("inf"), float("nan"), -float("inf"), float("inf")
    x[8, 2, 1] = float("nan")
    w = torch.from_numpy((1 + 0.5 * rng.standard_normal(D)).astype(np.float32))
    _, batch = batch_of([9], [9], [[0]])
    k = x[:, 4:].to(DEV)
    got = q8.q8_kv_append_norm(k[:, :1], k[:, 1:], q8.q8_kv_cache(1, 1, D, page=32, device=DEV), batch, q=x[:, :4].to(DEV),
                               q_weight=w.to(DEV)).cpu().float()
    with np.errstate(invalid="ignore"):
        want = torch.from_numpy(M.normalised(x[:, :4].float().numpy(), w.numpy(), 1e-6)).to(BF).float()
    assert want[0, 1].isnan().sum() == 1 and want[2, 0].isnan().all() and want[8, 2].isnan().all()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())


def test_append_zeros_and_no_tokens():
    cache = q8.q8_kv_cache(2, 1, 64, page=32, device=DEV)
    _, batch = batch_of([3], [3], [[0]])
    one = torch.ones(64, dtype=F32, device=DEV)
    z = torch.zeros(3, 1, 64, dtype=BF, device=DEV)
    q = q8.q8_kv_append_norm(z, z, cache, batch, q=z, q_weight=one, k_weight=one)
    assert (q == 0).all() and all((t == 0).all() for t in cache)
    _, batch = batch_of([0], [0], [[0]])
    assert q8.q8_kv_append_norm(z[:0], z[:0], cache, batch, q=z[:0], q_weight=one).shape == (0, 1, 64)
    _, batch = batch_of([3], [3], [[0]])
    x = torch.randn(3, 2, 64, device=DEV).to(BF)
    assert q8.q8_kv_append_norm(x[:, :1], x[:, 1:], cache, batch, k_weight=one) is None
    # in place, and what q8_kv_append gives where nothing is normalised
    cos, sin = (up(a) for a in tables_of_angles(3, 64))
    for turned in (False, True):
        a, b = (q8.q8_kv_cache(2, 1, 64, page=32, device=DEV) for _ in range(2))
        k = x[:, :1].contiguous()
        want = q8.q8_kv_append(k, k, a, batch, q=x, cos=cos, sin=sin, interleaved=turned)
        y = x.clone()
        assert torch.equal(q8.q8_kv_append_norm(k, k, b, batch, q=y, cos=cos, sin=sin, interleaved=turned, out=y), want)
        assert all(torch.equal(s, t) for s, t in zip(a, b))
    y = x.clone()
    want = q8.q8_kv_append_norm(k, k, a, batch, q=x, q_weight=one, cos=cos, sin=sin)
    assert torch.equal(q8.q8_kv_append_norm(k, k, a, batch, q=y, q_weight=one, cos=cos, sin=sin, out=y), want)


# ---------------------------------------------------------------- attention
def any_mask(rng, n, kind):
    if kind == "tree":
        return M.tree_of(rng, n)[1]
    if kind == "chain":
        return np.tril(np.ones((n, n), bool))
    if kind == "none":
        return np.zeros((n, n), bool)
    return rng.random((n, n)) < 0.4


def run_tree(rng, news, lens, Hq, Hk, D, page, dt, kind="tree", window=0, cache=None, table=None, scale=None, words=None,
             deep=True, max_q=None, max_kv=None, qscale=1.0, garbage=True, strided=False, beyond=0):
    if table is None:
        table, pages = table_of(rng, [max(n, 1) for n in lens], page)
    if cache is None:
        cache = random_cache(rng, pages, Hk, page, D)
    words = words or max(1, -(-max(news) // 64))
    sees = [any_mask(rng, n, kind) for n in news]
    sees = [s[:, :64 * words] for s in sees]
    start, batch = batch_of(news, lens, table, max_q, max_kv)
    T = int(start[-1])
    pos = None
    if deep:
        pos = np.concatenate([b - n + np.maximum(s.sum(1) - 1, 0) for n, b, s in zip(news, lens, sees)]).astype(np.int32)
        pos = pos + beyond
    mask = np.zeros((T, words), np.uint64)
    for s, a in enumerate(sees):
        mask[start[s]:start[s + 1]] = M.words_of(a, words)
        extra = rng.integers(0, 2, (len(a), 64 * words)).astype(bool)     # bits of tokens that are not there
        extra[:, :news[s]] = False
        mask[start[s]:start[s + 1]] |= M.words_of(extra, words)
    if garbage:
        # NaN codes in every slot that no query sees
        for s, (n, total) in enumerate(zip(news, lens)):
            seen = M.tree_seen(n, total, sees[s], None if pos is None else pos[start[s]:start[s + 1]], window).any(0)
            seen = np.concatenate([seen, np.zeros(table.shape[1] * page, bool)])
            for lp in range(table.shape[1]):
                at = table[s, lp]
                if 0 <= at < len(cache["ke"]):
                    hide = ~seen[lp * page:(lp + 1) * page]
                    cache["k"][at][:, hide] = 0x7F
                    cache["v"][at][:, :, hide] = 0xFF
    q = torch.from_numpy((rng.standard_normal((T, Hq + (2 if strided else 0), D)) * qscale).astype(np.float32)).to(dt)
    qd = q.to(DEV)[:, :Hq]
    out, lse = q8.q8_attention_kv8_tree(qd, device(cache), batch, up(mask.view(np.int64)), positions=up(pos), window=window,
                                        scale=scale, lse=True)
    want, wl, av, aqk = M.tree_attention(cache, table, start, lens, q[:, :Hq].double().numpy(), sees, pos, scale, window)
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
def test_tree_shapes(page, D, dt):
    """One block of 16 rows, several, and blocks of 128 and 256."""
    rng = np.random.default_rng(D + page)
    run_tree(rng, [3, 1, 4, 2], [3, 31, 129, 1000], 8, 2, D, page, dt)
    run_tree(rng, [12, 7, 16], [300, 16, 77], 8, 2, D, page, dt)
    run_tree(rng, [70, 33, 1, 0], [200, 40, 65, 9], 8, 2, D, page, dt)


@pytest.mark.parametrize("kind", ["tree", "chain", "none", "any"])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("D,page,dt", [(64, 32, HF), (128, 64, BF), (256, 128, HF)])
def test_tree_masks_and_windows(kind, window, D, page, dt):
    rng = np.random.default_rng(D + window)
    run_tree(rng, [5, 1, 9], [90, 1, 500], 4, 2, D, page, dt, kind=kind, window=window)
    run_tree(rng, [65, 130, 20], [300, 131, 20], 6, 2, D, page, dt, kind=kind, window=window, strided=True)
    run_tree(rng, [24, 64], [700, 64], 4, 1, D, page, dt, kind=kind, window=window, deep=False)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (2, 2), (5, 1), (12, 4), (17, 1), (48, 2)])
def test_tree_heads(Hq, Hk):
    rng = np.random.default_rng(Hq)
    run_tree(rng, [1, 12, 30], [300, 77, 31], Hq, Hk, 64, 32, BF, strided=True)


def test_tree_words_of_masks():
    rng = np.random.default_rng(2)
    # more words than tokens, fewer (later tokens are seen by nobody), masks that end inside a step of keys
    run_tree(rng, [5, 64], [40, 100], 4, 2, 64, 32, BF, kind="any", words=5)
    run_tree(rng, [200, 70], [260, 75], 4, 2, 64, 32, BF, kind="any", words=1)
    run_tree(rng, [200, 70], [260, 75], 4, 2, 128, 64, HF, kind="any", words=2)
    run_tree(rng, [333], [1000], 2, 1, 128, 64, BF, kind="any")
    for past in (0, 1, 15, 16, 17, 31, 33, 47, 63, 64, 65):
        run_tree(rng, [66, 3], [past + 66, past + 3], 2, 1, 64, 32, HF, kind="any")


@pytest.mark.parametrize("window", [1, 33, 700])
def test_tree_windows_of_long_sequences(window):
    rng = np.random.default_rng(window)
    run_tree(rng, [1, 4, 80], [2000, 1500, 900], 4, 1, 64, 32, BF, window=window)
    # positions that leave past .. past + n - 1 are taken at its ends
    run_tree(rng, [9, 40], [500, 900], 4, 1, 64, 32, BF, window=window, beyond=-300)
    run_tree(rng, [9, 40], [500, 900], 4, 1, 64, 32, BF, window=window, beyond=300)


def test_tree_rows_and_sequences_without_keys():
    rng = np.random.default_rng(1)
    table = np.array([[0, 1], [2, -1], [-1, -1], [-1, -1]], np.int32)
    cache = random_cache(rng, 3, 2, 32, 64)
    out = run_tree(rng, [70, 1, 3, 0], [40, 1, 0, 0], 4, 2, 64, 32, BF, cache=cache, table=table, kind="chain")
    assert (out[:30] == 0).all() and (out[71:] == 0).all()
    table, pages = table_of(rng, [9, 70], 32)
    out = run_tree(rng, [9, 70], [9, 70], 4, 2, 64, 32, BF, kind="none")
    assert (out == 0).all()


def test_tree_rows_behind_the_last_sequence_are_left():
    rng = np.random.default_rng(3)
    table, pages = table_of(rng, [50], 32)
    cache = device(random_cache(rng, pages, 1, 32, 64))
    _, batch = batch_of([6], [50], table)
    q = torch.randn(20, 4, 64, device=DEV).to(BF)
    mask = torch.ones(20, 1, dtype=torch.int64, device=DEV)
    out = torch.full((20, 4, 64), 7.0, dtype=BF, device=DEV)
    y = q8.q8_attention_kv8_tree(q, cache, batch, mask, out=out)
    assert y is out and (out[6:] == 7).all() and (out[:6] != 7).any()


def test_tree_long_keys_are_split_and_joined():
    run = lambda: run_tree(np.random.default_rng(3), [9, 2], [20011, 9000], 8, 2, 128, 128, BF)  # noqa: E731
    assert torch.equal(run(), run())                     # the same bits, run to run
    run_tree(np.random.default_rng(4), [40], [9000], 8, 2, 128, 64, HF)
    run_tree(np.random.default_rng(4), [66, 1], [5000, 12], 8, 2, 64, 32, HF, kind="any")
    run_tree(np.random.default_rng(4), [30], [6000], 4, 1, 256, 64, BF, window=3000)


@pytest.mark.parametrize("D,dt", [(64, HF), (128, BF), (256, BF)])
@pytest.mark.parametrize("S", [2, 40, 64, 65])
def test_tree_many_sequences(S, D, dt):
    """Batches whose workgroups follow each other, taken by length: lengths that are alike, empty sequences among
    them, up to 64 (one a lane) and more; bounds that ask for 16 rows a wave and for 32."""
    rng = np.random.default_rng(S)
    lens = rng.choice([0, 1, 33, 90, 90, 90, 150, 200], S)
    news = np.minimum(lens, rng.integers(0, 10, S))
    news[0], lens[0] = 9, 120
    for most in (None, 5000):
        for _ in range(2 if S == 2 else 1):
            run_tree(rng, news.tolist(), lens.tolist(), 32, 8, D, 32, dt, max_q=300 if S == 2 else None, max_kv=most)
    run_tree(rng, [3] * S, [40] * S, 32, 8, D, 32, dt, max_q=300 if S == 2 else 9)


def test_tree_bounds_that_are_too_small_and_scales():
    rng = np.random.default_rng(8)
    run_tree(rng, [70, 3], [600, 2000], 4, 2, 64, 64, BF, max_q=1, max_kv=1)
    run_tree(rng, [10, 1], [3000, 2000], 4, 2, 128, 64, BF, max_kv=100)
    for dt, kw in ((BF, dict(qscale=40.0)), (HF, dict(qscale=1e-3)), (BF, dict(scale=-0.05)), (BF, dict(scale=0.0))):
        run_tree(rng, [5, 70], [900, 500], 4, 2, 128, 64, dt, **kw)


def test_tree_values_of_very_different_size():
    rng = np.random.default_rng(6)
    lens = [512, 300]
    table, pages = table_of(rng, lens, 32)
    cache = random_cache(rng, pages, 1, 32, 64)
    cache["ve"][:] = rng.choice([90, 100, 118, 130], (pages, 1))
    cache["v"][table[0, 3]] = 0
    cache["ve"][table[0, 3]] = 0
    run_tree(rng, [6, 40], lens, 2, 1, 64, 32, BF, cache=cache, table=table)


@pytest.mark.parametrize("n,total,Hq,D,page", [(5, 70, 2, 64, 32), (30, 300, 4, 128, 64), (30, 300, 2, 256, 32), (130, 180, 4, 64, 32),
                                               (200, 400, 2, 256, 64), (40, 9000, 4, 128, 64), (70, 40, 2, 64, 32)])
def test_tree_nan_codes(n, total, Hq, D, page):
    """A NaN among the values reaches the rows that see its key, one among the keys their scores; no others."""
    rng = np.random.default_rng(n + D)
    table, pages = table_of(rng, [total], page)
    cache = random_cache(rng, pages, 1, page, D)
    _, batch = batch_of([n], [total], table)
    sees = any_mask(rng, n, "any")
    words = -(-n // 64)
    mask = up(M.words_of(sees, words).view(np.int64))
    seen = M.tree_seen(n, total, sees, None, 0)
    q = torch.randn(n, Hq, D, device=DEV).to(BF)
    call = lambda c: q8.q8_attention_kv8_tree(q, device(c), batch, mask, lse=True)  # noqa: E731
    clean, clean_lse = call(cache)
    for at in sorted({0, max(total - n - 1, 0), max(total - n, 0), total - n // 2, total - 1}):
        rows = torch.from_numpy(np.flatnonzero(seen[:, at])).to(DEV)
        c = {**cache, "v": cache["v"].copy()}
        c["v"][table[0, at // page], 0, [3, D - 1], at % page] = [0x7F, 0xFF]
        out, lse = call(c)
        want = clean.clone()
        for f in (3, D - 1):
            want[rows, :, f] = float("nan")
        assert torch.equal(torch.isnan(out), torch.isnan(want)), at
        assert torch.equal(out.nan_to_num(), want.nan_to_num()) and torch.equal(lse, clean_lse), at
        c = {**cache, "k": cache["k"].copy()}
        c["k"][table[0, at // page], 0, at % page, D - 2] = 0x7F
        out, lse = call(c)
        bad = torch.zeros(n, dtype=torch.bool, device=DEV)
        bad[rows] = True
        assert out[bad].isnan().all() and lse[bad].isnan().all(), at
        assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], clean_lse[~bad]), at


def test_offsets_past_32_bits():
    """A cache of over 2^32 bytes a tensor, used at its end."""
    page, D, Hk = 128, 128, 8
    pages = (1 << 32) // (page * D * Hk) + 40
    cache = q8.q8_kv_cache(pages, Hk, D, page=page, device=DEV)
    rng = np.random.default_rng(0)
    table = np.array([[pages - 1, pages - 7, 3]], np.int32)
    x = torch.from_numpy(rng.standard_normal((300, 4 + 2 * Hk, D)).astype(np.float32)).to(BF)
    w = torch.ones(D, dtype=BF)
    start, batch = batch_of([300], [300], table)
    xd = x.to(DEV)
    q8.q8_kv_append_norm(xd[:, 4:4 + Hk], xd[:, 4 + Hk:], cache, batch, k_weight=w.to(DEV))
    small = {"k": np.zeros((3, Hk, page, D), np.uint8), "ke": np.zeros((3, Hk), np.uint8),
             "v": np.zeros((3, Hk, D, page), np.uint8), "ve": np.zeros((3, Hk), np.uint8)}
    t3, xf = np.array([[0, 1, 2]], np.int32), x.float().numpy()
    P.append(small, t3, start, [300], M.normalised(xf[:, 4:4 + Hk], w.float().numpy(), 1e-6), xf[:, 4 + Hk:])
    for name, big in zip(("k", "ke", "v", "ve"), cache):
        assert np.array_equal(big[table[0].tolist()].cpu().numpy(), small[name]), name
    sees = [any_mask(rng, 40, "tree")]
    start, batch = batch_of([40], [300], table)
    qd = torch.from_numpy(rng.standard_normal((40, 8, D)).astype(np.float32)).to(BF)
    got = q8.q8_attention_kv8_tree(qd.to(DEV), cache, batch, up(M.words_of(sees[0], 1).view(np.int64)))
    want, lse, av, aqk = M.tree_attention(small, t3, start, [300], qd.double().numpy(), sees)
    tol, _ = bounds(av, aqk, lse, want, D, 300, BF)
    assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()


# ---------------------------------------------------------------- streams, graphs, the binding
def test_other_stream_and_graph():
    """On a stream of its own, and replayed from a graph with changed inputs between the replays."""
    rng = np.random.default_rng(21)
    news, lens = [9, 5], [700, 90]
    table, pages = table_of(rng, [2100, 800], 64)
    base = random_cache(rng, pages, 2, 64, 128)
    sees = [M.tree_of(rng, n)[1] for n in news]
    mask = up(np.concatenate([M.words_of(s, 1) for s in sees]).view(np.int64))
    pos = up(np.concatenate([b - n + s.sum(1) - 1 for n, b, s in zip(news, lens, sees)]).astype(np.int32))
    x = [torch.from_numpy(rng.standard_normal((14, 12, 128)).astype(np.float32)).to(BF).to(DEV) for _ in range(4)]
    cos, sin = (up(a) for a in tables_of_angles(2100, 128))
    w = torch.rand(128, device=DEV) + 0.5
    _, batch = batch_of(news, lens, table, 9, 2100)
    need = q8.q8_attention_tree_workspace_bytes(14, 8, 2, 128, 2, 9, 2100)
    ws = torch.empty(need + 16, dtype=torch.uint8, device=DEV)

    def step(xin, cache, out):
        q = q8.q8_kv_append_norm(xin[:, 8:10], xin[:, 10:], cache, batch, q=xin[:, :8], q_weight=w, k_weight=w, cos=cos, sin=sin,
                                 positions=pos, out=out[0])
        return q8.q8_attention_kv8_tree(q, cache, batch, mask, positions=pos, out=out[1], workspace=ws)

    outs = lambda: (torch.empty(14, 8, 128, dtype=BF, device=DEV), torch.empty(14, 8, 128, dtype=BF, device=DEV))  # noqa: E731
    eager_cache, eager = device(base), []
    for xin in x:
        eager.append(step(xin, eager_cache, outs()).clone())
    side = torch.cuda.Stream()
    cache, xin, out = device(base), x[0].clone(), outs()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(xin, cache, out)
    side.synchronize()
    assert torch.equal(out[1], eager[0])
    cache2 = device(base)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(xin, cache2, out)
    for i, want in enumerate(eager):
        xin.copy_(x[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[1], want), i
        (torch.randn(256, 256, device=DEV) @ torch.randn(256, 256, device=DEV)).sum().item()
    assert all(torch.equal(a, b) for a, b in zip(cache2, eager_cache))


def interpreted(f):
    hold = q8._FAST
    q8._FAST = type("none", (), {n: staticmethod(lambda *a: NotImplemented)
                                 for n in ("kv_append_norm", "attention_kv8_tree", "kv_compact", "kv_fork")})
    try:
        return f()
    finally:
        q8._FAST = hold


def test_compiled_and_interpreted_calls_agree():
    fast = q8._fast()
    rng = np.random.default_rng(4)
    table, pages = table_of(rng, [300, 90], 64)
    base = random_cache(rng, pages, 2, 64, 128)
    _, batch = batch_of([2, 1], [300, 90], table)
    qkv = torch.from_numpy(rng.standard_normal((3, 12, 128)).astype(np.float32)).to(BF).to(DEV)
    cos, sin = (up(a) for a in tables_of_angles(300, 128))
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    w, pos = torch.rand(128, device=DEV).to(HF), torch.tensor([5, 6, 7], dtype=torch.int32, device=DEV)
    mask = torch.tensor([[1], [3], [1]], dtype=torch.int64, device=DEV)

    def both(cache):
        r = q8.q8_kv_append_norm(k, v, cache, batch, q=q, q_weight=w, k_weight=w, cos=cos, sin=sin, positions=pos)
        return [r, q8.q8_attention_kv8_tree(r, cache, batch, mask, positions=pos, window=100),
                q8.q8_attention_kv8_tree(r, cache, batch, mask.view(torch.uint64)), *cache]

    for a, b in zip(both(device(base)), interpreted(lambda: both(device(base)))):
        assert torch.equal(a, b)
    assert isinstance(fast.kv_append_norm(k, v, device(base), batch, q, w, w, 1e-6, cos, sin, False, pos, None), torch.Tensor)
    assert fast.kv_append_norm(k, v, device(base), batch, q, w, w, 0.0, cos, sin, False, pos, None) == _lib.Q8_ERR_BAD_ARG
    assert fast.kv_append_norm(k, v, device(base), batch, q, w, w.float(), 1e-6, cos, sin, False, pos, None) is NotImplemented
    assert isinstance(fast.attention_kv8_tree(q, device(base), batch, mask, pos, None, 0, None), torch.Tensor)
    assert fast.attention_kv8_tree(q, device(base), batch, mask, pos, None, -1, None) == _lib.Q8_ERR_BAD_ARG
    assert fast.attention_kv8_tree(q, device(base), batch, mask.int(), pos, None, 0, None) is NotImplemented
    with pytest.raises(TypeError):
        fast.kv_append_norm(k, v)


def test_binding_refusals():
    cache = q8.q8_kv_cache(4, 2, 64, page=32, device=DEV)
    _, batch = batch_of([2], [2], [[0, 1]])
    q = torch.zeros(2, 4, 64, dtype=BF, device=DEV)
    k = torch.zeros(2, 2, 64, dtype=BF, device=DEV)
    w = torch.ones(64, dtype=BF, device=DEV)
    mask = torch.zeros(2, 1, dtype=torch.int64, device=DEV)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    att = lambda **kw: q8.q8_attention_kv8_tree(**{**dict(q=q, cache=cache, batch=batch, mask=mask), **kw})  # noqa: E731
    app = lambda **kw: q8.q8_kv_append_norm(**{**dict(k=k, v=k, cache=cache, batch=batch, k_weight=w), **kw})  # noqa: E731
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(mask=mask.int()), dict(mask=mask.cpu()), dict(mask=mask[0]),
                dict(positions=pos.long()), dict(batch=batch._replace(kv_len=batch.kv_len.long()))):
        with pytest.raises(TypeError):
            att(**bad)
    for bad in (dict(mask=mask[:1]), dict(positions=pos[:1]), dict(mask=mask.expand(2, 3)), dict(q=q.transpose(0, 1)), dict(out=q[:1]),
                dict(cache=cache._replace(v=cache.k))):
        with pytest.raises(ValueError):
            att(**bad)
    for bad in (dict(window=-1), dict(scale=float("nan")), dict(q=q[:, :3].contiguous()), dict(mask=mask[:, :0])):
        with pytest.raises(_lib.Q8Error):
            att(**bad)
    for bad in (dict(k_weight=w.double()), dict(k_weight=w.cpu()), dict(positions=pos.long()), dict(q=q, q_weight=w.float()), dict(v=k.half())):
        with pytest.raises(TypeError):
            app(**bad)
    for bad in (dict(k_weight=w[:32]), dict(positions=pos[:1]), dict(q_weight=w), dict(out=q), dict(v=k[:1]), dict(cos=torch.zeros(4, 16, device=DEV))):
        with pytest.raises(ValueError):
            app(**bad)
    for bad in (dict(eps=0.0), dict(eps=float("nan")), dict(cos=torch.zeros(4, 4, device=DEV), sin=torch.zeros(4, 4, device=DEV))):
        with pytest.raises(_lib.Q8Error):
            app(**bad)
